"""One decoder layer of a batch of running requests, step by step: block map,
INT4 fused QKV projection, rotary positions and cache append, attention over
the paged cache, INT4 output projection, routed SwiGLU experts.

    python examples/decode_step.py [--requests 4] [--steps 8] [--cache e4m3] [--graph]

Weights and requests are random; the requests begin with contexts of different
lengths, whose keys and values are put into the cache as a prompt's would be.
With --graph a step is captured once in a CUDA graph and replayed: lengths,
block tables and slots are all made on the GPU, so nothing of a step depends
on the host.  Needs the library built and a GB300.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from w4a16_int4_weight_gemv_gb300 import binding as w

GROUP = 128


def random_int4(gen, *shape):
    """(wq, scale, zero) of random INT4 weights [..., N, K]."""
    *lead, n, k = shape
    dev = gen.device
    wq = torch.randint(-2 ** 31, 2 ** 31, (*lead, n, k // 8), generator=gen, device=dev, dtype=torch.int64).int()
    scale = ((0.5 + torch.rand(*lead, n, k // GROUP, generator=gen, device=dev)) * 0.2 * k ** -0.5).bfloat16()
    return wq, scale, torch.full((*lead, n, k // GROUP), 8, dtype=torch.uint8, device=dev)


class Layer:
    """A decoder layer's weights: q_heads query heads over kv_heads key/value
    heads of dim, topk of `experts` SwiGLU experts of width ffn."""

    def __init__(self, hidden=4096, q_heads=32, kv_heads=8, dim=128, experts=8, topk=2, ffn=1024, theta=10000.0, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.q_heads, self.kv_heads, self.dim, self.topk = q_heads, kv_heads, dim, topk
        self.qkv = random_int4(gen, (q_heads + 2 * kv_heads) * dim, hidden)
        self.out = random_int4(gen, hidden, q_heads * dim)
        self.gate, self.up = (random_int4(gen, experts, ffn, hidden) for _ in range(2))
        self.down = random_int4(gen, experts, hidden, ffn)
        self.router = torch.randn(hidden, experts, generator=gen, device="cuda") * hidden ** -0.5
        half = dim // 2
        self.inv_freq = theta ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        self.inv_freq = self.inv_freq.float()


class Requests:
    """The running requests: their lengths, block table and share of the cache."""

    def __init__(self, layer: Layer, contexts, room, page=16, e4m3=False, seed=0):
        n = len(contexts)
        columns = -(-(max(contexts) + room) // page)
        self.blocks, self.page = n * columns, page
        shape = (self.blocks, page, layer.kv_heads, layer.dim)
        dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        scales = [torch.full((layer.kv_heads,), 1 / 32, device="cuda") for _ in range(2)] if e4m3 else [None, None]
        self.cache = w.PagedCache(torch.zeros(shape, dtype=dtype, device="cuda"), torch.zeros(shape, dtype=dtype, device="cuda"), *scales)
        self.table = torch.full((n, columns), -1, dtype=torch.int32, device="cuda")
        order = torch.randperm(self.blocks, generator=torch.Generator().manual_seed(seed))
        self.free = order.int().cuda()
        self.free_head = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.lengths = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.one = torch.ones(n, dtype=torch.int32, device="cuda")
        self.workspace = w.paged_attention_workspace(self.cache, layer.q_heads)
        # the contexts: keys and values as a prompt's projection would give them
        gen = torch.Generator(device="cuda").manual_seed(seed + 1)
        total = sum(contexts)
        self.advance(w.w4a16_paged_map(self.lengths, torch.tensor(contexts, dtype=torch.int32, device="cuda"), self.table, self.free,
                                       self.free_head, page, self.blocks, total))
        self.prompt = [torch.randn(total, layer.kv_heads, layer.dim, generator=gen, device="cuda").bfloat16() for _ in range(2)]
        w.w4a16_rope_append(None, *self.prompt, self.map.positions, layer.inv_freq, self.map.slots, self.cache)

    def advance(self, m):
        self.map = m
        self.lengths.copy_(m.kv_len)
        self.free_head.copy_(m.free_head)


def step(layer: Layer, req: Requests, x):
    """x bf16 [requests, hidden], one token of every request -> the layer's output."""
    n = x.shape[0]
    m = w.w4a16_paged_map(req.lengths, req.one, req.table, req.free, req.free_head, req.page, req.blocks, n)
    qkv = w.w4a16_gemv(x, *layer.qkv, GROUP, weights_static=True)
    q, k, v = (t.view(n, -1, layer.dim) for t in
               qkv.split([layer.q_heads * layer.dim, layer.kv_heads * layer.dim, layer.kv_heads * layer.dim], 1))
    w.w4a16_rope_append(q, k, v, m.positions, layer.inv_freq, m.slots, req.cache, q_out=q)
    a, _ = w.w4a16_paged_attention(q, req.cache, req.table, m.kv_len, workspace=req.workspace)
    x = x + w.w4a16_gemv(a.view(n, -1), *layer.out, GROUP, weights_static=True)
    top, ids = torch.topk(x.float() @ layer.router, layer.topk)
    y = x + w.moe_ffn(x, ids.int(), torch.softmax(top, 1), layer.gate, layer.up, layer.down, GROUP)
    req.advance(m)
    return y


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=4, help="1 to 16")
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    ap.add_argument("--graph", action="store_true")
    a = ap.parse_args()
    layer = Layer()
    contexts = [37 + 911 * i for i in range(a.requests)]
    req = Requests(layer, contexts, room=a.steps + 8, e4m3=a.cache == "e4m3")
    x = torch.randn(a.requests, 4096, device="cuda").bfloat16()
    step(layer, req, x)  # everything loaded before the capture and the clock
    if a.graph:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = step(layer, req, x)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    begin.record()
    for _ in range(a.steps):
        if a.graph:
            graph.replay()
        else:
            y = step(layer, req, x)
    end.record()
    torch.cuda.synchronize()
    error = w.w4a16_device_error()
    print("%d requests, lengths now %s, %.1f us a step, output norm %.3f, device error bits 0x%x"
          % (a.requests, req.lengths.tolist(), 1e3 * begin.elapsed_time(end) / a.steps, y.float().norm(), error))
    return 1 if error else 0


if __name__ == "__main__":
    sys.exit(main())
