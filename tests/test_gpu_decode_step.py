"""The paged-cache operators together with the INT4 projections and experts,
as examples/decode_step.py runs them: the keys, values and attention of
several steps against 64-bit forms, and a captured step against the same step
run call by call."""
import importlib.util
import os

import pytest
import torch

from . import paged_reference as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_weight_gemv_gb300 import build_ext
    build_ext.build()
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.w.w4a16_device_error(clear=True)
    return mod


def small(ex, e4m3=False):
    layer = ex.Layer(hidden=512, q_heads=8, kv_heads=2, dim=64, experts=4, topk=2, ffn=256, seed=3)
    req = ex.Requests(layer, [5, 0, 130, 31], room=8, page=16, e4m3=e4m3, seed=4)
    return layer, req


@pytest.mark.parametrize("e4m3", [False, True])
def test_steps_match_the_plain_form(ex, e4m3):
    layer, req = small(ex, e4m3)
    w = ex.w
    contexts = [5, 0, 130, 31]
    gen = torch.Generator(device="cuda").manual_seed(7)
    seen, scale = [], layer.dim ** -0.5
    original = w.w4a16_paged_attention
    for s in range(4):
        x = torch.randn(4, 512, generator=gen, device="cuda").bfloat16()
        y = ex.step(layer, req, x)
        assert not y.isnan().any()
        # the projection's rows, turned and stored in 64 bits
        qkv = ex.w.w4a16_gemv(x, *layer.qkv, ex.GROUP).double().cpu()
        q, k, v = (t.view(4, -1, 64) for t in qkv.split([512, 128, 128], 1))
        pos = torch.tensor([[c + s for c in contexts]], dtype=torch.int32)
        f = layer.inv_freq.cpu()
        qr, kr = ref.rope(q, pos, f, [32], False), ref.rope(k, pos, f, [32], False)
        seen.append((kr, v))
        lens = [c + s + 1 for c in contexts]
        assert req.lengths.tolist() == lens
        table = req.table.tolist()
        cache = [c.float().double().cpu() * (1 / 32 if e4m3 else 1) for c in (req.cache.k, req.cache.v)]
        # what is in the cache: every step's rows at their places, to the cache type's rounding
        step_tol = 2.0 ** -4 if e4m3 else 2.0 ** -8
        for i, (kk, vv) in enumerate(seen):
            for b in range(4):
                j = contexts[b] + i
                at = (table[b][j // 16], j % 16)
                for got, want in ((cache[0][at], kk[b]), (cache[1][at], vv[b])):
                    assert ((got - want).abs() <= step_tol * 1.001 * want.abs() + 2.0 ** -10 * (1 / 32 if e4m3 else 1) + 1e-5).all()
        # attention over that cache: rotated queries rounded to bf16 once more than the 64-bit form's
        out, lse = original(qr.bfloat16().cuda(), req.cache, req.table, req.lengths)
        want, want_lse, spread, reach = ref.attention(qr.bfloat16().double(), *cache, table, lens, scale, 0)
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2 * (64 + 16) * 2.0 ** -24 * reach[..., None]) * spread + 1e-30
        assert ((out.double().cpu() - want).abs() <= tol).all()
    assert w.w4a16_device_error(clear=True) == 0


def test_a_captured_step_repeats_the_calls(ex):
    layer, req = small(ex)
    layer2, req2 = small(ex)
    x = torch.randn(4, 512, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda").bfloat16()
    first = [ex.step(layer, req, x).clone() for _ in range(5)]
    assert torch.equal(ex.step(layer2, req2, x), first[0])  # everything loaded before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ex.step(layer2, req2, x)
    for i in range(1, 5):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, first[i]), i
    assert req.lengths.tolist() == req2.lengths.tolist()
    assert torch.equal(req.table, req2.table)
    assert torch.equal(req.cache.k, req2.cache.k) and torch.equal(req.cache.v, req2.cache.v)
    assert ex.w.w4a16_device_error(clear=True) == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_step_hands_the_right_things_on(ex, e4m3, monkeypatch):
    """What the step itself gives its attention and takes from it: the call's own
    queries, lengths and table, and the outputs that the rest of the step goes on with."""
    layer, req = small(ex, e4m3)
    w = ex.w
    contexts = [5, 0, 130, 31]
    calls = []
    plain = w.w4a16_paged_attention

    def recorded(q, cache, table, kv_len, **kw):
        out, lse = plain(q, cache, table, kv_len, **kw)
        calls.append((q.clone(), cache, table.clone(), kv_len.clone(), out.clone(), lse.clone()))
        return out, lse

    monkeypatch.setattr(w, "w4a16_paged_attention", recorded)
    gen = torch.Generator(device="cuda").manual_seed(11)
    u = 2.0 ** -8
    for s in range(3):
        x = torch.randn(4, 512, generator=gen, device="cuda").bfloat16()
        y = ex.step(layer, req, x)
        q, cache, table, kv_len, out, lse = calls[s]
        lens = [c + s + 1 for c in contexts]
        assert len(calls) == s + 1 and cache is req.cache and kv_len.tolist() == lens and torch.equal(table, req.table)
        # the queries: the projection's, turned in 64 bits, rounded once
        rows = w.w4a16_gemv(x, *layer.qkv, ex.GROUP).double().cpu()[:, :512].view(4, 8, 64)
        pos = torch.tensor([[n - 1 for n in lens]], dtype=torch.int32)
        turned = ref.rope(rows, pos, layer.inv_freq.cpu(), [32], False)
        size = rows.abs().amax(-1, keepdim=True)
        assert ((q.double().cpu() - turned).abs() <= u * turned.abs() + 2.0 ** -18 * size).all()
        # the outputs, over what is in the cache now
        factor = 1 / 32 if e4m3 else 1
        cached = [c.float().double().cpu() * factor for c in (req.cache.k, req.cache.v)]
        want, want_lse, spread, reach = ref.attention(q.double().cpu(), *cached, table.tolist(), lens, layer.dim ** -0.5, 0)
        score = (64 + 16) * 2.0 ** -24 * reach
        assert ((out.double().cpu() - want).abs() <= u * want.abs() + (u + 2 * score[..., None]) * spread + 1e-30).all()
        assert ((lse.double().cpu() - want_lse).abs() <= score + 2.0 ** -20 * (1 + want_lse.abs())).all()
        # and the rest of the step from them: the same calls on the same rows give the same bits
        h = x + w.w4a16_gemv(out.view(4, -1), *layer.out, ex.GROUP, weights_static=True)
        top, ids = torch.topk(h.float() @ layer.router, layer.topk)
        assert torch.equal(y, h + w.moe_ffn(h, ids.int(), torch.softmax(top, 1), layer.gate, layer.up, layer.down, ex.GROUP))
    assert w.w4a16_device_error(clear=True) == 0
