"""The 8-bit cache with scales by group in a decoder layer's step, as
examples/decode_step.py runs it, and the calls over it on a stream that is not the
current one (which make their outputs and workspaces themselves)."""
import pytest
import torch

from . import scaled_reference as ref
from .test_gpu_decode_step import ex  # noqa: F401  (the fixture)
from .test_gpu_paged import freqs, i32, w  # noqa: F401  (w: the fixture)
from .test_gpu_scaled import attention_problem, check_attention, make_cache, raw, read_problem
from .test_gpu_streams import BUSY, Raw, bits, tensors

pytestmark = pytest.mark.gpu
TYPES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def small(ex, dtype):
    layer = ex.Layer(hidden=512, q_heads=8, kv_heads=2, dim=64, experts=4, topk=2, ffn=256, seed=3)
    return layer, ex.Requests(layer, [5, 0, 130, 31], room=8, page=32, groups=dtype, seed=4)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_steps_match_the_plain_form(ex, w, dtype):
    layer, req = small(ex, TYPES[dtype])
    contexts, gen = [5, 0, 130, 31], torch.Generator(device="cuda").manual_seed(7)
    assert req.cache.group == 16
    seen = []
    for s in range(4):
        x = torch.randn(4, 512, generator=gen, device="cuda").bfloat16()
        y = ex.step(layer, req, x)
        assert not y.isnan().any()
        qkv = w.w4a16_gemv(x, *layer.qkv, ex.GROUP).double().cpu()
        q, k, v = (t.view(4, -1, 64) for t in qkv.split([512, 128, 128], 1))
        pos, f = torch.tensor([[c + s for c in contexts]], dtype=torch.int32), layer.inv_freq.cpu()
        seen.append((ref.rope(k, pos, f, [32], False), v))
        lens = [c + s + 1 for c in contexts]
        assert req.lengths.tolist() == lens
        # every step's rows stand for what the projection gave, however often a scale has grown since
        table = req.table.tolist()
        for i, rows in enumerate(seen):
            for b in range(4):
                j = contexts[b] + i
                block, place = table[b][j // 32], j % 32
                for codes, scales, want in ((req.cache.k, req.cache.k_scale, rows[0][b]), (req.cache.v, req.cache.v_scale, rows[1][b])):
                    S = scales[block, place // 16].double().cpu()[:, None]
                    got = codes[block, place].float().double().cpu() * S
                    bound = S if dtype == "int8" else 2.0 ** -4 * want.abs() + 2.0 ** -9 * S
                    assert ((got - want).abs() <= bound * (1 + 2.0 ** -16) + 2.0 ** -18 * want.abs().max()).all()
        qr = ref.rope(q, pos, f, [32], False).bfloat16()
        check_attention(w, qr[:, None], req.cache, table, lens, got=w.w4a16_scaled_attention(qr.cuda(), req.cache, req.table, req.lengths))
    assert w.w4a16_device_error(clear=True) == 0


def test_a_captured_step_repeats_the_calls(ex):
    layer, req = small(ex, torch.int8)
    layer2, req2 = small(ex, torch.int8)
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


def attention(w):
    lens = [3000, 1, 0, 777]
    q, cache, table = attention_problem(w, 41, lens, 2, 8, 2, 128, 16, 16, torch.int8, columns=4096)
    args = q.cuda(), cache, i32(table), i32(lens)
    return lambda stream: w.w4a16_scaled_attention(*args, stream=stream)


def append(w):
    cache = make_cache(w, torch.Generator().manual_seed(1), 40, 16, 8, 2, 64, torch.float8_e4m3fn)
    x = torch.randn(500, 8, 64, device="cuda").bfloat16()
    args = x[:, :4], x[:, 4:6], x[:, 6:], torch.arange(500).int().cuda(), freqs(64).cuda(), i32(list(range(500))), cache

    def call(stream):
        q = w.w4a16_scaled_append(*args, stream=stream)
        (stream or torch.cuda.current_stream()).synchronize() if not isinstance(stream, Raw) else torch.cuda.synchronize()
        return q, raw(cache.k)[:31], raw(cache.v)[:31], cache.k_scale[:31], cache.v_scale[:31]
    return call


def read(w):
    cache, table, start = read_problem(w, 3, [60, 40, 100], 2, 64, 16, 8, torch.int8)
    args = cache, i32(table), i32(start)
    return lambda stream: w.w4a16_scaled_read(*args, rows=start[-1] + 3, stream=stream)


@pytest.mark.parametrize("handle", [False, True], ids=["Stream", "handle"])
@pytest.mark.parametrize("call", [attention, append, read], ids=lambda f: f.__name__)
def test_calls_on_a_stream_that_is_not_the_current_one(w, call, handle):
    call = call(w)
    want = [bits(t.contiguous()) for t in tensors(call(None))]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            torch.cuda._sleep(BUSY)  # the call's kernels come later than what follows here
        got = tensors(call(Raw(s) if handle else s))
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (512, 4096, 1 << 16, 1 << 18, 1 << 20, 3 << 20, 10 << 20, 40 << 20)
                for _ in range(4)]
        torch.cuda.current_stream().synchronize()
        s.synchronize()
        assert len(junk) == 32
        for a, b in zip(got, want):
            assert torch.equal(bits(a.contiguous()), b)
    assert w.w4a16_device_error(clear=True) == 0


def test_two_captured_graphs_and_their_workspaces(w):
    # two graphs of one workspace, replayed one after another on one stream; and two of their own, on two
    lens = [2000, 0, 300]
    problems = [attention_problem(w, seed, lens, 2, 8, 2, 64, 16, 16, torch.int8, columns=4096) for seed in (1, 2)]
    args = [(q.cuda(), c, i32(t), i32(lens)) for q, c, t in problems]
    want = [[t.clone() for t in w.w4a16_scaled_attention(*a)] for a in args]
    for shared in (True, False):
        one = w.scaled_attention_workspace(problems[0][1], 8, 2)
        spaces = [one, one if shared else w.scaled_attention_workspace(problems[0][1], 8, 2)]
        graphs, outs = [], []
        for a, ws in zip(args, spaces):
            w.w4a16_scaled_attention(*a, workspace=ws)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs.append(w.w4a16_scaled_attention(*a, workspace=ws))
            graphs.append(g)
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(5):
            for g, s in zip(graphs, [streams[0]] * 2 if shared else streams):
                with torch.cuda.stream(s):
                    g.replay()
            torch.cuda.synchronize()
            for got, x in zip(outs, want):
                assert all(torch.equal(a, b) for a, b in zip(got, x))
