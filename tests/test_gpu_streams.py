"""Calls on a stream that is not the current one, which make their outputs and
workspaces themselves: that memory must not be given to anybody else while the
call's kernels run on that stream, nor, what the caller gets, while the current
stream still reads it."""
import pytest
import torch

from w4a16_int4_weight_gemv_gb300 import synth

from .test_gpu_moe_hmma import bank
from .test_gpu_paged import attention_problem, freqs, i32, w  # noqa: F401  (w: the fixture)
from .test_gpu_parity import dev

pytestmark = pytest.mark.gpu
BUSY = 4_000_000  # clock cycles that a stream is kept busy: about 2 ms


def attention(w):
    lens = [3000, 1, 0, 777]
    q, cache, table = attention_problem(w, 41, lens, 8, 2, 128, 16, "bf16", "token", columns=4096)
    args = q.cuda(), cache, i32(table), i32(lens)
    return lambda stream: w.w4a16_paged_attention(*args, stream=stream)


def rope(w):
    x = torch.randn(500, 4, 64, device="cuda").bfloat16()
    args = x, None, None, torch.arange(500).int().cuda(), freqs(64).cuda(), None, None
    return lambda stream: w.w4a16_rope_append(*args, stream=stream)


def block_map(w):
    args = i32([5, 0]), i32([300, 40]), i32([[29] + [-1] * 30] + [[-1] * 31]), i32(list(range(29))), i32([0]), 16, 32, 400
    return lambda stream: w.w4a16_paged_map(*args, stream=stream)  # the table's new entries are the same every time


def gemv(w, swiglu=False):
    p = synth.dense_problem(2, 512, 1024, 128, "const8", seed=1)
    args = [dev(p[k]) for k in ("x", "wq", "scale", "zero")]
    return lambda stream: w.w4a16_gemv(*args, 128, swiglu_output=swiglu, stream=stream)


def swiglu(w):
    g, u = (torch.randn(8, 512, device="cuda").bfloat16() for _ in range(2))
    return lambda stream: w.w4a16_swiglu(g, u, stream=stream)


def pack_and_dequant(w):
    p = synth.dense_problem(1, 256, 1024, 128, "const8", seed=2)
    codes = torch.randint(0, 16, (256, 1024), dtype=torch.uint8, device="cuda")
    wq, scale, zero = (dev(p[k]) for k in ("wq", "scale", "zero"))
    return lambda stream: (w.int4_pack(codes, stream=stream), w.int4_dequant(wq, scale, zero, 128, stream=stream))


def pack_and_dequant3(w):
    b = synth.expert_bank3(3, 1, 256, 1024)
    codes = torch.randint(0, 8, (256, 1024), dtype=torch.uint8, device="cuda")
    wq, scale, zero = (dev(a)[0] for a in b)
    return lambda stream: (w.int3_pack(codes, stream=stream), w.int3_dequant(wq, scale, zero, 128, stream=stream))


def experts(w, how):
    p = (synth.moe_problem3 if how.startswith("int3") else synth.moe_problem)(M=4, E=8, H=1024, F=512, topk=2, g=128, seed=5)
    x, ids, rw = dev(p["x"]), dev(p["ids"]), dev(p["route_w"])
    gate, up, down = bank(p["gate"]), bank(p["up"]), bank(p["down"])
    per_slot = torch.randn(4, 2, 512, device="cuda").bfloat16()
    return {
        "ffn": lambda stream: w.moe_ffn(x, ids, rw, gate, up, down, 128, stream=stream),
        "ffn from single calls": lambda stream: w.moe_ffn(x, ids, rw, gate, up, down, 128, stream=stream, fused=False),
        "slots": lambda stream: w.w4a16_moe_gemv(x, ids, *gate, 128, stream=stream),
        "routed sum": lambda stream: w.w4a16_moe_gemv(per_slot, ids, *down, 128, route_w=rw, x_per_slot=True, stream=stream),
        "routed sum, kernel 2": lambda stream: w.w4a16_moe_gemv(per_slot, ids, *down, 128, route_w=rw, x_per_slot=True, stream=stream, kernel_id=2),
        "int3 ffn": lambda stream: w.w3a16_moe_ffn(x, ids, rw, gate, up, down, 128, stream=stream),
        "int3 slots": lambda stream: w.w3a16_moe_gemv(x, ids, *gate, 128, stream=stream),
    }[how]


CALLS = {"attention": attention, "rope": rope, "map": block_map, "gemv": gemv, "gemv with swiglu": lambda w: gemv(w, True), "swiglu": swiglu,
         "pack, dequant": pack_and_dequant, "int3 pack, dequant": pack_and_dequant3}
for name in ("ffn", "ffn from single calls", "slots", "routed sum", "routed sum, kernel 2", "int3 ffn", "int3 slots"):
    CALLS[name] = lambda w, name=name: experts(w, name)


def tensors(x):
    return list(x) if isinstance(x, tuple) else [x]


def bits(t):
    return t.clone().view(torch.uint8)


class Raw:
    """A stream by its handle alone, as another library would name it."""

    def __init__(self, s):
        self.cuda_stream = s.cuda_stream


@pytest.mark.parametrize("raw", [False, True], ids=["Stream", "handle"])
@pytest.mark.parametrize("name", list(CALLS))
def test_own_buffers_are_not_given_away_before_the_call_is_done(w, name, raw):
    call = CALLS[name](w)
    want = [bits(t) for t in tensors(call(None))]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            torch.cuda._sleep(BUSY)  # the call's kernels come later than what follows here
        got = tensors(call(Raw(s) if raw else s))
        # the current stream takes memory of every size the call may have let go of, and writes it
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (512, 4096, 1 << 16, 1 << 18, 1 << 20, 3 << 20, 10 << 20, 40 << 20)
                for _ in range(4)]
        torch.cuda.current_stream().synchronize()
        s.synchronize()
        assert len(junk) == 32
        for a, b in zip(got, want):
            assert torch.equal(bits(a), b)
    assert w.w4a16_device_error(clear=True) == 0


@pytest.mark.parametrize("name", list(CALLS))
def test_results_are_not_given_away_while_they_are_read(w, name):
    call = CALLS[name](w)
    want = [bits(t) for t in tensors(call(None))]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = tensors(call(s))
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(BUSY)
        read = [bits(t) for t in got]  # after the wait, on the current stream
        sizes = [t.nbytes for t in got]
        del got
        with torch.cuda.stream(s):  # nothing says that this comes after the reading
            junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
        torch.cuda.synchronize()
        assert len(junk) == 4 * len(sizes)
        for a, b in zip(read, want):
            assert torch.equal(a, b)
    assert w.w4a16_device_error(clear=True) == 0


def test_the_current_stream_by_name_changes_nothing(w):
    call = CALLS["rope"](w)
    assert torch.equal(call(None), call(torch.cuda.current_stream()))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        a, b = call(None), call(s)
    s.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["attention", "rope", "ffn"])
def test_a_forked_stream_in_a_capture(w, name):
    call = CALLS[name](w)
    want = [bits(t) for t in tensors(call(None))]
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        got = tensors(call(s))
        torch.cuda.current_stream().wait_stream(s)
        read = [t.clone() for t in got]
    for _ in range(3):
        for t in got + read:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(read, want):
            assert torch.equal(bits(a), b)
    assert w.w4a16_device_error(clear=True) == 0
