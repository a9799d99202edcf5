"""The paged-cache entry points check their arguments before anything is
launched (no GPU needed), and the plain forms the GPU tests compare with agree
with hand-worked cases."""
import ctypes

import numpy as np
import pytest
import torch

from . import paged_reference as ref

P = ctypes.c_void_p
A16, MIS, ODD = P(0x1000), P(0x1008), P(0x1002)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def w():
    from w4a16_int4_weight_gemv_gb300 import build_ext
    build_ext.build()
    from w4a16_int4_weight_gemv_gb300 import binding
    return binding


def cache(w, **kw):
    d = dict(k=0x1000, v=0x1000, k_scale=None, v_scale=None, dtype=0, heads=8, dim=128, page=16, blocks=64, k_block=16 * 1024,
             k_token=1024, k_head=128, v_block=16 * 1024, v_token=1024, v_head=128)
    d.update(kw)
    return ctypes.byref(w._KvCache(**d))


def test_map_checks(w):
    S = w.Status
    def call(ctx=A16, new=P(0x2000), B=4, table=A16, stride=8, columns=8, free=A16, n_free=9, head=A16, page=16, blocks=64,
             slots=A16, pos=A16, tokens=5, start=A16, kv=P(0x3000), head_out=P(0x4000)):
        return w.load_library().w4a16_paged_map(ctx, new, B, table, stride, columns, free, n_free, head, page, blocks, slots, pos,
                                                tokens, start, kv, head_out, None)
    for bad in (dict(ctx=None), dict(new=None), dict(table=None), dict(head=None), dict(start=None), dict(kv=None), dict(head_out=None),
                dict(free=None), dict(slots=None), dict(pos=None)):
        assert call(**bad) == S.ERR_NULL, bad
    for bad in (dict(B=0), dict(columns=0), dict(stride=7), dict(n_free=-1), dict(page=0), dict(blocks=0), dict(tokens=-1)):
        assert call(**bad) == S.ERR_SHAPE, bad
    for bad in (dict(B=16385), dict(page=65537), dict(blocks=1 << 27), dict(tokens=1 << 31), dict(n_free=1 << 31), dict(kv=A16),
                dict(kv=P(0x2000)), dict(head_out=A16)):
        assert call(**bad) == S.ERR_UNSUPPORTED, bad
    for bad in (dict(ctx=ODD), dict(slots=ODD), dict(table=ODD), dict(head_out=ODD)):
        assert call(**bad) == S.ERR_ALIGN, bad
    if not torch.cuda.is_available():
        assert call() == S.ERR_CUDA
        assert call(free=None, n_free=0, slots=None, pos=None, tokens=0) == S.ERR_CUDA  # allowed: the device is the next check


def test_rope_append_checks(w):
    S = w.Status
    def call(q=A16, qt=4096, qh=128, qo=A16, qot=4096, qoh=128, hq=32, k=A16, kt=1024, kh=128, v=A16, vt=1024, vh=128, pos=A16, ax=0,
             f=A16, sec=None, axes=1, rotary=128, dim=128, flags=0, slots=A16, c=None, T=2):
        c = cache(w) if c is None else c
        return w.load_library().w4a16_rope_append(q, qt, qh, qo, qot, qoh, hq, k, kt, kh, v, vt, vh, pos, ax, f, sec, axes, rotary, dim,
                                                  flags, slots, c if c != "none" else None, T, None)
    sections = lambda *v: (ctypes.c_int32 * len(v))(*v)
    for bad in (dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(slots=None), dict(c="none"), dict(pos=None), dict(f=None),
                dict(q=None, qo=None, k=None, v=None, slots=None, c="none"), dict(axes=2), dict(c=cache(w, k=None)),
                dict(c=cache(w, dtype=1))):
        assert call(**bad) == S.ERR_NULL, bad
    for bad in (dict(T=-1), dict(axes=0, sec=sections(1)), dict(rotary=24), dict(rotary=-16), dict(rotary=144), dict(dim=120, rotary=64), dict(hq=0),
                dict(sec=sections(63)), dict(sec=sections(65)), dict(axes=2, sec=sections(-1, 65)), dict(axes=2, sec=sections(32, 31)),
                dict(c=cache(w, dim=64)), dict(c=cache(w, heads=0)), dict(c=cache(w, page=0)), dict(c=cache(w, dim=72))):
        assert call(**bad) == S.ERR_SHAPE, bad
    for bad in (dict(flags=4), dict(axes=5, sec=sections(64, 0, 0, 0, 0)), dict(dim=272, rotary=64), dict(c=cache(w, dtype=2)),
                dict(c=cache(w, blocks=1 << 27)), dict(c=cache(w, dim=512))):
        assert call(**bad) == S.ERR_UNSUPPORTED, bad
    for bad in (dict(q=MIS), dict(qo=MIS), dict(k=MIS), dict(v=MIS), dict(qt=4100), dict(qoh=4), dict(vh=-128), dict(pos=ODD), dict(slots=ODD),
                dict(c=cache(w, k=0x1008)), dict(c=cache(w, v_head=132)), dict(c=cache(w, dtype=1, k_scale=0x1000, v_scale=0x1000, k_token=1032))):
        assert call(**bad) == S.ERR_ALIGN, bad
    assert call(T=0) == S.OK
    if not torch.cuda.is_available():
        assert call() == S.ERR_CUDA
        assert call(rotary=0, pos=None, f=None) == S.ERR_CUDA


def test_attention_checks(w):
    S, lib = w.Status, w.load_library()
    need = lib.w4a16_paged_attention_workspace_bytes(32, 8, 128)
    assert need > 0
    for bad in ((0, 8, 128), (32, 0, 128), (30, 8, 128), (32, 8, 0), (32, 8, 72), (32, 8, 272)):
        assert lib.w4a16_paged_attention_workspace_bytes(*bad) == 0
    def call(q=A16, qr=4096, qh=128, c=None, table=A16, stride=8, columns=8, kv=A16, B=2, hq=32, scale=0.1, window=0, out=A16, outr=4096, outh=128,
             lse=None, ws=A16, n=need):
        return lib.w4a16_paged_attention(q, qr, qh, cache(w) if c is None else c if c != "none" else None, table, stride, columns, kv, B, hq, scale,
                                         window, out, outr, outh, lse, ws, n, None)
    for bad in (dict(q=None), dict(c="none"), dict(table=None), dict(kv=None), dict(out=None), dict(c=cache(w, v=None))):
        assert call(**bad) == S.ERR_NULL, bad
    for bad in (dict(B=0), dict(hq=0), dict(hq=30), dict(columns=0), dict(stride=7), dict(window=-1)):
        assert call(**bad) == S.ERR_SHAPE, bad
    assert call(B=1 << 19) == S.ERR_UNSUPPORTED
    for bad in (dict(q=MIS), dict(out=MIS), dict(qr=100), dict(outh=4), dict(table=ODD), dict(kv=ODD), dict(lse=ODD), dict(ws=MIS)):
        assert call(**bad) == S.ERR_ALIGN, bad
    for bad in (dict(ws=None), dict(n=need - 1)):
        assert call(**bad) == S.ERR_WORKSPACE, bad
    if not torch.cuda.is_available():
        assert call() == S.ERR_CUDA


def test_attention_refuses_tables_whose_tiles_pass_32_bits(w):
    # the launch counts a request's tiles, and two more a row, in 32 bits
    S, lib = w.Status, w.load_library()
    def call(columns, page, kv, hq, window=0, B=1):
        need = lib.w4a16_paged_attention_workspace_bytes(hq, kv, 64)
        c = cache(w, heads=kv, dim=64, page=page, blocks=1000, k_head=64, v_head=64)
        return lib.w4a16_paged_attention(A16, 64 * hq, 64, c, A16, columns, columns, A16, B, hq, 0.1, window, A16, 64 * hq, 64, None, A16, need, None)
    allowed = S.ERR_CUDA if not torch.cuda.is_available() else None  # with a GPU: not launched on these addresses
    #  tiles of a row, rows: 2^31 - 1024 tokens are 2^27 - 64 tiles
    for args, fits in (((1 << 27, 16, 16, 16), True), ((1 << 27, 16, 17, 17), False), ((1 << 15, 1 << 16, 17, 17), False),
                       ((1 << 27, 16, 2, 128), True), ((1 << 27, 16, 2, 2 * 129), False), ((1 << 27, 16, 8, 64), True), ((1 << 27, 16, 8, 72), True),
                       ((1 << 27, 16, 8, 8 * 17), True), ((1 << 27, 16, 8, 8 * 33), False), ((1 << 27, 16, 17, 17, 1 << 30), True),
                       ((1 << 27, 16, 64, 64, 1 << 30), False), ((1 << 26, 16, 31, 31), True), ((1 << 26, 16, 32, 32), False),
                       ((1 << 26, 16, 32, 32, 0, 1000), False)):
        if not fits:
            assert call(*args) == S.ERR_UNSUPPORTED, args
        elif allowed is not None:
            assert call(*args) == allowed, args


def test_binding_refuses_cpu_tensors(w):
    z = torch.zeros
    with pytest.raises(ValueError):
        w.PagedCache(z(2, 16, 1, 64).bfloat16(), z(2, 16, 1, 64).bfloat16())
    with pytest.raises(ValueError):
        w.w4a16_paged_map(z(2).int(), z(2).int(), z(2, 4).int(), z(8).int(), z(1).int(), 16, 8, 2)
    with pytest.raises(ValueError):
        w.w4a16_rope_append(z(2, 4, 64).bfloat16(), None, None, z(2).int(), z(32), None, None)


def test_reference_map_by_hand():
    # request 0 holds 5 of 4-token blocks [9, 7], adds 4: one new block; request 1 begins with 3 tokens
    got = ref.paged_map([5, 0], [4, 3], [[9, 7, -1], [-1, -1, -1]], [50, 2, 4, 6], 1, 4, 10, 8)
    assert got[0] == [[9, 7, 2], [4, -1, -1]]
    assert got[1] == [7 * 4 + 1, 7 * 4 + 2, 7 * 4 + 3, 2 * 4, 16, 17, 18, -1]
    assert got[2] == [5, 6, 7, 8, 0, 1, 2, -1]
    assert got[3:] == ([0, 4, 7], [9, 3], 3, set())


def test_reference_rope_by_hand():
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0, 5.0]]], dtype=torch.float64)
    quarter = torch.tensor([3.14159265358979 / 2, 0.0]).float()
    y = ref.rope(x, torch.tensor([[1]]), quarter, [2], False)
    assert torch.allclose(y, torch.tensor([[[-3.0, 2.0, 1.0, 4.0, 5.0]]], dtype=torch.float64), atol=1e-6)
    y = ref.rope(x, torch.tensor([[1]]), quarter, [2], True)
    assert torch.allclose(y, torch.tensor([[[-2.0, 1.0, 3.0, 4.0, 5.0]]], dtype=torch.float64), atol=1e-6)
    z = ref.rope(y, torch.tensor([[1]]), quarter, [2], True, inverse=True)
    assert torch.allclose(z, x, atol=1e-12)


def test_reference_attention_against_softmax():
    gen = torch.Generator().manual_seed(0)
    k, v = (torch.randn(4, 2, 1, 16, generator=gen, dtype=torch.float64) for _ in range(2))
    q = torch.randn(1, 2, 16, generator=gen, dtype=torch.float64)
    out, lse, spread, reach = ref.attention(q, k, v, [[3, 0, 1]], [5], 0.25, 3)
    rows = [(0, 0), (0, 1), (1, 0)]  # the last three of five tokens
    kk, vv = torch.stack([k[i, p, 0] for i, p in rows]), torch.stack([v[i, p, 0] for i, p in rows])
    s = 0.25 * q[0] @ kk.t()
    assert torch.allclose(out[0], torch.softmax(s, 1) @ vv)
    assert torch.allclose(lse[0], torch.logsumexp(s, 1))


def test_marshalling_module_is_of_these_sources_and_this_machine(w, monkeypatch, tmp_path):
    # a file made for another Python, machine, torch or interface has another name: it is neither taken for
    # fresh nor loaded, whatever its time stamp, also where no new one can be built
    import shutil
    import sysconfig

    from w4a16_int4_weight_gemv_gb300 import build_ext
    here = build_ext.fastcall_path()
    assert torch.__version__ in here and here.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    include = tmp_path / "include"
    shutil.copytree(build_ext.INCLUDE, include)
    build = tmp_path / "_build"
    build.mkdir()
    monkeypatch.setattr(build_ext, "INCLUDE", str(include))
    monkeypatch.setattr(build_ext, "BUILD_DIR", str(build))
    monkeypatch.setenv("CXX", "/bin/false")
    same = build_ext.fastcall_path()
    assert same.rsplit("/", 1)[1] == here.rsplit("/", 1)[1]
    open(same, "w").close()
    assert build_ext.build_fastcall() == same  # of these sources: as it is
    with open(include / "w4a16.h", "a") as f:
        f.write("/* changed */\n")
    changed = build_ext.fastcall_path()
    assert changed != same
    assert build_ext.build_fastcall() is None and w._load_fast() is None
    monkeypatch.setattr(build_ext.sysconfig, "get_config_var", lambda name: ".cpython-399-other-linux-gnu.so")
    assert build_ext.fastcall_path() not in (same, changed)


@pytest.mark.parametrize("fast", [True, False], ids=["marshalling module", "binding"])
@pytest.mark.filterwarnings("ignore:Accessing the data pointer")
def test_tensors_of_two_devices_are_refused(w, monkeypatch, fast):
    # tensors without memory stand in for those of two GPUs
    from torch._subclasses.fake_tensor import FakeTensorMode
    if not fast:
        monkeypatch.setattr(w, "_fast", None)
    with FakeTensorMode(allow_non_fake_inputs=True):
        def make(dtype, *shape, gpu=0):
            return torch.empty(shape, dtype=dtype, device="cuda:%d" % gpu)

        def other(t):
            return make(t.dtype, *t.shape, gpu=1)

        i32, f32, bf16, e4m3 = torch.int32, torch.float32, torch.bfloat16, torch.float8_e4m3fn

        def refused(call, args, names):
            for name in names:
                with pytest.raises(ValueError, match="device"):
                    call(**{**args, name: other(args[name])})

        kv = dict(k=make(e4m3, 8, 16, 2, 64), v=make(e4m3, 8, 16, 2, 64), k_scale=make(f32, 2), v_scale=make(f32, 2))
        refused(w.PagedCache, kv, ["v", "k_scale", "v_scale"])
        cache = w.PagedCache(make(bf16, 8, 16, 2, 64), make(bf16, 8, 16, 2, 64))

        out = w.PagedMap(make(i32, 5), make(i32, 5), make(i32, 4), make(i32, 3), make(i32, 1))
        args = dict(ctx_len=make(i32, 3), new_len=make(i32, 3), block_table=make(i32, 3, 4), free_blocks=make(i32, 6), free_head=make(i32, 1), page=16,
                    num_blocks=8, tokens=5, out=out)
        refused(w.w4a16_paged_map, args, ["new_len", "block_table", "free_blocks", "free_head"])
        for name in out._fields:
            with pytest.raises(ValueError, match="device"):
                w.w4a16_paged_map(**{**args, "out": out._replace(**{name: other(getattr(out, name))})})

        args = dict(q=make(bf16, 5, 4, 64), k=make(bf16, 5, 2, 64), v=make(bf16, 5, 2, 64), positions=make(i32, 5), inv_freq=make(f32, 32),
                    slots=make(i32, 5), cache=cache, q_out=make(bf16, 5, 4, 64))
        refused(w.w4a16_rope_append, args, ["q", "k", "v", "positions", "inv_freq", "slots", "q_out"])
        refused(w.w4a16_rope_append, {**args, "q": None, "q_out": None, "positions": make(i32, 1, 5), "sections": [32]},
                ["k", "v", "positions", "inv_freq", "slots"])
        refused(w.w4a16_rope_append, {**args, "k": None, "v": None, "slots": None, "cache": None}, ["positions", "inv_freq", "q_out"])

        args = dict(q=make(bf16, 3, 4, 64), cache=cache, block_table=make(i32, 3, 4), kv_len=make(i32, 3), out=make(bf16, 3, 4, 64),
                    lse=make(f32, 3, 4), workspace=make(torch.uint8, 1 << 22))
        refused(w.w4a16_paged_attention, args, ["q", "block_table", "kv_len", "out", "lse", "workspace"])


def test_sections_go_by_their_values(w):
    # one list of whole numbers that change in place, as numpy and torch have them
    for make in (lambda v: torch.tensor(v), lambda v: np.array(v)):
        lengths = [make(20), make(12)]
        assert list(w._section_array(lengths)) == [20, 12]
        for x in lengths:
            x[()] = 16
        assert list(w._section_array(lengths)) == [16, 16]
    with pytest.raises(TypeError):
        w._section_array([16.0, 16.0])
