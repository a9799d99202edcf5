"""The entry points over an 8-bit cache with scales by group check their arguments
before anything is launched (no GPU needed), and the plain forms that the GPU tests
compare with agree with hand-worked cases."""
import ctypes

import pytest
import torch

from . import scaled_reference as ref

P = ctypes.c_void_p
A16, MIS, ODD = P(0x1000), P(0x1008), P(0x1002)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def w():
    from w4a16_int4_weight_gemv_gb300 import build_ext
    build_ext.build()
    from w4a16_int4_weight_gemv_gb300 import binding
    return binding


def cache(w, **kw):
    d = dict(k=0x1000, v=0x1000, k_scale=0x1000, v_scale=0x1000, dtype=2, heads=8, dim=128, page=32, group=16, blocks=64, k_block=32 * 1024, k_token=1024, k_head=128,
             v_block=32 * 1024, v_token=1024, v_head=128, ks_block=16, ks_group=1, ks_head=2, vs_block=16, vs_group=1, vs_head=2)
    d.update(kw)
    return ctypes.byref(w._ScaledCache(**d))


# what every call finds wrong with a cache
def bad_caches(w):
    S = w.Status
    for status, bads in ((S.ERR_NULL, (dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None))),
                         (S.ERR_SHAPE, (dict(heads=0), dict(page=0), dict(blocks=0), dict(dim=72), dict(dim=0), dict(group=0), dict(group=24), dict(page=8, group=16))),
                         (S.ERR_UNSUPPORTED, (dict(dtype=0), dict(dtype=3), dict(dim=272), dict(page=65537), dict(blocks=1 << 26), dict(heads=65537),
                                              dict(page=256, group=256))),
                         (S.ERR_ALIGN, (dict(k=0x1008), dict(v=0x1008), dict(k_scale=0x1002), dict(k_token=1032), dict(v_head=-128), dict(v_block=8), dict(ks_block=-1),
                                        dict(vs_head=-2)))):
        for bad in bads:
            yield status, cache(w, **bad)


def test_append_checks(w):
    S = w.Status
    def call(q=A16, qt=4096, qh=128, qo=A16, qot=4096, qoh=128, hq=32, k=A16, kt=1024, kh=128, v=A16, vt=1024, vh=128, pos=A16, ax=0, f=A16, sec=None, axes=1,
             rotary=128, dim=128, flags=0, slots=A16, c=None, T=2):
        c = cache(w) if c is None else c
        return w.load_library().w4a16_scaled_append(q, qt, qh, qo, qot, qoh, hq, k, kt, kh, v, vt, vh, pos, ax, f, sec, axes, rotary, dim, flags, slots,
                                                    c if c != "none" else None, T, None)
    sections = lambda *v: (ctypes.c_int32 * len(v))(*v)
    for status, c in bad_caches(w):
        assert call(c=c) == status
    for bad in (dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(slots=None), dict(c="none"), dict(pos=None), dict(f=None), dict(axes=2)):
        assert call(**bad) == S.ERR_NULL, bad
    for bad in (dict(T=-1), dict(axes=0, sec=sections(1)), dict(rotary=24), dict(rotary=-16), dict(rotary=144), dict(dim=120, rotary=64), dict(hq=0), dict(ax=-1),
                dict(sec=sections(63)), dict(axes=2, sec=sections(-1, 65)), dict(axes=2, sec=sections(32, 31)), dict(c=cache(w, dim=64))):
        assert call(**bad) == S.ERR_SHAPE, bad
    for bad in (dict(flags=4), dict(flags=w.ROPE_INVERSE), dict(axes=5, sec=sections(64, 0, 0, 0, 0)), dict(dim=272, rotary=64), dict(T=1 << 31), dict(hq=65537),
                # places that are one cannot be written
                dict(c=cache(w, ks_block=0)), dict(c=cache(w, vs_group=0)), dict(c=cache(w, ks_head=0)), dict(c=cache(w, k_token=0)), dict(c=cache(w, v_head=0)),
                dict(c=cache(w, v_block=0))):
        assert call(**bad) == S.ERR_UNSUPPORTED, bad
    for bad in (dict(q=MIS), dict(qo=MIS), dict(k=MIS), dict(v=MIS), dict(qt=4100), dict(qoh=4), dict(vh=-128), dict(pos=ODD), dict(slots=ODD), dict(f=ODD)):
        assert call(**bad) == S.ERR_ALIGN, bad
    assert call(T=0) == S.OK
    if not torch.cuda.is_available():
        assert call() == S.ERR_CUDA
        assert call(rotary=0, pos=None, f=None) == S.ERR_CUDA
        assert call(q=None, qo=None) == S.ERR_CUDA
        assert call(c=cache(w, blocks=1, k_block=0, v_block=0, ks_block=0, vs_block=0)) == S.ERR_CUDA  # one of them: no stride


def test_read_checks(w):
    S = w.Status
    def call(c=None, table=A16, stride=8, columns=8, start=A16, first=None, B=2, k=A16, kr=1024, kh=128, v=A16, vr=1024, vh=128, dtype=0, rows=9):
        return w.load_library().w4a16_scaled_read(cache(w) if c is None else c if c != "none" else None, table, stride, columns, start, first, B, k, kr, kh, v, vr, vh,
                                                  dtype, rows, None)
    for status, c in bad_caches(w):
        assert call(c=c) == status
    for bad in (dict(c="none"), dict(table=None), dict(start=None), dict(k=None), dict(v=None)):
        assert call(**bad) == S.ERR_NULL, bad
    for bad in (dict(B=0), dict(columns=0), dict(stride=7), dict(rows=-1)):
        assert call(**bad) == S.ERR_SHAPE, bad
    for bad in (dict(B=16385), dict(rows=1 << 31), dict(dtype=2)):
        assert call(**bad) == S.ERR_UNSUPPORTED, bad
    for bad in (dict(k=MIS), dict(v=MIS), dict(kr=1028), dict(vh=4), dict(kh=-128), dict(dtype=1, vr=1026), dict(table=ODD), dict(start=ODD), dict(first=ODD)):
        assert call(**bad) == S.ERR_ALIGN, bad
    assert call(rows=0, k=None, v=None) == S.OK
    if not torch.cuda.is_available():
        assert call() == S.ERR_CUDA and call(dtype=1, kr=1028, first=A16) == S.ERR_CUDA


def test_attention_checks(w):
    S, lib = w.Status, w.load_library()
    size = lib.w4a16_scaled_attention_workspace_bytes
    need = size(32, 8, 128, 3)
    assert need > 0 and size(32, 8, 128, 1) == lib.w4a16_paged_attention_workspace_bytes(32, 8, 128)
    for bad in ((0, 8, 128, 1), (32, 0, 128, 1), (30, 8, 128, 1), (32, 8, 0, 1), (32, 8, 72, 1), (32, 8, 272, 1), (32, 8, 128, 0), (32, 8, 128, 17), (1 << 30, 1, 128, 16)):
        assert size(*bad) == 0
    def call(q=A16, qr=12288, qt=4096, qh=128, c=None, table=A16, stride=8, columns=8, kv=A16, B=2, new=3, hq=32, scale=0.1, window=0, out=A16, outr=12288, outt=4096,
             outh=128, lse=None, ws=A16, n=need):
        return lib.w4a16_scaled_attention(q, qr, qt, qh, cache(w) if c is None else c if c != "none" else None, table, stride, columns, kv, B, new, hq, scale, window,
                                          out, outr, outt, outh, lse, ws, n, None)
    for status, c in bad_caches(w):
        assert call(c=c) == status
    for bad in (dict(q=None), dict(c="none"), dict(table=None), dict(kv=None), dict(out=None)):
        assert call(**bad) == S.ERR_NULL, bad
    for bad in (dict(B=0), dict(hq=0), dict(hq=30), dict(columns=0), dict(stride=7), dict(window=-1), dict(new=0)):
        assert call(**bad) == S.ERR_SHAPE, bad
    for bad in (dict(new=17), dict(B=1 << 19), dict(B=1 << 18), dict(hq=1 << 30)):
        assert call(**bad) == S.ERR_UNSUPPORTED, bad
    for bad in (dict(q=MIS), dict(out=MIS), dict(qr=100), dict(qt=4), dict(outt=-8), dict(outh=4), dict(table=ODD), dict(kv=ODD), dict(lse=ODD), dict(ws=MIS)):
        assert call(**bad) == S.ERR_ALIGN, bad
    for bad in (dict(ws=None), dict(n=need - 1)):
        assert call(**bad) == S.ERR_WORKSPACE, bad
    if not torch.cuda.is_available():
        assert call() == S.ERR_CUDA and call(window=2 ** 31 - 1) == S.ERR_CUDA


@pytest.mark.parametrize("dim", [16, 64, 128, 144, 256])
@pytest.mark.parametrize("hq", [1, 3, 4, 5, 7, 9, 16, 40])
def test_workspace_serves_fewer_new_tokens(w, hq, dim):
    size = [w.load_library().w4a16_scaled_attention_workspace_bytes(hq, 1, dim, n) for n in range(1, 17)]
    assert size == sorted(size)


def test_attention_refuses_tables_whose_tiles_pass_32_bits(w):
    S, lib = w.Status, w.load_library()
    def call(columns, page, kv, hq, new, window=0):
        need = lib.w4a16_scaled_attention_workspace_bytes(hq, kv, 64, new)
        c = cache(w, heads=kv, dim=64, page=page, group=1, blocks=1000, k_head=64, v_head=64)
        return lib.w4a16_scaled_attention(A16, 64 * hq * new, 64 * hq, 64, c, A16, columns, columns, A16, 1, new, hq, 0.1, window, A16, 64 * hq * new, 64 * hq, 64, None,
                                          A16, need, None)
    #  a window of w tokens and N - 1 more lies in ceil((w + N - 1) / 16) + 1 tiles; 16 heads of 32 columns are 32 rows
    for args, fits in (((1 << 27, 16, 16, 16, 1), True), ((1 << 27, 16, 16, 16, 8), True), ((1 << 27, 16, 8, 8, 16), True), ((1 << 27, 16, 16, 32, 16), False),
                       ((1 << 27, 16, 17, 17, 1), False), ((1 << 27, 16, 16, 32, 16, (1 << 30) - 4096), True),
                       ((1 << 27, 16, 16, 32, 16, 1 << 30), False), ((1 << 27, 16, 16, 64, 16, 1 << 30), False)):
        if not fits:
            assert call(*args) == S.ERR_UNSUPPORTED, args
        elif not torch.cuda.is_available():  # with a GPU: not launched on these addresses
            assert call(*args) == S.ERR_CUDA, args


def test_the_other_cache_refuses_this_type(w):
    # int8 codes need scales by group
    c = w._KvCache(k=0x1000, v=0x1000, k_scale=0x1000, v_scale=0x1000, dtype=w.CACHE_INT8, heads=8, dim=128, page=16, blocks=64, k_block=16 * 1024, k_token=1024,
                   k_head=128, v_block=16 * 1024, v_token=1024, v_head=128)
    assert w.load_library().w4a16_paged_attention(A16, 4096, 128, ctypes.byref(c), A16, 8, 8, A16, 2, 32, 0.1, 0, A16, 4096, 128, None, A16, 1 << 26,
                                                  None) == w.Status.ERR_UNSUPPORTED


def test_binding_refuses_cpu_tensors(w):
    z = torch.zeros
    with pytest.raises(ValueError):
        w.ScaledCache(z(2, 16, 1, 64).to(torch.int8), z(2, 16, 1, 64).to(torch.int8), z(2, 2, 1), z(2, 2, 1))
    for call in (lambda c: w.w4a16_scaled_append(None, z(1), z(1), z(1), z(1), z(1), c), lambda c: w.w4a16_scaled_read(c, z(1), z(1)),
                 lambda c: w.w4a16_scaled_attention(z(1), c, z(1), z(1))):
        with pytest.raises(TypeError):
            call(None)


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

        def refused(call, args, names):
            for name in names:
                with pytest.raises(ValueError, match="device"):
                    call(**{**args, name: make(args[name].dtype, *args[name].shape, gpu=1)})

        i32, f32, bf16, i8 = torch.int32, torch.float32, torch.bfloat16, torch.int8
        kv = dict(k=make(i8, 8, 16, 2, 64), v=make(i8, 8, 16, 2, 64), k_scale=make(f32, 8, 2, 2), v_scale=make(f32, 8, 2, 2))
        refused(w.ScaledCache, kv, ["v", "k_scale", "v_scale"])
        c = w.ScaledCache(**kv)
        assert c.group == 8
        args = dict(q=make(bf16, 5, 4, 64), k=make(bf16, 5, 2, 64), v=make(bf16, 5, 2, 64), positions=make(i32, 5), inv_freq=make(f32, 32), slots=make(i32, 5), cache=c,
                    q_out=make(bf16, 5, 4, 64))
        refused(w.w4a16_scaled_append, args, ["q", "k", "v", "positions", "inv_freq", "slots", "q_out"])
        args = dict(cache=c, block_table=make(i32, 3, 4), row_start=make(i32, 4), first=make(i32, 3), k_out=make(bf16, 9, 2, 64), v_out=make(bf16, 9, 2, 64))
        refused(w.w4a16_scaled_read, args, ["block_table", "row_start", "first", "k_out", "v_out"])
        for q in (make(bf16, 3, 4, 64), make(bf16, 3, 2, 4, 64)):
            args = dict(q=q, cache=c, block_table=make(i32, 3, 4), kv_len=make(i32, 3), out=make(bf16, *q.shape), lse=make(f32, *q.shape[:-1]),
                        workspace=make(torch.uint8, 1 << 22))
            refused(w.w4a16_scaled_attention, args, ["q", "block_table", "kv_len", "out", "lse", "workspace"])


def test_reference_append_by_hand():
    # int8, group 4 of a page of 8: 126 holds at scale 1; 254 is 127 * 2, so that 126 becomes 63 of scale 2; 255 needs 4
    codes, scales = torch.full((1, 8, 1, 1), 99.0, dtype=torch.float64), torch.full((1, 2, 1), 3.0)
    def go(values, slots):
        nonlocal codes, scales
        x = torch.tensor(values).bfloat16().view(-1, 1, 1)
        codes, scales, _, bad = ref.append(codes, scales, x, x.double(), 0, False, slots, 8, 4, torch.int8)
        return bad
    assert not go([126.0], [0])
    assert codes.flatten().tolist() == [126] + [99] * 7 and scales.flatten().tolist() == [1, 3]
    assert not go([254.0, 5.0], [1, 2])
    assert codes.flatten().tolist() == [63, 127, 2] + [99] * 5 and scales.flatten().tolist() == [2, 3]  # 5 / 2: to even
    assert not go([255.0, 1.5, 0.25], [3, 4, 5])
    assert codes.flatten().tolist() == [32, 64, 1, 64, 96, 16, 99, 99] and scales.flatten().tolist() == [4, 2.0 ** -6]
    assert go([1.0, 1.0], [7, 6]) and codes.flatten()[6] == 99  # 6 does not follow 7: left out
    assert go([1.0], [8]) and not go([1.0], [-1])
    assert not go([0.0], [0]) and scales[0, 0, 0] == 2.0 ** -126 and codes.flatten().tolist()[:2] == [0, 64]  # begun anew


def test_reference_scale_takes_the_length_of_a_pair():
    assert ref.scale_for(ref.need_of(torch.tensor([[300.0, 400.0]]), 2, False), torch.float8_e4m3fn, 0.0) == 2
    assert ref.scale_for(ref.need_of(torch.tensor([[300.0, 400.0]]), 0, False), torch.float8_e4m3fn, 0.0) == 1
    assert ref.scale_for(ref.need_of(torch.tensor([[1.0, 0.0]]), 2, True), torch.int8, 0.3) == 0.5
    assert ref.scale_for(None, torch.int8, 0.0) != ref.scale_for(None, torch.int8, 0.0)  # NaN


def test_reference_codes():
    x = torch.tensor([0.0, 2.0 ** -10, 3 * 2.0 ** -10, 1.0625, 1.1875, 447.0, 463.0, -17.0])
    assert torch.equal(ref.nearest(x, torch.float8_e4m3fn), x.to(torch.float8_e4m3fn).float())
    y = torch.randn(4096) * torch.exp2(torch.randint(-12, 6, (4096,)).float())
    assert torch.equal(ref.nearest(y, torch.float8_e4m3fn), y.to(torch.float8_e4m3fn).float())


def test_reference_attention_against_softmax():
    gen = torch.Generator().manual_seed(0)
    ck, cv = (torch.randint(-127, 128, (4, 2, 1, 16), generator=gen).double() for _ in range(2))
    ks, vs = (torch.rand(4, 2, 1, generator=gen).double() * 0.02 for _ in range(2))
    q = torch.randn(1, 2, 2, 16, generator=gen, dtype=torch.float64)
    out, lse, *_ = ref.attention(q, ck, cv, ks, vs, [[3, 0, 1]], [5], 0.25, 3, 1)
    for i, rows in enumerate(([(3, 1), (0, 0), (0, 1)], [(0, 0), (0, 1), (1, 0)])):  # of the first four and of all five tokens the last three
        kk, vv = (torch.stack([c[b, p, 0] * s[b, p, 0] for b, p in rows]) for c, s in ((ck, ks), (cv, vs)))
        s = 0.25 * q[0, i] @ kk.t()
        assert torch.allclose(out[0, i], torch.softmax(s, 1) @ vv) and torch.allclose(lse[0, i], torch.logsumexp(s, 1))
