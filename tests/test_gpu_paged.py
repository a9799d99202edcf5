"""The paged-cache operators on the GPU against their plain 64-bit forms.

Tolerances (u = 2^-8: bf16 keeps 8 significant bits, so rounding to nearest
moves a value by at most 2^-8 of it):
  attention, out: |err| <= u |y| + u sum p|v| + (score error) sum p|v| -- one
      rounding of the result, one of each probability, and the fp32 scores'
      error, at most (dim + 16) 2^-24 of scale sum |q||k| (twice: once in the
      maximum's row, once in the token's), as a relative error of p;
  attention, lse: that score error, and a few fp32 roundings of the sum;
  rotation: u |y| + 2^-20 (|x1| + |x2|): the result's rounding, and cosine
      and sine to about 2^-21 each with the fp32 products;
  e4m3 codes: half a unit in the last place, 2^-4 relative above 2^-6 and
      2^-10 absolute below, next to the rotation's error.
Whole numbers are equal."""
import random

import pytest
import torch

from . import paged_reference as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(scope="module")
def w():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_weight_gemv_gb300 import build_ext
    build_ext.build()
    from w4a16_int4_weight_gemv_gb300 import binding
    binding.w4a16_device_error(clear=True)
    return binding


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# --------------------------------------------------------------------------
# block map
# --------------------------------------------------------------------------
def run_map(w, ctx, new, table, free, head, page, num_blocks, tokens, stride=0):
    t = i32(table)
    if stride:
        wide = torch.full((len(table), stride), 77, dtype=torch.int32, device="cuda")
        wide[:, :t.shape[1]] = t
        t = wide[:, :t.shape[1]]
    m = w.w4a16_paged_map(i32(ctx), i32(new), t, i32(free), i32([head]), page, num_blocks, tokens)
    flags = w.w4a16_device_error(clear=True)
    if stride:
        assert (wide[:, len(table[0]):] == 77).all()
    return t.tolist(), m, flags


def check_map(w, ctx, new, table, free, head, page, num_blocks, tokens, stride=0):
    t, m, flags = run_map(w, ctx, new, table, free, head, page, num_blocks, tokens, stride)
    want = ref.paged_map(ctx, new, table, free, head, page, num_blocks, tokens)
    assert t == want[0]
    assert m.slots.tolist() == want[1]
    assert m.positions.tolist() == want[2]
    assert m.row_start.tolist() == want[3]
    assert m.kv_len.tolist() == want[4]
    assert m.free_head.tolist() == [want[5]]
    bits = (w.DEVERR_SLOT if "slot" in want[6] else 0) | (w.DEVERR_BLOCKS if "blocks" in want[6] else 0)
    assert flags == bits


def map_problem(seed, B, page, longest_ctx, longest_new, decode=False):
    rng = random.Random(seed)
    ctx = [rng.choice([0, page, rng.randrange(longest_ctx + 1)]) for _ in range(B)]
    new = [1 if decode else rng.choice([0, 1, page, rng.randrange(longest_new + 1)]) for _ in range(B)]
    columns = -(-(longest_ctx + max(longest_new, page, 1)) // page) + 2
    blocks = sum(-(-(c + n) // page) for c, n in zip(ctx, new)) + 9
    ids = list(range(blocks))
    rng.shuffle(ids)
    table = []
    for c in ctx:
        k = -(-c // page)
        table.append([ids.pop() for _ in range(k)] + [-1] * (columns - k))
    return ctx, new, table, [-1, -1] + ids, 2, blocks


@pytest.mark.parametrize("page", [1, 7, 16, 24, 128])
@pytest.mark.parametrize("B", [1, 2, 31, 33, 511, 512, 513, 1100])
def test_map_matches_the_plain_form(w, B, page):
    ctx, new, table, free, head, blocks = map_problem(B * 131 + page, B, page, 90, 70)
    check_map(w, ctx, new, table, free, head, page, blocks, sum(new) + 3)


@pytest.mark.parametrize("B", [1, 16, 700])
def test_map_decode_step(w, B):
    ctx, new, table, free, head, blocks = map_problem(B, B, 16, 300, 1, decode=True)
    check_map(w, ctx, new, table, free, head, 16, blocks, B, stride=40)


def test_map_long_prompts(w):
    ctx, new, table, free, head, blocks = map_problem(5, 12, 16, 3000, 40000)
    check_map(w, ctx, new, table, free, head, 16, blocks, sum(new))


@pytest.mark.parametrize("tokens", [90001, 400000])
def test_map_buffers_off_16_bytes(w, tokens):
    # many tokens (four a thread), outputs that begin anywhere, requests without new tokens between
    rng = random.Random(tokens)
    new = [rng.choice([0, 0, 1, 3, rng.randrange(2 * tokens // 40)]) for _ in range(40)]
    ctx = [rng.randrange(50) for _ in new]
    ctx, new, tokens = ctx, new, max(tokens, sum(new) + 2)
    page, blocks = 24, sum(-(-(c + n) // 24) for c, n in zip(ctx, new)) + 5
    ids = list(range(blocks))
    rng.shuffle(ids)
    columns = max(-(-(c + n) // page) for c, n in zip(ctx, new)) + 1
    table = [[ids.pop() for _ in range(-(-c // page))] for c in ctx]
    table = [r + [-1] * (columns - len(r)) for r in table]
    want = ref.paged_map(ctx, new, table, ids, 0, page, blocks, tokens)
    for shift in (1, 2, 4):
        wide = [torch.full((tokens + 8,), 7, dtype=torch.int32, device="cuda") for _ in range(2)]
        out = w.paged_map_buffers(40, tokens, "cuda")._replace(slots=wide[0][shift:shift + tokens], positions=wide[1][shift:shift + tokens])
        m = w.w4a16_paged_map(i32(ctx), i32(new), i32(table), i32(ids), i32([0]), page, blocks, tokens, out=out)
        assert m.slots.tolist() == want[1] and m.positions.tolist() == want[2]
        for x in wide:
            assert (x[:shift] == 7).all() and (x[shift + tokens:] == 7).all()
    assert w.w4a16_device_error(clear=True) == 0


def test_map_most_requests(w):
    ctx, new, table, free, head, blocks = map_problem(6, 16384, 16, 5, 3)
    check_map(w, ctx, new, table, free, head, 16, blocks, sum(new) + 1)


def test_map_nothing_new(w):
    check_map(w, [5, 0, 16], [0, 0, 0], [[3, -1], [-1, -1], [1, -1]], [0, 2], 0, 16, 4, 4)
    check_map(w, [0], [0], [[-1]], [], 0, 16, 4, 0)


@pytest.mark.parametrize("case", ["free list", "columns", "places", "negative", "bad ids", "no free blocks"])
def test_map_runs_out(w, case):
    ctx, new, table, free, head, blocks = map_problem(11, 40, 16, 60, 80)
    tokens = sum(new) + 2
    if case == "free list":
        free = free[:20]
    elif case == "columns":
        table = [r[:5] for r in table]
    elif case == "places":
        tokens = sum(new) // 2
    elif case == "negative":
        ctx, new = [c if i % 5 else -3 for i, c in enumerate(ctx)], [n if i % 7 else -1 for i, n in enumerate(new)]
    elif case == "bad ids":
        free = [f if i % 6 else blocks + i for i, f in enumerate(free)]
        table = [[blocks if x >= 0 and i % 4 == 0 else x for x in r] for i, r in enumerate(table)]
    else:
        free, head = [], 0
    check_map(w, ctx, new, table, free, head, 16, blocks, tokens)


def test_map_refusals(w):
    a, t, f, h = i32([1, 2]), i32([[0, -1], [1, -1]]), i32([2, 3]), i32([0])
    ok = lambda **kw: w.w4a16_paged_map(**{**dict(ctx_len=a, new_len=a, block_table=t.clone(), free_blocks=f, free_head=h, page=16, num_blocks=4, tokens=3), **kw})
    ok()
    for bad in (dict(page=0), dict(num_blocks=0), dict(page=-4)):
        with pytest.raises(w.W4A16Error) as e:
            ok(**bad)
        assert e.value.status == w.Status.ERR_SHAPE
    with pytest.raises(w.W4A16Error) as e:
        ok(num_blocks=1 << 30)
    assert e.value.status == w.Status.ERR_UNSUPPORTED
    buf = w.paged_map_buffers(2, 3, a.device)
    with pytest.raises(w.W4A16Error) as e:
        ok(out=buf._replace(kv_len=a))
    assert e.value.status == w.Status.ERR_UNSUPPORTED
    with pytest.raises(w.W4A16Error) as e:
        ok(out=buf._replace(free_head=h))
    assert e.value.status == w.Status.ERR_UNSUPPORTED
    for bad in (dict(ctx_len=a.long()), dict(new_len=i32([1]))):
        with pytest.raises((TypeError, ValueError)):
            ok(**bad)
    for bad in (dict(block_table=t.t()), dict(block_table=t[:1]), dict(out=buf._replace(slots=i32([0]))), dict(ctx_len=a.cpu())):
        with pytest.raises(ValueError):
            ok(**bad)
    assert w.w4a16_device_error(clear=True) == 0


# --------------------------------------------------------------------------
# rotary + append
# --------------------------------------------------------------------------
def make_cache(w, gen, blocks, page, heads, dim, dtype, layout, fill=None):
    shape = (blocks, heads, page, dim) if layout == "head" else (blocks, page, heads, dim)
    pair = []
    for _ in range(2):
        x = torch.randn(shape, generator=gen)
        t = (x if dtype == "bf16" else (x * 20)).to(torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn).cuda()
        pair.append(t.permute(0, 2, 1, 3) if layout == "head" else t)
    scales = (None, None)
    if dtype == "fp8":
        scales = tuple((0.03 + 0.04 * torch.rand(heads, generator=gen)).cuda() for _ in range(2))
    return w.PagedCache(pair[0], pair[1], *scales)


def freqs(rotary):
    half = rotary // 2
    return torch.pow(torch.tensor(10000.0, dtype=torch.float64), -torch.arange(half, dtype=torch.float64) / max(half, 1)).float()


def check_codes(got, want, err, dtype):
    """Stored values (as cached, unscaled) against what they stand for."""
    if dtype == "bf16":
        tol = U * want.abs() + err
    else:
        want = want.clamp(-448, 448)
        tol = torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64)) * 1.0001 + err
    assert ((got - want).abs() <= tol).all(), float(((got - want).abs() - tol).max())


ROPE = [
    # T, q heads, kv heads, dim, rotary, sections, interleaved, page, dtype, layout, largest position
    (1, 32, 8, 128, 128, [64], False, 16, "bf16", "token", 30000),
    (3, 4, 4, 64, 64, [32], True, 16, "bf16", "head", 100),
    (37, 6, 2, 80, 64, [13, 19], False, 24, "bf16", "token", 5000),
    (65, 7, 1, 96, 96, [16, 16, 16], True, 7, "fp8", "token", 5000),
    (200, 8, 8, 256, 256, [40, 0, 60, 28], False, 64, "fp8", "head", 2 ** 31 - 1),
    (129, 2, 2, 16, 16, [8], False, 1, "bf16", "token", 2 ** 30),
    (50, 5, 5, 192, 16, [3, 5], True, 128, "bf16", "head", 1 << 25),
    (20, 3, 1, 128, 0, [0], False, 16, "fp8", "token", 10),
    (3000, 4, 1, 128, 96, [48], False, 32, "bf16", "token", 100000),
]


def rope_problem(w, case, seed):
    T, hq, hk, dim, rotary, sections, inter, page, dtype, layout, far = case
    gen = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, (hq + 2 * hk) * dim, generator=gen).bfloat16()
    pos = torch.randint(0, far, (len(sections), T), generator=gen, dtype=torch.int64).int()
    blocks = T // page + 3
    slots = torch.randperm(blocks * page, generator=gen)[:T].int()
    cache = make_cache(w, gen, blocks, page, hk, dim, dtype, layout)
    return qkv, pos, slots, cache


def split_qkv(qkv, hq, hk, dim):
    T = qkv.shape[0]
    q, k, v = qkv.split([hq * dim, hk * dim, hk * dim], 1)
    return q.view(T, hq, dim), k.view(T, hk, dim), v.view(T, hk, dim)


@pytest.mark.parametrize("case", ROPE, ids=lambda c: "T%d-q%d-kv%d-d%d-r%d-%s-%s" % (c[0], c[1], c[2], c[3], c[4], c[8], c[9]))
def test_rope_append_matches_the_plain_form(w, case):
    T, hq, hk, dim, rotary, sections, inter, page, dtype, layout, _ = case
    qkv, pos, slots, cache = rope_problem(w, case, 17 + T)
    slots[T // 2] = -1 if T > 1 else slots[T // 2]
    old = [c.clone() for c in (cache.k, cache.v)]
    q, k, v = split_qkv(qkv.cuda(), hq, hk, dim)
    f = freqs(rotary)
    got = w.w4a16_rope_append(q, k, v, pos.cuda(), f.cuda(), slots.cuda(), cache, sections=sections, interleaved=inter)
    assert w.w4a16_device_error(clear=True) == 0
    qd, kd, vd = (x.double() for x in split_qkv(qkv, hq, hk, dim))
    size = lambda x: 2.0 ** -20 * (x.abs() + ref.rope(x.abs(), torch.zeros_like(pos), f, sections, inter) + x.abs().amax(-1, keepdim=True))
    yq = ref.rope(qd, pos, f, sections, inter)
    assert ((got.double().cpu() - yq).abs() <= U * yq.abs() + size(qd)).all()
    yk = ref.rope(kd, pos, f, sections, inter)
    keep = slots >= 0
    at = slots[keep].long()
    for stored, before, want, err, scale in ((cache.k, old[0], yk, size(kd), cache.k_scale), (cache.v, old[1], vd, 0 * vd, cache.v_scale)):
        if scale is not None:
            s = scale.double().cpu()[:, None]
            want, err = want / s, err / s + 2.0 ** -22 * (want / s).abs()
        rows = stored.float().double().cpu()[at // page, at % page]
        check_codes(rows, want[keep], err[keep], dtype)
        untouched = torch.ones(cache.blocks * page, dtype=torch.bool)
        untouched[at] = False
        i = torch.arange(cache.blocks * page)[untouched]
        assert torch.equal(stored.float().cpu()[i // page, i % page], before.float().cpu()[i // page, i % page])


@pytest.mark.parametrize("case", [
    # several groups of tokens a thread block, the last one ragged; one and two tokens a thread
    (10007, 14, 1, 128, 128, [24, 20, 20], False, 16, "bf16", "token", 100000),
    (10007, 14, 1, 128, 48, [24], True, 24, "bf16", "head", 1 << 25),
    (10007, 14, 1, 128, 80, [40], True, 16, "fp8", "token", 100000),
    (12001, 6, 5, 112, 64, [32], False, 7, "bf16", "token", 5000),
    (9001, 1, 1, 48, 16, [8], False, 16, "fp8", "head", 5000),
    (9001, 33, 2, 64, 64, [32], True, 16, "fp8", "token", 5000),
    (7777, 5, 3, 80, 0, [0], False, 16, "bf16", "token", 10),
], ids=lambda c: "T%d-q%d-kv%d-d%d-r%d-%s-%s" % (c[0], c[1], c[2], c[3], c[4], c[8], c[9]))
def test_rope_append_of_many_tokens(w, case):
    test_rope_append_matches_the_plain_form(w, case)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_in_place_of_many_tokens(w, inter):
    x = torch.randn(40011, 4, 64, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    pos, f = torch.arange(40011).int().cuda(), freqs(64).cuda()
    y = w.w4a16_rope_append(x, None, None, pos, f, None, None, interleaved=inter)
    z = x.clone()
    w.w4a16_rope_append(z, None, None, pos, f, None, None, q_out=z, interleaved=inter)
    assert torch.equal(y, z)


def test_rope_in_place_and_without_keys(w):
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(9, 4, 64, generator=gen).bfloat16()
    pos, f = torch.arange(9).int(), freqs(64)
    y = w.w4a16_rope_append(x.cuda(), None, None, pos.cuda(), f.cuda(), None, None)
    z = x.cuda()
    assert w.w4a16_rope_append(z, None, None, pos.cuda(), f.cuda(), None, None, q_out=z) is z
    assert torch.equal(y, z)


def test_append_without_queries(w):
    case = (11, 2, 2, 64, 64, [32], False, 16, "bf16", "token", 99)
    qkv, pos, slots, cache = rope_problem(w, case, 5)
    q, k, v = split_qkv(qkv.cuda(), 2, 2, 64)
    f = freqs(64).cuda()
    assert w.w4a16_rope_append(None, k, v, pos.cuda(), f, slots.cuda(), cache) is None
    k1, v1 = cache.k.clone(), cache.v.clone()
    w.w4a16_rope_append(q, k, v, pos.cuda(), f, slots.cuda(), cache)
    assert torch.equal(k1, cache.k) and torch.equal(v1, cache.v)


def test_rope_no_tokens(w):
    x = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    y = w.w4a16_rope_append(x, None, None, i32([]), freqs(64).cuda(), None, None)
    assert y.shape == (0, 4, 64)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradient(w, inter):
    # the gradient of sum(g * rope(x)) is rope's inverse on g: against the formula's, and against differences
    gen = torch.Generator().manual_seed(8)
    T, H, D = 5, 3, 64
    g = torch.randn(T, H, D, generator=gen).bfloat16()
    pos = torch.randint(0, 3000, (2, T), generator=gen).int()
    f, sections = freqs(D), [20, 12]
    got = w.w4a16_rope_append(g.cuda(), None, None, pos.cuda(), f.cuda(), None, None, sections=sections, interleaved=inter,
                              inverse=True).double().cpu()
    gd = g.double()
    tol = U * got.abs() + 2.0 ** -19 * gd.abs().amax(-1, keepdim=True)
    assert ((got - ref.rope(gd, pos, f, sections, inter, inverse=True)).abs() <= tol).all()
    x = torch.randn(T, H, D, generator=gen, dtype=torch.float64)
    for t, h, d in ((0, 0, 0), (4, 2, 63), (2, 1, 31), (1, 0, 32), (3, 2, 33)):
        e = torch.zeros_like(x)
        e[t, h, d] = 1e-3
        fx = [(gd * ref.rope(x + s * e, pos, f, sections, inter)).sum() for s in (1, -1)]
        assert abs((fx[0] - fx[1]) / 2e-3 - got[t, h, d]) <= tol[t, h, d] + 1e-9


def test_append_saturates_and_keeps_nan(w):
    gen = torch.Generator().manual_seed(1)
    cache = make_cache(w, gen, 2, 4, 1, 16, "fp8", "token")
    k = torch.zeros(3, 1, 16, dtype=torch.bfloat16, device="cuda")
    k[0], k[1], k[2] = 1e4, -float("inf"), float("nan")
    w.w4a16_rope_append(None, k, k, i32([0, 0, 0]), freqs(16).cuda(), i32([0, 1, 2]), cache)
    v = cache.v.float().flatten(0, 1)
    assert (v[0] == 448).all() and (v[1] == -448).all() and v[2].isnan().all()


def test_append_flags_slots_outside(w):
    case = (8, 2, 2, 64, 64, [32], False, 16, "bf16", "token", 99)
    qkv, pos, slots, cache = rope_problem(w, case, 6)
    q, k, v = split_qkv(qkv.cuda(), 2, 2, 64)
    f = freqs(64).cuda()
    good = w.w4a16_rope_append(q, k, v, pos.cuda(), f, slots.cuda(), cache)
    want = cache.k.clone()
    for bad in (cache.blocks * 16, -2, 2 ** 31 - 1, -2 ** 31):
        s = slots.clone()
        s[3] = bad
        got = w.w4a16_rope_append(q, k, v, pos.cuda(), f, s.cuda(), cache)
        assert w.w4a16_device_error(clear=True) == w.DEVERR_SLOT
        assert torch.equal(got, good) and torch.equal(cache.k, want)


def test_rope_refusals(w):
    case = (4, 2, 2, 64, 64, [32], False, 16, "bf16", "token", 99)
    qkv, pos, slots, cache = rope_problem(w, case, 6)
    q, k, v = split_qkv(qkv.cuda(), 2, 2, 64)
    base = dict(q=q, k=k, v=v, positions=pos.cuda(), inv_freq=freqs(64).cuda(), slots=slots.cuda(), cache=cache)
    call = lambda **kw: w.w4a16_rope_append(**{**base, **kw})
    call()
    before = cache.k.clone()
    for bad, status in ((dict(inv_freq=freqs(64)[:12].cuda()), w.Status.ERR_SHAPE),       # rotary not a multiple of 16
                        (dict(inv_freq=torch.ones(40, device="cuda")), w.Status.ERR_SHAPE),  # rotary > dim
                        (dict(sections=[31]), w.Status.ERR_SHAPE)):
        with pytest.raises(w.W4A16Error) as e:
            call(**bad)
        assert e.value.status == status
    odd = torch.zeros(4, 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(w.W4A16Error) as e:
        call(q=odd[:, :128].view(4, 2, 64))
    assert e.value.status == w.Status.ERR_ALIGN
    with pytest.raises(w.W4A16Error) as e:
        call(positions=torch.zeros(5, 4, dtype=torch.int32, device="cuda"), sections=[8, 8, 8, 8, 0])
    assert e.value.status == w.Status.ERR_UNSUPPORTED
    for bad in (dict(k=k[:3]), dict(sections=[16, 16]), dict(cache=None), dict(q=q.float()), dict(q=q.transpose(1, 2)), dict(q=q.cpu()),
                dict(slots=slots.cuda().long()), dict(q_out=q[:2])):
        with pytest.raises((ValueError, TypeError)):
            call(**bad)
    assert torch.equal(cache.k, before)


# --------------------------------------------------------------------------
# attention
# --------------------------------------------------------------------------
def attention_problem(w, seed, lens, hq, hk, dim, page, dtype, layout, columns=None, sharp=1.5):
    gen = torch.Generator().manual_seed(seed)
    used = [-(-n // page) for n in lens]
    blocks = sum(used) + 3
    cache = make_cache(w, gen, blocks, page, hk, dim, dtype, layout)
    order = torch.randperm(blocks, generator=gen).tolist()
    columns = columns or max(max(used), 1)
    table = []
    for u in used:
        # past a request's blocks: ids that must not be followed
        table.append([order.pop() for _ in range(u)] + [10 ** 9] * (columns - u))
    q = (sharp * torch.randn(len(lens), hq, dim, generator=gen)).bfloat16()
    # whatever no request sees is not a number
    seen = torch.zeros(blocks, page, dtype=torch.bool)
    for r, n in zip(table, lens):
        for j in range(n):
            seen[r[j // page], j % page] = True
    for c in (cache.k, cache.v):
        hole = (~seen).cuda().view(blocks, page, 1, 1)
        c.view(torch.uint8 if dtype == "fp8" else torch.int16).masked_fill_(hole, 0x7F if dtype == "fp8" else 0x7FC0)
    return q, cache, table


def values_of(cache):
    k, v = cache.k.float().double().cpu(), cache.v.float().double().cpu()
    if cache.k_scale is not None:
        k, v = k * cache.k_scale.double().cpu()[:, None], v * cache.v_scale.double().cpu()[:, None]
    return k, v


def check_attention(w, q, cache, table, lens, scale=None, window=0, flags=0, got=None):
    dim = q.shape[2]
    scale = dim ** -0.5 if scale is None else scale
    if got is None:
        got = w.w4a16_paged_attention(q.cuda(), cache, i32(table), i32(lens), scale=scale, window=window)
    assert w.w4a16_device_error(clear=True) == flags
    out, lse = got[0].double().cpu(), got[1].double().cpu()
    want, want_lse, spread, reach = ref.attention(q.double(), *values_of(cache), table, lens, scale, window)
    score = (dim + 16) * 2.0 ** -24 * reach
    tol = U * want.abs() + (U + 2 * score[..., None]) * spread + 1e-30
    assert not out.isnan().any()
    assert ((out - want).abs() <= tol).all(), float(((out - want).abs() / tol.clamp(min=1e-30)).max())
    empty = want_lse == -float("inf")
    assert torch.equal(lse == -float("inf"), empty)
    d = (lse - want_lse)[~empty].abs()
    assert (d <= (score + 2.0 ** -21 * (1 + want_lse.abs()))[~empty].clamp(min=2.0 ** -21)).all(), float(d.max())
    assert (out[empty] == 0).all()


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200, 255, 257, 500]


@pytest.mark.parametrize("dtype,layout", [("bf16", "token"), ("bf16", "head"), ("fp8", "token"), ("fp8", "head")])
@pytest.mark.parametrize("dim,page", [(128, 16), (64, 24), (256, 64), (80, 8), (96, 7), (16, 1), (192, 128), (112, 48)])
def test_attention_lengths_dims_pages(w, dim, page, dtype, layout):
    q, cache, table = attention_problem(w, dim + page, LENS, 8, 2, dim, page, dtype, layout)
    check_attention(w, q, cache, table, LENS)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("hq,hk", [(1, 1), (5, 5), (2, 1), (6, 2), (4, 1), (7, 1), (8, 1), (9, 1), (16, 1), (17, 1), (24, 1), (34, 2), (64, 1), (40, 8)])
def test_attention_head_groups(w, hq, hk, dtype):
    lens = [3, 0, 90, 161]
    q, cache, table = attention_problem(w, hq * 7 + hk, lens, hq, hk, 64, 16, dtype, "token")
    check_attention(w, q, cache, table, lens)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 499, 1000000])
def test_attention_window(w, window, dtype):
    q, cache, table = attention_problem(w, window, LENS, 4, 2, 128, 16, dtype, "token")
    # what lies before the window is not read either
    for r, n in zip(table, LENS):
        for j in range(max(0, n - window)):
            for c in (cache.k, cache.v):
                c.view(torch.uint8 if dtype == "fp8" else torch.int16)[r[j // 16], j % 16] = 0x7F if dtype == "fp8" else 0x7FC0
    k, v = cache.k, cache.v
    got = w.w4a16_paged_attention(q.cuda(), cache, i32(table), i32(LENS), window=window)
    assert w.w4a16_device_error(clear=True) == 0
    check_attention(w, q, cache, table, LENS, window=window, got=got)


@pytest.mark.parametrize("dtype,dim,hq,hk,page", [("bf16", 128, 8, 2, 16), ("fp8", 128, 8, 2, 32), ("bf16", 64, 4, 4, 24), ("bf16", 256, 16, 1, 16)])
@pytest.mark.parametrize("lens", [[20000], [9001, 1], [0, 5000, 0, 12345, 3]], ids=str)
def test_attention_long(w, lens, dtype, dim, hq, hk, page):
    q, cache, table = attention_problem(w, 3, lens, hq, hk, dim, page, dtype, "token")
    check_attention(w, q, cache, table, lens)


def test_attention_many_requests(w):
    rng = random.Random(4)
    lens = [rng.choice([0, 1, 5, rng.randrange(120)]) for _ in range(1100)]
    q, cache, table = attention_problem(w, 9, lens, 4, 2, 64, 16, "bf16", "token")
    check_attention(w, q, cache, table, lens)


def test_attention_all_empty(w):
    q, cache, table = attention_problem(w, 9, [0, 0, 0], 4, 2, 64, 16, "bf16", "token")
    check_attention(w, q, cache, table, [0, 0, 0])


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_attention_strides(w, dtype):
    lens = [70, 5, 131]
    q, cache, table = attention_problem(w, 21, lens, 6, 2, 64, 16, dtype, "token")
    row = torch.full((3, 10 * 64), 9.0).bfloat16().cuda()   # a fused projection's rows: queries first
    row[:, :6 * 64] = q.reshape(3, -1).cuda()
    out = torch.full((3, 8, 6, 64), 5.0).bfloat16().cuda()
    wide = torch.full((3, 20), 10 ** 9, dtype=torch.int32, device="cuda")
    wide[:, :len(table[0])] = i32(table)
    got = w.w4a16_paged_attention(row[:, :6 * 64].view(3, 6, 64), cache, wide[:, :len(table[0])], i32([0] + lens)[1:], out=out[:, 2])
    check_attention(w, q, cache, table, lens, got=got)
    assert (out[:, :2] == 5).all() and (out[:, 3:] == 5).all()
    # heads before requests, in memory
    other = q.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    again = w.w4a16_paged_attention(other, cache, i32(table), i32(lens))
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


def test_attention_strided_cache(w):
    # keys and values interleaved in one allocation, with room between the heads
    lens = [40, 3]
    q, cache, table = attention_problem(w, 2, lens, 4, 2, 64, 16, "bf16", "token")
    both = torch.full((cache.blocks, 16, 2, 2, 96), float("nan")).bfloat16().cuda()
    both[:, :, 0, :, :64], both[:, :, 1, :, :64] = cache.k, cache.v
    view = w.PagedCache(both[:, :, 0, :, :64], both[:, :, 1, :, :64])
    check_attention(w, q, view, table, lens)


def test_attention_bad_blocks_are_left_out(w):
    lens = [70, 100, 33]
    q, cache, table = attention_problem(w, 12, lens, 4, 2, 64, 16, "bf16", "token")
    for bad in (-1, cache.blocks, 2 ** 31 - 1, -2 ** 31):
        t = [list(r) for r in table]
        t[1][2] = bad
        t[2] = [bad] * len(t[2])
        check_attention(w, q, cache, t, lens, flags=w.DEVERR_SLOT)


def test_attention_bad_lengths(w):
    lens = [70, 100, 33]
    q, cache, table = attention_problem(w, 12, [112, 112, 33], 4, 2, 64, 16, "bf16", "token")
    check_attention(w, q, cache, table, [70, 112 + 9, -4], flags=w.DEVERR_SLOT)
    assert lens


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_attention_large_scores(w, dtype):
    # one token far above the rest, and scores to about +-1e4: nothing overflows
    lens = [300, 17]
    q, cache, table = attention_problem(w, 31, lens, 8, 2, 128, 16, dtype, "token", sharp=600.0)
    check_attention(w, q, cache, table, lens)
    q, cache, table = attention_problem(w, 32, lens, 8, 2, 128, 16, dtype, "token", sharp=1e-20)
    check_attention(w, q, cache, table, lens)


def test_attention_infinite_scores(w):
    # keys that score -infinity have no weight; a request of nothing else counts as empty
    lens = [50, 20, 35]
    q, cache, table = attention_problem(w, 13, lens, 4, 2, 64, 16, "bf16", "token")
    q = q.abs() + 0.1
    for b, js in ((0, range(0, 50, 3)), (1, range(20)), (2, range(16, 35))):
        for j in js:
            cache.k[table[b][j // 16], j % 16, :, 5] = -float("inf")
    got = w.w4a16_paged_attention(q.bfloat16().cuda(), cache, i32(table), i32(lens))
    k, v = values_of(cache)
    want, want_lse, spread, _ = ref.attention(q.bfloat16().double(), k, v, table, lens, 0.125, 0)
    assert ((got[0].double().cpu() - want).abs() <= U * want.abs() + (U + 1e-4) * spread).all()
    assert (got[0][1] == 0).all() and (got[1][1] == -float("inf")).all()
    assert torch.allclose(got[1][::2].double().cpu(), want_lse[::2], rtol=1e-5, atol=1e-5)


def test_attention_nan_is_kept(w):
    lens = [50, 20]
    q, cache, table = attention_problem(w, 14, lens, 4, 2, 64, 16, "bf16", "token")
    cache.v[table[0][1], 3, 0, 7] = float("nan")
    cache.k[table[1][0], 3, 1, 7] = float("nan")
    out, lse = w.w4a16_paged_attention(q.cuda(), cache, i32(table), i32(lens))
    nan = torch.zeros(2, 4, 64, dtype=torch.bool)
    nan[0, :2, 7] = True
    nan[1, 2:] = True
    assert torch.equal(out.isnan().cpu(), nan)
    assert torch.equal(lse.isnan().cpu(), nan.all(-1))


def test_attention_of_tables_too_wide_for_one_launch(w):
    # rows of 2^26 blocks: the costs of two requests would pass 32 bits, so each is launched by itself
    lens = [70, 0, 700, 15]
    q, cache, table = attention_problem(w, 77, lens, 16, 16, 64, 16, "bf16", "token")
    wide = torch.empty(4, 1 << 26, dtype=torch.int32, device="cuda")
    wide[:, :len(table[0])] = i32(table)
    got = w.w4a16_paged_attention(q.cuda(), cache, wide, i32(lens))
    check_attention(w, q, cache, table, lens, got=got)


@pytest.mark.parametrize("lens", [[4000], [9, 7000, 0], [1500] * 6, [600] * 30], ids=str)
@pytest.mark.parametrize("page", [16, 24])
def test_attention_rows_over_clusters(w, lens, page):
    # few rows: one to eight CTAs for each; with a window, and with a block that is not there
    for dtype, dim, hq, hk in (("bf16", 128, 4, 2), ("fp8", 64, 3, 1), ("bf16", 256, 12, 1)):
        q, cache, table = attention_problem(w, len(lens) + page, lens, hq, hk, dim, page, dtype, "token")
        check_attention(w, q, cache, table, lens)
        check_attention(w, q, cache, table, lens, window=333)
    bad = [list(r) for r in table]
    bad[lens.index(max(lens))][3] = -7
    check_attention(w, q, cache, bad, lens, flags=w.DEVERR_SLOT)


@pytest.mark.parametrize("B", [128, 129, 300])
def test_attention_many_long_requests(w, B):
    # more requests than one scan of the lengths holds, long enough to be dealt in shares
    rng = random.Random(B)
    lens = [rng.choice([0, 1, 160, rng.randrange(400)]) for _ in range(B)]
    q, cache, table = attention_problem(w, B, lens, 8, 4, 64, 16, "bf16", "token")
    check_attention(w, q, cache, table, lens)
    check_attention(w, q, cache, table, [0] * (B - 1) + lens[-1:])


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_attention_offsets_past_32_bits(w, dtype):
    # element offsets beyond 2^32: only the blocks in use are written
    hk, dim, page = 8, 128, 16
    blocks = (1 << 32) // (hk * dim * page) + 300
    t = torch.empty((blocks, page, hk, dim), dtype=torch.uint8 if dtype == "fp8" else torch.bfloat16, device="cuda")
    big = t.view(torch.float8_e4m3fn) if dtype == "fp8" else t
    lens = [200, 77]
    q, small, table = attention_problem(w, 3, lens, 16, hk, dim, page, dtype, "token")
    far = blocks - small.blocks
    cache = w.PagedCache(big, big, small.v_scale, small.v_scale)  # one memory for both, so one scale
    raw = (lambda c: c.view(torch.uint8)) if dtype == "fp8" else (lambda c: c)
    raw(big)[far:] = raw(small.k)
    one = w.PagedCache(small.k, small.k, small.v_scale, small.v_scale)
    a = w.w4a16_paged_attention(q.cuda(), one, i32(table), i32(lens))
    b = w.w4a16_paged_attention(q.cuda(), cache, i32([[x + far if x < 10 ** 9 else x for x in r] for r in table]), i32(lens))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # and the append into them
    x = torch.randn(5, hk, dim, device="cuda").bfloat16()
    slots = torch.tensor([far * page + 3, 7, blocks * page - 1, far * page - 5, 100], dtype=torch.int32)
    w.w4a16_rope_append(None, x, x, torch.zeros(5, dtype=torch.int32, device="cuda"), freqs(128).cuda(), slots.cuda(), cache)
    rows = raw(big)[(slots // page).long(), (slots % page).long()]
    want = x if dtype == "bf16" else (x.float() / small.v_scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(rows, want)
    assert w.w4a16_device_error(clear=True) == 0


def test_attention_repeats_and_leaves_its_workspace(w):
    lens = [3000, 1, 0, 777]
    q, cache, table = attention_problem(w, 41, lens, 8, 2, 128, 16, "bf16", "token")
    ws = w.paged_attention_workspace(cache, 8)
    args = (q.cuda(), cache, i32(table), i32(lens))
    first = w.w4a16_paged_attention(*args, workspace=ws)
    for n in ([3000, 1, 0, 777], [5, 2000, 1500, 700]):
        w.w4a16_paged_attention(q.cuda(), cache, i32(table), i32([min(a, b) for a, b in zip(n, lens)]), workspace=ws)
        again = w.w4a16_paged_attention(*args, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    check_attention(w, q, cache, table, lens, got=first)


def test_attention_on_another_stream(w):
    lens = [900, 300]
    q, cache, table = attention_problem(w, 42, lens, 8, 2, 128, 16, "bf16", "token")
    dq, dt, dl = q.cuda(), i32(table), i32(lens)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = w.w4a16_paged_attention(dq, cache, dt, dl)
    s.synchronize()
    check_attention(w, q, cache, table, lens, got=got)
    got = w.w4a16_paged_attention(dq, cache, dt, dl, workspace=w.paged_attention_workspace(cache, 8))
    check_attention(w, q, cache, table, lens, got=got)


def test_attention_refusals(w):
    lens = [40, 3]
    q, cache, table = attention_problem(w, 2, lens, 4, 2, 64, 16, "bf16", "token")
    base = dict(q=q.cuda(), cache=cache, block_table=i32(table), kv_len=i32(lens), workspace=w.paged_attention_workspace(cache, 4))
    call = lambda **kw: w.w4a16_paged_attention(**{**base, **kw})
    call()
    for bad, status in ((dict(q=q[:, :3].cuda()), w.Status.ERR_SHAPE), (dict(window=-1), w.Status.ERR_SHAPE),
                        (dict(workspace=torch.zeros(8, dtype=torch.uint8, device="cuda")), w.Status.ERR_WORKSPACE),
                        (dict(q=torch.zeros(2, 4 * 64 + 4, dtype=torch.bfloat16, device="cuda")[:, :256].view(2, 4, 64)), w.Status.ERR_ALIGN)):
        with pytest.raises(w.W4A16Error) as e:
            call(**bad)
        assert e.value.status == status
    for bad in (dict(q=q), dict(q=q.cuda().half()), dict(q=q.cuda()[:, :, :32]), dict(kv_len=i32([1])), dict(kv_len=i32(lens).long()),
                dict(block_table=i32(table).t()), dict(block_table=i32(table)[:1]), dict(out=torch.empty(1, 4, 64, dtype=torch.bfloat16, device="cuda")),
                dict(lse=torch.empty(2, 3, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            call(**bad)
    with pytest.raises(TypeError):
        w.PagedCache(cache.k.float(), cache.v.float())
    with pytest.raises(ValueError):
        w.PagedCache(cache.k, cache.v[:1])
    with pytest.raises(ValueError):
        w.PagedCache(cache.k.cpu(), cache.v.cpu())
    with pytest.raises(ValueError):
        w.PagedCache(cache.k, cache.v, torch.ones(2, device="cuda"), torch.ones(2, device="cuda"))
    with pytest.raises(TypeError):
        w.PagedCache(cache.k.to(torch.float8_e4m3fn), cache.v.to(torch.float8_e4m3fn))
    assert w.w4a16_device_error(clear=True) == 0


# --------------------------------------------------------------------------
# the two ways of marshalling the arguments
# --------------------------------------------------------------------------
def test_both_marshallings_make_the_same_calls(w, monkeypatch):
    if w._fast is None:
        pytest.skip("the extension module was not built")
    results = []
    for fast in (w._fast, None):
        monkeypatch.setattr(w, "_fast", fast)
        ctx, new, table, free, head, blocks = map_problem(3, 9, 16, 60, 40)
        t = i32(table)
        m = w.w4a16_paged_map(i32(ctx), i32(new), t, i32(free), i32([head]), 16, blocks, sum(new) + 2,
                              out=w.paged_map_buffers(9, sum(new) + 2, "cuda"))
        case = (40, 6, 2, 64, 64, [20, 12], True, 16, "fp8", "head", 300)
        qkv, pos, slots, cache = rope_problem(w, case, 5)
        q, k, v = split_qkv(qkv.cuda(), 6, 2, 64)
        out = torch.empty(40, 6, 64, dtype=torch.bfloat16, device="cuda")
        assert w.w4a16_rope_append(q, k, v, pos.cuda(), freqs(64).cuda(), slots.cuda(), cache, sections=[20, 12], interleaved=True,
                                   q_out=out) is out
        lens = [30, 0, 77]
        qa, ca, ta = attention_problem(w, 8, lens, 4, 2, 64, 16, "bf16", "token")
        got = [torch.empty(3, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 4, device="cuda")]
        w.w4a16_paged_attention(qa.cuda(), ca, i32(ta), i32(lens), window=50, out=got[0], lse=got[1],
                                workspace=w.paged_attention_workspace(ca, 4), stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
        results.append([t, *m, out, cache.k.float(), cache.v.float(), *got])
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert w.w4a16_device_error(clear=True) == 0
