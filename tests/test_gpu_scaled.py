"""The operators over an 8-bit paged cache with scales by group, on the GPU against
their plain forms.

Scales are equal, bit for bit: they are powers of two decided by magnitudes that are
exact (or one fp32 sum of two exact squares).  So are the codes of values and of keys
that are not turned, codes that a grown scale shifts, and what is read back (one fp32
product, one rounding).  Tolerances of the rest:
  keys that are turned: |code - y / S| <= half a step (int8: 1/2; e4m3: 2^-4 of the
      code's magnitude, at least 2^-10) + 2^-20 (|x1| + |x2|) / S, the rotation's
      error: cosine and sine to about 2^-21 each with the fp32 products;
  queries: 2^-8 |y| + 2^-20 (|x1| + |x2|);
  attention, out: 2^-8 |y| + 2^-11 sum p|v| + 2^-33 max_j(p_j |s_j|) sum |c_j| (the
      rounding of the result and of the weights in fp16, normal and below), and as a
      relative error of each weight the fp32 scores' error, (dim + 16) 2^-24 of scale
      sum |q||k| (twice: in the maximum's row and in the token's own), and 2^-22 (8 +
      |log2 of the scales|) for the weight's exponent and its two powers of two;
  attention, lse: that score error, and a few fp32 roundings of the sum."""
import itertools
import random

import pytest
import torch

from . import scaled_reference as ref
from .test_gpu_paged import freqs, i32, split_qkv, w  # noqa: F401  (w: the fixture)

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
INT8, E4M3 = torch.int8, torch.float8_e4m3fn
TYPES = {"int8": INT8, "e4m3": E4M3}


def raw(t):
    return t.view(torch.uint8)


def code_values(t):
    return t.float().double().cpu()


def make_cache(w, gen, blocks, page, group, heads, dim, dtype, layout="token", spread=2):
    """A cache full of random codes and scales (powers of two; those of the values 2^-spread to 2^spread apart)."""
    kept = []
    for most in (2, spread):
        x = torch.randn(blocks, page, heads, dim, generator=gen)
        c = (x * 40).round().clamp(-127, 127).to(INT8) if dtype is INT8 else (x * 90).clamp(-448, 448).to(E4M3)
        c = c.cuda()
        if layout == "head":
            c = raw(c).permute(0, 2, 1, 3).contiguous().view(dtype).permute(0, 2, 1, 3)
        e = torch.randint(-most, most + 1, (blocks, heads, page // group), generator=gen).float()
        s = torch.exp2(e - (5 if dtype is INT8 else 7)).cuda()
        kept += [c, s.transpose(1, 2) if layout == "head" else s.transpose(1, 2).contiguous()]
    return w.ScaledCache(kept[0], kept[2], kept[1], kept[3])


def state_of(cache):
    return [raw(cache.k).clone(), raw(cache.v).clone(), cache.k_scale.clone(), cache.v_scale.clone()]


def same_bits(a, b):
    return all(torch.equal(x.view(torch.uint8) if x.dtype is torch.uint8 else x.contiguous().view(torch.int32),
                           y.view(torch.uint8) if y.dtype is torch.uint8 else y.contiguous().view(torch.int32)) for x, y in zip(a, b))


# --------------------------------------------------------------------------
# append
# --------------------------------------------------------------------------
def slots_of(rng, ctx, new, page, blocks):
    """Slots of requests that hold ctx[b] tokens and add new[b], their blocks in no order."""
    ids = list(range(blocks))
    rng.shuffle(ids)
    slots = []
    for c, n in zip(ctx, new):
        mine = [ids.pop() for _ in range(-(-(c + n) // page))]
        slots += [mine[p // page] * page + p % page for p in range(c, c + n)]
    return slots


def check_append(w, cache, qkv, hq, pos, f, sections, inter, slots, flags=0, slack_codes=0.0):
    """Appends to `cache` and looks at everything that the call may write."""
    hk, dim, page, group, dtype = cache.heads, cache.dim, cache.page, cache.group, cache.k.dtype
    q, k, v = split_qkv(qkv.cuda(), hq, hk, dim)
    before = [code_values(cache.k), code_values(cache.v), cache.k_scale.cpu(), cache.v_scale.cpu()]
    got = w.w4a16_scaled_append(q if hq else None, k, v, pos.cuda(), f.cuda(), i32(slots), cache, sections=sections, interleaved=inter)
    assert w.w4a16_device_error(clear=True) == flags
    half, rotary = f.numel(), 2 * f.numel()
    pos2 = pos if pos.dim() == 2 else pos[None]
    sections = sections or [half]

    def sums(x):  # |x1| + |x2| where a pair is turned
        m = torch.zeros_like(x)
        if half:
            a, b = (x[..., 0:rotary:2], x[..., 1:rotary:2]) if inter else (x[..., :half], x[..., half:rotary])
            t = a.abs() + b.abs()
            m[..., :rotary] = t.repeat_interleave(2, -1) if inter else torch.cat([t, t], -1)
        return m

    x = [t.double().cpu() for t in (q, k, v)]
    if hq:
        y = ref.rope(x[0], pos2, f, sections, inter)
        assert ((got.double().cpu() - y).abs() <= U * y.abs() + 2.0 ** -20 * sums(x[0])).all()
    else:
        assert got is None
    for codes, scales, old, olds, values, turned, rot in (
            (cache.k, cache.k_scale, before[0], before[2], k, ref.rope(x[1], pos2, f, sections, inter) if half else x[1], rotary),
            (cache.v, cache.v_scale, before[1], before[3], v, x[2], 0)):
        want, want_s, exact, bad = ref.append(old, olds, values.cpu(), turned, rot, inter, slots, page, group, dtype)
        assert bad == bool(flags)
        s = scales.cpu()
        assert torch.equal(torch.nan_to_num(s, nan=-1.0), torch.nan_to_num(want_s, nan=-1.0))
        have = code_values(codes)
        fresh = ~exact.isnan()
        void = s.isnan().repeat_interleave(group, 1)[..., None].expand_as(have)  # codes of no meaning
        fresh &= ~void
        still = ~fresh & ~void
        same = lambda a, b: (a == b) | (a.isnan() & b.isnan())
        assert same(have, want)[still].all()
        if rot:
            place = torch.full((codes.shape[0] * page,), -1)
            place[torch.tensor([i for i in slots if 0 <= i < len(place)], dtype=torch.long)] = torch.tensor([t for t, i in enumerate(slots) if 0 <= i < len(place)])
            at = place.view(-1, page)
            err = sums(x[1])[at.clamp(min=0)] * 2.0 ** -20 / s.double().repeat_interleave(group, 1)[..., None]
            step = torch.full_like(have, 0.5) if dtype is INT8 else (2.0 ** -4 * exact.abs()).clamp(min=2.0 ** -10)
            assert ((have - exact).abs() <= step * (1 + 2.0 ** -20) + err)[fresh].all()
        else:
            assert torch.equal(have[fresh], want[fresh])
    return got


def append_problem(w, seed, ctx, new, hq, hk, dim, rotary, axes, page, group, dtype, layout="token", pad=False):
    rng, gen = random.Random(seed), torch.Generator().manual_seed(seed)
    blocks = sum(-(-(c + n) // page) for c, n in zip(ctx, new)) + 2
    cache = make_cache(w, gen, blocks, page, group, hk, dim, dtype, layout)
    slots = slots_of(rng, ctx, new, page, blocks)
    if pad:
        for b in range(len(new) - 1, -1, -1):
            at = sum(new[:b])
            slots[at:at] = [-1] * rng.choice([0, 1, 3])
    T = len(slots)
    # values of very different size from token to token: scales that grow, and some that do not
    size = torch.exp2(torch.randint(-4, 5, (T, 1, 1), generator=gen).float())
    qkv = (torch.randn(T, hq + 2 * hk, dim, generator=gen) * size).bfloat16().view(T, -1)
    pos = torch.randint(0, 40000, (axes, T), generator=gen).int()
    half = rotary // 2
    sections = [half - (axes - 1) * (half // axes)] + [half // axes] * (axes - 1)
    return cache, qkv, pos, freqs(rotary) if rotary else torch.empty(0), sections, slots


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("page,group", [(16, 16), (16, 1), (32, 8), (24, 12), (24, 24), (128, 128), (7, 7), (64, 2)])
def test_append_groups(w, page, group, dtype):
    ctx, new = [0, 5, 37, 130, 3, 0, page - 1, page], [17, 1, 40, 3, 1, 150, 2, 1]
    p = append_problem(w, page + group, ctx, new, 3, 2, 64, 64, 1, page, group, TYPES[dtype], "head" if group % 8 else "token", pad=True)
    cache, qkv, pos, f, sections, slots = p
    check_append(w, cache, qkv, 3, pos[0], f, None, False, slots)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("dim,rotary,axes", [(16, 16, 1), (64, 0, 1), (80, 48, 3), (96, 96, 2), (128, 64, 4), (192, 192, 1), (256, 256, 2), (112, 16, 1), (256, 32, 1)])
def test_append_heads(w, dim, rotary, axes, inter, dtype):
    for hq, hk in ((4, 2), (0, 3), (7, 1)):
        cache, qkv, pos, f, sections, slots = append_problem(w, dim + rotary + hq, [3, 30, 0], [1, 20, 33], hq, hk, dim, rotary, axes, 32, 16, TYPES[dtype])
        check_append(w, cache, qkv, hq, pos, f, sections, inter, slots)


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 152, 700, 5000])
def test_append_numbers_of_tokens(w, T):
    cache, qkv, pos, f, sections, slots = append_problem(w, T, [9, 0], [T // 3, T - T // 3], 2, 1, 64, 64, 1, 48, 16, INT8)
    check_append(w, cache, qkv, 2, pos[0], f, None, True, slots)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_append_token_by_token(w, dtype):
    # a group filled one token at a time, its scale growing: codes stand for the values within the stated bounds
    dtype, gen = TYPES[dtype], torch.Generator().manual_seed(4)
    cache = make_cache(w, gen, 3, 16, 16, 2, 64, dtype)
    x = torch.randn(16, 2, 64, generator=gen) * torch.exp2(torch.linspace(-6, 6, 16))[torch.randperm(16, generator=gen)][:, None, None]
    x = x.bfloat16()
    for t in range(16):
        check_append(w, cache, torch.cat([x[t], x[t]]).view(1, -1), 0, torch.tensor([t]).int(), torch.empty(0), None, False, [16 + t])
    S = cache.v_scale[1, 0].double().cpu()[:, None]
    assert torch.equal(cache.k_scale[1], cache.v_scale[1])
    back = code_values(cache.v)[1] * S
    xd = x.double()
    bound = S.expand_as(xd) if dtype is INT8 else 2.0 ** -4 * xd.abs() + 2.0 ** -9 * S
    assert ((back - xd).abs() <= bound).all()
    top = xd.abs().amax((0, 2))[:, None]
    most = ref.MOST[dtype]
    assert (top <= most * S).all() and (top > most * S / 2).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "neighbours"])
def test_append_scales_at_their_borders(w, inter, dtype):
    # magnitudes that are just most * 2^e and the next above; pairs whose length passes it though neither value does
    dtype = TYPES[dtype]
    most = ref.MOST[dtype]
    rows = []
    for e in (-120, -20, 0, 3, 100):
        for a, b in ((most, 0.0), (most * (1 + 2.0 ** -6), 0.0), (most * 0.75, most * 0.75), (most * 0.6015625, most * 0.796875), (most / 2, 0.0), (0.0, 0.0)):
            rows.append((a * 2.0 ** e, b * 2.0 ** e))
    x = torch.zeros(len(rows), 1, 32)
    for t, (a, b) in enumerate(rows):
        x[t, 0, 2], x[t, 0, 3 if inter else 10] = a, -b
    x = x.bfloat16()
    cache = make_cache(w, torch.Generator().manual_seed(1), len(rows), 4, 2, 1, 32, dtype)
    pos = torch.arange(len(rows)).int()
    check_append(w, cache, torch.cat([x, x], 1).view(len(rows), -1), 0, pos, freqs(16), None, inter, [4 * t for t in range(len(rows))])


@pytest.mark.parametrize("dtype", list(TYPES))
def test_append_values_out_of_the_ordinary(w, dtype):
    # not finite: the group stands for NaN until it is begun anew, other groups and heads are as ever
    dtype, gen = TYPES[dtype], torch.Generator().manual_seed(2)
    inf, nan = float("inf"), float("nan")
    for odd in (inf, -inf, nan):
        cache = make_cache(w, gen, 4, 16, 8, 2, 32, dtype)
        x = torch.randn(12, 4, 32, generator=gen).bfloat16()
        x[3, 1, 5] = odd  # key head 1, group 0
        x[9, 2, 30] = odd  # value head 0, group 1
        f = freqs(32)
        check_append(w, cache, x.view(12, -1), 0, torch.arange(12).int(), f, None, False, list(range(16, 28)))
        assert cache.k_scale[1, 0, 1].isnan() and cache.v_scale[1, 1, 0].isnan()
        assert cache.k_scale[1].isnan().sum() == 1 and cache.v_scale[1].isnan().sum() == 1
        y = torch.randn(1, 4, 32, generator=gen).bfloat16()
        check_append(w, cache, y.view(1, -1), 0, torch.tensor([4]).int(), f, None, False, [28])
        assert cache.v_scale[1, 1, 0].isnan()
        check_append(w, cache, x[:3].reshape(3, -1), 0, torch.arange(3).int(), f, None, False, [16, 17, 18])
        assert not cache.k_scale[1, 0].isnan().any()
    # the largest and the smallest numbers, and nothing but zeros
    cache = make_cache(w, gen, 4, 16, 4, 1, 32, dtype)
    x = torch.zeros(16, 2, 32)
    x[0:4], x[4:8], x[8:12] = 3.3e38, 1e-40, 2.0 ** -126
    check_append(w, cache, x.bfloat16().view(16, -1), 0, torch.arange(16).int(), torch.empty(0), None, False, list(range(16)))


@pytest.mark.parametrize("dtype", list(TYPES))
def test_append_onto_scales_of_another_maker(w, dtype):
    # scales so far that are no powers of two, negative, zero, tiny, huge or no number
    dtype, gen = TYPES[dtype], torch.Generator().manual_seed(3)
    given = [0.03, 1.0, 1e-3, 0.0, -0.02, 1e-42, 2.0 ** -126, 3e38, float("inf"), float("nan"), 1.17e-38, 2.0 ** 127]
    cache = make_cache(w, gen, len(given), 8, 8, 1, 32, dtype)
    s = torch.tensor(given).view(-1, 1, 1).cuda()
    cache.k_scale.copy_(s), cache.v_scale.copy_(s)
    x = torch.randn(len(given), 2, 32, generator=gen).bfloat16()
    check_append(w, cache, x.view(len(given), -1), 0, torch.arange(len(given)).int(), torch.empty(0), None, False, [8 * b + 5 for b in range(len(given))])


def test_append_flags_slots(w):
    cache, qkv, pos, f, sections, slots = append_problem(w, 6, [0], [12], 2, 1, 32, 32, 1, 16, 4, INT8)
    base, block = state_of(cache), slots[0] - slots[0] % 16
    for at, bad in ((0, cache.blocks * 16), (5, -2), (11, 2 ** 31 - 1), (3, -2 ** 31)):
        s = list(slots)
        s[at] = bad
        check_append(w, cache, qkv, 2, pos[0], f, None, False, s, flags=w.DEVERR_SLOT)
    # a token in the group of the one before it that does not follow it, with what follows; the same slot twice
    for s in ([block, block + 2, block + 3, block + 4], [block + 5, block + 5], [block + 3, block + 2], [block + 1, block + 3, -1, block + 8]):
        check_append(w, cache, qkv[:len(s)], 2, pos[0, :len(s)].contiguous(), f, None, False, s, flags=w.DEVERR_SLOT)
    assert not same_bits(base, state_of(cache))


def test_append_twice_is_once(w):
    cache, qkv, pos, f, sections, slots = append_problem(w, 8, [5, 0], [1, 33], 2, 2, 64, 64, 1, 16, 16, E4M3)
    first = check_append(w, cache, qkv, 2, pos[0], f, None, False, slots)
    state = state_of(cache)
    again = check_append(w, cache, qkv, 2, pos[0], f, None, False, slots)
    assert torch.equal(first, again) and same_bits(state, state_of(cache))


def test_append_in_place_and_strides(w):
    # queries turned where they are; codes and scales inside larger allocations, what lies around them left alone
    gen = torch.Generator().manual_seed(5)
    both = torch.full((5, 16, 2, 3, 96), 77, dtype=INT8, device="cuda")
    scales = torch.full((5, 4, 2, 5), 9.0, device="cuda")
    cache = w.ScaledCache(both[:, :, 0, :, :64], both[:, :, 1, :, :64], scales[:, :, 0, :3], scales[:, :, 1, :3])
    T = 21
    qkv = torch.randn(T, (2 + 6) * 64, generator=gen).bfloat16()
    slots = list(range(20, 20 + T))
    got = check_append(w, cache, qkv, 2, torch.arange(T).int(), freqs(64), None, False, slots)
    assert (both[..., 64:] == 77).all() and (scales[..., 3:] == 9).all()
    rows = qkv.cuda()
    q, k, v = split_qkv(rows, 2, 3, 64)
    out = w.w4a16_scaled_append(q, k, v, torch.arange(T).int().cuda(), freqs(64).cuda(), i32(slots), cache, q_out=q)
    assert out is q and torch.equal(q, got)


# --------------------------------------------------------------------------
# read
# --------------------------------------------------------------------------
def check_read(w, cache, table, row_start, rows, first=None, dtype=torch.bfloat16, flags=0):
    got = [torch.full((rows, cache.heads, cache.dim), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    out = w.w4a16_scaled_read(cache, i32(table), i32(row_start), None if first is None else i32(first), *got)
    assert out[0] is got[0] and out[1] is got[1]
    assert w.w4a16_device_error(clear=True) == flags
    for codes, scales, have in ((cache.k, cache.k_scale, got[0]), (cache.v, cache.v_scale, got[1])):
        values = codes.float().cpu() * scales.cpu().repeat_interleave(cache.group, 1)[..., None]
        want = torch.full((rows, cache.heads, cache.dim), 7.0, dtype=dtype)
        for b, (i, j) in enumerate(zip(row_start, row_start[1:])):
            for r in range(i, min(j, rows)):
                p = r - i + (first[b] if first else 0)
                x = table[b][p // cache.page] if 0 <= p < len(table[b]) * cache.page else -1
                want[r] = values[x, p % cache.page].to(dtype) if 0 <= x < cache.blocks else 0
        assert torch.equal(have.cpu(), want)
    return got


def read_problem(w, seed, lens, hk, dim, page, group, dtype, layout="token", columns=0):
    rng, gen = random.Random(seed), torch.Generator().manual_seed(seed)
    blocks = sum(-(-n // page) for n in lens) + 2
    cache = make_cache(w, gen, blocks, page, group, hk, dim, dtype, layout)
    ids = list(range(blocks))
    rng.shuffle(ids)
    columns = max(columns, max(-(-n // page) for n in lens), 1)
    table = [[ids.pop() for _ in range(-(-n // page))] for n in lens]
    return cache, [r + [10 ** 9] * (columns - len(r)) for r in table], list(itertools.accumulate([0] + lens))


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dim,hk,page,group,layout", [(128, 8, 16, 16, "token"), (64, 1, 24, 8, "head"), (16, 3, 7, 1, "token"), (256, 5, 64, 64, "head"),
                                                      (80, 2, 128, 4, "token"), (96, 40, 16, 2, "token")])
def test_read(w, dim, hk, page, group, layout, dtype, out):
    lens = [1, 0, 33, page, 0, 0, 130, 0]
    cache, table, start = read_problem(w, dim + page, lens, hk, dim, page, group, TYPES[dtype], layout)
    check_read(w, cache, table, start, start[-1] + 3, dtype=out)


def test_read_parts_and_gaps(w):
    lens = [60, 40, 100]
    cache, table, _ = read_problem(w, 3, lens, 2, 64, 16, 8, INT8)
    check_read(w, cache, table, [5, 25, 25, 90], 95, first=[7, 0, 35])  # rows before the first request too
    check_read(w, cache, table, [0, 0, 0, 0], 4)
    new = w.w4a16_scaled_read(cache, i32(table), i32([0, 60, 100, 200]), rows=203, dtype=torch.float32)
    have = check_read(w, cache, table, [0, 60, 100, 200], 203, dtype=torch.float32)
    assert (new[0][200:] == 0).all() and all(torch.equal(a[:200], b[:200]) for a, b in zip(new, have))
    wide = torch.full((200, 2, 2, 96), 3.0, device="cuda").bfloat16()
    w.w4a16_scaled_read(cache, i32(table), i32([0, 60, 100, 200]), k_out=wide[:, 0, :, :64], v_out=wide[:, 1, :, :64])
    want = check_read(w, cache, table, [0, 60, 100, 200], 200)
    assert torch.equal(wide[:, 0, :, :64], want[0]) and torch.equal(wide[:, 1, :, :64], want[1]) and (wide[..., 64:] == 3).all()


@pytest.mark.parametrize("B", [255, 256, 257, 1000, 16384])
def test_read_many_requests(w, B):
    rng = random.Random(B)
    lens = [rng.choice([0, 0, 1, 2, rng.randrange(20)]) if B < 5000 else rng.choice([0, 1]) for _ in range(B)]
    cache, table, start = read_problem(w, B, lens, 1, 16, 16, 16, E4M3)
    check_read(w, cache, table, start, start[-1] + 1)


def test_read_what_is_not_there(w):
    lens = [40, 33]
    cache, table, start = read_problem(w, 4, lens, 2, 32, 16, 16, INT8)
    for bad in (-1, cache.blocks, 2 ** 31 - 1, -2 ** 31):
        t = [list(r) for r in table]
        t[0][1] = bad
        check_read(w, cache, t, start, start[-1], flags=w.DEVERR_SLOT)
    check_read(w, cache, table, start, start[-1], first=[0, -2], flags=w.DEVERR_SLOT)
    check_read(w, cache, table, start, start[-1], first=[2 ** 31 - 1, 0], flags=w.DEVERR_SLOT)
    check_read(w, cache, table, start, 50, flags=w.DEVERR_BLOCKS)  # fewer rows than tokens


# --------------------------------------------------------------------------
# attention
# --------------------------------------------------------------------------
def attention_problem(w, seed, lens, new, hq, hk, dim, page, group, dtype, layout="token", columns=None, sharp=1.5, spread=2):
    gen = torch.Generator().manual_seed(seed)
    used = [-(-n // page) for n in lens]
    blocks = sum(used) + 3
    cache = make_cache(w, gen, blocks, page, group, hk, dim, dtype, layout, spread)
    order = torch.randperm(blocks, generator=gen).tolist()
    columns = columns or max(max(used), 1)
    table = [[order.pop() for _ in range(u)] + [10 ** 9] * (columns - u) for u in used]
    q = (sharp * torch.randn(len(lens), new, hq, dim, generator=gen)).bfloat16()
    forget(cache, table, [range(n) for n in lens])
    return q, cache, table


def forget(cache, table, seen):
    """What no request sees is not a number: e4m3 codes, and scales of groups nobody sees any of."""
    page, group = cache.page, cache.group
    mark = torch.zeros(cache.blocks, page, dtype=torch.bool)
    for r, js in zip(table, seen):
        for j in js:
            mark[r[j // page], j % page] = True
    hole = (~mark).cuda().view(cache.blocks, page, 1, 1)
    lost = (~mark.view(cache.blocks, -1, group).any(2)).cuda()[:, :, None]
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        raw(c).masked_fill_(hole, 0x7F)
        s.masked_fill_(lost, float("nan"))


def check_attention(w, q, cache, table, lens, scale=None, window=0, flags=0, got=None):
    dim, new = q.shape[3], q.shape[1]
    scale = dim ** -0.5 if scale is None else scale
    if got is None:
        got = w.w4a16_scaled_attention(q.cuda(), cache, i32(table), i32(lens), scale=scale, window=window)
    assert w.w4a16_device_error(clear=True) == flags
    out, lse = got[0].double().cpu().view(q.shape), got[1].double().cpu().view(q.shape[:3])
    ks, vs = cache.k_scale.double().cpu(), cache.v_scale.double().cpu()
    want, want_lse, spread, reach, low = ref.attention(q.double(), code_values(cache.k), code_values(cache.v), ks, vs, table, lens, scale, window, cache.group)
    score = (dim + 16) * 2.0 ** -24 * reach
    logs = torch.log2(torch.where(vs.isfinite() & (vs != 0), vs, 1.0).abs()).abs().max()
    tol = U * want.abs() + (2.0 ** -11 + 2 * score[..., None] + 2.0 ** -22 * (8 + logs)) * spread + 2.0 ** -33 * low + 1e-37
    assert not out.isnan().any()
    assert ((out - want).abs() <= tol).all(), float(((out - want).abs() / tol).max())
    empty = want_lse == -float("inf")
    assert torch.equal(lse == -float("inf"), empty)
    d = (lse - want_lse)[~empty].abs()
    assert (d <= (score + 2.0 ** -21 * (1 + want_lse.abs()))[~empty].clamp(min=2.0 ** -21)).all(), float(d.max())
    assert (out[empty] == 0).all()
    return got


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 64, 65, 127, 129, 200, 257]
SHAPES = [(128, 16, 16), (64, 24, 8), (256, 64, 64), (80, 8, 4), (96, 7, 7), (16, 1, 1), (192, 128, 32), (112, 48, 1)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("new", [1, 3])
@pytest.mark.parametrize("dim,page,group", SHAPES)
def test_attention_lengths_dims_pages(w, dim, page, group, new, dtype):
    for layout in ("token", "head"):
        q, cache, table = attention_problem(w, dim + page, LENS, new, 4, 2, dim, page, group, TYPES[dtype], layout)
        check_attention(w, q, cache, table, LENS)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("new", [1, 2, 5, 16])
@pytest.mark.parametrize("hq,hk", [(1, 1), (5, 5), (6, 2), (4, 1), (8, 1), (9, 1), (16, 1), (17, 1), (40, 8)])
def test_attention_head_groups(w, hq, hk, new, dtype):
    lens = [3, 0, 90, 161]
    q, cache, table = attention_problem(w, hq * 7 + hk, lens, new, hq, hk, 64, 16, 8, TYPES[dtype])
    check_attention(w, q, cache, table, lens)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("new", [1, 4])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 1000000, 2 ** 31 - 1])
def test_attention_window(w, window, new, dtype):
    lens = [0, 1, 2, 3, 15, 17, 33, 64, 129, 500]
    q, cache, table = attention_problem(w, window % 997, lens, new, 4, 2, 128, 16, 4, TYPES[dtype])
    # what lies before every window is not read either
    forget(cache, table, [range(max(0, n - (new - 1) - window), n) for n in lens])
    check_attention(w, q, cache, table, lens, window=window)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dim,hq,hk,page,group,new", [(128, 8, 2, 16, 16, 1), (64, 4, 4, 24, 8, 2), (256, 16, 1, 16, 1, 1), (128, 8, 2, 64, 64, 5), (192, 3, 1, 32, 16, 4)])
@pytest.mark.parametrize("lens", [[20000], [9001, 1], [0, 5000, 0, 12345, 3]], ids=str)
def test_attention_long(w, lens, dim, hq, hk, page, group, new, dtype):
    q, cache, table = attention_problem(w, 3, lens, new, hq, hk, dim, page, group, TYPES[dtype])
    check_attention(w, q, cache, table, lens)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("group,new", [(1, 1), (3, 1), (8, 1), (9, 1), (16, 1), (17, 1), (3, 4), (5, 3)])
@pytest.mark.parametrize("dim", [16, 64, 80, 96, 128, 160, 192, 256])
def test_attention_shares_and_join(w, dim, group, new, dtype):
    # wide tables: the rows' tiles are dealt in shares and joined
    lens = [0, 1, 700, 33, 1500]
    page, of, layout = (16, 16, "token") if (dim + group) % 3 else (24, 8, "head")
    q, cache, table = attention_problem(w, dim * 32 + group, lens, new, 2 * group if dim < 128 else group, 2 if dim < 128 else 1, dim, page, of, TYPES[dtype], layout,
                                        columns=4096)
    check_attention(w, q, cache, table, lens)
    check_attention(w, q, cache, table, lens, window=9000)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dim,group,new", [(64, 9, 1), (128, 4, 4), (240, 10, 1), (256, 16, 1)])
def test_attention_shares_inside_a_window(w, dim, group, new, dtype):
    lens = [12000, 9005]
    q, cache, table = attention_problem(w, dim + group, lens, new, group, 1, dim, 16, 16, TYPES[dtype])
    check_attention(w, q, cache, table, lens, window=8999)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("group,new", [(4, 6), (8, 3), (4, 8), (2, 16)])
def test_attention_24_and_32_columns_together(w, group, new, dim, dtype):
    # long rows: a CTA's warps join inside of one; short ones: in their CTA
    lens = [20011, 5, 0, 1999]
    q, cache, table = attention_problem(w, dim + group, lens, new, group, 1, dim, 32, 8, TYPES[dtype])
    check_attention(w, q, cache, table, lens)
    check_attention(w, q, cache, table, lens, window=1000)
    # the workspace of more new tokens serves fewer
    ws = w.scaled_attention_workspace(cache, group, 16)
    got = w.w4a16_scaled_attention(q.cuda(), cache, i32(table), i32(lens), workspace=ws, out=torch.empty_like(q, device="cuda"),
                                   lse=torch.empty(q.shape[:3], device="cuda"))
    check_attention(w, q, cache, table, lens, got=got)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("dim,hq,hk,requests", [(128, 16, 8, 5), (64, 20, 20, 3), (192, 7, 7, 4), (128, 6, 3, 9), (256, 9, 9, 200), (64, 4, 2, 130), (128, 8, 8, 320), (16, 17, 17, 2)])
def test_attention_teams(w, dim, hq, hk, requests, dtype):
    # a token's heads next to one another, wide tables: the warps of an SM take the same shares of a
    # request's heads; warps are left over where the heads do not divide them
    rng = random.Random(dim + hk)
    some = [0, 1, 700, 33, 0, 1500, 64, 2100, 31, 32]
    lens = [some[i] if i < 10 else rng.choice([0, 3, 17, 40, 90]) for i in range(requests)]
    q, cache, table = attention_problem(w, dim + hq, lens, 1, hq, hk, dim, 16, 16, TYPES[dtype], columns=4096)
    check_attention(w, q, cache, table, lens)
    check_attention(w, q, cache, table, lens, window=32769)


def test_attention_many_requests(w):
    rng = random.Random(4)
    lens = [rng.choice([0, 1, 5, rng.randrange(120)]) for _ in range(700)]
    q, cache, table = attention_problem(w, 9, lens, 2, 4, 2, 64, 16, 16, INT8)
    check_attention(w, q, cache, table, lens)
    q, cache, table = attention_problem(w, 9, [0, 0, 0], 2, 4, 2, 64, 16, 16, INT8)
    check_attention(w, q, cache, table, [0, 0, 0])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("group", [1, 16, 32])
def test_attention_scales_far_apart(w, group, dtype):
    # values' scales from 2^-47 to 2^35: weights by the largest p would pass fp16's range or vanish in it
    for lens, columns, sharp in (([300, 17, 90], None, 1.5), ([900, 1200], 4096, 1.5), ([300, 90], None, 15.0)):
        q, cache, table = attention_problem(w, 31, lens, 1, 4, 2, 64, 32, group, TYPES[dtype], columns=columns, sharp=sharp, spread=40)
        check_attention(w, q, cache, table, lens)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_attention_scales_of_another_maker(w, dtype):
    # any scales: no powers of two, negative, zero, subnormal
    lens = [80, 33]
    q, cache, table = attention_problem(w, 33, lens, 2, 4, 2, 64, 16, 4, TYPES[dtype])
    gen = torch.Generator().manual_seed(1)
    for s in (cache.k_scale, cache.v_scale):
        x = 0.05 * torch.randn(s.shape, generator=gen).cuda()
        x[torch.rand(s.shape, generator=gen).cuda() < 0.1] = 0
        x[torch.rand(s.shape, generator=gen).cuda() < 0.1] = 1e-41
        s.copy_(torch.where(s.isnan(), s, x))
    check_attention(w, q, cache, table, lens)
    cache.v_scale.copy_(torch.where(cache.v_scale.isnan(), cache.v_scale, 0.0))
    out, lse = w.w4a16_scaled_attention(q.cuda(), cache, i32(table), i32(lens))
    assert (out == 0).all() and lse.isfinite().all()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_attention_large_scores(w, dtype):
    lens = [300, 17]
    for sharp in (600.0, 1e-20):
        q, cache, table = attention_problem(w, 31, lens, 2, 8, 2, 128, 16, 16, TYPES[dtype], sharp=sharp)
        check_attention(w, q, cache, table, lens)


@pytest.mark.parametrize("columns", [None, 4096])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_attention_nan_stays_with_those_that_see_it(w, dtype, columns):
    # new tokens 0..3 see 47, 48, 49, 50 tokens; window 20 begins at 27, 28, 29, 30
    for where, window, hit in ((48, 0, [2, 3]), (49, 0, [3]), (10, 0, [0, 1, 2, 3]), (28, 20, [0, 1]), (27, 20, [0]), (26, 20, []), (30, 20, [0, 1, 2, 3])):
        for part in ("k code", "v code", "k scale", "v scale"):
            if part.endswith("code") and dtype == "int8":
                continue
            q, cache, table = attention_problem(w, 14, [50, 20], 4, 4, 2, 64, 16, 1, TYPES[dtype], columns=columns)
            block, place = table[0][where // 16], where % 16
            if part.endswith("code"):
                raw(cache.k if part[0] == "k" else cache.v)[block, place, 0, 7] = 0xFF
            else:
                (cache.k_scale if part[0] == "k" else cache.v_scale)[block, place, 0] = float("nan")
            out, lse = w.w4a16_scaled_attention(q.cuda(), cache, i32(table), i32([50, 20]), window=window)
            nan = torch.zeros(2, 4, 4, 64, dtype=torch.bool)
            nan[0, hit, :2, slice(7, 8) if part == "v code" else slice(None)] = True
            if part == "v code":  # the weight of a token with a NaN is NaN where others do not see it: all of its head's values
                assert (out.isnan().cpu() | ~nan).all() and not out[1].isnan().any() and not out[:, :, 2:].isnan().any()
                assert torch.equal(out[0].isnan().any(-1).cpu()[:, :2], nan[0].any(-1)[:, :2])
            else:
                assert torch.equal(out.isnan().cpu(), nan), (part, where, window)
            assert torch.equal(lse.isnan().cpu(), nan.any(-1) if part[0] == "k" else torch.zeros_like(nan[..., 0]))


def test_attention_strides(w):
    lens = [70, 5, 131]
    q, cache, table = attention_problem(w, 21, lens, 2, 6, 2, 64, 16, 8, INT8)
    want = check_attention(w, q, cache, table, lens)
    row = torch.full((3, 2, 10 * 64), 9.0).bfloat16().cuda()  # a fused projection's rows: queries first
    row[..., :6 * 64] = q.flatten(2).cuda()
    out = torch.full((3, 2, 8, 6, 64), 5.0).bfloat16().cuda()
    wide = torch.full((3, 20), 10 ** 9, dtype=torch.int32, device="cuda")
    wide[:, :len(table[0])] = i32(table)
    got = w.w4a16_scaled_attention(row[..., :6 * 64].view(3, 2, 6, 64), cache, wide[:, :len(table[0])], i32([0] + lens)[1:], out=out[:, :, 3])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and (out[:, :, :3] == 5).all() and (out[:, :, 4:] == 5).all()
    # new tokens before requests, and heads before both, in memory
    for order in ((1, 0, 2, 3), (2, 1, 0, 3)):
        other = q.cuda().permute(order).contiguous().permute(order)
        again = w.w4a16_scaled_attention(other, cache, i32(table), i32(lens))
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    # one token without the dimension of new ones
    a = w.w4a16_scaled_attention(q[:, 0].cuda(), cache, i32(table), i32(lens))
    b = w.w4a16_scaled_attention(q[:, :1].cuda(), cache, i32(table), i32(lens))
    assert a[0].shape == (3, 6, 64) and a[1].shape == (3, 6) and torch.equal(a[0], b[0][:, 0]) and torch.equal(a[1], b[1][:, 0])
    # scales that all groups share (a stride of 0)
    one = torch.full((1, 1, 2), 0.03, device="cuda").expand(cache.blocks, 2, 2)
    check_attention(w, q, w.ScaledCache(cache.k, cache.v, one, one), table, lens)


def test_attention_bad_blocks_and_lengths(w):
    lens = [70, 100, 33]
    q, cache, table = attention_problem(w, 12, [112, 112, 33], 2, 4, 2, 64, 16, 16, E4M3)
    for bad in (-1, cache.blocks, 2 ** 31 - 1, -2 ** 31):
        t = [list(r) for r in table]
        t[1][2] = bad
        t[2] = [bad] * len(t[2])
        check_attention(w, q, cache, t, lens, flags=w.DEVERR_SLOT)
    check_attention(w, q, cache, table, [70, 112 + 9, -4], flags=w.DEVERR_SLOT)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_offsets_past_32_bits(w, dtype):
    # element offsets beyond 2^32: only the blocks in use are written
    hk, dim, page, dtype = 8, 128, 16, TYPES[dtype]
    blocks = (1 << 32) // (hk * dim * page) + 300
    t = torch.empty((blocks, page, hk, dim), dtype=torch.uint8, device="cuda").view(dtype)
    scales = torch.empty(blocks, 1, hk, device="cuda")
    lens = [200, 77]
    q, small, table = attention_problem(w, 3, lens, 2, 16, hk, dim, page, page, dtype)
    far = blocks - small.blocks
    cache = w.ScaledCache(t, t, scales, scales)  # one memory for both
    raw(t)[far:], scales[far:] = raw(small.k), small.k_scale
    one = w.ScaledCache(small.k, small.k, small.k_scale, small.k_scale)
    moved = [[x + far if x < 10 ** 9 else x for x in r] for r in table]
    a = w.w4a16_scaled_attention(q.cuda(), one, i32(table), i32(lens))
    b = w.w4a16_scaled_attention(q.cuda(), cache, i32(moved), i32(lens))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = w.w4a16_scaled_read(one, i32(table), i32([0, 200, 277]), rows=277)
    b = w.w4a16_scaled_read(cache, i32(moved), i32([0, 200, 277]), rows=277)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x = torch.randn(5, hk, dim, device="cuda").bfloat16()
    args = x, x, torch.zeros(5, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda")
    w.w4a16_scaled_append(None, *args, i32([(far + b) * page for b in range(5)]), cache)
    w.w4a16_scaled_append(None, *args, i32([b * page for b in range(5)]), one)
    assert torch.equal(raw(t)[far:far + 5, 0], raw(small.k)[:5, 0]) and torch.equal(scales[far:far + 5], small.k_scale[:5])
    assert w.w4a16_device_error(clear=True) == 0


# --------------------------------------------------------------------------
# the three together
# --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", list(TYPES))
def test_a_request_from_prompt_to_drafts(w, dtype):
    """Map, append, read and attention as a serving loop runs them: prompts, single tokens, then drafts of which some are
    taken back; what attention gives is that of the keys and values read back."""
    dtype, gen = TYPES[dtype], torch.Generator().manual_seed(11)
    hq, hk, dim, page, group, B = 8, 2, 64, 16, 8, 3
    blocks, columns = 40, 12
    cache = w.ScaledCache(*(torch.empty(blocks, page, hk, dim, dtype=dtype, device="cuda") for _ in range(2)),
                          *(torch.empty(blocks, page // group, hk, device="cuda") for _ in range(2)))
    table = torch.full((B, columns), -1, dtype=torch.int32, device="cuda")
    free, head = torch.randperm(blocks, generator=gen).int().cuda(), i32([0])
    lengths, f = i32([0] * B), freqs(dim).cuda()
    keys = [[torch.empty(0, hk, dim, dtype=torch.float64) for _ in range(2)] for _ in range(B)]
    for step, new in enumerate(([37, 5, 0], [1, 1, 1], [1, 1, 1], [4, 4, 4], [1, 1, 1], [4, 4, 4])):
        T = sum(new)
        m = w.w4a16_paged_map(lengths, i32(new), table, free, head, page, blocks, T + 2)
        qkv = torch.randn(T + 2, (hq + 2 * hk) * dim, generator=gen).bfloat16()
        q, k, v = split_qkv(qkv.cuda(), hq, hk, dim)
        q = w.w4a16_scaled_append(q, k, v, m.positions, f, m.slots, cache)
        at = 0
        turned = ref.rope(k.double().cpu(), m.positions.cpu()[None].clamp(min=0), f.cpu(), [dim // 2], False)
        for b, n in enumerate(new):
            keys[b] = [torch.cat([old, x[at:at + n]]) for old, x in zip(keys[b], (turned, v.double().cpu()))]
            at += n
        total = [len(x[0]) for x in keys]
        assert m.kv_len.tolist() == total
        start = list(itertools.accumulate([0] + total))
        read = [x.double().cpu() for x in w.w4a16_scaled_read(cache, table, i32(start), rows=start[-1], dtype=torch.float32)]
        for b, (i, j) in enumerate(zip(start, start[1:])):
            for have, want, scales in ((read[0][i:j], keys[b][0], cache.k_scale), (read[1][i:j], keys[b][1], cache.v_scale)):
                S = torch.stack([scales[table[b, p // page], p % page // group] for p in range(j - i)]).double().cpu()[..., None] if j > i else 0
                bound = S * torch.ones_like(want) if dtype is INT8 else 2.0 ** -4 * want.abs() + 2.0 ** -9 * S
                assert ((have - want).abs() <= bound * (1 + 2.0 ** -16)).all(), (step, b)
        if min(new) == max(new):
            n = new[0]
            check_attention(w, q[:T].view(B, n, hq, dim).cpu(), cache, table.tolist(), total,
                            got=w.w4a16_scaled_attention(q[:T].view(B, n, hq, dim), cache, table, m.kv_len))
        lengths, head = m.kv_len.clone(), m.free_head.clone()
        if step == 3:  # two of each request's drafts are not taken; their blocks stay in the table
            lengths -= 2
            keys = [[x[:-2] for x in pair] for pair in keys]
            before = -(-(lengths + 2) // page)
            after = -(-lengths // page)
            head -= (before - after).sum().int()
            taken = [int(table[b, c]) for b in range(B) for c in range(int(after[b]), int(before[b]))]
            free[int(head):int(head) + len(taken)] = i32(taken)
    assert w.w4a16_device_error(clear=True) == 0


def test_graph_capture_and_replay(w):
    lens = [300, 40, 0]
    q, cache, table = attention_problem(w, 8, lens, 2, 4, 2, 64, 16, 16, INT8)
    x = torch.randn(3, 4 + 4, 64).bfloat16().cuda()
    slots, pos = i32([table[b][n // 16] * 16 + n % 16 if n else -1 for b, n in enumerate(lens)]), i32(lens)
    f, dq, t, n = freqs(64).cuda(), q.cuda(), i32(table), i32(lens)
    ws = w.scaled_attention_workspace(cache, 4, 2)

    start = i32([0, 300, 340, 340])

    def step(stream=None):
        y = w.w4a16_scaled_append(x[:, :4], x[:, 4:6], x[:, 6:], pos, f, slots, cache, stream=stream)
        return [y, *w.w4a16_scaled_attention(dq, cache, t, n, workspace=ws, stream=stream), *w.w4a16_scaled_read(cache, t, start, rows=341, stream=stream)]

    want = step()
    state = state_of(cache)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for g in got:
            g.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and same_bits(state, state_of(cache))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and same_bits(state, state_of(cache))


def test_attention_repeats_and_leaves_its_workspace(w):
    lens = [3000, 1, 0, 777]
    q, cache, table = attention_problem(w, 41, lens, 3, 8, 2, 128, 16, 16, INT8)
    ws = w.scaled_attention_workspace(cache, 8, 3)
    args = (q.cuda(), cache, i32(table), i32(lens))
    first = w.w4a16_scaled_attention(*args, workspace=ws)
    for n in ([3000, 1, 0, 777], [5, 1, 0, 700]):
        w.w4a16_scaled_attention(q.cuda(), cache, i32(table), i32(n), workspace=ws)
        again = w.w4a16_scaled_attention(*args, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    check_attention(w, q, cache, table, lens, got=first)


# --------------------------------------------------------------------------
# refusals
# --------------------------------------------------------------------------
def test_refusals(w):
    lens = [40, 3]
    q, cache, table = attention_problem(w, 2, lens, 2, 4, 2, 64, 16, 8, INT8)
    x = torch.randn(5, 2, 64, device="cuda").bfloat16()
    S = w.Status
    before = state_of(cache)
    bases = {
        w.w4a16_scaled_attention: dict(q=q.cuda(), cache=cache, block_table=i32(table), kv_len=i32(lens), workspace=w.scaled_attention_workspace(cache, 4, 2)),
        w.w4a16_scaled_append: dict(q=x, k=x, v=x, positions=i32(range(5)), inv_freq=freqs(64).cuda(), slots=i32(range(5)), cache=cache),
        w.w4a16_scaled_read: dict(cache=cache, block_table=i32(table), row_start=i32([0, 40, 43]), rows=43),
    }
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")
    shared = w.ScaledCache(cache.k, cache.v, cache.k_scale[:1, :, :].expand(cache.blocks, 2, 2), cache.v_scale)
    for call, bad, status in (
            (w.w4a16_scaled_attention, dict(q=q[:, :, :3].cuda()), S.ERR_SHAPE), (w.w4a16_scaled_attention, dict(window=-1), S.ERR_SHAPE),
            (w.w4a16_scaled_attention, dict(workspace=z(8, dtype=torch.uint8)), S.ERR_WORKSPACE),
            (w.w4a16_scaled_attention, dict(q=z(2, 17, 4, 64)), S.ERR_UNSUPPORTED),
            (w.w4a16_scaled_attention, dict(q=z(2, 2, 4 * 64 + 4)[..., :256].view(2, 2, 4, 64)), S.ERR_ALIGN),
            (w.w4a16_scaled_append, dict(inv_freq=freqs(64)[:12].cuda()), S.ERR_SHAPE), (w.w4a16_scaled_append, dict(sections=[31]), S.ERR_SHAPE),
            (w.w4a16_scaled_append, dict(cache=shared), S.ERR_UNSUPPORTED),
            (w.w4a16_scaled_append, dict(q=z(5, 2 * 64 + 4)[:, :128].view(5, 2, 64)), S.ERR_ALIGN),
            (w.w4a16_scaled_read, dict(block_table=i32([[0]] * 16385), row_start=i32([0] * 16386)), S.ERR_UNSUPPORTED)):
        with pytest.raises(w.W4A16Error) as e:
            call(**{**bases[call], **bad})
        assert e.value.status == status, bad
    for call, bad in (
            (w.w4a16_scaled_attention, dict(q=q)), (w.w4a16_scaled_attention, dict(q=q.cuda().half())), (w.w4a16_scaled_attention, dict(kv_len=i32([1]))),
            (w.w4a16_scaled_attention, dict(out=z(2, 1, 4, 64))), (w.w4a16_scaled_attention, dict(out=z(2, 4, 64))), (w.w4a16_scaled_attention, dict(lse=z(2, 4))),
            (w.w4a16_scaled_attention, dict(q=q[..., :32].cuda())), (w.w4a16_scaled_attention, dict(block_table=i32(table)[:1])),
            (w.w4a16_scaled_append, dict(k=x[:3])), (w.w4a16_scaled_append, dict(q=x[:3])), (w.w4a16_scaled_append, dict(sections=[16, 16])),
            (w.w4a16_scaled_append, dict(slots=i32(range(5)).long())), (w.w4a16_scaled_append, dict(v=x.float())), (w.w4a16_scaled_append, dict(q_out=x[:2])),
            (w.w4a16_scaled_read, dict(rows=None)), (w.w4a16_scaled_read, dict(dtype=torch.float16)), (w.w4a16_scaled_read, dict(row_start=i32([0, 40]))),
            (w.w4a16_scaled_read, dict(k_out=z(43, 2, 64))), (w.w4a16_scaled_read, dict(k_out=z(43, 2, 64), v_out=z(43, 2, 64, dtype=torch.float32))),
            (w.w4a16_scaled_read, dict(k_out=z(43, 2, 32), v_out=z(43, 2, 32))), (w.w4a16_scaled_read, dict(k_out=z(44, 2, 64), v_out=z(44, 2, 64)))):
        with pytest.raises((ValueError, TypeError)):
            call(**{**bases[call], **bad})
    other = w.PagedCache(z(2, 16, 2, 64), z(2, 16, 2, 64))
    for call, base in bases.items():
        with pytest.raises(TypeError):
            call(**{**base, "cache": other})
    k, s = cache.k, cache.k_scale
    for bad in ((k.float(), k.float(), s, s), (k, k[:1], s, s), (k.cpu(), k.cpu(), s, s), (k, k, s[:, :, :1], s), (k, k, s, s.double()), (k, k, s[:1], s[:1]),
                (k, k, z(cache.blocks, 3, 2, dtype=torch.float32), z(cache.blocks, 3, 2, dtype=torch.float32)), (k, k, s, None), (k.transpose(2, 3), k, s, s)):
        with pytest.raises((ValueError, TypeError)):
            w.ScaledCache(*bad)
    assert same_bits(before, state_of(cache)) and w.w4a16_device_error(clear=True) == 0
