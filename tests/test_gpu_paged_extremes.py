"""The paged-cache operators at the ends of the number ranges.

Attention with scores of 2^20 to 2^30: there fp32 scores are whole numbers or
coarser, so a test with arbitrary keys says nothing.  Here every query and key
value is 2^a or 1.25 * 2^a, so products, their sums and the scores are exact,
the tokens at the top score exactly alike and all others at least 2^18 lower.
The weights are then 1/n and 0, and out is the mean of n values:
  out: one rounding to bf16 (2^-8), and the fp32 sums of up to 20 tiles with
       their joining and quotient (32 roundings of 2^-22 of the mean size);
  lse: score + log n, from a few fp32 roundings (2^-21 of it)."""
import pytest
import torch

from .test_gpu_paged import U, i32, w  # noqa: F401  (w: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("columns", [0, 4096], ids=["own table", "wide table"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("top", [2.0 ** 20, 2.0 ** 23, 2.0 ** 24, 1.25 * 2.0 ** 24, 2.0 ** 25, 1.25 * 2.0 ** 26, 2.0 ** 28, 1.25 * 2.0 ** 28, 2.0 ** 30])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_attention_very_large_scores(w, dtype, top, sign, columns):
    dim, page, hk, group, lens = 64, 16, 2, 3, [1, 7, 40, 300]
    gen = torch.Generator().manual_seed(int(top) % 1000)
    used = [-(-n // page) for n in lens]
    blocks = sum(used)
    order = torch.randperm(blocks, generator=gen).tolist()
    width = columns or max(used)
    table = [[order.pop() for _ in range(u)] + [-1] * (width - u) for u in used]
    kind = torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn
    k = torch.zeros(blocks, page, hk, dim)
    v = torch.randn(blocks, page, hk, dim, generator=gen).mul(8).to(kind)
    # key values of sign * 1 or sign * 1/2 (of the row's largest score: 1 where positive, 1/2 where negative)
    best = {}
    for b, n in enumerate(lens):
        first = torch.rand(n, hk, generator=gen) < 0.3
        first[n // 2] = True
        for j in range(n):
            large = first[j] if sign > 0 else ~first[j]
            k[table[b][j // page], j % page] = torch.where(large, 1.0, 0.5)[:, None] * sign
        best[b] = first
    scores = top if sign > 0 else -top / 2
    q = torch.full((len(lens), hk * group, dim), top / dim).bfloat16()
    assert (q.double() * dim == top).all()
    cache = w.PagedCache(k.to(kind).cuda(), v.cuda(), *([torch.ones(hk, device="cuda") for _ in range(2)] if dtype == "fp8" else []))
    out, lse = w.w4a16_paged_attention(q.cuda(), cache, i32(table), i32(lens), scale=1.0)
    assert w.w4a16_device_error(clear=True) == 0
    values = v.float().double()
    for b, n in enumerate(lens):
        rows = torch.stack([values[table[b][j // page], j % page] for j in range(n)])  # [n, hk, dim]
        for h in range(hk * group):
            mine = rows[best[b][:, h // group], h // group]
            want, size = mine.mean(0), mine.abs().mean(0)
            got = out[b, h].double().cpu()
            assert ((got - want).abs() <= U * want.abs() + 2.0 ** -17 * size).all(), (b, h)
            exact = scores + torch.log(torch.tensor(float(len(mine)), dtype=torch.float64))
            assert abs(lse[b, h].double().cpu() - exact) <= 2.0 ** -21 * abs(exact), (b, h)


SCALES = [0.0, -0.0, 2.0 ** -149, 2.0 ** -130, 1.5 * 2.0 ** -127, 2.0 ** -126, 1.1 * 2.0 ** -100, 2.0 ** -60, 0.037, -0.25, 2.0 ** 60, 1.3 * 2.0 ** 100,
          1.7 * 2.0 ** 120, 2.0 ** 127, float("inf"), float("nan")]


def test_append_of_any_scale(w):
    # a head for every scale; codes equal to those of the fp32 quotient, not-a-numbers where that is none
    heads, dim, tokens = len(SCALES), 64, 24
    scale = torch.tensor(SCALES)
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(tokens, heads, dim, generator=gen) * 2.0 ** torch.randint(-12, 9, (tokens, heads, dim), generator=gen)
    near = torch.where(scale.isfinite() & (scale != 0), scale.abs(), 1.0)[:, None]
    x[:16] *= near  # quotients of a size that the codes hold
    x[16, :, 32:40] = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), 3e38, -1e-40, 2.0 ** -133])
    x = x.bfloat16()
    kv = [torch.zeros(2, 16, heads, dim, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    cache = w.PagedCache(*kv, scale.cuda(), scale.cuda())
    w.w4a16_rope_append(None, x.cuda(), x.cuda(), i32([0] * tokens), torch.ones(0, device="cuda"), i32(list(range(tokens))), cache)
    assert w.w4a16_device_error(clear=True) == 0
    quotient = x.float() / scale[:, None]
    want = quotient.clamp(-448, 448).to(torch.float8_e4m3fn)
    for c in kv:  # no pair is turned: keys are stored as values are
        got = c.cpu().view(32, heads, dim)[:tokens]
        nan = quotient.isnan()
        assert torch.equal(got.float().isnan(), nan)
        differ = (got.view(torch.uint8) != want.view(torch.uint8)) & ~nan
        assert not differ.any(), differ.nonzero()[:8]
