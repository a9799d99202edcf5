"""Calls over an 8-bit paged cache with scales by group whose inputs lie at the edge of
what the interface allows."""
import pytest
import torch

from .scaled_slots import stored
from .test_gpu_paged import freqs, i32, split_qkv, w  # noqa: F401  (w: the fixture)
from .test_gpu_scaled import E4M3, TYPES, U, attention_problem, check_append, code_values, make_cache, raw, same_bits, state_of

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------
# attention: value codes that are no number
# --------------------------------------------------------------------------
def with_code(w, q, cache, table, lens, window, where, code):
    """Attention with one value code (token `where` of request 0, head 0, dim 7) set to `code`, and that code put back."""
    at = raw(cache.v)[table[0][where // cache.page], where % cache.page, 0, 7:8]
    before = at.clone()
    at.fill_(code)
    got = w.w4a16_scaled_attention(q.cuda(), cache, i32(table), i32(lens), window=window)
    at.copy_(before)
    return got


# (dim, page, group): a scale a box, a scale or two tokens, one by one beside tensor copies, no boxes; rows of 64, 128 and 256 bytes
@pytest.mark.parametrize("columns", [None, 4096], ids=["one launch", "shares"])
@pytest.mark.parametrize("dim,page,group", [(64, 16, 16), (128, 32, 32), (96, 16, 1), (128, 32, 2), (64, 24, 12), (80, 7, 7), (256, 16, 16), (192, 64, 4)])
def test_a_nan_value_reaches_the_one_new_token_that_sees_it(w, dim, page, group, columns):
    # 150 tokens: the last step partly filled from 128 or 144 on; window 45 begins at 105, inside a step
    lens = [150, 20]
    q, cache, table = attention_problem(w, dim + page, lens, 1, 4, 2, dim, page, group, E4M3, columns=columns)
    for window, seen, unseen in ((0, (0, 10, 127, 128, 144, 149), ()), (45, (105, 111, 130, 149), (104, 96, 3))):
        for where in seen + unseen:
            want = with_code(w, q, cache, table, lens, window, where, 0x00)
            for code in (0x7F, 0xFF):
                out, lse = with_code(w, q, cache, table, lens, window, where, code)
                nan = torch.zeros_like(out, dtype=torch.bool)
                nan[0, 0, :2, 7] = where in seen
                assert torch.equal(out.isnan(), nan), (where, window)
                # the rest is what it is with a code of 0, bit for bit
                assert torch.equal(out.masked_fill(nan, 0.0), want[0].masked_fill(nan, 0.0)) and torch.equal(lse, want[1])
    assert w.w4a16_device_error(clear=True) == 0


@pytest.mark.parametrize("columns", [None, 4096], ids=["one launch", "shares"])
@pytest.mark.parametrize("dim,page,group", [(64, 16, 16), (128, 32, 2), (80, 7, 7), (256, 16, 16)])
@pytest.mark.parametrize("new,hq", [(4, 4), (8, 8), (7, 8)])
def test_a_nan_value_reaches_all_new_tokens_that_see_it(w, new, hq, dim, page, group, columns):
    # new token i of N sees 150 - (N - 1 - i) tokens
    lens = [150, 20]
    q, cache, table = attention_problem(w, dim + page, lens, new, hq, 2, dim, page, group, E4M3, columns=columns)
    most = 448 * float(cache.v_scale.nan_to_num(0.0).abs().max())
    for window in (0, 45):
        for where in (10, 128, 150 - new, 149, 105, 102, 96):
            want = with_code(w, q, cache, table, lens, window, where, 0x00)[0]
            out = with_code(w, q, cache, table, lens, window, where, 0x7F)[0]
            ends = [150 - (new - 1 - i) for i in range(new)]
            hit = torch.tensor([where < end and (not window or where >= end - window) for end in ends]).cuda()
            half = hq // 2  # query heads of head 0
            assert out[0, hit, :half, 7].isnan().all()
            assert not out[1].isnan().any() and not out[0, ~hit].isnan().any() and not out[0, :, half:].isnan().any()
            if where < 150 - new and (not window or where >= 150 - window):  # all of them see it: nothing but its dim
                assert int(out.isnan().sum()) == new * half
            # whoever does not see it: twice the error of one call, 2^-8 of the result and 2^-10 of a value at most
            for a, b in ((out[1], want[1]), (out[0, ~hit], want[0, ~hit]), (out[0, :, half:], want[0, :, half:])):
                assert ((a - b).abs().double() <= 2 * (U * b.abs().double() + 2.0 ** -10 * most)).all()
    assert w.w4a16_device_error(clear=True) == 0


# --------------------------------------------------------------------------
# append: pairs longer than the largest float
# --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("rotary", [32, 64])
def test_keys_longer_than_a_float_holds_are_turned(w, rotary, inter, dtype):
    gen = torch.Generator().manual_seed(rotary)
    T, hk, dim = 40, 2, 64
    x = torch.randn(T, 2 * hk, dim, generator=gen).sign() * 3.3e38
    x[5:9] *= torch.rand(4, 2 * hk, dim, generator=gen)
    x[20] = 1.0  # beside values of ordinary size, in one group and alone
    x[24:28] = torch.randn(4, 2 * hk, dim, generator=gen)
    cache = make_cache(w, gen, 4, 16, 4, hk, dim, TYPES[dtype])
    check_append(w, cache, x.bfloat16().view(T, -1), 0, torch.arange(T).int() * 997, freqs(rotary), None, inter, list(range(16, 16 + T)))


# --------------------------------------------------------------------------
# append: slots that do not follow one another
# --------------------------------------------------------------------------
def check_slots(w, page, group, hk, dim, slots, blocks, seed, dtype):
    """What the tokens that are stored give, and nothing of the others: the same cache, bit for bit, as
    with -1 in their places, which is compared with the plain form."""
    kept, bad = stored(slots, group, blocks * page)
    T = len(slots)
    qkv = torch.randn(T, 2 * hk * dim, generator=torch.Generator().manual_seed(seed)).bfloat16()
    pos, f = torch.arange(T).int(), freqs(dim)
    clean, cache = (make_cache(w, torch.Generator().manual_seed(seed), blocks, page, group, hk, dim, dtype) for _ in range(2))
    assert same_bits(state_of(clean), state_of(cache))
    check_append(w, clean, qkv, 0, pos, f, None, False, kept)
    _, k, v = split_qkv(qkv.cuda(), 0, hk, dim)
    for _ in range(3):
        again = make_cache(w, torch.Generator().manual_seed(seed), blocks, page, group, hk, dim, dtype)
        w.w4a16_scaled_append(None, k, v, pos.cuda(), f.cuda(), i32(slots), again)
        assert w.w4a16_device_error(clear=True) == (w.DEVERR_SLOT if bad else 0)
        assert same_bits(state_of(clean), state_of(again))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("group,slots", [(4, [17, 16]), (4, [16, 16]), (4, [19, 16, 17, 18, 19, 20, 21]), (4, [16, 17, 16, 17, 18]), (4, [18, 17, 16]),
                                         (4, [16, 18, 19, 20]), (16, [31, 16]), (16, [16, 16, 17]), (1, [16, 16]), (1, [17, 17, 18, 18, 18, 17 + 16]),
                                         (8, [24, 16, 24 + 8, 24 + 8]), (2, [3, 2, 1, 0])], ids=str)
def test_a_slot_in_the_group_of_the_token_before_has_to_follow_it(w, group, slots, dtype):
    check_slots(w, 16, group, 3, 64, slots, 4, 5, TYPES[dtype])


@pytest.mark.parametrize("T", [40, 700, 6000])
@pytest.mark.parametrize("group", [1, 4, 16])
def test_slots_out_of_order_in_calls_of_many_tokens(w, group, T):
    # such pairs between the tokens of neighbouring groups, in blocks of their own: inside of what a CTA
    # takes (a power of two of tokens, 32 at most) and across two CTAs
    slots, spare = list(range(16, 16 + T)), (T // 16 + 4) * 16
    for t in range(15, T - 1, 16):
        slots[t], slots[t + 1] = spare + group - 1, spare  # a group's last place, then its first (group 1: the same again)
        spare += 16
    check_slots(w, 16, group, 2, 32, slots, spare // 16, T + group, TYPES["int8"])


# --------------------------------------------------------------------------
# append: tokens that are taken back
# --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", list(TYPES))
def test_drafts_taken_back_leave_their_scale(w, dtype):
    gen = torch.Generator().manual_seed(9)
    cache = make_cache(w, gen, 2, 16, 8, 1, 32, TYPES[dtype])
    x = torch.randn(16, 2, 32, generator=gen).bfloat16()

    def write(values, at):
        n = len(values)
        check_append(w, cache, values.reshape(n, -1), 0, torch.arange(n).int(), freqs(32), None, False, list(range(at, at + n)))
        return [s[0, :, 0].cpu() for s in (cache.k_scale, cache.v_scale)]

    def off():  # the accepted values, by the header's bound; e4m3: 2^-4 of the value besides
        have = (code_values(cache.v)[0] * cache.v_scale[0].double().cpu().repeat_interleave(8, 0)[..., None])[:, 0]
        want, S = x[:, 1].double(), cache.v_scale[0].double().cpu().repeat_interleave(8, 0)
        return (have - want).abs(), S if dtype == "int8" else 2.0 ** -9 * S + 2.0 ** -4 * want.abs()

    first = write(x[:3], 0)
    grown = write(64 * x[3:5], 3)  # drafts, 64 times as large
    assert all(g[0] >= 16 * f[0] for f, g in zip(first, grown))
    kept = write(x[3:16], 3)  # others take their places, and go on into the next group
    assert all(k[0] == g[0] for k, g in zip(kept, grown))  # as far as it grew
    assert all(k[1] <= 4 * f[0] for k, f in zip(kept, first))  # the group that began since then has its own
    e, bound = off()
    assert (e <= bound).all()
    # written from its first place on, the group has a scale of its own tokens again
    again = write(x[:8], 0)
    assert all(a[0] < g[0] / 8 and a[1] == k[1] for a, g, k in zip(again, grown, kept))
    e, bound = off()
    assert (e <= bound).all()
    # a draft that is not finite
    bad = x[5:6].clone()
    bad[0, :, 7] = float("inf")
    assert all(s[0].isnan() and not s[1].isnan() for s in write(bad, 5))
    assert all(s[0].isnan() for s in write(x[5:8], 5))
    assert all(s[0] == a[0] for s, a in zip(write(x[:8], 0), again))
    e, bound = off()
    assert (e <= bound).all()


def test_an_append_without_keys_values_or_slots_is_refused(w):
    cache = make_cache(w, torch.Generator().manual_seed(1), 2, 16, 8, 2, 64, TYPES["int8"])
    before = state_of(cache)
    x = torch.randn(5, 2, 64, device="cuda").bfloat16()
    args = dict(q=x, k=x, v=x, positions=i32(range(5)), inv_freq=freqs(64).cuda(), slots=i32(range(5)), cache=cache)
    for name in ("k", "v", "slots"):
        for q_out in (None, torch.empty_like(x)):
            with pytest.raises(TypeError):
                w.w4a16_scaled_append(**{**args, name: None, "q_out": q_out})
    assert same_bits(before, state_of(cache)) and w.w4a16_device_error(clear=True) == 0
