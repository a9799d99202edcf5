"""Plain forms of the operators over an 8-bit paged cache with scales by group
(torch, CPU), that the GPU tests compare with.  Loops over runs, requests, tokens
and heads; nothing of the library is used."""
import math

import torch

from . import paged_reference as paged

MOST = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
NAN = float("nan")


def nearest(x, dtype):
    """The code next to each value of x (float32 or double, in range), ties to even, as a value."""
    if dtype is torch.int8:
        return x.round().clamp(-127, 127)
    step = torch.ldexp(torch.ones_like(x), torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 4)
    return ((x / step).round() * step).clamp(-448, 448)


def power_of_two_above(x):
    """The smallest power of two >= x > 0 (a Python float, exact)."""
    m, e = math.frexp(x)
    return math.ldexp(1.0, e - 1 if m == 0.5 else e)


def need_of(x, rotary, interleaved):
    """x [tokens, dim] float32 of one head: the largest magnitude, of pairs that are turned their
    length, as the square that the scale is compared with (its sum rounded to fp32)."""
    half = rotary // 2
    a, b = (x[:, 0:rotary:2], x[:, 1:rotary:2]) if interleaved else (x[:, :half], x[:, half:rotary])
    if not torch.isfinite(x).all():
        return None
    top = x[:, rotary:].abs().double().square().amax().item() if rotary < x.shape[1] else 0.0
    if half:
        # scaled by a power of two first, so that the squares are in fp32's range
        big = float(x.abs().max())
        f = 2.0 ** -math.frexp(big)[1] if big else 1.0
        top = max(top, float(((a.double() * f).float().square() + (b.double() * f).float().square()).max()) / f / f)
    return top


def scale_for(square, dtype, old):
    """The group's scale: of the largest squared magnitude, and of the scale so far (0: none)."""
    if square is None or not math.isfinite(old):
        return NAN
    s = 2.0 ** -126
    while square > (MOST[dtype] * s) ** 2:
        s *= 2
    if old:
        s = max(s, power_of_two_above(abs(old)))
    return s if s <= 2.0 ** 127 else NAN


def append(codes, scales, x, turned, rotary, interleaved, slots, page, group, dtype):
    """codes double [blocks, page, heads, dim] (the values codes are), scales float32 [blocks, groups, heads],
    x bf16 [T, heads, dim], turned double: x after its rotation.  Returns the state after the append, the
    values of the new tokens over their scale before rounding (NaN elsewhere), and whether a slot was bad."""
    codes, scales, bad = codes.clone(), scales.clone(), False
    exact = torch.full_like(codes, NAN)
    limit = codes.shape[0] * page
    t, T = 0, len(slots)
    while t < T:
        s, before = slots[t], slots[t - 1] if t else -1
        if not 0 <= s < limit:
            bad |= s != -1
            t += 1
            continue
        n = 1
        while t + n < T and (s + n) % group and slots[t + n] == s + n:
            n += 1
        if s % group and before >= 0 and before // group == s // group:
            bad = True
            t += n
            continue
        block, place, held = s // page, s % page, s % group
        g = place // group
        for h in range(codes.shape[2]):
            old = float(scales[block, g, h]) if held else 0.0
            S = scale_for(need_of(x[t:t + n, h].float(), rotary, interleaved), dtype, old)
            if held and S != old:
                ratio = torch.tensor(old, dtype=torch.float32) / torch.tensor(S, dtype=torch.float32)
                rows = slice(place - held, place)
                codes[block, rows, h] = nearest(codes[block, rows, h].float() * ratio, dtype).double()
            scales[block, g, h] = S
            rows = slice(place, place + n)
            exact[block, rows, h] = turned[t:t + n, h] / S
            codes[block, rows, h] = nearest(exact[block, rows, h], dtype)
        t += n
    return codes, scales, exact, bad


def attention(q, codes_k, codes_v, ks, vs, table, lens, scale, window, group):
    """q [B, N, Hq, D] double; codes [blocks, page, Hk, D] and scales [blocks, groups, Hk] double.  Returns
    out, lse, and what the tolerances go by: spread = sum p |v|, reach = max |scale| sum |q| |k|, and
    low = max_j (p_j |s_j|) sum_j |c_j|."""
    B, N, Hq, D = q.shape
    blocks, page, Hk, _ = codes_k.shape
    G = Hq // Hk
    shape = (B, N, Hq)
    out, spread, low = (torch.zeros(*shape, D, dtype=torch.float64) for _ in range(3))
    lse, reach = torch.full(shape, -math.inf, dtype=torch.float64), torch.zeros(shape, dtype=torch.float64)
    most = len(table[0]) * page
    for b in range(B):
        length = min(max(int(lens[b]), 0), most)
        for i in range(N):
            end = length - (N - 1 - i)
            first = max(0, end - window) if window else 0
            at = [(table[b][j // page], j % page) for j in range(first, end)]
            at = [(x, p) for x, p in at if 0 <= x < blocks]
            if not at:
                continue
            x, p = (torch.tensor(z) for z in zip(*at))
            for h in range(Hq):
                fk, fv = ks[x, p // group, h // G], vs[x, p // group, h // G]
                kk, cv = codes_k[x, p, h // G] * fk[:, None], codes_v[x, p, h // G]
                s = scale * (kk @ q[b, i, h])
                e = torch.exp(s - s.max())
                w = e / e.sum()
                lse[b, i, h] = e.sum().log() + s.max()
                out[b, i, h], spread[b, i, h] = w @ (cv * fv[:, None]), w @ (cv * fv[:, None]).abs()
                low[b, i, h] = (w * fv.abs()).max() * cv.abs().sum(0)
                reach[b, i, h] = (abs(scale) * (kk.abs() @ q[b, i, h].abs())).max()
    return out, lse, spread, reach, low


rope = paged.rope
