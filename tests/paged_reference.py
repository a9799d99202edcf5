"""Plain 64-bit forms of the paged-cache operators (torch, CPU, double) that
the GPU tests compare with.  Loops over requests, tokens and heads; nothing of
the library is used."""
import torch


def paged_map(ctx, new, table, free, head, page, num_blocks, tokens):
    """As w4a16_paged_map on lists; returns (table, slots, positions, row_start, kv_len, head, flags)
    with flags a set of "slot" and "blocks"."""
    table = [list(r) for r in table]
    columns, flags = len(table[0]), set()
    slots, positions, row_start, kv_len = [], [], [0], []
    taken = 0

    def valid(i):
        if 0 <= i < num_blocks:
            return i
        flags.add("slot")
        return -1

    for b, (c, n) in enumerate(zip(ctx, new)):
        if c < 0 or n < 0:
            flags.add("blocks")
        c, n = max(c, 0), max(n, 0)
        before, after = min(-(-c // page), columns), -(-(c + n) // page)
        if after > columns:
            flags.add("blocks")
            after = columns
        for col in range(before, after):
            at = head + taken
            taken += 1
            if at >= len(free):
                flags.add("blocks")
                table[b][col] = -1
            else:
                table[b][col] = valid(free[at])
        for pos in range(c, c + n):
            col = pos // page
            block = -1
            if col < columns:
                block = table[b][col]
                if col < -(-c // page):
                    block = valid(block)
            positions.append(pos)
            slots.append(block * page + pos % page if block >= 0 else -1)
        row_start.append(row_start[-1] + n)
        kv_len.append(c + n)
    if len(slots) > tokens:
        flags.add("blocks")
    pad = [-1] * max(0, tokens - len(slots))
    return (table, (slots + pad)[:tokens], (positions + pad)[:tokens], row_start, kv_len,
            min(head + taken, max(len(free), head)), flags)


def rope(x, positions, inv_freq, sections, interleaved, inverse=False):
    """x [T, heads, dim] double; positions [axes, T]; the rotation of the first 2 * len(inv_freq) values."""
    half = inv_freq.numel()
    axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections))
    a = positions.double()[axis].t() * inv_freq.double()  # [T, half]
    c, s = a.cos()[:, None], (-a if inverse else a).sin()[:, None]
    y = x.clone()
    if interleaved:
        x1, x2 = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = x1 * c - x2 * s, x2 * c + x1 * s
    else:
        x1, x2 = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = x1 * c - x2 * s, x2 * c + x1 * s
    return y


def attention(q, k, v, table, lens, scale, window):
    """q [B, Hq, D], k and v [blocks, page, Hk, D], all double.  Returns out, lse, and per output what the
    tolerances go by: spread = sum p |v| and reach = max |scale| sum |q| |k| of a row."""
    B, Hq, D = q.shape
    blocks, page, Hk, _ = k.shape
    G = Hq // Hk
    out = torch.zeros(B, Hq, D, dtype=torch.float64)
    lse = torch.full((B, Hq), -float("inf"), dtype=torch.float64)
    spread = torch.zeros(B, Hq, D, dtype=torch.float64)
    reach = torch.zeros(B, Hq, dtype=torch.float64)
    for b in range(B):
        n = min(max(int(lens[b]), 0), len(table[b]) * page)
        first = max(0, n - window) if window else 0
        at = [(table[b][j // page], j % page) for j in range(first, n)]
        at = [(i, p) for i, p in at if 0 <= i < blocks]
        if not at:
            continue
        i, p = (torch.tensor(z) for z in zip(*at))
        for h in range(Hq):
            kk, vv = k[i, p, h // G], v[i, p, h // G]
            s = scale * (kk @ q[b, h])
            top = s.max()
            if top == -float("inf"):
                continue
            e = torch.exp(s - top)
            lse[b, h] = e.sum().log() + top
            w = e / e.sum()
            out[b, h], spread[b, h] = w @ vv, w @ vv.abs()
            reach[b, h] = (abs(scale) * (kk.abs() @ q[b, h].abs())).max()
    return out, lse, spread, reach
