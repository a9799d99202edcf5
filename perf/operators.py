"""The paged-cache operators of a decode step, as cases that can be timed and compared.

Three operators that follow one another between the fused QKV projection and
the output projection of a decoder layer:

  map     block tables and slot maps from the lengths of the requests
  append  rotary positions (one or several axes) on q and k, and the write of
          k and v into the paged cache
  attend  attention of one new token per request over that cache

`run` computes a case either from elementary torch operations in 32 bits (the
plain form) or, with `own` set, through this package.  Lengths are a fixed
multiset per case, dealt to the requests by the seed, so a case's work does
not depend on the seed.
"""
import math

import numpy as np
import torch

own = False


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    # 32 query heads over 8 key/value heads of 128: the 6144 rows of the fused
    # QKV projection over a hidden size of 4096 that the benchmark sweeps.
    gqa = dict(q_heads=32, kv_heads=8, dim=128)
    return [
        # sixteen running requests each add one token: the scheduler's work of every decode step
        dict(name="map decode 16", op="map", requests=16, longest_ctx=4096, longest_new=1, page=16),
        # a wave of ragged prompts, some continuing a cached prefix
        dict(name="map prompts 96", op="map", requests=96, longest_ctx=2048, longest_new=8191, page=16),
        # one token of one request: latency only
        dict(name="append 1", op="append", tokens=1, rotary=128, axes=1, pairs="halves", page=16, cache="bf16", blocks=64, **gqa),
        # an odd-sized prompt chunk into an 8-bit cache, half of each head rotated, neighbouring pairs
        dict(name="append 4095 fp8", op="append", tokens=4095, rotary=64, axes=1, pairs="neighbours", page=32, cache="fp8", blocks=160, **gqa),
        # the tokens of a video clip: time, height and width axes
        dict(name="append video 16384", op="append", tokens=16384, rotary=128, axes=3, pairs="halves", page=16, cache="bf16", blocks=1280, **gqa),
        # one stream, short context: latency
        dict(name="attend 1 x 300", op="attend", requests=1, longest=300, spread="even", page=16, cache="bf16", window=0, layout="token", **gqa),
        # a small ragged batch, one empty request in it
        dict(name="attend 16 ragged", op="attend", requests=16, longest=4096, spread="ragged", page=16, cache="bf16", window=0, layout="token", **gqa),
        # one stream over a very long context: the cache's length has to be split
        dict(name="attend 1 x 131072", op="attend", requests=1, longest=131072, spread="even", page=64, cache="bf16", window=0, layout="token", **gqa),
        # a serving batch over an 8-bit cache whose blocks keep each head's tokens together
        dict(name="attend 128 fp8", op="attend", requests=128, longest=8192, spread="ragged", page=32, cache="fp8", window=0, layout="head", **gqa),
        # one shared key/value head, wide heads, a sliding window
        dict(name="attend window", op="attend", requests=8, longest=20000, spread="ragged", page=16, cache="bf16", window=4096, layout="token", q_heads=16, kv_heads=1, dim=256),
        # a head of its own for every query head, narrow heads, pages that do not divide a tile
        dict(name="attend own heads 64", op="attend", requests=24, longest=1500, spread="ragged", page=24, cache="bf16", window=0, layout="token", q_heads=20, kv_heads=20, dim=64),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(["map", "append", "attend", "attend"])
    if op == "map":
        requests = _log_int(rng, 1, 512)
        new = 1 if rng.random() < 0.4 else _log_int(rng, 2, max(2, min(8191, 700000 // requests)))
        return dict(op="map", requests=requests, longest_ctx=_log_int(rng, 1, 16384), longest_new=new, page=rng.choice([8, 16, 24, 32, 64, 128]))
    kv_heads = rng.choice([1, 2, 4, 5, 8, 16])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8, 16])
    while q_heads > 64:
        q_heads -= kv_heads
    dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
    page = rng.choice([8, 16, 16, 24, 32, 64, 128])
    cache = rng.choice(["bf16", "bf16", "fp8"])
    if op == "append":
        # at most the largest listed case's bytes
        most = 16384 * (4 * 32 + 8 * 8) * 128 // ((4 * q_heads + 8 * kv_heads) * dim)
        tokens = _log_int(rng, 1, most)
        axes = rng.choice([1, 1, 2, 3, 4])
        rotary = rng.choice([r for r in (32, 64, 96, 128, 192, 256) if r <= dim])
        return dict(op="append", tokens=tokens, rotary=rotary, axes=axes, pairs=rng.choice(["halves", "neighbours"]), page=page, cache=cache,
                    blocks=tokens // page + 1 + rng.randrange(1, 64), q_heads=q_heads, kv_heads=kv_heads, dim=dim)
    requests = _log_int(rng, 1, 160)
    # at most the longest listed context, and no more cached values than the largest listed case holds
    longest = _log_int(rng, 1, min(131072, 128 * 8192 * 8 * 128 // (6 * requests * max(kv_heads, q_heads // 4) * dim)))
    window = rng.choice([0, 0, 0, _log_int(rng, 1, longest)])
    return dict(op="attend", requests=requests, longest=longest, spread=rng.choice(["even", "ragged", "ragged"]), page=page, cache=cache, window=window,
                layout=rng.choice(["token", "head"]), q_heads=q_heads, kv_heads=kv_heads, dim=dim)


def _lengths(n, longest, spread):
    """The multiset of lengths of a case: all the same, or from empty to the longest."""
    if spread == "even" or n == 1:
        return np.full(n, longest, dtype=np.int64)
    at = np.arange(1, n + 1) / n
    v = np.maximum(1, np.round(longest * at ** 2)).astype(np.int64)
    if n >= 8:
        v[0] = 0
    return v


def _sections(rotary, axes):
    """How many of the rotary / 2 frequencies go by each axis."""
    half = rotary // 2
    each = [half // axes] * axes
    each[0] += half - sum(each)
    return each


def _map_lengths(case):
    n = case["requests"]
    ctx = _lengths(n, case["longest_ctx"], "ragged")
    if n >= 3:
        ctx[1] = 0
    new = _lengths(n, case["longest_new"], "even" if case["longest_new"] == 1 else "ragged")
    return ctx, new


def work(case):
    if case["op"] == "map":
        _, new = _map_lengths(case)
        tokens, n = int(new.sum()), case["requests"]
        fresh = tokens / case["page"]
        # lengths read and written, a slot and a position a token, a table entry and a free block a new block
        return {"bytes": 16.0 * n + 8.0 * tokens + 8.0 * fresh, "flops": 0.0}
    width = 2 if case["cache"] == "bf16" else 1
    if case["op"] == "append":
        t, d = case["tokens"], case["dim"]
        return {"bytes": float(t * d * (4 * case["q_heads"] + 2 * (2 + width) * case["kv_heads"]) + t * (4 * case["axes"] + 4)),
                "flops": float(3 * t * case["rotary"] * (case["q_heads"] + case["kv_heads"]))}
    n = _lengths(case["requests"], case["longest"], case["spread"])
    seen = int((np.minimum(n, case["window"]) if case["window"] else n).sum())
    return {"bytes": float(2 * seen * case["kv_heads"] * case["dim"] * width + 4 * case["requests"] * case["q_heads"] * (case["dim"] + 1)),
            "flops": 4.0 * seen * case["q_heads"] * case["dim"]}


# --------------------------------------------------------------------------
# what a program has in hand before the call
# --------------------------------------------------------------------------
def _rng(seed):
    return np.random.RandomState(seed % (1 << 31)), torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def _int32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _cache(case, blocks, gen, filled):
    """k and v [blocks, page, heads, dim] (in memory by token or by head), and the scales of an 8-bit cache."""
    page, heads, dim = case["page"], case["kv_heads"], case["dim"]
    by_head = case.get("layout") == "head"
    shape = (blocks, heads, page, dim) if by_head else (blocks, page, heads, dim)
    dtype = torch.bfloat16 if case["cache"] == "bf16" else torch.float8_e4m3fn
    pair = []
    for _ in range(2):
        t = torch.zeros(shape, dtype=dtype, device="cuda")
        if filled:
            for part in t.view(torch.uint8 if dtype != torch.bfloat16 else dtype).split(max(1, (1 << 26) // (page * heads * dim))):
                x = _randn(gen, *part.shape)
                part.copy_(x if dtype == torch.bfloat16 else (x * 24).to(dtype).view(torch.uint8))
        pair.append(t.permute(0, 2, 1, 3) if by_head else t)
    scales = (None, None)
    if case["cache"] == "fp8":
        scales = tuple(0.03 + 0.02 * torch.rand(heads, device="cuda", generator=gen) for _ in range(2))
    return pair[0], pair[1], scales[0], scales[1]


def prepare(case, seed):
    rs, gen = _rng(seed)
    s = dict(case)
    if case["op"] == "map":
        n, page = case["requests"], case["page"]
        ctx, new = _map_lengths(case)
        rs.shuffle(ctx)
        rs.shuffle(new)
        before, after = -(-ctx // page), -(-(ctx + new) // page)
        columns = -(-(case["longest_ctx"] + case["longest_new"]) // page) + 1
        # enough for the worst deal of the lengths, so that shapes go by the case alone
        blocks = int((-(-np.sort(ctx) // page)).sum() + new.sum() // page + 2 * n + 8)
        order = rs.permutation(blocks)
        table = np.full((n, columns), -1)
        place = np.arange(columns)[None, :] < before[:, None]
        table[place] = order[: int(before.sum())]
        free = np.full(blocks, -1)
        head = 3  # taken by earlier steps
        left = order[int(before.sum()):]
        free[head: head + len(left)] = left[: blocks - head]
        assert head + int((after - before).sum()) <= min(blocks, head + len(left))
        s.update(ctx_len=_int32(ctx), new_len=_int32(new), block_table=_int32(table), free_blocks=_int32(free), free_head=_int32([head]), blocks=blocks,
                 tokens=int(new.sum()) + 5)
        if own:  # output buffers that a serving loop keeps from step to step
            from w4a16_int4_weight_gemv_gb300 import binding
            s["out"] = binding.paged_map_buffers(n, s["tokens"], s["ctx_len"].device)
        return s
    if case["op"] == "append":
        t, page, axes, half = case["tokens"], case["page"], case["axes"], case["rotary"] // 2
        hq, hk, dim = case["q_heads"], case["kv_heads"], case["dim"]
        qkv = _randn(gen, t, (hq + 2 * hk) * dim).to(torch.bfloat16)  # one row a token: what the fused projection gives
        q, k, v = qkv.split([hq * dim, hk * dim, hk * dim], dim=1)
        positions = rs.randint(0, 64, size=(axes, t))
        positions[0] = rs.randint(0, 30000) + np.arange(t)
        slots = rs.permutation(case["blocks"] * page)[:t]
        if t >= 8:
            slots[rs.randint(t)] = -1  # a padded place of the batch
        k_cache, v_cache, k_scale, v_scale = _cache(case, case["blocks"], gen, False)
        freq = torch.pow(torch.tensor(10000.0, dtype=torch.float64), -torch.arange(half, dtype=torch.float64) / half)
        s.update(q=q.view(t, hq, dim), k=k.view(t, hk, dim), v=v.view(t, hk, dim), positions=_int32(positions), slots=_int32(slots),
                 inv_freq=freq.to(torch.float32).cuda(), sections=_sections(case["rotary"], axes),
                 axis=torch.from_numpy(np.repeat(np.arange(axes), _sections(case["rotary"], axes))).cuda(), k_cache=k_cache, v_cache=v_cache, k_scale=k_scale,
                 v_scale=v_scale, q_out=torch.empty(t, hq, dim, dtype=torch.bfloat16, device="cuda"))
        if own:  # the handle of a cache is made once, when the cache is
            from w4a16_int4_weight_gemv_gb300 import binding
            s["cache_handle"] = binding.PagedCache(k_cache, v_cache, k_scale, v_scale)
        return s
    n, page, longest = case["requests"], case["page"], case["longest"]
    lengths = _lengths(n, longest, case["spread"])
    rs.shuffle(lengths)
    used = -(-lengths // page)
    blocks = int(used.sum()) + 3
    columns = -(-longest // page)
    order = rs.permutation(blocks)
    table = np.full((n, columns), -1)
    table[np.arange(columns)[None, :] < used[:, None]] = order[: int(used.sum())]
    k_cache, v_cache, k_scale, v_scale = _cache(case, blocks, gen, True)
    # places that no request has written hold whatever was there: not-a-numbers among it
    rows = torch.arange(columns * page, device="cuda").view(1, columns, page) < torch.from_numpy(lengths).cuda().view(n, 1, 1)
    written = torch.zeros(blocks, page, dtype=torch.bool, device="cuda")
    tab = torch.from_numpy(table).cuda()
    written[tab[tab >= 0]] = rows[tab >= 0]
    nan = 0x7F if case["cache"] == "fp8" else 0x7FC0
    for c in (k_cache, v_cache):
        c.view(torch.uint8 if case["cache"] == "fp8" else torch.int16).masked_fill_(~written.view(blocks, page, 1, 1), nan)
    q = (1.5 * _randn(gen, n, case["q_heads"], case["dim"])).to(torch.bfloat16)
    s.update(q=q, k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale, block_table=_int32(table), kv_len=_int32(lengths),
             scale=case["dim"] ** -0.5, out=torch.empty_like(q), lse=torch.empty(n, case["q_heads"], device="cuda"))
    if own:  # the handle of the cache and the scratch memory, kept from step to step
        from w4a16_int4_weight_gemv_gb300 import binding
        s["cache_handle"] = binding.PagedCache(k_cache, v_cache, k_scale, v_scale)
        s["workspace"] = binding.paged_attention_workspace(s["cache_handle"], case["q_heads"])
    return s


# --------------------------------------------------------------------------
# the operators through this package
# --------------------------------------------------------------------------
def _run_own(s):
    from w4a16_int4_weight_gemv_gb300 import binding
    if s["op"] == "map":
        m = binding.w4a16_paged_map(s["ctx_len"], s["new_len"], s["block_table"], s["free_blocks"], s["free_head"], s["page"], s["blocks"], s["tokens"],
                                    out=s["out"])
        return {"block_table": s["block_table"], "slots": m.slots, "positions": m.positions, "row_start": m.row_start, "kv_len": m.kv_len,
                "free_head": m.free_head}
    if s["op"] == "append":
        q = binding.w4a16_rope_append(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["slots"], s["cache_handle"], sections=s["sections"],
                                      interleaved=s["pairs"] == "neighbours", q_out=s["q_out"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    out, lse = binding.w4a16_paged_attention(s["q"], s["cache_handle"], s["block_table"], s["kv_len"], scale=s["scale"], window=s["window"], out=s["out"],
                                             lse=s["lse"], workspace=s["workspace"])
    return {"out": out, "lse": lse}


# --------------------------------------------------------------------------
# the plain form
# --------------------------------------------------------------------------
def _plain_map(s):
    ctx, new, table, page, cap = s["ctx_len"].long(), s["new_len"].long(), s["block_table"], s["page"], s["tokens"]
    n, columns = table.shape
    before, after = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    need = after - before
    ends, taken = new.cumsum(0), need.cumsum(0)
    first = taken - need + s["free_head"]
    c = torch.arange(columns, device=ctx.device)
    fresh = (c >= before[:, None]) & (c < after[:, None])
    at = (first[:, None] + c - before[:, None]).clamp(0, s["free_blocks"].numel() - 1)
    table.copy_(torch.where(fresh, s["free_blocks"][at], table))
    t = torch.arange(cap, device=ctx.device)
    r = torch.searchsorted(ends, t, right=True).clamp(max=n - 1)
    live = t < ends[-1]
    pos = torch.where(live, ctx[r] + t - (ends - new)[r], 0)
    slot = table[r, pos // page].long() * page + pos % page
    return {"block_table": table, "slots": torch.where(live, slot, -1).int(), "positions": torch.where(live, pos, -1).int(),
            "row_start": torch.cat([ends.new_zeros(1), ends]).int(), "kv_len": (ctx + new).int(), "free_head": (s["free_head"] + taken[-1]).int()}


def _turn(x, cos, sin, rotary, pairs):
    """The rotation of the first `rotary` values of each head, in 32 bits."""
    x = x.float()
    r, rest = x[..., :rotary], x[..., rotary:]
    a, b = (r[..., : rotary // 2], r[..., rotary // 2:]) if pairs == "halves" else (r[..., 0::2], r[..., 1::2])
    y, z = a * cos - b * sin, b * cos + a * sin
    r = torch.cat([y, z], -1) if pairs == "halves" else torch.stack([y, z], -1).flatten(-2)
    return torch.cat([r, rest], -1)


def _store(cache, x, scale, slots):
    """cache[slots[t]] = x[t] wherever slots[t] >= 0, the slots all different."""
    page, heads, dim = cache.shape[1:]
    rows = cache.shape[0] * page
    token = torch.full((rows + 1,), -1, device=x.device)
    token[torch.where(slots >= 0, slots.long(), rows)] = torch.arange(x.shape[0], device=x.device)
    token = token[:rows]
    y = x.to(cache.dtype) if scale is None else (x.float() / scale[:, None]).clamp(-448, 448).to(cache.dtype)
    new = _bytes_of(y)[token.clamp(min=0)].view(cache.shape)
    old = _bytes_of(cache)
    old.copy_(torch.where((token >= 0).view(-1, page, 1, 1), new, old))


def _plain_append(s):
    angle = s["positions"].float()[s["axis"]].t() * s["inv_freq"]
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    q = _turn(s["q"], cos, sin, s["rotary"], s["pairs"]).to(torch.bfloat16)
    _store(s["k_cache"], _turn(s["k"], cos, sin, s["rotary"], s["pairs"]), s["k_scale"], s["slots"])
    _store(s["v_cache"], s["v"], s["v_scale"], s["slots"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _bytes_of(cache):
    """An 8-bit cache as bytes, which every indexing operation takes."""
    return cache.view(torch.uint8) if cache.element_size() == 1 else cache


def _gathered(cache, scale, blocks, places, seen):
    """The cached rows of every request, [requests, heads, longest, dim] in 32 bits, zero where nothing is seen."""
    x = _bytes_of(cache)[blocks, places].view(cache.dtype)
    x = torch.where(seen[:, :, None, None], x.float(), 0.0)
    return (x if scale is None else x * scale[:, None]).permute(0, 2, 1, 3)


def _plain_attend(s):
    n, hq, dim = s["q"].shape
    t = torch.arange(s["longest"], device="cuda")
    length = s["kv_len"][:, None]
    seen = t < length
    if s["window"]:
        seen = seen & (t >= length - s["window"])
    blocks, places = s["block_table"].clamp(min=0).long()[:, t // s["page"]], t % s["page"]
    hk = s["kv_heads"]
    q = s["q"].float().view(n, hk, hq // hk, dim) * s["scale"]
    k = _gathered(s["k_cache"], s["k_scale"], blocks, places, seen)
    score = torch.matmul(q, k.transpose(2, 3)).masked_fill(~seen[:, None, None], -math.inf)
    del k
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    v = _gathered(s["v_cache"], s["v_scale"], blocks, places, seen)
    out = torch.matmul(e, v) / total.clamp(min=1e-30)
    return {"out": out.view(n, hq, dim).to(torch.bfloat16), "lse": (total.log() + top).view(n, hq)}


def run(state):
    if own:
        return _run_own(state)
    return {"map": _plain_map, "append": _plain_append, "attend": _plain_attend}[state["op"]](state)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "map":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        sections, half = s["sections"], case["rotary"] // 2
        angle = torch.cat([s["positions"][a].double()[:, None] * f.double() for a, f in enumerate(s["inv_freq"].split(sections))], 1)
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]  # e^(i angle)

        def rotated(x):
            x = x.double().clone()
            part = x[..., : case["rotary"]]
            re, im = (slice(0, half), slice(half, None)) if case["pairs"] == "halves" else (slice(0, None, 2), slice(1, None, 2))
            z = torch.complex(part[..., re], part[..., im]) * turn
            part[..., re], part[..., im] = z.real, z.imag
            return x

        def stored(cache, x, scale):
            c = torch.zeros(cache.shape, dtype=torch.float64, device="cuda")
            kept = s["slots"] >= 0
            c.flatten(0, 1)[s["slots"][kept].long()] = (x if scale is None else x / scale.double()[:, None])[kept]
            return c

        return {"q": rotated(s["q"]), "k_cache": stored(s["k_cache"], rotated(s["k"]), s["k_scale"]),
                "v_cache": stored(s["v_cache"], s["v"].double(), s["v_scale"])}
    n, hq, dim = s["q"].shape
    hk, page = case["kv_heads"], case["page"]
    out = torch.zeros(n, hq, dim, dtype=torch.float64, device="cuda")
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device="cuda")
    one = torch.ones(hk, device="cuda")
    ks, vs = (one, one) if s["k_scale"] is None else (s["k_scale"], s["v_scale"])
    for b, length in enumerate(s["kv_len"].tolist()):
        if length == 0:
            continue
        first = max(0, length - case["window"]) if case["window"] else 0
        ids = s["block_table"][b, : -(-length // page)].long()
        for h in range(hk):
            k, v = (_bytes_of(c)[:, :, h][ids].view(c.dtype).flatten(0, 1)[first:length].double() * f[h].double()
                    for c, f in ((s["k_cache"], ks), (s["v_cache"], vs)))
            rows = slice(h * (hq // hk), (h + 1) * (hq // hk))
            score = s["q"][b, rows].double() @ k.T * s["scale"]
            lse[b, rows] = torch.logsumexp(score, 1)
            out[b, rows] = torch.softmax(score, 1) @ v
    return {"out": out, "lse": lse}
