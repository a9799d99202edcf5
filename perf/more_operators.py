"""The operators of an 8-bit paged cache with a scale for each group of tokens and head, as cases that can be timed and compared.

  write   rotary positions on q and k, and the write of k and v into the
          cache, which finds the scales: powers of two, one for each group of
          `group` tokens of a block and head, that grow with the group
  chunk   the same followed by the read of the whole requests back into bf16
  read    the keys and values of requests back into bf16 or fp32
  attend  attention of one or several new tokens per request over that cache

`run` computes a case either from elementary torch operations (the plain form)
or, with `own` set, through this package.  Lengths are a fixed multiset per
case, dealt to the requests by the seed, so a case's work does not depend on
the seed.
"""
import math

import numpy as np
import torch

own = False

# largest magnitude of a code
_MOST = {"int8": 127, "e4m3": 448}
_TYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    # 32 query heads over 8 key/value heads of 128: the 6144 rows of the fused
    # QKV projection over a hidden size of 4096 that the benchmark sweeps.
    gqa = dict(q_heads=32, kv_heads=8, dim=128)
    turn = dict(rotary=128, axes=1, pairs="halves")
    return [
        # one token of one request: latency only
        dict(name="write 1", op="write", requests=1, longest_ctx=300, longest_new=1, page=16, group=16, code="e4m3", layout="token", **turn, **gqa),
        # the decode step of a serving batch: every request adds a token to a group that it has begun
        dict(name="write decode 128", op="write", requests=128, longest_ctx=4096, longest_new=1, page=32, group=32, code="e4m3", layout="head", **turn, **gqa),
        # ragged prompts of text and image tokens: three axes
        dict(name="write prompts", op="write", requests=24, longest_ctx=0, longest_new=1999, page=16, group=16, code="e4m3", layout="token", rotary=128, axes=3,
             pairs="halves", **gqa),
        # an odd-sized chunk of a long prompt, half of each head turned, neighbouring pairs; the prompt so far is read back
        dict(name="chunk 4095 int8", op="chunk", requests=1, longest_ctx=8195, longest_new=4095, page=64, group=16, code="int8", layout="token", rotary=64, axes=1,
             pairs="neighbours", **gqa),
        # a short context leaves the cache: latency
        dict(name="read 1 x 300", op="read", requests=1, longest=300, spread="even", page=16, group=16, code="int8", layout="token", wide=False, kv_heads=8, dim=128),
        # a batch's contexts move to another engine
        dict(name="read 64 ragged", op="read", requests=64, longest=8192, spread="ragged", page=32, group=32, code="e4m3", layout="head", wide=False, kv_heads=8, dim=128),
        # one stream, short context: latency
        dict(name="attend 1 x 300", op="attend", requests=1, new=1, longest=300, spread="even", page=16, group=16, code="int8", layout="token", window=0, **gqa),
        # a small ragged batch with an empty request in it, a scale for every token
        dict(name="attend 16 ragged", op="attend", requests=16, new=1, longest=4096, spread="ragged", page=16, group=1, code="e4m3", layout="token", window=0, **gqa),
        # one stream over a very long context: the cache's length has to be split
        dict(name="attend 1 x 131072", op="attend", requests=1, new=1, longest=131072, spread="even", page=64, group=16, code="int8", layout="token", window=0, **gqa),
        # a serving batch whose blocks keep each head's tokens together, a scale for each block
        dict(name="attend 128 int8", op="attend", requests=128, new=1, longest=8192, spread="ragged", page=32, group=32, code="int8", layout="head", window=0, **gqa),
        # five drafted tokens of each request verified together
        dict(name="attend drafts", op="attend", requests=16, new=5, longest=16384, spread="ragged", page=64, group=64, code="e4m3", layout="token", window=0, **gqa),
        # a head of its own for every query head, narrow heads, a sliding window, pages that do not divide a tile
        dict(name="attend own heads 64", op="attend", requests=24, new=1, longest=3000, spread="ragged", page=24, group=8, code="int8", layout="token", window=1500,
             q_heads=20, kv_heads=20, dim=64),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(["write", "chunk", "read", "attend", "attend", "attend"])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 16])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8, 16])
    while q_heads > 64:
        q_heads -= kv_heads
    dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
    page = rng.choice([8, 16, 16, 24, 32, 64, 128])
    group = rng.choice([g for g in (1, 4, 8, 12, 16, 24, 32, 64, 128) if page % g == 0])
    case = dict(op=op, page=page, group=group, code="e4m3" if op == "write" else rng.choice(["int8", "e4m3"]), layout=rng.choice(["token", "head"]), kv_heads=kv_heads,
                dim=dim)
    if op in ("write", "chunk"):
        # at most the bytes of the largest listed case
        most = 16384 * (4 * 32 + 8 * 8) * 128 // ((4 * q_heads + 12 * kv_heads) * dim) // 2
        requests = _log_int(rng, 1, 128)
        new = 1 if rng.random() < 0.4 else _log_int(rng, 1, max(1, most // requests))
        ctx = rng.choice([0, _log_int(rng, 1, max(1, min(8192, most // requests)))])
        return dict(case, requests=requests, longest_ctx=ctx, longest_new=new, q_heads=q_heads, rotary=rng.choice([r for r in (0, 32, 64, 96, 128, 192, 256) if r <= dim]),
                    axes=rng.choice([1, 1, 2, 3, 4]), pairs=rng.choice(["halves", "neighbours"]))
    requests = _log_int(rng, 1, 160)
    if op == "read":
        longest = _log_int(rng, 1, min(131072, 64 * 8192 * 8 * 128 // (6 * requests * kv_heads * dim)))
        return dict(case, requests=requests, longest=longest, spread=rng.choice(["even", "ragged", "ragged"]), wide=rng.random() < 0.25)
    new = rng.choice([1, 1, 1, 2, 3, 5, 8])
    # at most the longest listed context, and no more cached values than the largest listed case holds
    longest = _log_int(rng, 1, min(131072, 128 * 8192 * 8 * 128 // (6 * requests * max(kv_heads, new * q_heads // 4) * dim)))
    window = rng.choice([0, 0, 0, _log_int(rng, 1, longest)])
    return dict(case, requests=requests, new=new, longest=longest, spread=rng.choice(["even", "ragged", "ragged"]), window=window, q_heads=q_heads)


def _lengths(n, longest, spread):
    """The multiset of lengths of a case: all the same, or from empty to the longest."""
    if spread == "even" or n == 1:
        return np.full(n, longest, dtype=np.int64)
    at = np.arange(1, n + 1) / n
    v = np.maximum(1, np.round(longest * at ** 2)).astype(np.int64)
    if n >= 8:
        v[0] = 0
    return v


def _write_lengths(case):
    n = case["requests"]
    ctx = _lengths(n, case["longest_ctx"], "ragged") if case["longest_ctx"] else np.zeros(n, dtype=np.int64)
    new = _lengths(n, case["longest_new"], "even" if case["longest_new"] == 1 else "ragged")
    return ctx, new


def _sections(rotary, axes):
    """How many of the rotary / 2 frequencies go by each axis."""
    half = rotary // 2
    each = [half // axes] * axes
    each[0] += half - sum(each)
    return each


def work(case):
    d, hk, group = case["dim"], case["kv_heads"], case["group"]
    if case["op"] in ("write", "chunk"):
        ctx, new = _write_lengths(case)
        t = int(new.sum())
        # q read and written, k and v read, their codes written; a scale for each group and head
        b = t * (4 * case["q_heads"] * d + 6 * hk * d + 4 * case["axes"] + 4) + 8 * hk * int((-(-new // group)).sum())
        if case["op"] == "chunk":
            n = int((ctx + new).sum())
            b += 6 * n * hk * d + 8 * hk * n // group
        return {"bytes": float(b), "flops": float(3 * t * case["rotary"] * (case["q_heads"] + hk) + 2 * t * hk * d)}
    lengths = _lengths(case["requests"], case["longest"], case["spread"])
    if case["op"] == "read":
        n = int(lengths.sum())
        return {"bytes": float(2 * n * hk * d * (1 + (4 if case["wide"] else 2)) + 8 * hk * n // group), "flops": 2.0 * n * hk * d}
    new, window = case["new"], case["window"]
    seen = np.minimum(lengths, window + new - 1) if window else lengths  # by one at least of a request's new tokens
    each = [np.clip(lengths - i, 0, window or None) for i in range(new)]
    return {"bytes": float(int(seen.sum()) * hk * (2 * d + 8 / group) + 4 * case["requests"] * new * case["q_heads"] * (d + 1)),
            "flops": 4.0 * int(sum(e.sum() for e in each)) * case["q_heads"] * d}


# --------------------------------------------------------------------------
# what a program has in hand before the call
# --------------------------------------------------------------------------
def _rng(seed):
    return np.random.RandomState(seed % (1 << 31)), torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def _power_of_two(e):
    """2^e of whole numbers e from -126 on."""
    return ((e + 127).int() << 23).view(torch.float32)


def _int32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _cache(case, blocks, gen):
    """k, v [blocks, page, heads, dim] (in memory by token or by head) and their scales [blocks, page / group, heads]: what earlier steps left."""
    page, heads, dim, groups = case["page"], case["kv_heads"], case["dim"], case["page"] // case["group"]
    by_head = case["layout"] == "head"
    shape = (blocks, heads, page, dim) if by_head else (blocks, page, heads, dim)
    dtype, found = _TYPE[case["code"]], []
    for _ in range(2):
        t = torch.empty(shape, dtype=dtype, device="cuda")
        for part in t.view(torch.uint8).split(max(1, (1 << 26) // (page * heads * dim))):
            x = _randn(gen, *part.shape)
            x = (x * 32).round().clamp(-127, 127).to(dtype) if case["code"] == "int8" else (x * 100).clamp(-448, 448).to(dtype)
            part.copy_(x.view(torch.uint8))
        # powers of two, of most groups about the same, of some much larger
        power = torch.randint(-1, 2, (blocks, heads, groups), device="cuda", generator=gen) + 4 * (torch.rand(blocks, heads, groups, device="cuda", generator=gen) < 0.02)
        scale = _power_of_two(power - (5 if case["code"] == "int8" else 7))
        found += [t.permute(0, 2, 1, 3) if by_head else t, scale.transpose(1, 2)]
    return {"k_cache": found[0], "k_scale": found[1], "v_cache": found[2], "v_scale": found[3]}


def _table(rs, lengths, page, spare):
    """Block ids of requests of these lengths, in no order."""
    used = -(-lengths // page)
    blocks, columns = int(used.sum()) + spare, max(1, int(used.max()))
    table = np.full((len(lengths), columns), -1)
    table[np.arange(columns)[None, :] < used[:, None]] = rs.permutation(blocks)[: int(used.sum())]
    return table, blocks


def _handle(s):
    """The handle of a cache is made once, when the cache is."""
    from w4a16_int4_weight_gemv_gb300 import binding
    return binding.ScaledCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])


def prepare(case, seed):
    rs, gen = _rng(seed)
    s = dict(case)
    page, hk, dim = case["page"], case["kv_heads"], case["dim"]
    if case["op"] in ("write", "chunk"):
        ctx, new = _write_lengths(case)
        # dealt together, so that shapes go by the case alone
        order = rs.permutation(case["requests"])
        ctx, new = ctx[order], new[order]
        table, blocks = _table(rs, ctx + new, page, 3)
        t, axes, half, hq = int(new.sum()), case["axes"], case["rotary"] // 2, case["q_heads"]
        request = np.repeat(np.arange(len(new)), new)
        place = np.arange(t) - np.repeat(np.cumsum(new) - new, new) + ctx[request]
        slots = table[request, place // page] * page + place % page
        if t >= 8 and case["op"] == "write" and case["longest_new"] == 1:
            slots[rs.randint(t)] = -1  # a padded place of the batch
        positions = rs.randint(0, 64, size=(axes, t))
        positions[0] = place + (rs.randint(0, 30000) if axes == 1 else 0)
        qkv = _randn(gen, t, (hq + 2 * hk) * dim).to(torch.bfloat16)  # one row a token: what the fused projection gives
        q, k, v = qkv.split([hq * dim, hk * dim, hk * dim], dim=1)
        freq = torch.pow(torch.tensor(10000.0, dtype=torch.float64), -torch.arange(half, dtype=torch.float64) / max(1, half))
        total = np.concatenate([[0], np.cumsum(ctx + new)])
        s.update(_cache(case, blocks, gen), q=q.view(t, hq, dim), k=k.view(t, hk, dim), v=v.view(t, hk, dim), positions=_int32(positions), slots=_int32(slots),
                 inv_freq=freq.to(torch.float32).cuda(), sections=_sections(case["rotary"], axes), block_table=_int32(table), row_start=_int32(total),
                 axis=torch.from_numpy(np.repeat(np.arange(axes), _sections(case["rotary"], axes))).cuda(), ctx=ctx, new_of=new, tokens=int(total[-1]),
                 q_out=torch.empty(t, hq, dim, dtype=torch.bfloat16, device="cuda"))
        if case["op"] == "chunk":
            s.update(k_out=torch.zeros(s["tokens"], hk, dim, dtype=torch.bfloat16, device="cuda"), v_out=torch.zeros(s["tokens"], hk, dim, dtype=torch.bfloat16, device="cuda"))
        if own:
            s["cache_handle"] = _handle(s)
        return s
    lengths = _lengths(case["requests"], case["longest"], case["spread"])
    rs.shuffle(lengths)
    table, blocks = _table(rs, lengths, page, 3)
    s.update(_cache(case, blocks, gen), block_table=_int32(table), kv_len=_int32(lengths))
    if case["op"] == "read":
        start = np.concatenate([[0], np.cumsum(lengths)])
        shape, dtype = (int(start[-1]) + 5, hk, dim), torch.float32 if case["wide"] else torch.bfloat16  # five rows behind the last request
        s.update(row_start=_int32(start), tokens=int(start[-1]), k_out=torch.zeros(shape, dtype=dtype, device="cuda"), v_out=torch.zeros(shape, dtype=dtype, device="cuda"))
        if own:
            s["cache_handle"] = _handle(s)
        return s
    # places that no request has written hold whatever was there, and groups without any a scale that is no number
    columns = table.shape[1]
    rows = torch.arange(columns * page, device="cuda").view(1, columns, page) < torch.from_numpy(lengths).cuda().view(-1, 1, 1)
    written = torch.zeros(blocks, page, dtype=torch.bool, device="cuda")
    tab = torch.from_numpy(table).cuda()
    written[tab[tab >= 0]] = rows[tab >= 0]
    for c in ("k_cache", "v_cache"):
        s[c].view(torch.uint8).masked_fill_(~written.view(blocks, page, 1, 1), 0x7F)
    some = written.view(blocks, -1, case["group"]).any(2)
    for c in ("k_scale", "v_scale"):
        s[c].masked_fill_(~some[:, :, None], math.nan)
    n, new, hq = case["requests"], case["new"], case["q_heads"]
    q = (1.5 * _randn(gen, n, new, hq, dim)).to(torch.bfloat16)
    s.update(q=q, scale=dim ** -0.5, out=torch.empty_like(q), lse=torch.empty(n, new, hq, device="cuda"))
    if own:  # the handle of the cache and the scratch memory, kept from step to step
        from w4a16_int4_weight_gemv_gb300 import binding
        s["cache_handle"] = _handle(s)
        s["workspace"] = binding.scaled_attention_workspace(s["cache_handle"], hq, new)
    return s


# --------------------------------------------------------------------------
# the operators through this package
# --------------------------------------------------------------------------
def _run_own(s):
    from w4a16_int4_weight_gemv_gb300 import binding
    if s["op"] == "attend":
        out, lse = binding.w4a16_scaled_attention(s["q"], s["cache_handle"], s["block_table"], s["kv_len"], scale=s["scale"], window=s["window"], out=s["out"],
                                                  lse=s["lse"], workspace=s["workspace"])
        return {"out": out, "lse": lse}
    found = {}
    if s["op"] != "read":
        q = binding.w4a16_scaled_append(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["slots"], s["cache_handle"], sections=s["sections"],
                                        interleaved=s["pairs"] == "neighbours", q_out=s["q_out"])
        found = {"q": q, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
        if s["op"] == "write":
            return {**found, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    k, v = binding.w4a16_scaled_read(s["cache_handle"], s["block_table"], s["row_start"], k_out=s["k_out"], v_out=s["v_out"])
    return {**found, "k": k, "v": v}


# --------------------------------------------------------------------------
# the plain form
# --------------------------------------------------------------------------
def _pairs_of(x, rotary, pairs):
    r = x[..., :rotary]
    return (r[..., : rotary // 2], r[..., rotary // 2:]) if pairs == "halves" else (r[..., 0::2], r[..., 1::2])


def _turn(x, cos, sin, rotary, pairs):
    """The rotation of the first `rotary` values of each head, in 32 bits."""
    x = x.float()
    a, b = _pairs_of(x, rotary, pairs)
    y, z = a * cos - b * sin, b * cos + a * sin
    r = torch.cat([y, z], -1) if pairs == "halves" else torch.stack([y, z], -1).flatten(-2)
    return torch.cat([r, x[..., rotary:]], -1)


def _codes(x, code):
    """To the nearest code, as its byte."""
    if code == "int8":
        return x.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _store(cache, scale, y, square, s):
    """Values y [tokens, heads, dim] into the cache; square [tokens, heads]: of the largest length in each token."""
    page, group, code = s["page"], s["group"], s["code"]
    blocks, _, heads, dim = cache.shape
    groups, slots = blocks * page // group, s["slots"].long()
    live = slots >= 0
    at = torch.where(live, slots // group, groups)  # one group more, for tokens that are not stored
    place = torch.where(live, slots % group, 0)
    first = torch.full((groups + 1,), group, device=y.device).scatter_reduce(0, at, place, "amin")
    top = torch.zeros(groups + 1, heads, device=y.device).scatter_reduce(0, at[:, None].expand(-1, heads), square, "amax")[:groups]
    touched, first = first[:groups] < group, first[:groups]
    # the smallest power of two whose codes hold it: 4^e most^2 >= square
    part, power = torch.frexp(top.double() / _MOST[code] ** 2)
    power = torch.where(part == 0.5, power - 1, torch.where(part > 0, power, -252))
    fresh = _power_of_two((power + 1).div(2, rounding_mode="floor").clamp(min=-126))
    old = torch.where((touched & (first > 0))[:, None], scale.reshape(groups, heads), 0.0)
    part, power = torch.frexp(old)
    whole = torch.where(old > 0, _power_of_two(torch.where(part == 0.5, power - 1, power)), 0.0)
    grown = torch.where(touched[:, None], torch.maximum(fresh, whole), scale.reshape(groups, heads))
    # what the group holds, under the new scale
    ratio = torch.where(touched[:, None], old / grown, 1.0)
    held = cache.view(torch.uint8).reshape(groups, group, heads, dim)
    earlier = (torch.arange(group, device=y.device) < first[:, None]) & touched[:, None]
    again = _codes(held.view(cache.dtype).float() * ratio[:, None, :, None], code)
    held = torch.where((earlier[:, :, None] & (ratio != 1.0)[:, None])[..., None], again, held).view(-1, heads, dim)
    # and the new tokens
    token = torch.full((groups * group + 1,), -1, device=y.device)
    token[torch.where(live, slots, groups * group)] = torch.arange(y.shape[0], device=y.device)
    token = token[: groups * group]
    new = _codes(y / grown[at.clamp(max=groups - 1)][..., None], code)
    held = torch.where((token >= 0)[:, None, None], new[token.clamp(min=0)], held)
    cache.view(torch.uint8).copy_(held.view(cache.shape))
    scale.copy_(grown.view(scale.shape))


def _plain_write(s):
    # angles of far positions lose their low bits in 32
    angle = s["positions"].double()[s["axis"]].t() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _turn(s["q"], cos, sin, s["rotary"], s["pairs"]).to(torch.bfloat16)
    k, v = s["k"].float(), s["v"].float()
    a, b = _pairs_of(k, s["rotary"], s["pairs"])
    length = torch.cat([a * a + b * b, k[..., s["rotary"]:].square()], -1).amax(-1)
    _store(s["k_cache"], s["k_scale"], _turn(k, cos, sin, s["rotary"], s["pairs"]), length, s)
    _store(s["v_cache"], s["v_scale"], v, v.square().amax(-1), s)
    return {"q": q, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_read(s):
    group, page, start = s["group"], s["page"], s["row_start"].long()
    t = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(start, t, right=True) - 1
    place = t - start[b]
    slot = s["block_table"][b, place // page].long() * page + place % page
    for out, c, f in (("k_out", "k_cache", "k_scale"), ("v_out", "v_cache", "v_scale")):
        x = s[c].view(torch.uint8)[slot // page, slot % page].view(s[c].dtype).float()
        s[out][: s["tokens"]] = (x * s[f][slot // page, slot % page // group][..., None]).to(s[out].dtype)
    return {"k": s["k_out"], "v": s["v_out"]}


def _gathered(s, c, f, blocks, places, seen):
    """The cached rows of every request, [requests, heads, longest, dim] in 32 bits, zero where nothing is seen."""
    x = s[c].view(torch.uint8)[blocks, places].view(s[c].dtype).float() * s[f][blocks, places // s["group"]][..., None]
    return torch.where(seen[:, :, None, None], x, 0.0).permute(0, 2, 1, 3)


def _plain_attend(s):
    n, new, hq, dim = s["q"].shape
    hk = s["kv_heads"]
    t = torch.arange(s["longest"], device="cuda")
    length = s["kv_len"][:, None, None] - torch.arange(new - 1, -1, -1, device="cuda")[:, None]  # of each new token
    seen = t < length
    if s["window"]:
        seen = seen & (t >= length - s["window"])
    blocks, places = s["block_table"].clamp(min=0).long()[:, t // s["page"]], t % s["page"]
    some = seen.any(1)
    q = s["q"].float().view(n, new, hk, hq // hk, dim).transpose(1, 2).reshape(n, hk, -1, dim) * s["scale"]
    seen = seen[:, None, :, None].expand(n, hk, new, hq // hk, -1).reshape(n, hk, -1, s["longest"])
    k = _gathered(s, "k_cache", "k_scale", blocks, places, some)
    score = torch.matmul(q, k.transpose(2, 3)).masked_fill(~seen, -math.inf)
    del k
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    v = _gathered(s, "v_cache", "v_scale", blocks, places, some)
    out = torch.matmul(e, v) / total.clamp(min=1e-30)
    by_token = lambda x: x.view(n, hk, new, hq // hk, -1).transpose(1, 2).reshape(n, new, hq, -1)  # noqa: E731
    return {"out": by_token(out).to(torch.bfloat16), "lse": by_token(total.log() + top)[..., 0]}


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "attend":
        return _plain_attend(state)
    found = {} if state["op"] == "read" else _plain_write(state)
    if state["op"] == "write":
        return {**found, "k_cache": state["k_cache"], "v_cache": state["v_cache"]}
    return {**found, **_plain_read(state)}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _nearest(x, code):
    """The code value next to x (ties to even)."""
    if code == "int8":
        return x.round().clamp(-127, 127)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return ((x / step).round() * step).clamp(-448, 448)


def _exact_write(s):
    """The state after the write, in 64 bits: {"q", "k_scale", "v_scale", "k_cache", "v_cache"} (codes as the values they are)."""
    code, group, page, rotary = s["code"], s["group"], s["page"], s["rotary"]
    half = rotary // 2
    angle = torch.cat([s["positions"][a].double()[:, None] * f.double() for a, f in enumerate(s["inv_freq"].split(s["sections"]))], 1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]  # e^(i angle)
    re, im = (slice(0, half), slice(half, rotary)) if s["pairs"] == "halves" else (slice(0, rotary, 2), slice(1, rotary, 2))

    def rotated(x):
        """x turned, and the largest length in each head."""
        x = x.double().clone()
        z = torch.complex(x[..., re], x[..., im])
        longest = torch.cat([z.abs(), x[..., rotary:].abs()], -1).amax(-1)
        x[..., re], x[..., im] = (z * turn).real, (z * turn).imag
        return x, longest

    found = {"q": rotated(s["q"])[0]}
    for name, (x, longest) in (("k", rotated(s["k"])), ("v", (s["v"].double(), s["v"].double().abs().amax(-1)))):
        codes, scale = s[name + "_cache"].to(torch.float32).double(), s[name + "_scale"].double().clone()
        begin = 0
        for b, (ctx, new) in enumerate(zip(s["ctx"].tolist(), s["new_of"].tolist())):
            mine = range(begin, begin + new)
            begin += new
            if new == 0 or int(s["slots"][mine[0]]) < 0:
                continue
            # the request's tokens from the beginning of the group that the first new one lies in
            low = ctx // group * group
            ids = s["block_table"][b].long()
            place = torch.arange(low, ctx + new, device="cuda")
            where, inside = ids[place // page], place % page
            gap = -(ctx + new) % group
            need = torch.nn.functional.pad(longest[mine[0]: mine[0] + new], (0, 0, ctx - low, gap)).view(-1, group, longest.shape[1]).amax(1) / _MOST[code]
            block, of = ids[place[::group] // page], place[::group] % page // group
            if ctx > low:
                need[0] = torch.maximum(need[0], scale[block[0], of[0]])
            part, power = torch.frexp(need)
            fresh = ((torch.where(part == 0.5, power - 1, power).clamp(min=-126).long() + 1023) << 52).view(torch.float64)
            if ctx > low:
                old = codes[where[: ctx - low], inside[: ctx - low]]
                codes[where[: ctx - low], inside[: ctx - low]] = torch.where((fresh[0] == scale[block[0], of[0]])[:, None], old,
                                                                             _nearest(old * (scale[block[0], of[0]] / fresh[0])[:, None], code))
            scale[block, of] = fresh
            each = fresh.repeat_interleave(group, 0)[ctx - low: ctx - low + new]
            codes[where[ctx - low:], inside[ctx - low:]] = _nearest(x[mine[0]: mine[0] + new] / each[..., None], code)
        found[name + "_cache"], found[name + "_scale"] = codes, scale
    return found


def exact(case, seed):
    s = prepare(case, seed)
    group, page, hk = case["group"], case["page"], case["kv_heads"]
    if case["op"] in ("write", "chunk"):
        s.update(_exact_write(s))
        if case["op"] == "write":
            return {name: s[name] for name in ("q", "k_scale", "v_scale", "k_cache", "v_cache")}
    if case["op"] != "attend":
        found = {name: s[name] for name in ("q", "k_scale", "v_scale")} if case["op"] == "chunk" else {}
        for name in ("k", "v"):
            full = torch.zeros(s[name + "_out"].shape, dtype=torch.float64, device="cuda")
            start = s["row_start"].tolist()
            for b, (i, j) in enumerate(zip(start, start[1:])):
                ids = s["block_table"][b, : -(-(j - i) // page)].long()
                x = s[name + "_cache"].view(torch.uint8)[ids].view(s[name + "_cache"].dtype) if case["op"] == "read" else s[name + "_cache"][ids]
                full[i:j] = (x.to(torch.float32).double() * s[name + "_scale"][ids].double().repeat_interleave(group, 1)[..., None]).flatten(0, 1)[: j - i]
            found[name] = full
        return found
    n, new, hq, dim = s["q"].shape
    out = torch.zeros(n, new, hq, dim, dtype=torch.float64, device="cuda")
    lse = torch.full((n, new, hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, length in enumerate(s["kv_len"].tolist()):
        ids = s["block_table"][b, : -(-length // page)].long()
        for h in range(hk):
            k, v = ((s[c].view(torch.uint8)[:, :, h][ids].view(s[c].dtype).to(torch.float32).double()
                     * s[f][:, :, h][ids].double().repeat_interleave(group, 1)[..., None]).flatten(0, 1) for c, f in (("k_cache", "k_scale"), ("v_cache", "v_scale")))
            rows = slice(h * (hq // hk), (h + 1) * (hq // hk))
            for i in range(new):
                end = length - (new - 1 - i)
                first = max(0, end - case["window"]) if case["window"] else 0
                if end <= 0:
                    continue
                score = s["q"][b, i, rows].double() @ k[first:end].T * s["scale"]
                lse[b, i, rows] = torch.logsumexp(score, 1)
                out[b, i, rows] = torch.softmax(score, 1) @ v[first:end]
    return {"out": out, "lse": lse}
