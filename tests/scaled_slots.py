"""Which tokens an append with scales by group stores, from the definition: the slots of
a call, one after another (no GPU, nothing of the library)."""


def stored(slots, group, limit):
    """The slots with -1 for every token that is not stored, and whether any was refused.

    A token lies outside the cache (limit: slots of it), in the group of the token before it
    without following that token's slot, or goes on from one that is refused."""
    kept, bad = [], False
    for t, s in enumerate(slots):
        before = slots[t - 1] if t else -1
        out = s != -1 and not 0 <= s < limit
        if 0 <= s < limit and before >= 0 and before // group == s // group:
            out = before != s - 1 or kept[-1] == -1
        kept.append(-1 if out else s)
        bad |= out
    return kept, bad
