"""The rule by which the GPU tests know which tokens an append with scales by group stores,
against cases worked by hand (no GPU needed)."""
import random

import pytest

from .scaled_slots import stored

LIMIT = 64
CASES = [
    # group 4: in order, over a group's end, a later group first
    (4, [4, 5, 6, 7, 8], None), (4, [6, 7, 8, 9, 2, 3], None), (4, [8, 9, 4, 5], None), (4, [-1, 5, -1, 8], None),
    # the group's first place after another of its places: descending, the same again, with what goes on from it
    (4, [5, 4], [5, -1]), (4, [4, 4], [4, -1]), (4, [7, 4, 5, 6, 7, 8, 9], [7, -1, -1, -1, -1, 8, 9]), (4, [4, 5, 4, 5, 6], [4, 5, -1, -1, -1]),
    # other places: a gap, the same again, descending
    (4, [4, 6, 7, 8], [4, -1, -1, 8]), (4, [5, 5, 6], [5, -1, -1]), (4, [7, 6], [7, -1]), (4, [4, 5, 7, 4], [4, 5, -1, -1]),
    # a group of one token: only the same slot again is in the group of the token before
    (1, [3, 2, 1, 0], None), (1, [3, 3, 4, 4, 4, 3], [3, -1, 4, -1, -1, 3]),
    # outside the cache
    (4, [64, 0], [-1, 0]), (4, [3, -2, 2 ** 31 - 1, 4], [3, -1, -1, 4]), (4, [63, 64], [63, -1]),
]


@pytest.mark.parametrize("group,slots,want", CASES, ids=lambda x: str(x).replace(" ", ""))
def test_stored_by_hand(group, slots, want):
    assert stored(slots, group, LIMIT) == (want or slots, want is not None)


def test_tokens_of_a_map_are_all_stored():
    # requests' tokens in order, padded places between them
    rng = random.Random(0)
    for group in (1, 2, 8, 16):
        ids, slots = list(range(40)), []
        rng.shuffle(ids)
        for _ in range(8):
            begin, n = rng.randrange(16), rng.randrange(1, 40)
            mine = [ids.pop() for _ in range(-(-(begin + n) // 16))]
            slots += [mine[p // 16] * 16 + p % 16 for p in range(begin, begin + n)] + [-1] * rng.choice([0, 1])
        assert stored(slots, group, 640) == (slots, False)
