"""Block tables of steps large enough for a cluster of CTAs, with requests of
one warp that take every way through the resize before the cluster's barrier."""
import numpy as np
import pytest

from tests.fill_util import PAGE, check_tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [32, 70, 1100])
@pytest.mark.parametrize("fixed", [False, True])
def test_lanes_that_part_before_the_cluster_barrier(B, fixed):
    """Neighbouring requests that are refused (length, page id, empty list),
    finish, stay, shrink and grow by a few pages or by many, beside prompts
    whose tokens fill the whole cluster."""
    rng = np.random.default_rng(B)
    cached, new = rng.integers(0, 80, B), rng.integers(0, 4, B)
    cached[::7], new[::7] = 0, 0                            # finished
    new[1::9] = rng.integers(60, 900, len(new[1::9]))       # prompts, long runs of pages
    new[3], new[B - 2] = 9000, 8000
    owned = -(-cached // PAGE) + rng.integers(0, 3, B)
    owned[::7] += 20
    width = int(max(owned.max(), (-(-(cached + new) // PAGE)).max())) + 1
    used = int(owned.sum())
    pages = used + int((-(-new // PAGE)).sum()) // 2         # the list runs out
    ids = rng.permutation(pages)
    table = np.full((B, width), -1)
    table[np.arange(width)[None] < owned[:, None]] = ids[:used]
    free = np.concatenate([ids[used:], np.full(used + 5, -1)])
    table[7, 3] = pages + 5                                  # a foreign page in a returned run
    cached[5], new[11] = -1, -3                              # lengths out of range
    room = int(np.maximum(new, 0).sum()) + 100
    if fixed:
        got = check_tables(table, pages, cached, new, room)
        assert got["flag"] & 16
    else:
        got = check_tables(table, pages, cached, new, room, owned, free, pages - used)
        # (the finished requests of 1100 give back more pages than the others ask for)
        assert got["flag"] == (17 if B == 1100 else 49)
