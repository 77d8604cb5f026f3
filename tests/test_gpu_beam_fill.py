"""Block tables of beams in steps in which copies are asked for and no page goes
back, so that nothing but the copies stands between reading the old entries and
writing new ones: rows that were empty are filled, every other one goes on."""
import numpy as np
import pytest

from oracle import beam_oracle as O
from tests.beam_util import run_beam_tables
from tests.fill_util import PAGE

pytestmark = pytest.mark.gpu


def _pages(n):
    return -(-n // PAGE)


def parted(rng, B, W, live, lens, apart, width, spare):
    """The first `live` rows of each request share their pages up to `apart` columns
    from their end; the others are empty.  All pages that stand nowhere are free,
    `spare` places are left."""
    table = np.full((B * W, width), -1)
    n = np.zeros(B * W, int)
    need = sum(_pages(x) * (live + 1) for x in lens)
    pool = need + B * W + 5
    ids, at = rng.permutation(pool), 0
    for b in range(B):
        cols = _pages(lens[b])
        common = max(0, cols - apart)
        shared, at = ids[at:at + common], at + common
        for j in range(live):
            r = b * W + j
            table[r, :common] = shared
            table[r, common:cols] = ids[at:at + cols - common]
            at += cols - common
            n[r] = lens[b]
    count = pool - at
    free = np.concatenate([ids[at:], np.full(spare, -1)])
    return dict(lens=n, table=table, num_pages=pool, owned=-(-n // PAGE), free=free, count=count)


def check(c, parents, repeat):
    given = {"free_pages" if k == "free" else "free_count" if k == "count" else k: v for k, v in c.items()}
    want = O.beam_tables(parents, **given)
    asked = int((want["copies"][:, 2] > 0).sum())
    assert asked > 0 and want["count"] == c["count"] - asked and want["flag"] == 0, "not such a step"
    for _ in range(repeat):
        got = run_beam_tables(parents, **c)
        for k in want:
            np.testing.assert_array_equal(got[k], want[k], err_msg=k)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("row", [2, 7])
def test_a_prompt_of_another_row_among_requests_that_go_on(row, seed):
    """31 requests go on as they are; one is admitted whose prompt does not lie in row 0,
    so that the row itself is to get a copy of its last page."""
    rng = np.random.default_rng(seed)
    B, W = 32, 8
    lens = rng.integers(20000, 32001, B)
    one = int(rng.integers(B))
    lens[one] = 32000 + 5
    c = parted(rng, B, W, W, lens, 12, _pages(32768), 9)
    rows = np.arange(one * W, (one + 1) * W)
    others = rows[rows != rows[row]]
    gone = np.setdiff1d(c["table"][others], np.append(c["table"][rows[row]], -1))
    c["table"][others], c["lens"][others], c["owned"][others] = -1, 0, 0
    c["free"] = np.concatenate([gone, c["free"]])           # their own pages are free
    c["count"] += len(gone)
    parents = np.tile(np.arange(W), (B, 1))
    parents[one] = row
    check(c, parents, 4)


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("B,length,apart", [(1, 200, 9), (1, 9000, 500), (16, 9000, 300), (64, 2000, 90), (256, 400, 20)])
def test_live_rows_fill_empty_ones(B, length, apart, seed):
    """Rows 0 - 3 of 8 live and go on, parted long ago; each is taken twice, by rows
    that precede it and by rows that follow."""
    rng = np.random.default_rng(100 * B + seed)
    lens = PAGE * rng.integers(length // PAGE - 5, length // PAGE, B) + rng.integers(1, PAGE, B)
    c = parted(rng, B, 8, 4, lens, apart, _pages(length) + 2, 3)
    check(c, np.tile([1, 1, 0, 0, 3, 3, 2, 2], (B, 1)), 4)


@pytest.mark.parametrize("W", [3, 17, 32])
@pytest.mark.parametrize("B,apart,width", [(1, 600, 700), (12, 600, 700), (12, 40, 1300)])
def test_chains_of_parents(B, apart, width, W):
    """The last row is empty; parents 0, 0, 1, 2 ...: row 1 is to get a copy in the
    column from which row 2 takes row 1's old page, and so on.  Many columns a warp,
    one CTA and several."""
    rng = np.random.default_rng(1000 * W + B)
    lens = PAGE * (width - 10 - rng.integers(0, 5, B)) + rng.integers(1, PAGE, B)
    c = parted(rng, B, W, W - 1, lens, apart, width, 3)
    check(c, np.tile(np.maximum(np.arange(W) - 1, 0), (B, 1)), 8)


@pytest.mark.parametrize("seed", range(8))
def test_any_order_of_parents(seed):
    """Every live row goes on, in any order; the rows that were empty take any of them."""
    rng = np.random.default_rng(seed)
    B, W = int(rng.integers(1, 40)), int(rng.integers(3, 33))
    live = int(rng.integers(1, W))
    lens = PAGE * rng.integers(60, 120, B) + rng.integers(1, PAGE, B)
    c = parted(rng, B, W, live, lens, int(rng.integers(1, 100)), 125, 3)
    parents = np.stack([rng.permutation(np.concatenate([np.arange(live), rng.integers(0, live, W - live)]))
                        for _ in range(B)])
    check(c, parents, 4)
