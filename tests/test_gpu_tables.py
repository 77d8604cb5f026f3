"""Block tables and slot maps on the GPU against the request-by-request oracle
(whole numbers: equal)."""
import numpy as np
import pytest
import torch

from tests.fill_util import PAGE, check_tables, i32, run_tables

pytestmark = pytest.mark.gpu


def _pool(rng, B, cached, extra_owned, spare, width=None, new=None):
    """Tables, owned counts and a free list of `spare` pages."""
    owned = np.array([-(-c // PAGE) + e for c, e in zip(cached, extra_owned)])
    used = int(owned.sum())
    ids = rng.permutation(used + spare)
    w = width or int(max(owned.max(), max(-(-(c + n) // PAGE) for c, n in zip(cached, new)))) + 1
    table = np.full((B, w), -1)
    table[np.arange(w)[None] < owned[:, None]] = ids[:used]
    free = np.concatenate([ids[used:], np.full(used + 7, -1)])
    return table, owned, free, spare, used + spare


@pytest.mark.parametrize("B", [1, 2, 31, 33, 300, 1023, 1024, 1025, 2500, 8192])
def test_mixed_steps(B):
    rng = np.random.default_rng(B)
    cached = rng.integers(0, 200, B)
    new = rng.integers(0, 8, B)
    new[rng.integers(0, B, max(1, B // 10))] = rng.integers(0, 150)
    extra = rng.integers(0, 3, B) * (rng.random(B) < 0.3)
    if B > 3:
        cached[B // 2] = new[B // 2] = 0            # a finished request gives everything back
        extra[B // 2] = 40
    table, owned, free, n, pool = _pool(rng, B, cached, extra, 15 * B + 40, new=new)
    check_tables(table, pool, cached, new, int(new.sum()) + int(rng.integers(0, 40)), owned, free, n)


@pytest.mark.parametrize("tokens", [(4096,), (4097,), (5000, 1, 0, 20000), (0,), (1,)])
def test_many_tokens(tokens):
    """Both sides of the single-kernel limit, and no tokens at all."""
    rng = np.random.default_rng(len(tokens))
    cached = rng.integers(0, 100, len(tokens))
    table, owned, free, n, pool = _pool(rng, len(tokens), cached, [0] * len(tokens),
                                        sum(tokens) // PAGE + 60, new=tokens)
    check_tables(table, pool, cached, list(tokens), sum(tokens), owned, free, n)


@pytest.mark.parametrize("B,tokens", [(127, 511), (128, 512), (128, 513), (129, 512), (1, 512),
                                      (1, 513), (40, 1025)])
def test_both_sides_of_the_small_call(B, tokens):
    """Where the number of threads changes: shrinking, growing, finished and
    untouched requests, and a token buffer with rows left over."""
    rng = np.random.default_rng(1000 * B + tokens)
    cached, new = rng.integers(0, 90, B), rng.multinomial(tokens - min(tokens, 3), np.ones(B) / B)
    extra = rng.integers(0, 4, B)
    cached[B // 2] = new[B // 2] = 0
    table, owned, free, n, pool = _pool(rng, B, cached, extra, 2 * B + tokens, new=new)
    check_tables(table, pool, cached, new, tokens, owned, free, n)


@pytest.mark.parametrize("B", [100, 400, 1100])
def test_long_runs_of_pages(B):
    """Requests that give back or take 4, 5, 255, 256, 257 and more pages: more
    long runs than the CTA shares at once, of both kinds, and none at all."""
    rng = np.random.default_rng(B)
    sizes = np.array([0, 1, 4, 5, 12, 31, 32, 33, 255, 256, 257, 700])
    move = rng.choice(sizes, B, p=[.1, .1, .1, .2, .15, .1, .1, .05, .03, .02, .03, .02])
    grows = rng.random(B) < 0.5
    cached = rng.integers(0, 60, B)
    new = np.where(grows, np.maximum(16 * move - rng.integers(0, 15, B), 0), rng.integers(0, 3, B))
    extra = np.where(grows, 0, move + (-(-(cached + new) // PAGE)) - (-(-cached // PAGE)))
    table, owned, free, n, pool = _pool(rng, B, cached, extra, int(move.sum()) + B, new=new)
    check_tables(table, pool, cached, new, int(new.sum()), owned, free, n)


@pytest.mark.parametrize("where", [0, 128, 255, 256, 699])
def test_a_foreign_page_in_a_long_run(where):
    """A run with a page id that is none stays where it is; the others move."""
    rng = np.random.default_rng(where)
    cached, new, extra = [16, 5, 64, 0], [0, 3, 0, 4000], [700, 300, 0, 0]
    table, owned, free, n, pool = _pool(rng, 4, cached, extra, 300, new=new)
    table[0, 1 + where] = pool + where
    check_tables(table, pool, cached, new, sum(new), owned, free, n)


@pytest.mark.parametrize("spare", [0, 1, 2, 3, 4, 5, 9])
def test_pool_runs_out(spare):
    """Requests are served in order until the list is short; one that needs no
    page is served all the same, and returned pages are handed out again."""
    rng = np.random.default_rng(7)
    cached, new = [16, 31, 5, 64, 0, 48], [16, 2, 1, 17, 33, 0]
    table, owned, free, n, pool = _pool(rng, 6, cached, [0, 0, 2, 0, 0, 1], spare, new=new)
    check_tables(table, pool, cached, new, sum(new), owned, free, n)


def test_refused_requests():
    """Lengths out of range, a table row too short, rows past the token
    buffer, impossible page counts and foreign page ids: flagged, unchanged."""
    rng = np.random.default_rng(3)
    base = dict(cached=[20, 33, 7, 100], new=[5, 6, 1, 3])
    for cached, new, edit, room in (
            ([-1, 33, 7, 100], base["new"], None, 99),
            (base["cached"], [5, -6, 1, 3], None, 99),
            ([20, 33, 7, 2 ** 31 - 1], base["new"], None, 99),
            (base["cached"], [5, 6, 1, 2 ** 31 - 1], None, 99),
            ([20, 2000, 7, 100], base["new"], None, 99),
            (base["cached"], base["new"], None, 11),
            (base["cached"], base["new"], ("owned", 1, -1), 99),
            (base["cached"], base["new"], ("owned", 2, 999), 99),
            (base["cached"], base["new"], ("table", (2, 2), 10 ** 6), 99),
            (base["cached"], base["new"], ("free", 49, -5), 99),
            (base["cached"], base["new"], ("table", (1, 2), -1), 99),
            (base["cached"], [5, 60, 1, 3], ("free", 49, -5), 99)):
        table, owned, free, n, pool = _pool(rng, 4, base["cached"], [0, 0, 2, 0], 50, width=12,
                                            new=base["new"])
        arrays = dict(table=table, owned=owned, free=free)
        if edit:
            arrays[edit[0]][edit[1]] = edit[2]
        got = check_tables(table, pool, cached, new, room, owned, free, n)
        # nobody takes a page with the base lengths, so the bad entry of the
        # free list is met in the last case only
        assert got["flag"] != 0 or (edit[0] == "free" and new == base["new"])
    for count in (-1, 10 ** 6):      # a free list that is not one
        table, owned, free, n, pool = _pool(rng, 4, base["cached"], [0, 0, 2, 0], 50, new=base["new"])
        got = check_tables(table, pool, base["cached"], [5, 16, 1, 13], 99, owned, free, count)
        assert got["flag"] == 32


@pytest.mark.parametrize("B,most", [(1, 1), (5, 40), (1200, 3)])
def test_fixed_table(B, most):
    """Without a free list the table stays; a missing page leaves its tokens
    without a slot."""
    rng = np.random.default_rng(B)
    cached, new = rng.integers(0, 60, B), rng.integers(0, most + 1, B)
    table = rng.integers(0, 900, (B, 8))
    table[rng.random((B, 8)) < 0.1] = -1
    table[0, 0] = 900
    got = check_tables(table, 900, cached, new, int(new.sum()) + 3)
    np.testing.assert_array_equal(got["table"], table)


def test_repeat_is_idle_and_streams_and_graphs_agree():
    """A second call with the same lengths moves no page; a captured call
    replays on other lengths; a call on another stream gives the same."""
    from self_speculative_sparse_vg_gb300 import vg
    rng = np.random.default_rng(11)
    cached, new = [100, 3, 64, 31], [6, 6, 6, 6]
    table, owned, free, n, pool = _pool(rng, 4, cached, [0, 1, 0, 0], 30, width=16, new=new)
    first = run_tables(table, pool, cached, new, 30, owned, free, n)
    again = run_tables(first["table"], pool, cached, new, 30, first["owned"], first["free"],
                       first["count"])
    for k in first:
        np.testing.assert_array_equal(first[k], again[k], err_msg=k)
    side = torch.cuda.Stream()
    other = run_tables(table, pool, cached, new, 30, owned, free, n, stream=None)
    with torch.cuda.stream(side):
        other = run_tables(table, pool, cached, new, 30, owned, free, n)
    for k in first:
        np.testing.assert_array_equal(first[k], other[k], err_msg=k)

    t, o, f, c = i32(table), i32(owned), i32(free), i32([n])
    ca, ne = i32(cached), i32(new)
    cu, lens = (torch.zeros(m, dtype=torch.int32, device="cuda") for m in (5, 4))
    pos, slots = (torch.zeros(30, dtype=torch.int32, device="cuda") for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vg.step_tables(t, pool, ca, ne, cu, lens, pos, slots, owned=o, free_pages=f, free_count=c)
    ca.copy_(i32([x + 3 for x in cached]))
    graph.replay()
    torch.cuda.synchronize()
    from oracle import fill_oracle as F
    want = F.step_tables(table, pool, [x + 3 for x in cached], new, 30, owned, free, n)
    np.testing.assert_array_equal(t.cpu().numpy(), want["table"])
    np.testing.assert_array_equal(slots.cpu().numpy(), want["slots"])
    np.testing.assert_array_equal(f.cpu().numpy(), want["free"])


def test_without_an_error_flag():
    from self_speculative_sparse_vg_gb300 import vg
    cu, lens = (torch.zeros(m, dtype=torch.int32, device="cuda") for m in (2, 1))
    pos, slots = (torch.full((4,), 5, dtype=torch.int32, device="cuda") for _ in range(2))
    vg.step_tables(i32([[0, 1]]), 2, i32([-4]), i32([2]), cu, lens, pos, slots)
    assert lens.tolist() == [0] and slots.tolist() == [-1] * 4 and pos.tolist() == [0] * 4
