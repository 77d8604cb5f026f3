"""Block tables of beams and page copies on the GPU against the oracle (whole
numbers and bits: equal)."""
import numpy as np
import pytest
import torch

from oracle import beam_oracle as O
from tests.beam_util import check_beam_tables, run_beam_tables
from tests.fill_util import PAGE, i32

pytestmark = pytest.mark.gpu


def _pages(n):
    return -(-n // PAGE)


def make(rng, B, W, lo, hi, apart, spare=40, extra=0.2, width=None):
    """Requests whose rows share pages up to a point and then part; some rows
    hold a page past their length, some are empty."""
    width = width or _pages(hi) + 3
    lens = np.zeros(B * W, int)
    owned = np.zeros(B * W, int)
    table = np.full((B * W, width), -1)
    pool = B * W * (apart + 3) + B * (_pages(hi) + 3) + spare
    ids = rng.permutation(pool)
    at = 0
    for b in range(B):
        n = int(rng.integers(lo, hi + 1))
        cols, tail = _pages(n), n % PAGE
        for j in range(W):
            r = b * W + j
            if rng.random() < 0.1:
                continue                                   # an empty row
            part = 0
            mates = [i for i in range(b * W, r) if owned[i]]
            if mates:
                part = int(rng.integers(max(0, cols - apart), cols + 1))
                part = min(part, cols - 1 if tail else cols)
                table[r, :part] = table[mates[rng.integers(len(mates))], :part]
            more = int(rng.random() < extra)
            k = cols - part + more
            table[r, part:part + k] = ids[at:at + k]
            at += k
            lens[r], owned[r] = n, cols + more
    free = np.concatenate([ids[at:], np.full(at + 3, -1)])
    parents = np.minimum(rng.geometric(0.5, (B, W)) - 1, W - 1)
    return dict(parents=parents, lens=lens, table=table, num_pages=pool, owned=owned, free=free, count=pool - at)


@pytest.mark.parametrize("B,W", [(1, 1), (1, 2), (1, 4), (3, 5), (8, 8), (2, 32), (64, 4), (128, 32), (4096, 1), (700, 3)])
def test_steps(B, W):
    rng = np.random.default_rng(B * 100 + W)
    c = make(rng, B, W, 0, 300 if B < 500 else 40, 6)
    if B > 2:
        c["parents"][B // 2] = -1                           # a finished request
        c["parents"][B // 3, ::2] = -1
    check_beam_tables(**c)


@pytest.mark.parametrize("width", [4, 40, 300, 1025, 4200, 9000])
@pytest.mark.parametrize("B", [1, 5])
def test_table_widths(width, B):
    """From one small CTA to a cluster whose threads own several columns."""
    rng = np.random.default_rng(width)
    c = make(rng, B, 4, max(1, (width - 3) * PAGE // 2), (width - 3) * PAGE, min(width - 3, 50), width=width)
    check_beam_tables(**c)


def test_long_tables_apart_from_the_beginning():
    """Rows that share nothing: every page of the rows that end goes back."""
    rng = np.random.default_rng(5)
    c = make(rng, 9, 8, 30000, 40000, 2500)
    got = check_beam_tables(**c)
    assert got["count"] > c["count"] + 10000


@pytest.mark.parametrize("n", [1, 15, 16, 17, 4096])
def test_a_new_request_is_one_rows_prompt(n):
    """All rows take row 0; its full pages are shared, its last is copied."""
    W, cols = 6, _pages(n)
    table = np.full((W, cols + 2), -1)
    table[0, :cols] = np.arange(cols) + 7
    free = np.concatenate([np.arange(cols + 7, cols + 27), np.zeros(9)])
    got = check_beam_tables(np.zeros((1, W), int), [n] + [0] * (W - 1), table, cols + 40, [cols] + [0] * (W - 1),
                            free, 20)
    assert got["count"] == 20 - (W - 1 if n % PAGE else 0)
    assert (got["copies"][1:, 2] == n % PAGE).all() and got["copies"][0, 2] == 0


@pytest.mark.parametrize("spare", [0, 1, 2, 3, 6])
def test_the_list_runs_out(spare):
    """Rows are served in order, from the returned pages too; the rest is emptied."""
    rng = np.random.default_rng(spare)
    c = make(rng, 3, 4, 33, 60, 3, extra=0.0)
    c["parents"][:] = [[0, 0, 0, 0], [1, 1, 1, 1], [3, 2, 2, 2]]
    c["free"] = np.concatenate([c["free"][:spare], np.full(200, -1)])
    c["count"] = spare
    check_beam_tables(**c)


@pytest.mark.parametrize("spare", [0, 2, 7])
@pytest.mark.parametrize("B", [2, 12])
def test_the_list_runs_out_of_long_tables(B, spare):
    """The rows that are emptied lose their entries of columns that would stay."""
    rng = np.random.default_rng(10 * B + spare)
    W, width = 8, 600
    lens = np.repeat(rng.integers(8000, 9001, B), W)
    owned = -(-lens // PAGE)
    table = np.full((B * W, width), -1)
    for b in range(B):                                      # all rows were given one row's table
        rows = slice(b * W, (b + 1) * W)
        table[rows, :owned[b * W]] = 600 * b + rng.permutation(600)[:owned[b * W]]
    parents = rng.integers(0, W, (B, W))
    free = np.concatenate([600 * B + np.arange(spare), np.full(50, -1)])
    got = check_beam_tables(parents, lens, table, 600 * B + spare, owned, free, spare)
    assert got["flag"] == 32 and (got["owned"] == 0).any()


@pytest.mark.parametrize("W", [1, 3, 8, 17, 32])
@pytest.mark.parametrize("B,hi,apart", [(6, 33000, 30), (40, 33000, 3), (3, 9000, 560), (300, 1500, 2)])
def test_requests_that_begin_and_end_among_others(B, W, hi, apart):
    """Long runs of columns with one page at most, of which all, some or none go
    back, between columns where the rows part; foreign ids among the returned."""
    if B * W > 4096:
        B = 4096 // W
    rng = np.random.default_rng(1000 * B + W)
    c = make(rng, B, W, 1, hi, apart)
    rows = lambda b: slice(b * W, (b + 1) * W)              # noqa: E731
    for b in range(B):
        kind = b % 6
        if kind == 0:                                       # finished
            c["parents"][b] = -1
        elif kind == 1:                                     # a prompt that one row holds, not always the first
            one = int(rng.integers(W))
            for r in range(b * W, (b + 1) * W):
                if r != b * W + one:
                    c["lens"][r] = c["owned"][r] = 0
                    c["table"][r] = -1
            c["parents"][b] = one
        elif kind == 2:                                     # one row goes on, the others are emptied
            c["parents"][b] = -1
            c["parents"][b, rng.integers(W)] = rng.integers(W)
        elif kind == 3:                                     # rows cut back to a part of their pages
            c["lens"][rows(b)] //= 2
        elif kind == 4:
            c["parents"][b] = -1
            c["table"][rows(b), 5:9] = [-3, 2 ** 30, c["num_pages"], -1]
    check_beam_tables(**c)


def test_refused_requests_stay_as_they_were():
    rng = np.random.default_rng(1)
    for edit in (("parents", (1, 2), 4), ("parents", (1, 0), -2), ("parents", (0, 0), 2 ** 31 - 1),
                 ("lens", 5, -1), ("lens", 5, 10 ** 6), ("lens", 6, 2 ** 31 - 1), ("owned", 5, -1), ("owned", 4, 99),
                 ("owned", 7, 0)):
        c = make(rng, 3, 4, 33, 60, 3, width=9)
        c["lens"][c["lens"] == 0] = 0
        c[edit[0]][edit[1]] = edit[2]
        got = check_beam_tables(**c)
        assert got["flag"] & (2 | 16) or edit == ("owned", 7, 0)


def test_a_list_that_is_none_changes_nothing():
    rng = np.random.default_rng(2)
    c = make(rng, 3, 4, 33, 60, 3)
    c["parents"][:] = [[0, 0, 0, 0]] * 3
    for count in (-1, 10 ** 6, len(c["free"])):
        got = check_beam_tables(**{**c, "count": count})
        assert got["flag"] == 32 and (got["table"] == c["table"]).all()


def test_foreign_page_ids():
    """Returned ones are dropped, kept ones stay, popped ones leave no page."""
    rng = np.random.default_rng(4)
    for where, value in ((("table", (1, 0)), -7), (("table", (1, 1)), 10 ** 6), (("table", (0, 2)), -1),
                         (("free", -1), 0)):
        c = make(rng, 2, 4, 40, 47, 3, extra=0.0)
        c["parents"][:] = [[0, 0, 2, 0], [2, 2, 2, 3]]
        if where[0] == "free":
            c["free"][max(c["count"] - 2, 0)] = -5
        else:
            c["table"][where[1]] = value
        check_beam_tables(**c)


def test_a_shared_last_page_stays_with_one_row():
    """Rows that were given one row's whole table, the partly filled page too."""
    table = np.full((4, 5), -1)
    table[:, :3] = [4, 9, 2]
    free = np.arange(20, 40)
    got = check_beam_tables([[3, 1, 1, 0]], [40] * 4, table, 50, [3] * 4, np.concatenate([free, [0] * 9]), 20)
    assert len(set(got["table"][:, 2].tolist())) == 4 and got["count"] == 17


@pytest.mark.parametrize("B,W,steps", [(2, 4, 60), (5, 3, 40)])
def test_a_search_with_growing_tables(B, W, steps):
    """beam_tables and step_tables in turn, as a search runs them: after every
    step a page is free, or stands in rows of one request at one column, the page
    that a row writes next is its own, and the cache holds each row's history."""
    from self_speculative_sparse_vg_gb300 import vg
    rng = np.random.default_rng(B)
    R, width, pool = B * W, 40, B * W * 12 + 30
    table, owned, lens = i32(np.full((R, width), -1)), i32([0] * R), i32([0] * R)
    free, count = i32(np.concatenate([rng.permutation(pool), np.zeros(4)])), i32([pool])
    copies, flag = i32(np.zeros((R, 3))), i32([0])
    cache = torch.zeros(pool, 2, PAGE, 64, dtype=torch.bfloat16, device="cuda")
    kv = vg.PagedKV(cache, cache.clone(), table)
    out = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    history = [[] for _ in range(R)]

    def append(new):
        n = int(np.sum(new))
        cu, kvl, pos, slots = out(R + 1), out(R), out(n), out(n)
        vg.step_tables(table, pool, lens, i32(new), cu, kvl, pos, slots, owned=owned, free_pages=free,
                       free_count=count, error_flag=flag)
        lens.copy_(kvl)
        token = rng.integers(1, 250, n)
        rows = torch.from_numpy(token).cuda().bfloat16()[:, None, None].expand(n, 2, 64).contiguous()
        vg.rope_append(kv, None, rows, rows, slots, error_flag=flag)
        at = 0
        for r in range(R):
            history[r] += token[at:at + new[r]].tolist()
            at += new[r]

    def reorder(parents):
        nonlocal history
        vg.beam_tables(table, pool, i32(parents), lens, owned, free, count, copies, error_flag=flag)
        vg.copy_pages(kv, copies, error_flag=flag)
        history = [list(history[b * W + p]) if p >= 0 else [] for b in range(B) for p in parents[b]]

    prompts = np.zeros(R, int)
    prompts[::W] = rng.integers(1, 100, B)
    append(prompts)
    reorder(np.zeros((B, W), int))
    for step in range(steps):
        append(np.array([1 if h else 0 for h in history]))
        parents = np.minimum(rng.geometric(0.5, (B, W)) - 1, W - 1)
        if step == steps // 2:
            parents[0] = -1
        reorder(parents)
        torch.cuda.synchronize()
        assert int(flag.item()) == 0
        t, o, n = table.cpu().numpy(), owned.cpu().numpy(), int(count.item())
        assert lens.cpu().tolist() == [len(h) for h in history]
        held = {}
        for r in range(R):
            for c in range(o[r]):
                held.setdefault(int(t[r, c]), set()).add((r // W, c))
        assert all(len(where) == 1 for where in held.values())
        loose = free.cpu().numpy()[:n].tolist()
        assert sorted(loose + list(held)) == list(range(pool))
        tails = [int(t[r, o[r] - 1]) for r in range(R) if len(history[r]) % PAGE]
        assert len(tails) == len(set(tails))
        for r, h in enumerate(history):
            for pool_ in (kv.k_pages, kv.v_pages):
                rows = pool_[t[r, :o[r]].tolist(), 1, :, 5].flatten().tolist()[:len(h)]
                assert rows == h, r


@pytest.mark.parametrize("Hkv,d", [(1, 64), (2, 128), (8, 128), (5, 64), (16, 64)])
@pytest.mark.parametrize("n", [1, 7, 60])
def test_copies(n, Hkv, d):
    from self_speculative_sparse_vg_gb300 import vg
    rng = np.random.default_rng(n + Hkv)
    ids = rng.permutation(2 * n + 3)
    copies = np.stack([ids[:n], ids[n:2 * n], rng.integers(0, 17, n)], 1)
    copies[rng.random(n) < 0.3] = (-1, -1, 0)
    for layers in (1, 3):
        pools = [torch.randn(2, 2 * n + 3, Hkv, PAGE, d).bfloat16() for _ in range(layers)]
        dev = [p.cuda() for p in pools]
        kv = [vg.PagedKV(p[0], p[1], i32([[0]])) for p in dev]
        flag = i32([0])
        vg.copy_pages(kv[0] if layers == 1 else kv, i32(copies), error_flag=flag)
        torch.cuda.synchronize()
        assert int(flag.item()) == 0
        for p, x in zip(pools, dev):
            for v in range(2):
                want = O.copy_pages(p[v].view(torch.int16).numpy(), copies)
                np.testing.assert_array_equal(x[v].cpu().view(torch.int16).numpy(), want)


def test_copies_of_more_layers_than_a_launch_takes():
    from self_speculative_sparse_vg_gb300 import vg
    x = torch.randn(130, 2, 4, 1, PAGE, 64).bfloat16().cuda()
    before = x.clone()
    kv = [vg.PagedKV(p[0], p[1], i32([[0]])) for p in x]
    vg.copy_pages(kv, i32([[2, 0, 9]]))
    before[:, :, 0, :, :9] = before[:, :, 2, :, :9]
    assert torch.equal(x, before)


def test_copies_that_are_none_are_flagged_and_skipped():
    from self_speculative_sparse_vg_gb300 import vg
    x = torch.randn(2, 6, 2, PAGE, 64).bfloat16().cuda()
    before = x.clone()
    for bad in ([-1, 2, 3], [6, 2, 3], [0, -1, 3], [0, 6, 3], [0, 1, 17], [0, 1, -1]):
        flag = i32([0])
        vg.copy_pages(vg.PagedKV(x[0], x[1], i32([[0]])), i32([bad]), error_flag=flag)
        assert int(flag.item()) == vg.DEVERR_PAGE and torch.equal(x, before)
    vg.copy_pages(vg.PagedKV(x[0], x[1], i32([[0]])), i32(np.zeros((0, 3))))


def test_on_a_stream_of_its_own_and_captured():
    rng = np.random.default_rng(8)
    c = make(rng, 6, 5, 100, 900, 9)
    a, b = run_beam_tables(**c), run_beam_tables(**c, stream=torch.cuda.Stream())
    for k in a:
        np.testing.assert_array_equal(a[k], b[k])
    from self_speculative_sparse_vg_gb300 import vg
    dev = {k: i32([c[k]] if k == "count" else c[k]) for k in ("table", "lens", "owned", "free", "count", "parents")}
    kept = {k: v.clone() for k, v in dev.items()}
    copies = i32(np.zeros((30, 3)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vg.beam_tables(dev["table"], c["num_pages"], dev["parents"], dev["lens"], dev["owned"], dev["free"],
                       dev["count"], copies)
    for _ in range(2):
        for k, v in kept.items():
            dev[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for k in ("table", "lens", "owned", "free"):
            np.testing.assert_array_equal(dev[k].cpu().numpy(), a[k])
        np.testing.assert_array_equal(copies.cpu().numpy(), a["copies"])


def test_binding_refusals():
    from self_speculative_sparse_vg_gb300 import vg
    i = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    good = dict(page_table=i(6, 4), num_pages=9, parents=i(2, 3), lens=i(6), owned=i(6), free_pages=i(9),
                free_count=i(1), copies=i(6, 3))
    vg.beam_tables(**good)
    for bad in (dict(page_table=i(24)), dict(page_table=i(5, 4)), dict(parents=i(6)), dict(parents=i(2, 4)),
                dict(lens=i(5)), dict(owned=i(7)), dict(free_count=i(2)), dict(copies=i(6, 2)), dict(num_pages=-1),
                dict(num_pages="x"), dict(lens=i(6).long()), dict(owned=i(6).cpu()), dict(page_table=i(4, 6).T),
                dict(error_flag=i(1).float())):
        with pytest.raises(ValueError):
            vg.beam_tables(**{**good, **bad})
    with pytest.raises(vg.VGError) as e:
        vg.beam_tables(i(33, 4), 9, i(1, 33), i(33), i(33), i(9), i(1), i(33, 3))
    assert e.value.status == 2
    p = torch.zeros(4, 2, PAGE, 64, dtype=torch.bfloat16, device="cuda")
    kv = vg.PagedKV(p, p.clone(), i(1, 1))
    other = vg.PagedKV(p[:3].clone(), p[:3].clone(), i(1, 1))
    for bad in (([kv, other], i(2, 3)), (kv, i(6)), (kv, i(2, 4)), (kv, i(2, 3).cpu()), ([], i(2, 3))):
        with pytest.raises(ValueError):
            vg.copy_pages(*bad)
