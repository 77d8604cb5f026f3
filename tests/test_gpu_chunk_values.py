"""Chunk attention over values that are not finite: where they show, whatever
units the CTAs' shares make of the rows, and nowhere else."""
import numpy as np
import pytest
import torch

from tests.fill_util import Cache, check_chunk, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
def test_notes_of_one_unit_do_not_reach_later_ones(d):
    """Every CTA takes many units: pairs of short chunks whose last value is NaN
    in some dimensions, then a longer chunk (mostly cut, its front part without
    a position tile that needs a look), which uses the first pair's slot."""
    from self_speculative_sparse_vg_gb300 import vg
    lens, new = [], []
    for i in range(330):
        lens += [40 + i % 7, 33 + i % 5, 1500 + 37 * (i % 23)]
        new += [3, 2, 6]
    c = Cache(lens, 1, d, seed=31)
    qd, want, want_lse = check_chunk(c, new, 4)
    cu = np.concatenate([[0], np.cumsum(new)])
    w = want.clone()
    for b in range(len(new)):
        if new[b] < 6:
            v = c.v[b].clone()
            dims = [b % d, (b * 7 + d // 2) % d]
            v[-1, 0, dims] = float("nan")
            c.write(b, c.k[b], v)
            for x in dims:
                w[int(cu[b + 1]) - 1, :, x] = float("nan")
    for _ in range(3):
        out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
        vg.chunk_attention(c.gpu(), qd, i32(cu), i32(lens), d ** -0.5, out, lse=lse)
        assert torch.equal(out.isnan(), w.isnan())
        assert torch.equal(out[~w.isnan()], w[~w.isnan()]) and torch.equal(lse, want_lse)


INF, NAN = float("inf"), float("nan")


def _special(c, Hq, new, want, values=(), keys=(), seed=5):
    """One call over sequence 0 of `c` after values[(position, dim)] and
    keys[(position, dim)] were put into V and K; (out, want) with what the
    formula gives: a value that is not finite adds to every row that attends it,
    a NaN in a key makes NaN of every row that attends it."""
    from self_speculative_sparse_vg_gb300 import vg
    L, d = c.lens[0], c.kp.shape[3]
    k, v, w = c.k[0].clone(), c.v[0].clone(), want.clone()
    for (p, x), value in dict(values).items():
        v[p, 0, x] = value
        w[max(0, p - (L - new)):, :Hq, x] += value
    for (p, x), value in dict(keys).items():
        k[p, 0, x] = value
        w[max(0, p - (L - new)):, :Hq] = NAN
    c.write(0, k, v)
    q = torch.randn(new, Hq, d, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
    out = torch.zeros_like(q)
    vg.chunk_attention(c.gpu(), q, i32([0, new]), i32([L]), d ** -0.5, out)
    return out, w


def _same(out, want):
    assert torch.equal(out.isnan(), want.isnan())
    assert torch.equal(out[~out.isnan()], want[~want.isnan()])


# one tile, which no cut divides, of one row tile or two; a few tiles, each in a
# part of its own; long ones
SHAPES = [(64, 100, 30, 4), (128, 120, 50, 4), (128, 128, 3, 8), (64, 200, 60, 4), (128, 300, 9, 4), (64, 30011, 90, 4), (128, 20003, 5, 2), (64, 9001, 1, 8)]


@pytest.mark.parametrize("d,L,new,Hq", SHAPES)
def test_values_of_both_kinds_add_up(d, L, new, Hq):
    """In one dimension, a value before the chunk (in a tile that needs no look,
    and in the one that does) and another inside it."""
    c = Cache([L], 1, d, seed=32)
    _, want, _ = check_chunk(c, [new], Hq)
    pos0 = L - new
    inside = pos0 + new // 2
    values = {}
    for at, (a, b) in enumerate([(NAN, INF), (-INF, INF), (INF, -INF), (INF, INF), (NAN, -INF), (-INF, -INF),
                                 (INF, NAN)]):
        values[(3, 2 * at)] = a                     # a far position
        values[(pos0, d - 2 - 2 * at)] = a          # the first row's own
        if new > 1:
            values[(inside, 2 * at)] = b
            values[(inside, d - 2 - 2 * at)] = b
    _same(*_special(c, Hq, new, want, values))


@pytest.mark.parametrize("d,L,new,Hq", SHAPES)
def test_rows_of_nan_scores_stay_nan(d, L, new, Hq):
    """A NaN in a key makes all of a row NaN, dimensions of an infinite value too."""
    c = Cache([L], 1, d, seed=33)
    _, want, _ = check_chunk(c, [new], Hq)
    _same(*_special(c, Hq, new, want, {(L - 1, 5): INF, (L - 1, d - 1): -INF}, {(1, 3): NAN}))


# a CTA per row merges up to 32 rows, one per 32 rows more of them
@pytest.mark.parametrize("falls", [False, True])
@pytest.mark.parametrize("d,new,Hq", [(64, 1, 4), (128, 1, 8), (64, 40, 4), (128, 33, 2), (64, 1, 1)])
def test_a_part_of_no_weight_still_shows_what_is_not_finite(d, new, Hq, falls):
    """Scores that rise or fall by hundreds along the positions: the first or
    the last parts weigh nothing, but a NaN or an infinity that a row attends
    there shows, and a NaN score makes the row NaN."""
    from self_speculative_sparse_vg_gb300 import vg
    L = 20000
    c = Cache([L], 1, d, seed=34)
    ramp = (torch.arange(L) * ((-400.0 if falls else 400.0) / L) / (0.5 * d ** 0.5))[:, None, None]
    c.k[0] = (c.k[0].float() * 0.1 + ramp).bfloat16()
    c.write(0, c.k[0], c.v[0])
    q = torch.full((new, Hq, d), 0.5, dtype=torch.bfloat16)
    _, want, want_lse = check_chunk(c, [new], Hq, q=q)

    def call():
        out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
        vg.chunk_attention(c.gpu(), q.cuda(), i32([0, new]), i32([L]), d ** -0.5, out, lse=lse)
        return out, lse
    v = c.v[0].clone()
    at = (lambda p: L - 1 - new - p) if falls else (lambda p: p)  # noqa: E731
    v[at(3), 0, 2], v[at(5), 0, 4], v[at(9000), 0, d - 1] = NAN, INF, -INF
    c.write(0, c.k[0], v)
    out, lse = call()
    bad = [2, 4, d - 1]
    rest = [x for x in range(d) if x not in bad]
    assert torch.equal(out[..., rest], want[..., rest]) and torch.equal(lse, want_lse)
    assert out[..., 2].isnan().all() and not out[..., bad].isfinite().any()
    k = c.k[0].clone()
    k[at(7), 0, 1] = NAN
    c.write(0, k, c.v[0])
    out, lse = call()
    assert out.isnan().all() and lse.isnan().all()


@pytest.mark.parametrize("L,new", [(1, 1), (100, 7), (20000, 3), (5000, 80)])
def test_rows_whose_scores_are_all_minus_infinity(L, new):
    """Zero, with a log-sum-exp of -infinity, as rows that attend nothing.  (The
    heads whose queries are zero in that dimension have NaN scores.)"""
    from self_speculative_sparse_vg_gb300 import vg
    c = Cache([L], 1, 64, seed=35)
    g = torch.Generator().manual_seed(6)
    q = torch.randn(new, 4, 64, generator=g).bfloat16()
    q[:, :, 9] = 0                       # the dimension that is -infinity in every key
    _, want, want_lse = check_chunk(c, [new], 4, q=q)
    q[:, 1, 9] = 1.0
    k = c.k[0].clone()
    k[:, 0, 9] = -INF
    c.write(0, k, c.v[0])
    out, lse = torch.full_like(want, 3.0), torch.full_like(want_lse, 3.0)
    vg.chunk_attention(c.gpu(), q.cuda(), i32([0, new]), i32([L]), 0.125, out, lse=lse)
    assert (out[:, 1] == 0).all() and torch.isneginf(lse[:, 1]).all()
    assert out[:, [0, 2, 3]].isnan().all()
