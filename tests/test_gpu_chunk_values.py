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
