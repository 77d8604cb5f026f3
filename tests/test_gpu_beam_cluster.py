"""Block tables of beams whose CTAs of one cluster have unequal work: wide tables of
few columns, so that most CTAs find no tile and exchange their counts at once, and
tables whose columns all lie in the last requests."""
import numpy as np
import pytest

from oracle import beam_oracle as O
from tests.beam_util import run_beam_tables
from tests.fill_util import PAGE

pytestmark = pytest.mark.gpu


def _case(rng, B, W, cols, width):
    """Request b has cols[b] columns, of which its rows share all but the last two."""
    lens, table = np.zeros(B * W, int), np.full((B * W, width), -1)
    pool = sum(c + 2 * W for c in cols) + B * W + 3
    ids, at = rng.permutation(pool), 0
    for b, c in enumerate(cols):
        common = max(0, c - 2)
        shared, at = ids[at:at + common], at + common
        for r in range(b * W, (b + 1) * W):
            table[r, :common] = shared
            table[r, common:c] = ids[at:at + c - common]
            at += c - common
            lens[r] = max(0, PAGE * c - int(rng.integers(0, PAGE)))
    free = np.concatenate([ids[at:], np.full(at + 3, -1)])
    return dict(lens=lens, table=table, num_pages=pool, owned=-(-lens // PAGE), free=free, count=pool - at)


@pytest.mark.parametrize("B,cols", [(2, [1, 0]), (2, [0, 3]), (5, [0, 0, 0, 0, 2000]), (5, [2000, 0, 0, 0, 0]),
                                    (16, [0] * 15 + [40]), (64, [1] * 64), (3, [0, 0, 0])])
@pytest.mark.parametrize("width", [2100, 40000])
def test_ctas_without_columns(B, cols, width):
    rng = np.random.default_rng(B + width)
    W = 4
    c = _case(rng, B, W, cols, width)
    want, parents = None, None
    for turn in range(20):
        if turn % 10 == 0:
            parents = rng.integers(-1, W, (B, W))
            want = O.beam_tables(parents, c["lens"], c["table"], c["num_pages"], c["owned"], c["free"], c["count"])
        got = run_beam_tables(parents, **c)
        for k in want:
            np.testing.assert_array_equal(got[k], want[k], err_msg=k)


def test_calls_in_a_row():
    """Two hundred calls with nothing between them, each on what the last one left."""
    import torch
    from self_speculative_sparse_vg_gb300 import vg
    from tests.fill_util import i32
    rng = np.random.default_rng(7)
    B, W, width = 6, 4, 6000
    c = _case(rng, B, W, [0, 5, 0, 900, 2, 3000], width)
    parents = [rng.integers(0, W, (B, W)) for _ in range(200)]
    dev = {k: i32([c[k]] if k == "count" else c[k]) for k in ("table", "lens", "owned", "free", "count")}
    copies, flag, par = i32(np.zeros((B * W, 3))), i32([0]), [i32(x) for x in parents]
    torch.cuda.synchronize()
    for x in par:
        vg.beam_tables(dev["table"], c["num_pages"], x, dev["lens"], dev["owned"], dev["free"], dev["count"], copies,
                       error_flag=flag)
    torch.cuda.synchronize()
    at = [c[k] for k in ("lens", "table", "owned", "free", "count")]
    for x in parents:
        w = O.beam_tables(x, at[0], at[1], c["num_pages"], at[2], at[3], at[4])
        at = [w[k] for k in ("lens", "table", "owned", "free", "count")]
    assert int(flag.item()) == 0 == w["flag"]
    for k, v in zip(("lens", "table", "owned", "free"), at):
        np.testing.assert_array_equal(dev[k].cpu().numpy(), v, err_msg=k)
    assert int(dev["count"].item()) == at[4]
    np.testing.assert_array_equal(copies.cpu().numpy(), w["copies"])
