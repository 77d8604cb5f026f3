"""Cross attention of rows of which one state has a far larger score than all others,
that together still matter: weights that lie below fp16's normal range beside the
largest."""
import numpy as np
import pytest
import torch

from oracle import beam_oracle as O
from tests.beam_util import HALF_STEP
from tests.fill_util import i32

pytestmark = pytest.mark.gpu


def bounds(out, lse, A, S, count, d, dtype, vmax):
    """The output is rounded once and each weight may be, by half a step or, in fp16, by
    2^-32 of the largest weight, which is a row's unit here; an fp16 output below 2^-14
    by 2^-25.  Scores are float32 sums of d products (S bounds their magnitudes) and
    shift a weight by that much; `count` float32 additions make the sums."""
    rel = 2.0 * (d + 8) * 2.0 ** -23 * (S + 1.0) + 2.0 * count * 2.0 ** -23 + 2.0 ** -20
    tol = HALF_STEP[dtype] * (np.abs(out) + A) * 1.01 + rel[..., None] * A + 1e-30
    if dtype == torch.float16:
        tol += count * vmax * 2.0 ** -32 + 2.0 ** -25
    return tol, rel + 2.0 ** -22 * np.abs(lse)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("powers", [21.0, 25.5, 27.0, 31.0])
@pytest.mark.parametrize("rows,Hq,Hkv,d", [(1, 2, 2, 64), (3, 4, 1, 128), (1, 3, 1, 64), (33, 1, 1, 128), (50, 2, 2, 64),
                                           (200, 1, 1, 64)])
@pytest.mark.parametrize("where", ["first", "last", "any"])
def test_one_state_far_above_the_others(where, rows, Hq, Hkv, d, powers, dtype):
    """Each of 160 sequences has 1500 states or so whose weights are 2^-powers of the one
    largest and nearby, and whose values that one does not hide (its own are zeros)."""
    from self_speculative_sparse_vg_gb300 import vg
    batch = 160 if rows < 100 else 40
    rng = np.random.default_rng(int(powers * 10) + rows)
    lens = rng.integers(1300, 1700, batch)
    starts = np.concatenate([[0], np.cumsum(lens)[:-1]])
    total = int(lens.sum())
    g = torch.Generator().manual_seed(rows + d)
    k = torch.zeros(total, Hkv, d)
    # scores 4 k0 in natural units: ln 2 per power
    k[:, :, 0] = -powers * np.log(2.0) / 4 + 0.2 * torch.rand(total, Hkv, generator=g)
    v = 0.5 + torch.rand(total, Hkv, d, generator=g)
    at = {"first": starts, "last": starts + lens - 1, "any": starts + rng.integers(0, lens)}[where]
    k[torch.from_numpy(at), :, 0] = 0.0
    v[torch.from_numpy(at)] = 0.0
    q = torch.zeros(batch * rows, Hq, d)
    q[:, :, 0] = 4.0
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    out = torch.zeros(batch * rows, Hq, d, dtype=dtype, device="cuda")
    lse = torch.zeros(batch * rows, Hq, device="cuda")
    flag = i32([0])
    vg.cross_attention(q.cuda(), k.cuda(), v.cuda(), i32(np.arange(batch + 1) * rows), i32(starts), i32(lens), 1.0,
                       out, lse=lse, error_flag=flag)
    torch.cuda.synchronize()
    assert int(flag.item()) == 0
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for e in range(batch):
        r, s = slice(e * rows, (e + 1) * rows), slice(int(starts[e]), int(starts[e] + lens[e]))
        n = int(lens[e])
        # all rows of a sequence are alike
        ro, rl, A, S = O.cross_attention(q[r][:1].double().numpy(), k[s].double().numpy(), v[s].double().numpy(),
                                         np.ones(n, bool), 1.0)
        tol, tol_l = bounds(ro, rl, A, S, n, d, dtype, 1.5)
        worst = np.max(np.abs(got[r] - ro) / tol)
        assert worst <= 1.0, f"sequence {e}: {worst:.2f} times the bound"
        assert (np.abs(gl[r] - rl) <= tol_l).all(), f"lse of sequence {e}"
