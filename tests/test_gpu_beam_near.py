"""Selection among logits of one beam that are too near to one another for their
scores to differ."""
import numpy as np
import pytest
import torch

from tests.beam_util import run_select

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("W,K,V", [(1, 8, 20000), (1, 64, 120001), (4, 8, 50000), (5, 40, 9000), (32, 64, 20000)])
@pytest.mark.parametrize("order", ["rising", "any"])
def test_logits_nearer_than_their_scores(order, W, K, V, dtype):
    """64 logits of i 1e-20 (in bfloat16 still different ones) in a row of -5s beside a
    score of -10: the differences are 2^-63 of the score and more lists than one hold
    them.  Equal rows have equal scores, so all places go to the lowest beams, 64
    tokens each, larger logits first."""
    rng = np.random.default_rng(V + K)
    at = np.sort(rng.choice(V, 64, replace=False))
    if order == "any":
        at = rng.permutation(at)
    x = torch.full((2 * W, V), -5.0)
    x[:, torch.from_numpy(at)] = torch.arange(1, 65) * 1e-20
    x = x.to(dtype)
    assert len(set(x[0, torch.from_numpy(at)].tolist())) == 64
    score, token, parent, _, flag = run_select(x, np.full((2, W), -10.0, np.float32), K)
    assert flag == 0
    for b in range(2):
        assert parent[b].tolist() == [0] * K
        assert token[b].tolist() == at[::-1][:K].tolist()
        assert (np.diff(score[b]) == 0).all()


def test_near_logits_of_ended_and_living_beams():
    """The same among beams of other scores: the places of each beam hold its first
    tokens in the order of their logits, whatever lies between."""
    rng = np.random.default_rng(3)
    W, V, K = 6, 30000, 24
    x = torch.full((W, V), -7.0)
    at = [rng.permutation(V)[:10] for _ in range(W)]
    for w in range(W):
        x[w, torch.from_numpy(at[w])] = torch.arange(1, 11) * 1e-19
    s = np.array([[-3.0, -3.0, -3.0000002, -2.9999998, -3.0, -3.0]], np.float32)
    _, token, parent, marks, flag = run_select(x, s, K, ended=np.array([[0, 0, 0, 0, 1, 0]]), end_token=5)
    assert flag == 0
    for w in range(W):
        mine = token[0][parent[0] == w].tolist()
        assert mine == ([5] if w == 4 else at[w][::-1].tolist())[:len(mine)]
