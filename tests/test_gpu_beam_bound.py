"""Scores of the selection under the bound that a slice's size allows."""
import numpy as np
import pytest
import torch

from tests.beam_util import run_select

pytestmark = pytest.mark.gpu

SLICE_WORDS, THREADS = 32 * 1024 // 4, 256


def bound(spread, vocab, size, score):
    """How far a score may be from the exact one.  A slice holds 32 KB at most, of which
    a thread adds SLICE_WORDS / THREADS words of two logits; 5 + 8 + 5 + 1 sums follow;
    an exponential is off by 2^-22 and by its argument's three roundings, 2^-24 of the
    distance from the maximum each, under the softmax `spread`; expf (2 ulp), its sum
    and the logarithm's parts 2^-22; the result is rounded once."""
    words = min(-(-vocab * size // 4), SLICE_WORDS)
    adds = 2 * -(-words // THREADS) + 19
    return 2.0 ** -24 * (adds + 4 + 3 * spread + 8 + abs(score)) + 1e-37


@pytest.mark.parametrize("dtype,V", [(torch.float32, 786432), (torch.float32, 128256), (torch.bfloat16, 1572864),
                                     (torch.bfloat16, 128256), (torch.float16, 600001), (torch.float32, 8192)])
@pytest.mark.parametrize("spread", [0.0, 0.01, 2.5, 8.0, 40.0])
def test_scores(spread, dtype, V):
    """Full slices of equal, nearly equal and far apart logits: in the first the error is
    that of the sums alone."""
    W, K = 3, 6
    x = (torch.randn(2 * W, V, generator=torch.Generator().manual_seed(V)) * spread).to(dtype)
    s = -np.arange(2 * W, dtype=np.float32).reshape(2, W) - 4
    score, token, parent, _, flag = run_select(x, s, K)
    assert flag == 0 and (token >= 0).all()
    y = x.double().numpy()
    m = y.max(1, keepdims=True)
    e = np.exp(y - m)
    z = e.sum(1, keepdims=True)
    distance = (e * (m - y)).sum(1) / z[:, 0]
    for b in range(2):
        for i in range(K):
            w, t = int(parent[b, i]), int(token[b, i])
            r = b * W + w
            want = float(s[b, w]) + y[r, t] - m[r, 0] - np.log(z[r, 0])
            off = abs(score[b, i] - want)
            assert off <= bound(distance[r], V, x.element_size(), want), (b, i, off)
