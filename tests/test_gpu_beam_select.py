"""The selection over beams and vocabulary on the GPU against the float64
oracle: types, odd vocabularies, strides, ties, bans, beams that ended or do not
live, values that are not finite, refusals, graphs."""
import numpy as np
import pytest
import torch

from tests.beam_util import check_select, run_select

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
INF = float("inf")


def _logits(rows, V, dtype, seed, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, V, generator=g) * spread).to(dtype)


def _scores(B, W, seed):
    rng = np.random.default_rng(seed)
    return (-rng.random((B, W)).cumsum(1) * 2 - 3).astype(np.float32)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1, 2, 3, 7, 15, 16, 17, 31, 63, 255, 256, 511, 513, 1000, 4097, 16385, 50257, 128256])
def test_vocabularies(V, dtype):
    B, W = 2, 3
    check_select(_logits(B * W, V, dtype, V), _scores(B, W, V), 4)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("W,K", [(1, 1), (1, 64), (2, 5), (4, 8), (5, 10), (8, 16), (9, 33), (16, 32), (32, 64), (32, 1)])
def test_beams_and_places(W, K, dtype):
    check_select(_logits(2 * W, 5003, dtype, W), _scores(2, W, K), K)


@pytest.mark.parametrize("B", [1, 30, 400])
def test_batches(B):
    check_select(_logits(B * 3, 3001, torch.bfloat16, B), _scores(B, 3, B), 6)


@pytest.mark.parametrize("dtype,V", [(torch.float32, 786432), (torch.bfloat16, 1572864), (torch.float16, 600001)])
def test_the_longest_rows(dtype, V):
    check_select(_logits(2, V, dtype, 3), _scores(1, 2, 1), 8)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shift", [1, 2, 3, 5, 8])
def test_slices_of_wider_rows(shift, dtype):
    """Rows that begin anywhere, in a buffer with NaN around them."""
    V, rows = 1237, 6
    wide = torch.full((rows, V + 20 + shift), float("nan"), dtype=dtype)
    x = _logits(rows, V, dtype, shift)
    wide[:, shift:shift + V] = x
    dev = wide.cuda()[:, shift:shift + V]
    a = run_select(dev, _scores(2, 3, 5), 7)
    b = run_select(x, _scores(2, 3, 5), 7)
    for u, w in zip(a, b):
        np.testing.assert_array_equal(u, w)
    check_select(dev, _scores(2, 3, 5), 7)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [40, 2000, 33001])
@pytest.mark.parametrize("value", ["equal", "lowest", "few", "steps", "zeros"])
def test_ties_go_to_the_lowest(value, V, dtype):
    """Rows of equal values, most of a row at the type's lowest or -inf, a few
    different values, and zeros of both signs: more candidates than a slice lists."""
    g = torch.Generator().manual_seed(V)
    x = torch.full((4, V), 0.75)
    if value == "lowest":
        x[:] = torch.finfo(dtype).min
        x[:, torch.randint(0, V, (9,), generator=g)] = 3.0
    elif value == "few":
        x = torch.randint(0, 3, (4, V), generator=g).float()
    elif value == "steps":
        x = torch.randint(0, 3, (4, V), generator=g).float()
        x[torch.rand(4, V, generator=g) < 0.7] = -INF
    elif value == "zeros":
        x = torch.where(torch.rand(4, V, generator=g) < 0.5, 0.0, -0.0)
    for K in (1, 6, 20, 50):
        check_select(x.to(dtype), _scores(2, 2, K), K)


@pytest.mark.parametrize("dtype", TYPES)
def test_equal_beams_go_to_the_lower(dtype):
    """Beams of the same logits and score, in rows that begin on different bytes."""
    V = 12345
    x = _logits(1, V, dtype, 4).expand(8, V).contiguous()
    check_select(x, np.full((2, 4), -2.5, np.float32), 10, exactly=True)


@pytest.mark.parametrize("dtype", TYPES)
def test_beams_that_do_not_live_or_have_ended(dtype):
    V, W = 3333, 5
    s = _scores(6, W, 2)
    s[0, 1:] = -INF                          # a first step
    s[1, 1:] = -1e9
    s[2, 2:] = np.finfo(np.float32).min      # so low that sums may leave float's range
    s[3, :] = -INF                           # nothing lives
    s[4, 3] = -INF
    ended = np.zeros((6, W), bool)
    ended[4, [0, 3]] = True                  # an ended beam at -inf offers nothing
    ended[5, :] = True
    x = _logits(6 * W, V, dtype, 9)
    x[4 * W] = float("nan")                  # an ended beam's logits are not read
    x[3 * W + 1] = INF                       # nor those of a beam at -inf
    for K in (5, 10, 20):
        check_select(x, s, K, ended=ended, end_token=7)
        check_select(x, s, K, ended=ended, end_token=2 * V, with_ended=False)


@pytest.mark.parametrize("dtype", TYPES)
def test_bans(dtype):
    """-infinity bans tokens: of a row, of most, of all but one, of all."""
    V = 2222
    x = _logits(8, V, dtype, 1)
    g = torch.Generator().manual_seed(3)
    x[0, torch.rand(V, generator=g) < 0.5] = -INF
    x[1, 1:] = -INF
    x[2, :-1] = -INF
    x[3] = -INF
    x[4:, 5:] = -INF                         # a request with fewer candidates than places
    check_select(x, _scores(2, 4, 3), 24, end_token=1)


@pytest.mark.parametrize("dtype", TYPES)
def test_values_that_are_not_finite_are_flagged(dtype):
    """The beam offers nothing, the others are served."""
    V = 5000
    for at, bad in ((0, float("nan")), (V - 1, INF), (2500, float("nan")), (17, INF)):
        x = _logits(4, V, dtype, at)
        x[1, at] = bad
        check_select(x, _scores(1, 4, at), 8)
        x[1] = -INF
        x[1, at] = bad
        check_select(x, _scores(1, 4, at), 8)
    for bad in (float("nan"), INF):
        s = _scores(2, 2, 1)
        s[1, 0] = bad
        check_select(_logits(4, V, dtype, 5), s, 8)
        check_select(_logits(4, V, dtype, 5), s, 8, ended=np.array([[0, 0], [1, 0]]))


def test_large_and_small_spreads():
    for spread in (1e-6, 0.01, 30.0, 1000.0):
        check_select(_logits(6, 7001, torch.float32, 2, spread), _scores(2, 3, 4), 6)
        check_select(_logits(6, 7001, torch.bfloat16, 3, spread), _scores(2, 3, 4) * 100, 6)


def test_in_place_and_captured():
    """out_scores over scores and out_ended over ended, three steps in one graph."""
    from self_speculative_sparse_vg_gb300 import vg
    B, W, V = 3, 4, 9001
    xs = [_logits(B * W, V, torch.bfloat16, i).cuda() for i in range(3)]
    s0 = torch.from_numpy(_scores(B, W, 0)).cuda()
    ended0 = torch.zeros(B, W, dtype=torch.bool, device="cuda")
    ended0[1, 2] = True

    def steps(s, ended, apart):
        seen = []
        for x in xs:
            o, e = (torch.empty_like(s), torch.empty_like(ended)) if apart else (s, ended)
            t, p = (torch.zeros(B, W, dtype=torch.int32, device="cuda") for _ in range(2))
            vg.beam_select(x, s, o, t, p, ended=ended, end_token=5, out_ended=e)
            s, ended = o, e
            seen += [t, p]
        return [s, ended] + seen
    want = steps(s0, ended0, True)
    s, ended = s0.clone(), ended0.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = steps(s, ended, False)
    for _ in range(2):
        s.copy_(s0)
        ended.copy_(ended0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_on_a_stream_of_its_own():
    x, s = _logits(8, 60000, torch.float16, 2), _scores(2, 4, 1)
    a, b = run_select(x, s, 8), run_select(x, s, 8, stream=torch.cuda.Stream())
    for u, w in zip(a, b):
        np.testing.assert_array_equal(u, w)


def test_binding_refusals():
    from self_speculative_sparse_vg_gb300 import vg
    f = lambda *n, dt=torch.float32: torch.zeros(*n, dtype=dt, device="cuda")  # noqa: E731
    i = lambda *n: f(*n, dt=torch.int32)  # noqa: E731
    good = dict(logits=f(6, 50), scores=f(2, 3), out_scores=f(2, 4), out_tokens=i(2, 4), out_parents=i(2, 4))
    vg.beam_select(**good)
    for bad in (dict(logits=f(6, 50, dt=torch.float64)), dict(logits=f(5, 50)), dict(logits=f(50, 6).T),
                dict(logits=f(300)), dict(scores=f(6)), dict(scores=f(2, 3, dt=torch.float16)),
                dict(out_scores=f(3, 4)), dict(out_scores=f(2, 4).double()), dict(out_tokens=i(2, 3)),
                dict(out_tokens=f(2, 4)), dict(out_parents=i(2, 5)), dict(ended=f(2, 2, dt=torch.bool)),
                dict(ended=f(2, 3)), dict(out_ended=f(2, 3, dt=torch.bool)), dict(end_token="x"),
                dict(end_token=1 << 40), dict(scores=f(2, 3).cpu()), dict(error_flag=f(1))):
        with pytest.raises((ValueError, TypeError)):
            vg.beam_select(workspace=f(1 << 20, dt=torch.uint8), **{**good, **bad})
    for shape, K, status in (((33, 1), 4, 2), ((3, 2), 65, 2), ((3, 2), 0, 1)):
        W, B = shape
        with pytest.raises(vg.VGError) as e:
            vg.beam_select(f(B * W, 50), f(B, W), f(B, K), i(B, K), i(B, K), workspace=f(1 << 20, dt=torch.uint8))
        assert e.value.status == status
    with pytest.raises(vg.VGError) as e:
        vg.beam_select(**good, workspace=f(16, dt=torch.uint8))
    assert e.value.status == 3
    with pytest.raises(vg.VGError) as e:
        vg.beam_select(**good, workspace=f(1 << 20, dt=torch.uint8)[1:])
    assert e.value.status == 1
