"""Refusals of the calls for beams and encoder states (no GPU), and pins of
their oracle."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

from oracle import beam_oracle as O
from tests.conftest import ensure_lib

FAKE = 0x4000
INF = float("inf")


@pytest.fixture(scope="module")
def vg():
    ensure_lib()
    from self_speculative_sparse_vg_gb300 import vg
    return vg


def test_cross_attention_refusals(vg):
    def call(**kw):
        a = dict(q=FAKE, qs=4096, k=FAKE, ks=1024, v=FAKE, vs=1024, type=1, cu=FAKE, starts=FAKE, lens=FAKE,
                 mask=None, b=2, n=5, s=100, hq=32, hkv=8, d=128, scale=0.1, o=FAKE, os=4096, lse=None, ws=None,
                 wsb=0, flag=None, stream=None)
        a.update(kw)
        return vg._lib.vg_cross_attention(*a.values())
    for name in ("q", "k", "v", "cu", "starts", "lens", "o"):
        assert call(**{name: None}) == 1, name
    for name in ("q", "k", "v", "o"):
        assert call(**{name: FAKE + 8}) == 1, name          # not on 16 bytes
    for name in ("qs", "os"):
        assert call(**{name: 4088}) == 1 and call(**{name: 4100}) == 1, name
    for name in ("ks", "vs"):
        assert call(**{name: 1016}) == 1 and call(**{name: 1028}) == 1, name
    for name in ("b", "hq", "hkv", "d"):
        assert call(**{name: 0}) == 1 and call(**{name: -1}) == 1, name
    assert call(n=-1) == 1 and call(s=-1) == 1 and call(hq=33) == 1
    for scale in (0.0, -1.0, float("nan"), INF):
        assert call(scale=scale) == 1, scale
    assert call(type=0) == 2 and call(type=3) == 2 and call(d=96) == 2 and call(b=4097) == 2
    assert call(hq=129 * 8, qs=1 << 20, os=1 << 20) == 2 and call(s=(1 << 30) + 1) == 2
    assert call(n=0) == 0                                   # nothing to do, nothing launched
    need = vg._lib.vg_cross_workspace_bytes(2, 5, 32, 8, 128)
    assert need > 0 and call() == 3 and call(ws=FAKE, wsb=need - 1) == 3
    assert call(s=0, k=None, v=None) == 3                   # without states there is nothing to read
    for off in (1, 4, 8):
        assert call(ws=FAKE + off, wsb=need + 64) == 1, off
    for bad in ((0, 5, 32, 8, 128), (2, 0, 32, 8, 128), (2, 5, 33, 8, 128), (2, 5, 32, 8, 96), (2, 5, 1032, 8, 128)):
        assert vg._lib.vg_cross_workspace_bytes(*bad) == 0, bad


def test_beam_select_refusals(vg):
    def call(**kw):
        a = dict(x=FAKE, type=1, stride=1000, s=FAKE, e=None, end=2, b=2, w=4, v=1000, k=8, os=FAKE, ot=FAKE, op=FAKE,
                 oe=None, ws=None, wsb=0, flag=None, stream=None)
        a.update(kw)
        return vg._lib.vg_beam_select(*a.values())
    for name in ("x", "s", "os", "ot", "op"):
        assert call(**{name: None}) == 1, name
    for name in ("b", "w", "v", "k"):
        assert call(**{name: 0}) == 1 and call(**{name: -1}) == 1, name
    assert call(stride=999) == 1 and call(stride=-1000) == 1
    assert call(x=FAKE + 1) == 1 and call(x=FAKE + 2, type=0) == 1
    assert call(type=3) == 2 and call(type=-1) == 2 and call(w=33) == 2 and call(k=65) == 2
    assert call(v=2_000_000, stride=2_000_000) == 2         # rows of more than 3 MB
    assert call(v=800_000, stride=800_000, type=0) == 2
    need = vg._lib.vg_beam_select_workspace_bytes(2, 4, 1000, 1, 8)
    assert need > 0 and call() == 3 and call(ws=FAKE, wsb=need - 1) == 3
    assert call(ws=FAKE + 8, wsb=need + 64) == 1
    for bad in ((0, 4, 1000, 1, 8), (2, 33, 1000, 1, 8), (2, 4, 0, 1, 8), (2, 4, 1000, 4, 8), (2, 4, 1000, 1, 65),
                (2, 4, 2_000_000, 1, 8)):
        assert vg._lib.vg_beam_select_workspace_bytes(*bad) == 0, bad


def test_beam_tables_refusals(vg):
    good = [FAKE, 4, 3, FAKE, FAKE, 64, 100, FAKE, FAKE, 100, FAKE, FAKE, None, None]

    def call(**kw):
        a = list(good)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return vg._lib.vg_beam_tables(*a)
    for i in (0, 3, 4, 7, 8, 10, 11):
        assert call(**{f"a{i}": None}) == 1, i
    for i in (1, 2, 5, 6, 9):
        assert call(**{f"a{i}": 0}) == 1 and call(**{f"a{i}": -1}) == 1, i
    assert call(a2=33) == 2 and call(a1=1366) == 2 and call(a6=1 << 28) == 2 and call(a5=1 << 28) == 2
    assert call(a1=1000, a5=1 << 22) == 2


def test_copy_pages_refusals(vg):
    def call(layers=2, pages=10, heads=8, d=128, copies=FAKE, n=3, k=(0x1000, 0x2000), v=(0x3000, 0x4000)):
        arr = lambda x: None if x is None else (ctypes.c_void_p * len(x))(*x)  # noqa: E731
        return vg._lib.vg_copy_pages(arr(k), arr(v), layers, pages, heads, d, copies, n, None, None)
    assert call(n=0) == 0 and call(layers=0) == 0           # nothing to do, nothing launched
    assert call(k=None) == 1 and call(v=None) == 1 and call(copies=None) == 1
    for kw in (dict(layers=-1), dict(pages=0), dict(heads=0), dict(d=0), dict(n=-1), dict(k=(0x1000, 0)),
               dict(v=(0x3000, 0x4008))):
        assert call(**kw) == 1, kw
    assert call(d=96) == 2


def test_what_is_no_tensor_or_not_on_a_gpu_is_refused(vg):
    i = torch.zeros(1, dtype=torch.int32)
    f, h = torch.zeros(1, 1), torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    for bad in (None, 3, "x", i):
        with pytest.raises(ValueError):
            vg.cross_attention(bad, h, h, i, i, i, 1.0, h, workspace=i)
        with pytest.raises(ValueError):
            vg.beam_select(bad, f, f, i, i, workspace=i)
        with pytest.raises(ValueError):
            vg.beam_tables(bad, 3, i, i, i, i, i, i)
    with pytest.raises(ValueError):
        vg.beam_tables(i.view(1, 1), 3, i.view(1, 1), i, i, i, i, torch.zeros(1, 3, dtype=torch.int32))
    p = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        vg.copy_pages(vg.PagedKV(p, p, i.view(1, 1)), torch.zeros(1, 3, dtype=torch.int32))
    assert vg.beam_select_workspace_bytes(1, 1, 10, torch.float64, 1) == 0


@pytest.mark.parametrize("name", ["cross_attention", "beam_select", "beam_tables", "copy_pages"])
def test_a_wrong_number_of_arguments_is_a_type_error(vg, name):
    from self_speculative_sparse_vg_gb300 import vg_binding
    with pytest.raises(TypeError):
        getattr(vg_binding, name)(1, 2)


# ------------------------------------------------------------------ the oracle
def test_cross_oracle_is_softmax_of_the_attended():
    from scipy.special import log_softmax, softmax
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(3, 4, 8)), rng.normal(size=(9, 2, 8)), rng.normal(size=(9, 2, 8))
    keep = np.array([1, 0, 1, 1, 1, 0, 0, 1, 1], bool)
    out, lse, A, S = O.cross_attention(q, k, v, keep, 0.3)
    kk, vv = np.repeat(k, 2, 1), np.repeat(v, 2, 1)
    s = np.where(keep, 0.3 * np.einsum("thd,jhd->thj", q, kk), -np.inf)
    np.testing.assert_allclose(out, np.einsum("thj,jhd->thd", softmax(s, -1), vv), atol=1e-12)
    np.testing.assert_allclose(lse, s[..., 0] - log_softmax(s, -1)[..., 0], atol=1e-12)
    assert (np.abs(out) <= A + 1e-12).all() and (np.abs(s[..., keep]).max(-1) <= S + 1e-12).all()
    out, lse, _, _ = O.cross_attention(q, k, v, np.zeros(9, bool), 0.3)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_beam_oracle_by_probabilities():
    """exp(score) of a beam's tokens add up to exp of its own; order and ties."""
    rng = np.random.default_rng(1)
    x, s = rng.normal(size=(3, 50)), np.array([-1.0, -2.5, -INF])
    cand, flag, _ = O.beam_candidates(x, s, None, 7)
    assert flag == 0 and len(cand) == 100 and all(a[0] >= b[0] for a, b in itertools.pairwise(cand))
    for w in (0, 1):
        assert np.isclose(sum(np.exp(c[0]) for c in cand if c[1] == w), np.exp(s[w]))
    assert [c[3] for c in cand if c[2] == 7] == [True, True]
    cand, flag, _ = O.beam_candidates(np.zeros((2, 4)), [-1.0, -1.0], [False, False], 0)
    assert [(c[1], c[2]) for c in cand] == [(0, 0), (0, 1), (0, 2), (0, 3), (1, 0), (1, 1), (1, 2), (1, 3)]
    cand, flag, _ = O.beam_candidates(np.array([[np.nan, 0], [0, -INF]]), [-1.0, -3.0], [True, False], 9)
    assert [(c[0], c[1], c[2]) for c in cand] == [(-1.0, 0, 9), (-3.0, 1, 0)] and flag == 0
    cand, flag, _ = O.beam_candidates(np.array([[np.nan, 0], [0, INF]]), [-1.0, -3.0], None, 9)
    assert cand == [] and flag == O.DEVERR_VALUE


def test_beam_tables_oracle_by_hand():
    # three rows share page 4; rows 0 and 2 hold 20 positions, row 1 has parted
    table = [[4, 6, -1], [4, 8, -1], [4, 9, 3]]
    got = O.beam_tables([[1, 1, 0]], [20, 20, 20], table, 20, [2, 2, 3], [11, 12, 0, 0, 0], 2)
    # 9 and the page past row 2's length go back, 3 is popped for row 1's copy of 8
    assert got["table"].tolist() == [[4, 8, -1], [4, 3, -1], [4, 6, -1]]
    assert got["copies"].tolist() == [[-1, -1, 0], [8, 3, 4], [-1, -1, 0]]
    assert got["free"][:3].tolist() == [11, 12, 9] and got["count"] == 3
    assert got["lens"].tolist() == [20] * 3 and got["owned"].tolist() == [2] * 3 and got["flag"] == 0
    got = O.beam_tables([[-1, -1, -1]], [20, 20, 20], table, 20, [2, 2, 3], [0] * 9, 0)
    assert got["free"][:5].tolist() == [4, 6, 8, 9, 3] and got["count"] == 5 and (got["table"] == -1).all()


def test_the_measured_cases_draw_and_count():
    import random

    from perf import more_operators as m
    names = [c["name"] for c in m.listed()]
    assert len(set(names)) == len(names) and 4 <= len(names) <= 12
    rng = random.Random(1)
    for case in m.listed() + [m.draw(rng) for _ in range(40)]:
        w = m.work(case)
        assert w["bytes"] > 0 and w["flops"] >= 0
