"""Refusals of the cache-filling calls (no GPU), and pins of their oracle."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import fill_oracle as F
from tests.conftest import ensure_lib

FAKE = 0x4000


@pytest.fixture(scope="module")
def vg():
    ensure_lib()
    from self_speculative_sparse_vg_gb300 import vg
    return vg


def _kv(vg, head_dim=128, heads=8, page_size=16, k=0x1000, pages=100, width=64):
    return vg.PagedKVStruct(k, 0x2000, 0x3000, pages, page_size, width, heads, head_dim)


def test_step_tables_refusals(vg):
    f = vg._lib.vg_step_tables
    good = [FAKE, FAKE, 4, FAKE, 64, 100, FAKE, FAKE, 100, FAKE, 10, FAKE, FAKE, FAKE, FAKE, None, None]

    def call(**kw):
        a = list(good)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)
    for i in (0, 1, 3, 11, 12, 13, 14):
        assert call(**{f"a{i}": None}) == 1, i
    for i, v in ((2, 0), (2, -1), (4, 0), (5, 0), (8, 0), (10, -1)):
        assert call(**{f"a{i}": v}) == 1, (i, v)
    for i in (6, 7, 9):                     # a free list in part
        assert call(**{f"a{i}": None}) == 1, i
    assert call(a2=8193) == 2 and call(a5=1 << 28) == 2 and call(a4=1 << 28) == 2


def test_rope_append_refusals(vg):
    kv = _kv(vg)

    def call(kv=kv, **kw):
        a = dict(q=FAKE, qs=4096, k=FAKE, ks=1024, v=FAKE, vs=1024, o=FAKE, os=4096, n=5, hq=32,
                 pos=FAKE, ps=5, axes=1, freq=FAKE, axis=None, rot=128, il=0, slots=FAKE, flag=None,
                 stream=None)
        a.update(kw)
        return vg._lib.vg_rope_append(ctypes.byref(kv), *a.values())
    for name in ("q", "k", "v", "o", "slots", "pos", "freq"):
        assert call(**{name: None}) == 1, name
    for name in ("q", "k", "v", "o"):
        assert call(**{name: FAKE + 8}) == 1, name          # not on 16 bytes
    for name in ("qs", "ks", "vs", "os"):
        assert call(**{name: 8}) == 1 and call(**{name: 4100}) == 1, name
    assert call(n=-1) == 1 and call(hq=-1) == 1 and call(rot=-16) == 1 and call(rot=144) == 1
    assert call(axes=0) == 1 and call(axes=3, ps=4) == 1 and call(axes=-2) == 1
    assert call(rot=24) == 2 and call(axes=9) == 2
    assert call(kv=_kv(vg, head_dim=96)) == 2 and call(kv=_kv(vg, page_size=32)) == 2
    assert call(kv=_kv(vg, pages=1 << 28)) == 2 and call(kv=_kv(vg, k=0x1008)) == 1
    assert call(n=0) == 0                                   # nothing to do, nothing launched


def test_chunk_attention_refusals(vg):
    kv = _kv(vg)

    def call(kv=kv, **kw):
        a = dict(q=FAKE, qs=4096, cu=FAKE, lens=FAKE, b=2, n=5, hq=32, scale=0.1, o=FAKE, os=4096,
                 lse=None, ws=None, wsb=0, flag=None, stream=None)
        a.update(kw)
        return vg._lib.vg_chunk_attention(ctypes.byref(kv), *a.values())
    for name in ("q", "cu", "lens", "o"):
        assert call(**{name: None}) == 1, name
    for name in ("q", "o"):
        assert call(**{name: FAKE + 2}) == 1, name
    for name in ("qs", "os"):
        assert call(**{name: 4088}) == 1 and call(**{name: 4100}) == 1, name
    assert call(b=0) == 1 and call(n=-1) == 1 and call(hq=0) == 1 and call(hq=33) == 1
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == 1, scale
    assert call(hq=136, qs=136 * 128, os=136 * 128) == 2 and call(b=4097) == 2
    assert call(kv=_kv(vg, head_dim=256)) == 2 and call(kv=_kv(vg, k=0x1008)) == 1
    assert call(n=0) == 0
    need = vg._lib.vg_chunk_workspace_bytes(2, 5, 32, 8, 128)
    assert need > 0 and call() == 3 and call(ws=FAKE, wsb=need - 1) == 3
    for off in (1, 4, 8):
        assert call(ws=FAKE + off, wsb=need + 64) == 1, off
    for bad in ((0, 5, 32, 8, 128), (2, 0, 32, 8, 128), (2, 5, 33, 8, 128), (2, 5, 32, 8, 96),
                (2, 5, 136, 8, 128)):
        assert vg._lib.vg_chunk_workspace_bytes(*bad) == 0, bad


def test_binding_refusals(vg):
    """Wrong types, shapes and places are refused before the library is called."""
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    h = lambda *n: torch.zeros(*n, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError):
        vg.step_tables(i(2, 4), 8, i(2), i(2), i(3), i(2), i(9), i(9))       # not on a GPU
    with pytest.raises(ValueError):
        vg.step_tables(i(2, 4), 8, i(2), i(2), i(3), i(2), i(9), i(8))
    with pytest.raises(ValueError):
        vg.step_tables(i(8), 8, i(2), i(2), i(3), i(2), i(9), i(9))
    kv = vg.PagedKV(h(4, 2, 16, 64), h(4, 2, 16, 64), i(1, 4))
    with pytest.raises(ValueError):
        vg.rope_append(kv, None, h(3, 2, 64), h(3, 2, 64), i(3))
    with pytest.raises(ValueError):
        vg.chunk_attention(kv, h(3, 4, 64), i(2), i(1), 0.1, h(3, 4, 64))
    with pytest.raises(ValueError):
        vg.chunk_attention(kv, torch.zeros(3, 4, 64), i(2), i(1), 0.1, h(3, 4, 64))


# ---------------------------------------------------------------- oracle pins
def test_oracle_tables_by_hand():
    # 20 + 6 tokens on pages [7, 5]: the block starts in page 5; request 1 gives page 9 back, which
    # request 2 then takes, before the last page of the free list
    r = F.step_tables([[7, 5, -1], [4, 9, -1], [-1, -1, -1]], 12, [20, 3, 0], [6, 1, 17], 26,
                      [2, 2, 0], [0, 1, 2, -1, -1], 3)
    assert r["flag"] == 0 and r["count"] == 2 and r["cu"].tolist() == [0, 6, 7, 24]
    assert r["table"].tolist() == [[7, 5, -1], [4, -1, -1], [9, 2, -1]]
    assert r["owned"].tolist() == [2, 1, 2] and r["lens"].tolist() == [26, 4, 17]
    assert r["slots"][:7].tolist() == [84, 85, 86, 87, 88, 89, 67]
    assert r["slots"][7:24].tolist() == list(range(144, 160)) + [32]
    assert r["slots"][24:].tolist() == [-1, -1]
    assert r["positions"][:7].tolist() == [20, 21, 22, 23, 24, 25, 3]


def test_oracle_tables_refuse_in_order():
    r = F.step_tables([[-1] * 4] * 3, 9, [0, 0, 0], [17, 33, 16], 99, [0, 0, 0], [5, 6, 7, 8], 4)
    # 2 pages, then 3 that no longer fit, and one after it that would
    assert r["lens"].tolist() == [17, 0, 0] and r["flag"] == 32 and r["count"] == 2


def test_oracle_rope_turns_relative():
    """Scores of turned pairs depend on the distance of the positions only."""
    rng = np.random.default_rng(0)
    x, y = rng.normal(size=(2, 1, 1, 32))
    f = 100.0 ** (-np.arange(8) / 8)
    for inter in (False, True):
        dots = []
        for a, b in ((0, 5), (40, 45), (1000, 1005)):
            u = F.rope(x, [[a]], f, [0] * 8, inter)
            w = F.rope(y, [[b]], f, [0] * 8, inter)
            dots.append((u * w).sum())
        np.testing.assert_allclose(dots, dots[0], atol=1e-10)
        np.testing.assert_array_equal(F.rope(x, [[0]], f, [0] * 8, inter), x)


def test_oracle_chunk_is_the_verify_oracle():
    """k + 1 rows at the end of a sequence: the same definition as verification."""
    from oracle import vg_oracle as O
    rng = np.random.default_rng(1)
    L, R = 37, 4
    q = rng.normal(size=(1, R, 4, 8))
    k, v = rng.normal(size=(2, 2, L + R, 8))
    want, _ = O.verify_attention(q, [k], [v], [L], 0.3)
    got, lse, A, S = F.chunk_attention(q[0], k.transpose(1, 0, 2), v.transpose(1, 0, 2), R, 0.3)
    np.testing.assert_allclose(got, want[0], atol=1e-12)
    got, lse, A, S = F.chunk_attention(q[0], k.transpose(1, 0, 2)[:2], v.transpose(1, 0, 2)[:2], R, 0.3)
    assert (got[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2:]).all()
