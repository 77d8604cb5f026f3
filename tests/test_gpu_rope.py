"""Rotary positions and the append to the paged cache against float64."""
import numpy as np
import pytest
import torch

from oracle import fill_oracle as F
from tests.fill_util import PAGE, i32

pytestmark = pytest.mark.gpu


def _case(T, Hq, Hkv, d, rot, axes=1, interleaved=False, far=2000, fused=False, seed=0, theta=1e4):
    g = torch.Generator().manual_seed(seed)
    r = lambda *n: torch.randn(*n, generator=g).bfloat16()  # noqa: E731
    if fused:
        x = r(T, (Hq + 2 * Hkv) * d).cuda()
        q, k, v = (y.unflatten(1, (-1, d)) for y in x.split([Hq * d, Hkv * d, Hkv * d], 1))
    else:
        q, k, v = r(T, Hq, d).cuda(), r(T, Hkv, d).cuda(), r(T, Hkv, d).cuda()
    pages = T // PAGE + 3
    slots = torch.randperm(pages * PAGE, generator=g)[:T].int()
    pos = torch.randint(0, far, (axes, T), generator=g, dtype=torch.int32)
    freq = (theta ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / max(rot, 1))).float()
    axis = torch.randint(0, axes, (rot // 2,), generator=g).int()
    kp, vp = r(pages, Hkv, PAGE, d), r(pages, Hkv, PAGE, d)
    return dict(q=q, k=k, v=v, slots=slots, pos=pos, freq=freq, axis=axis, kp=kp, vp=vp,
                interleaved=interleaved)


def _want(c):
    args = (c["pos"].numpy(), c["freq"].double().numpy(), c["axis"].numpy(), c["interleaved"])
    turn = lambda x: F.rope(x.double().cpu().numpy(), *args)  # noqa: E731
    return turn(c["q"]), turn(c["k"])


def _tolerance(x, y, rot, interleaved):
    """One rounding to bf16 (half a step: 2^-8) of a float32 rotation: two
    products and a sum of the pair's values, the sine and cosine good to 2^-21."""
    x = np.abs(x)
    p = x.copy()
    h = rot // 2
    if rot:
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, h), slice(h, rot))
        p[..., a] = p[..., b] = x[..., a] + x[..., b]
    return 2.0 ** -8 * np.abs(y) * 1.001 + 2.0 ** -20 * p


def _run(c, in_place=False, **kw):
    from self_speculative_sparse_vg_gb300 import vg
    kv = vg.PagedKV(c["kp"].cuda(), c["vp"].cuda(), torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
    q = c["q"].clone() if in_place else c["q"]
    out = None if in_place else torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = vg.rope_append(kv, q, c["k"], c["v"], c["slots"].cuda(), out,
                       positions=c["pos"].cuda() if len(c["freq"]) else None,
                       inv_freq=c["freq"].cuda() if len(c["freq"]) else None,
                       freq_axis=c["axis"].cuda() if len(c["pos"]) > 1 else None,
                       interleaved=c["interleaved"], error_flag=flag, **kw)
    torch.cuda.synchronize()
    return r, kv, int(flag.item())


def _check(c, **kw):
    r, kv, flag = _run(c, **kw)
    assert flag == 0
    rot, inter = 2 * len(c["freq"]), c["interleaved"]
    wq, wk = _want(c)
    assert (np.abs(r.double().cpu().numpy() - wq)
            <= _tolerance(c["q"].double().cpu().numpy(), wq, rot, inter)).all()
    kp, vp = kv.k_pages.cpu(), kv.v_pages.cpu()
    live = c["slots"] >= 0
    s = c["slots"][live].long()
    k = kp[s // PAGE, :, s % PAGE].double().numpy()
    n = live.numpy()
    assert (np.abs(k - wk[n]) <= _tolerance(c["k"].double().cpu().numpy(), wk, rot, inter)[n]).all()
    assert torch.equal(vp[s // PAGE, :, s % PAGE], c["v"].cpu()[live])
    # dims that do not turn, and slots that no token names, are untouched
    assert torch.equal(r[..., rot:].cpu(), c["q"][..., rot:].cpu())
    rest = torch.ones(kp.shape[0] * PAGE, dtype=torch.bool)
    rest[s] = False
    for got, was in ((kp, c["kp"]), (vp, c["vp"])):
        flat = lambda x: x.transpose(1, 2).flatten(0, 1)[rest]  # noqa: E731
        assert torch.equal(flat(got), flat(was))
    return r, kv


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,d,rot,axes", [
    (1, 32, 8, 128, 128, 1), (7, 40, 8, 128, 128, 1), (33, 8, 2, 64, 64, 3), (65, 8, 2, 64, 32, 2),
    (5, 1, 1, 128, 16, 1), (19, 6, 3, 64, 48, 8), (130, 4, 4, 128, 96, 3), (3, 16, 1, 64, 64, 1)])
def test_against_float64(T, Hq, Hkv, d, rot, axes, interleaved):
    _check(_case(T, Hq, Hkv, d, rot, axes, interleaved, seed=T))


@pytest.mark.parametrize("T", [1, 2, 50])
def test_slices_of_a_fused_projection(T):
    _check(_case(T, 8, 2, 128, 128, fused=True, seed=T))
    _check(_case(T, 8, 2, 64, 32, 3, True, fused=True, seed=T + 1))


@pytest.mark.parametrize("far", [2 ** 20, 2 ** 27, 2 ** 31 - 1])
def test_far_positions(far):
    """Angles of positions whose product with a frequency has no exact float32."""
    c = _case(24, 4, 2, 128, 128, far=far, seed=3, theta=5e5)
    c["pos"][0, :4] = torch.tensor([far, 0, -far, -1])
    _check(c)


def test_nothing_turns_is_a_copy():
    c = _case(37, 8, 2, 128, 0, seed=4)
    r, kv = _check(c)
    assert torch.equal(r, c["q"])


def test_in_place_and_without_queries():
    from self_speculative_sparse_vg_gb300 import vg
    c = _case(21, 8, 2, 128, 128, seed=6)
    a, kva = _check(c)
    b, kvb = _check(c, in_place=True)
    assert torch.equal(a, b)
    kv = vg.PagedKV(c["kp"].cuda(), c["vp"].cuda(), torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
    assert vg.rope_append(kv, None, c["k"], c["v"], c["slots"].cuda(), positions=c["pos"][0].cuda(),
                          inv_freq=c["freq"].cuda()) is None
    assert torch.equal(kv.k_pages, kva.k_pages) and torch.equal(kv.v_pages, kva.v_pages)


def test_padding_and_bad_slots():
    """Negative slots write nothing; slots past the pool and axes out of range
    are flagged."""
    c = _case(40, 8, 2, 128, 128, seed=7)
    c["slots"][[0, 13, 39]] = torch.tensor([-1, -2 ** 31, -7], dtype=torch.int32)
    _check(c)
    kp, vp = c["kp"].clone(), c["vp"].clone()
    c["slots"][5] = c["kp"].shape[0] * PAGE
    c["slots"][6] = 2 ** 31 - 1
    r, kv, flag = _run(c)
    assert flag == 2
    c["slots"][[5, 6]] = -1
    r2, kv2, flag2 = _run(c)
    assert flag2 == 0 and torch.equal(kv.k_pages, kv2.k_pages) and torch.equal(kv.v_pages, kv2.v_pages)
    assert torch.equal(r, r2)
    assert torch.equal(c["kp"], kp) and torch.equal(c["vp"], vp)
    c = _case(9, 8, 2, 64, 64, 3, seed=8)
    c["axis"][3], c["axis"][4] = 3, -1
    r, kv, flag = _run(c)
    assert flag == 2
    c["axis"][3] = c["axis"][4] = 0
    r2, kv2, flag2 = _run(c)
    assert flag2 == 0 and torch.equal(r, r2) and torch.equal(kv.k_pages, kv2.k_pages)


def test_values_pass_through_whatever_they_hold():
    """NaN and infinities of the values and of dims that do not turn arrive as
    they are; a NaN in a pair stays in that pair."""
    c = _case(6, 2, 1, 64, 32, seed=9)
    c["v"][1, 0, 3], c["v"][2, 0, 5] = float("nan"), float("inf")
    c["k"][3, 0, 40], c["k"][4, 0, 2] = float("inf"), float("nan")
    r, kv, flag = _run(c)
    s = c["slots"].long()
    v = kv.v_pages.cpu()[s // PAGE, :, s % PAGE]
    assert torch.equal(v.view(torch.int16), c["v"].cpu().view(torch.int16))
    k = kv.k_pages.cpu()[s // PAGE, :, s % PAGE]
    bad = torch.isnan(k)
    assert bad.sum() == 2 and bad[4, 0, 2] and bad[4, 0, 18] and k[3, 0, 40] == float("inf")


def test_large_pool_offsets():
    """Slots whose byte offset passes 32 bits."""
    from self_speculative_sparse_vg_gb300 import vg
    pages, Hkv, d = 150_000, 8, 128                # 4.9 GB a pool
    kp = torch.zeros(pages, Hkv, PAGE, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    kv = vg.PagedKV(kp, vp, torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(3, Hkv, d, generator=g).bfloat16().cuda() for _ in range(2))
    slots = i32([pages * PAGE - 1, 17, (pages - 9) * PAGE + 3])
    vg.rope_append(kv, None, k, v, slots)
    s = slots.long()
    assert torch.equal(kp[s // PAGE, :, s % PAGE], k) and torch.equal(vp[s // PAGE, :, s % PAGE], v)
    assert int((kp != 0).any(-1).any(1).sum()) == 3
