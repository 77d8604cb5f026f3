"""Cross attention on the GPU against the float64 oracle: sizes, types, head
groups, strides, masks, empty rows, refused sequences, graphs and streams."""
import numpy as np
import pytest
import torch

from tests.beam_util import States, check_cross
from tests.fill_util import i32

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("states", [1, 2, 127, 128, 129, 255, 256, 257, 1500, 9000])
def test_one_row_over_states(states, dtype, d):
    check_cross(States([states], 2, d, dtype, seed=states), [1], 8)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("rows", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700])
def test_rows_of_one_sequence(rows, dtype):
    check_cross(States([333], 1, 64, dtype, seed=rows), [rows], 1)


@pytest.mark.parametrize("Hq,Hkv,d", [(1, 1, 128), (8, 8, 64), (5, 1, 128), (40, 8, 128), (7, 1, 64), (32, 2, 64),
                                      (33, 1, 64), (64, 1, 128), (100, 1, 64), (128, 1, 128), (256, 2, 64)])
@pytest.mark.parametrize("rows", [1, 3, 26, 70])
def test_head_groups(Hq, Hkv, d, rows):
    check_cross(States([270, 5], Hkv, d, seed=Hq, gap=3), [rows, 2], Hq)


@pytest.mark.parametrize("masked", [0.0, 0.2, 0.97, 1.0])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (FP, 64)])
def test_ragged_batch(masked, dtype, d):
    """Sequences of any number of rows and states, none among them, in slots with
    NaN between them and in masked places."""
    lens = [700, 0, 1, 128, 255, 64, 1300, 3]
    new = [5, 4, 0, 130, 1, 300, 2, 6]
    check_cross(States(lens, 2, d, dtype, seed=3, room=1301, masked=masked), new, 8, rows_after=3)
    check_cross(States(lens, 2, d, dtype, seed=4, gap=1, masked=masked, fused=True), new, 8, strided=True)


@pytest.mark.parametrize("masked", [0.0, 0.3])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 4, 64), (16, 2, 64), (6, 2, 64), (34, 2, 64), (64, 2, 64), (66, 2, 64),
                                      (10, 10, 64), (8, 2, 128), (9, 3, 64)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_few_rows(Hq, Hkv, d, dtype, masked):
    """Sequences of at most 32 rows of a head, with one that has more: heads of 64
    go in pairs where their number is even."""
    rng = np.random.default_rng(Hq)
    lens = [1, 128, 700, 0, 129, 2000, 5, 300, 1111, 40]
    few = max(1, 32 * Hkv // Hq)
    new = rng.integers(0, few + 1, 10)
    new[:4] = [few, 1, few, min(few, 2)]
    new[7] = min(5 * few + 1, int(10 * few - new.sum() + new[7]))
    check_cross(States(lens, Hkv, d, dtype, seed=Hq, gap=2, masked=masked, fused=True), new, Hq, rows_after=1)


@pytest.mark.parametrize("batch", [31, 32, 33, 100, 400, 4096])
def test_many_sequences(batch):
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, 200 if batch < 500 else 20, batch)
    new = rng.integers(0, 4, batch)
    check_cross(States(lens, 1, 64, seed=batch), new, 2)


def test_infinities_in_states_that_nobody_attends():
    for junk in (float("inf"), float("-inf"), 3e38):
        check_cross(States([130, 77, 300], 2, 128, seed=1, gap=5, masked=0.3, junk=junk), [3, 70, 1], 4)


@pytest.mark.parametrize("rows", [1, 200])
@pytest.mark.parametrize("where", [0, 129, 700])
def test_non_finite_values_that_are_attended_show(where, rows):
    """As in the formula: a NaN or an infinity of V in its dimension of every row,
    one of K in the whole row."""
    from self_speculative_sparse_vg_gb300 import vg
    st = States([701, 50], 2, 64, seed=2)
    q = torch.randn(rows + 1, 4, 64, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    cu, starts, lens = i32([0, rows, rows + 1]), i32(st.starts), i32(st.lens)

    def call(k, v):
        out = torch.zeros_like(q)
        vg.cross_attention(q, k, v, cu, starts, lens, 0.125, out)
        return out
    k, v = st.gpu()
    clean = call(k, v)
    for bad in (float("nan"), float("inf")):
        v2 = v.clone()
        v2[where, 1, 5] = bad
        out = call(k, v2)
        assert not torch.isfinite(out[:rows, 2:, 5]).any()
        out[:rows, 2:, 5] = clean[:rows, 2:, 5]
        assert torch.equal(out, clean)
        k2 = k.clone()
        k2[where, 0, 7] = bad
        out = call(k2, v)
        # an infinite key makes a score of either sign: NaN, or a weight of zero
        some = torch.isnan(out[:rows, :2]).all(-1)
        assert some.all() if bad != bad else some.any()
        assert torch.equal(out[:rows, 2:], clean[:rows, 2:]) and torch.equal(out[rows:], clean[rows:])


@pytest.mark.parametrize("dtype", [BF, FP])
def test_scores_far_apart(dtype):
    """Large scores in rising and falling order: the reference of the exponent
    moves many times, or never."""
    st = States([900], 1, 64, dtype, seed=6)
    q = torch.randn(40, 2, 64, generator=torch.Generator().manual_seed(7)).to(dtype)
    for sign in (1.0, -1.0):
        ramp = torch.linspace(0.2, 4.0, 900)[:, None, None] * sign
        s2 = States([900], 1, 64, dtype, seed=6)
        s2.k.copy_((ramp * q[0, 0].float()).to(dtype))
        check_cross(s2, [40], 2, q=q, scale=0.5)
    check_cross(st, [40], 2, q=q, scale=3.0)


def test_sequences_that_share_states():
    """Two sequences may attend the same states, or parts of each other's."""
    st = States([600], 2, 128, seed=9)
    st.lens, st.starts = [600, 600, 100, 300], [0, 0, 450, 7]
    st.attended = [np.ones(n, bool) for n in st.lens]
    check_cross(st, [3, 150, 1, 40], 8)


def test_refused_sequences_are_left_as_they_were():
    from self_speculative_sparse_vg_gb300 import vg
    st = States([100, 60, 80], 2, 64, seed=1)
    k, v = st.gpu()
    q = torch.randn(9, 4, 64, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    want = torch.full_like(q, 7.0)
    vg.cross_attention(q, k, v, i32([0, 3, 6, 9]), i32(st.starts), i32(st.lens), 0.125, want)
    total = sum(st.lens)
    for starts, lens, cu, fine in (
            ([0, -1, 160], [100, 60, 80], [0, 3, 6, 9], [1, 0, 1]),
            ([0, 100, 160], [100, -60, 80], [0, 3, 6, 9], [1, 0, 1]),
            ([0, 100, 160], [100, 60, 81], [0, 3, 6, 9], [1, 1, 0]),
            ([0, total, 160], [100, 1, 80], [0, 3, 6, 9], [1, 0, 1]),
            ([2 ** 31 - 1, 100, 160], [2 ** 31 - 1, 60, 80], [0, 3, 6, 9], [0, 1, 1]),
            ([0, 100, 160], [100, 60, 80], [0, 3, 6, 10], [1, 1, 0]),
            ([0, 100, 160], [100, 60, 80], [-3, 3, 6, 9], [0, 1, 1])):
        out = torch.full_like(q, 7.0)
        flag = i32([0])
        vg.cross_attention(q, k, v, i32(cu), i32(starts), i32(lens), 0.125, out, error_flag=flag)
        assert int(flag.item()) == vg.DEVERR_LENGTH
        for e, good in enumerate(fine):
            r = slice(3 * e, 3 * e + 3)
            if good:
                assert torch.allclose(out[r].float(), want[r].float(), atol=2e-2)
            else:
                assert (out[r] == 7.0).all()


def test_no_states_and_no_rows():
    from self_speculative_sparse_vg_gb300 import vg
    q = torch.randn(3, 4, 64, device="cuda").bfloat16()
    none = torch.zeros(0, 2, 64, dtype=BF, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.zeros(3, 4, device="cuda")
    vg.cross_attention(q, none, none, i32([0, 2, 3]), i32([0, 0]), i32([0, 0]), 0.125, out, lse=lse)
    assert (out == 0).all() and torch.isneginf(lse).all()
    vg.cross_attention(q[:0], none, none, i32([0, 0]), i32([0]), i32([0]), 0.125, out[:0])
    out.fill_(7.0)
    kv = torch.randn(5, 2, 64, device="cuda").bfloat16()
    vg.cross_attention(q, kv, kv, i32([0, 0, 0]), i32([0, 0]), i32([5, 5]), 0.125, out)
    assert (out == 7.0).all()


@pytest.mark.parametrize("masked", [0.0, 0.4])
def test_long_states_far_in_a_large_buffer(masked):
    """Byte offsets past 32 bits: states at the end of a 9 GB projection."""
    from self_speculative_sparse_vg_gb300 import vg
    S, n = 1 << 22, 5000
    wide = torch.empty(S, 17, 64, dtype=BF, device="cuda")     # 2176 bytes a row
    wide[S - n:] = torch.randn(n, 17, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).to(BF)
    mask = None
    if masked:
        mask = torch.zeros(S, dtype=torch.bool, device="cuda")
        mask[S - n:] = torch.rand(n, device="cuda", generator=torch.Generator("cuda").manual_seed(4)) >= masked
    q = torch.randn(6, 16, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(BF)
    out, near = torch.zeros_like(q), torch.zeros_like(q)
    cu = i32([0, 6])
    vg.cross_attention(q, wide[:, :8], wide[:, 8:16], cu, i32([S - n]), i32([n]), 0.125, out, mask=mask)
    tail = wide[S - n:].contiguous()
    vg.cross_attention(q, tail[:, :8], tail[:, 8:16], cu, i32([0]), i32([n]), 0.125, near,
                       mask=None if mask is None else mask[S - n:].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(out, near) and out.abs().max() > 0


def test_same_bits_every_time_and_on_a_stream_of_its_own():
    st = States([1500, 700, 90], 4, 64, FP, seed=8, masked=0.1)
    _, a, la = check_cross(st, [5, 300, 1], 8)
    _, b, lb = check_cross(st, [5, 300, 1], 8, stream=torch.cuda.Stream())
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_two_graphs_share_a_workspace_as_lengths_change():
    """Captured once, replayed with other lengths, rows and masks."""
    from self_speculative_sparse_vg_gb300 import vg
    E, room, T, Hq, Hkv, d = 5, 600, 64, 8, 2, 128
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(E * room, Hkv, d, generator=g).bfloat16().cuda() for _ in range(2))
    mask = torch.ones(E * room, dtype=torch.bool, device="cuda")
    starts, lens, cu = i32(np.arange(E) * room), i32([0] * E), i32([0] * (E + 1))
    qs = [torch.randn(T, Hq, d, generator=g).bfloat16().cuda() for _ in range(2)]
    ws = torch.empty(vg.cross_workspace_bytes(E, T, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(q) for q in qs]
    call = lambda i, out, ws=ws: vg.cross_attention(qs[i], k, v, cu, starts, lens, 0.09, out, mask=mask,  # noqa: E731
                                                    workspace=ws)
    call(0, outs[0])
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            call(i, outs[i])
    rng = np.random.default_rng(2)
    for _ in range(5):
        lens.copy_(i32(rng.integers(0, room + 1, E)))
        cu.copy_(i32(np.concatenate([[0], np.sort(rng.integers(0, T + 1, E))])))
        mask.copy_(torch.from_numpy(rng.random(E * room) < 0.8).cuda())
        ws.fill_(255)
        for i in range(2):
            outs[i].fill_(3.0)
            graphs[i].replay()
        for i in range(2):
            want = torch.full_like(qs[i], 3.0)
            call(i, want, torch.empty_like(ws))
            torch.cuda.synchronize()
            assert torch.equal(outs[i], want)


def test_a_short_report_bound_is_reported_and_the_result_complete():
    from self_speculative_sparse_vg_gb300 import vg
    st = States([40000], 8, 128, seed=4, junk=0.0)
    q, want, _ = check_cross(st, [2], 32)
    k, v = st.gpu()
    flag, out = i32([0]), torch.zeros_like(want)
    vg.set_wait_limit_ns(1)
    try:
        vg.cross_attention(q, k, v, i32([0, 2]), i32([0]), i32([40000]), 128 ** -0.5, out, error_flag=flag)
        torch.cuda.synchronize()
    finally:
        vg.set_wait_limit_ns(0)
    assert int(flag.item()) == vg.DEVERR_TIMEOUT
    assert torch.equal(out, want)


def test_binding_refusals():
    """Wrong types, shapes and places, with tensors on the GPU."""
    from self_speculative_sparse_vg_gb300 import vg
    t = lambda *n, dt=BF: torch.zeros(*n, dtype=dt, device="cuda")  # noqa: E731
    good = dict(q=t(3, 4, 64), k=t(9, 2, 64), v=t(9, 2, 64), cu_q=i32([0, 3]), state_starts=i32([0]),
                state_lens=i32([9]), softmax_scale=0.1, out=t(3, 4, 64))
    vg.cross_attention(**good)
    for bad in (dict(q=t(3, 4, 64, dt=torch.float32)), dict(q=t(3, 4, 64, dt=FP)), dict(k=t(9, 2, 64, dt=FP)),
                dict(v=t(8, 2, 64)), dict(v=t(9, 1, 64)), dict(k=t(9, 2, 128)), dict(out=t(2, 4, 64)),
                dict(out=t(3, 4, 64, dt=FP)), dict(cu_q=i32([0])), dict(cu_q=i32([0, 3]).long()),
                dict(state_starts=i32([0, 0])), dict(state_lens=i32([9]).cpu()), dict(mask=t(8, dt=torch.bool)),
                dict(mask=t(9, dt=torch.int32)), dict(lse=t(3, 4)), dict(softmax_scale="x"), dict(softmax_scale=None),
                dict(k=t(9, 2, 64).transpose(0, 1)), dict(q=t(3, 64, 4).transpose(1, 2)), dict(k=t(9, 128)),
                dict(error_flag=t(1)), dict(workspace=t(9).cpu())):
        with pytest.raises(ValueError):
            vg.cross_attention(**{**good, **bad})
    for bad, status in ((dict(softmax_scale=0.0), 1), (dict(softmax_scale=float("nan")), 1),
                        (dict(workspace=t(16, dt=torch.uint8)), 3), (dict(q=t(3, 3, 64), out=t(3, 3, 64)), 1),
                        (dict(q=t(3, 4, 32), k=t(9, 2, 32), v=t(9, 2, 32), out=t(3, 4, 32)), 3),
                        (dict(k=t(9 * 128 + 4)[4:].view(9, 2, 64)), 1)):
        with pytest.raises(vg.VGError) as e:
            vg.cross_attention(**{"workspace": t(1 << 27, dt=torch.uint8) if status != 3 else None, **good, **bad})
        assert e.value.status in (status, 2), bad
