"""Attention of a chunk of new tokens over the paged cache against float64.

The bounds come from the arithmetic alone (fill_util.chunk_bounds); cache
slots that a row may not see hold NaN unless a test says otherwise."""
import numpy as np
import pytest
import torch

from tests.fill_util import PAGE, Cache, check_chunk, i32

pytestmark = pytest.mark.gpu

HEADS = [(32, 8, 128), (40, 8, 128), (8, 2, 64)]


@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000])
def test_single_token(Hq, Hkv, d, length):
    check_chunk(Cache([length], Hkv, d, seed=length), [1], Hq)


@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
@pytest.mark.parametrize("new,length", [
    (2, 2), (6, 300), (31, 31), (32, 32), (33, 33), (63, 200), (64, 64), (65, 130), (128, 128),
    (129, 400), (200, 200), (257, 700)])
def test_one_chunk(Hq, Hkv, d, new, length):
    check_chunk(Cache([length], Hkv, d, seed=new), [new], Hq)


@pytest.mark.parametrize("group,Hkv,d", [(1, 3, 128), (2, 1, 64), (3, 2, 128), (6, 1, 64), (7, 2, 64),
                                         (8, 1, 128), (12, 1, 64), (16, 2, 128), (16, 1, 64)])
def test_groups(group, Hkv, d):
    """Every group size packs its rows differently."""
    check_chunk(Cache([90, 260], Hkv, d, seed=group), [50, 3], group * Hkv)


@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
def test_ragged_batch(Hq, Hkv, d):
    lens = [1, 130, 700, 16, 0, 257, 384, 45]
    new = [1, 130, 6, 0, 0, 1, 150, 45]
    check_chunk(Cache(lens, Hkv, d, seed=2), new, Hq, strided=True, rows_after=5)


def test_many_short_sequences():
    """More sequences than multiprocessors, a few tokens each."""
    rng = np.random.default_rng(0)
    new = rng.integers(0, 4, 333)
    lens = new + rng.integers(0, 60, 333)
    check_chunk(Cache(lens.tolist(), 2, 64, seed=3), new.tolist(), 8, rows_after=2)


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (4, 1, 128)])
@pytest.mark.parametrize("new", [1, 5, 40])
def test_long_context(Hq, Hkv, d, new):
    """Few rows over many positions: the positions are shared out and merged."""
    check_chunk(Cache([20011], Hkv, d, seed=4), [new], Hq)


def test_rows_that_attend_nothing():
    """Sequences whose new tokens outnumber their positions, down to none."""
    lens, new = [0, 3, 17, 5, 140], [4, 9, 17, 5, 150]
    qd, out, lse = check_chunk(Cache(lens, 2, 128, seed=5), new, 8)
    assert (out[:4] == 0).all() and torch.isneginf(lse[:4]).all()
    assert (out[4:10] == 0).all() and not (out[10:13] == 0).all()


def test_nothing_to_do():
    c = Cache([10, 20], 2, 64, seed=6)
    check_chunk(c, [0, 0], 8, rows_after=3)
    check_chunk(c, [0, 0], 8)


@pytest.mark.parametrize("scale", [1e-3, 1.0, 7.0])
def test_scales(scale):
    """From nearly uniform weights to a single position that takes all."""
    check_chunk(Cache([300, 70], 2, 128, seed=7), [40, 70], 8, scale=scale)


def test_rising_and_falling_scores():
    """Logits that grow along the positions move the softmax reference again
    and again; logits that fall never move it and underflow to nothing."""
    for sign in (1.0, -1.0):
        c = Cache([900], 1, 64, seed=8)
        ramp = (sign * torch.arange(900) * 0.05)[:, None, None]
        c.k[0] = (c.k[0].float() * 0.1 + ramp).bfloat16()
        c.write(0, c.k[0], c.v[0])
        q = torch.full((70, 4, 64), 0.5, dtype=torch.bfloat16)
        check_chunk(c, [70], 4, q=q)


def test_masked_positions_hold_anything():
    """NaN, infinities and the type's extremes in K and V behind a row's own
    position, in the chunk itself and past the length, do not reach the row."""
    clean = Cache([300], 2, 128, seed=9)
    _, want, want_lse = check_chunk(clean, [170], 8)
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(torch.bfloat16).min,
                torch.finfo(torch.bfloat16).max):
        c = Cache([300], 2, 128, seed=9, junk=bad)
        k, v = c.k[0].clone(), c.v[0].clone()
        k[215:] = bad
        v[215:] = bad                       # positions 215 .. 299: the chunk's last 85 tokens
        c.write(0, k, v)
        from self_speculative_sparse_vg_gb300 import vg
        g = torch.Generator().manual_seed(5)
        q = torch.randn(170, 8, 128, generator=g).bfloat16().cuda()
        out = torch.zeros_like(q)
        lse = torch.zeros(170, 8, device="cuda")
        vg.chunk_attention(c.gpu(), q, i32([0, 170]), i32([300]), 128 ** -0.5, out, lse=lse)
        assert torch.equal(out[:85], want[:85]), bad
        assert torch.equal(lse[:85], want_lse[:85]), bad


def test_values_that_are_not_finite_reach_the_rows_that_attend_them():
    """A NaN or an infinity in V shows in its dimension of every row at or
    after its position and nowhere else, as in the formula."""
    from self_speculative_sparse_vg_gb300 import vg
    c = Cache([200], 1, 64, seed=10)
    _, want, _ = check_chunk(c, [200], 4)
    v = c.v[0].clone()
    v[50, 0, 3] = float("nan")
    v[150, 0, 7] = float("inf")
    v[130, 0, 9] = -float("inf")
    v[140, 0, 9] = float("inf")
    v[190, 0, 63] = -float("inf")
    c.write(0, c.k[0], v)
    g = torch.Generator().manual_seed(5)
    q = torch.randn(200, 4, 64, generator=g).bfloat16().cuda()
    out = torch.zeros_like(q)
    vg.chunk_attention(c.gpu(), q, i32([0, 200]), i32([200]), 0.125, out)
    w = want.clone()
    w[50:, :, 3] = float("nan")
    w[150:, :, 7] = float("inf")
    w[130:, :, 9] = -float("inf")
    w[140:, :, 9] = float("nan")
    w[190:, :, 63] = -float("inf")
    assert torch.equal(out.isnan(), w.isnan())
    assert torch.equal(out[~w.isnan()], w[~w.isnan()])


def test_pages_out_of_range():
    """A page id outside the pool is flagged; its positions count as zeros."""
    from self_speculative_sparse_vg_gb300 import vg
    for page in (-1, 10 ** 6):
        c = Cache([100, 40], 2, 128, seed=11)
        c.table[0, 2] = page
        kv = c.gpu()
        g = torch.Generator().manual_seed(5)
        q = torch.randn(41, 8, 128, generator=g).bfloat16()
        out = torch.zeros(41, 8, 128, dtype=torch.bfloat16, device="cuda")
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        vg.chunk_attention(kv, q.cuda(), i32([0, 40, 41]), i32([100, 40]), 128 ** -0.5, out,
                           error_flag=flag)
        assert int(flag.item()) == 1
        z = Cache([100, 40], 2, 128, seed=11)
        z.k[0][32:48] = 0
        z.v[0][32:48] = 0
        z.write(0, z.k[0], z.v[0])
        _, want, _ = check_chunk(z, [40, 1], 8, q=q)
        assert torch.equal(out, want)


def test_lengths_out_of_range():
    """Sequences whose rows or lengths make no sense are flagged and their
    rows stay; the others are served (rows that offsets out of order give to
    two sequences hold either's)."""
    from self_speculative_sparse_vg_gb300 import vg
    c = Cache([60, 50, 40], 2, 64, seed=12)
    kv = c.gpu()
    g = torch.Generator().manual_seed(5)
    q = torch.randn(30, 8, 64, generator=g).bfloat16()
    _, want, _ = check_chunk(c, [10, 10, 10], 8, q=q)
    for cu, lens, good in (([0, 10, 20, 30], [-1, 50, 40], (1, 2)),
                           ([0, 10, 20, 30], [60, 10 ** 6, 40], (0, 2)),
                           ([0, 10, 20, 31], [60, 50, 40], (0, 1)),
                           ([-1, 10, 20, 30], [60, 50, 40], (1, 2)),
                           ([0, 10, 5, 30], [60, 50, 40], ()),
                           ([0, 10, 2 ** 31 - 1, 30], [60, 50, 40], ())):
        out = torch.full_like(want, 3.0)
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        vg.chunk_attention(kv, q.cuda(), i32(cu), i32(lens), 0.125, out, error_flag=flag)
        assert int(flag.item()) == 16, (cu, lens)
        for b in good:
            assert torch.equal(out[10 * b:10 * b + 10], want[10 * b:10 * b + 10]), (cu, lens, b)
        for b in set(range(3)) - set(good):
            if cu == [0, 10, 20, 30]:
                assert (out[10 * b:10 * b + 10] == 3.0).all(), (cu, lens, b)


def test_two_calls_share_nothing_and_repeat_exactly():
    """The same call twice, a smaller call in between with the same workspace,
    another stream, and a captured call on new inputs give the same bits."""
    from self_speculative_sparse_vg_gb300 import vg
    c = Cache([5000, 700, 33], 2, 128, seed=13)
    kv = c.gpu()
    need = vg.chunk_workspace_bytes(3, 160, 8, 2, 128)
    ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device="cuda")
    new = [6, 150, 1]
    qd, first, lse = check_chunk(c, new, 8, workspace=ws, kv=kv)
    small = Cache([64], 2, 128, seed=1)
    check_chunk(small, [2], 8, workspace=ws)
    _, again, lse2 = check_chunk(c, new, 8, workspace=ws, kv=kv)
    assert torch.equal(first, again) and torch.equal(lse, lse2)
    cu, lens = i32([0, 6, 156, 157]), i32([5000, 700, 33])
    side = torch.cuda.Stream()
    outs = [torch.zeros_like(first) for _ in range(2)]
    torch.cuda.synchronize()
    wss = [torch.full_like(ws, 255) for _ in range(2)]
    with torch.cuda.stream(side):
        vg.chunk_attention(kv, qd, cu, lens, 128 ** -0.5, outs[0], workspace=wss[0])
    vg.chunk_attention(kv, qd, cu, lens, 128 ** -0.5, outs[1], workspace=wss[1])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first) and torch.equal(outs[1], first)
    out = torch.zeros_like(first)
    graph = torch.cuda.CUDAGraph()
    q2, cu2, lens2 = torch.zeros_like(qd), i32([0, 0, 0, 0]), i32([0, 0, 0])
    with torch.cuda.graph(graph):
        vg.chunk_attention(kv, q2, cu2, lens2, 128 ** -0.5, out, workspace=ws)
    q2.copy_(qd)
    cu2.copy_(cu)
    lens2.copy_(lens)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)


def test_rows_do_not_depend_on_the_batch():
    """A prompt in one piece, in chunks and beside others: the same rows up to
    the rounding of the merge."""
    from self_speculative_sparse_vg_gb300 import vg
    c = Cache([500, 900], 2, 64, seed=14)
    kv = c.gpu()
    g = torch.Generator().manual_seed(2)
    q = torch.randn(500, 8, 64, generator=g).bfloat16().cuda()
    whole = torch.zeros_like(q)
    one = vg.PagedKV(kv.k_pages, kv.v_pages, kv.page_table[:1].contiguous())
    vg.chunk_attention(one, q, i32([0, 500]), i32([500]), 0.125, whole)
    parts = torch.zeros_like(q)
    at = 0
    for n in (1, 100, 37, 250, 112):
        vg.chunk_attention(one, q[at:at + n], i32([0, n]), i32([at + n]), 0.125, parts[at:at + n])
        at += n
    torch.cuda.synchronize()
    # each side is within the bounds of one weight rounding and one output
    # rounding; |v| <= 5 and its weighted mean is below 1.5 here
    assert (whole.float() - parts.float()).abs().max() <= 2 * 2.0 ** -8 * (1.5 + 5.0)
    assert (whole.float() - parts.float()).abs().mean() <= 2.0 ** -8


def test_offsets_past_32_bits():
    """A pool whose byte offsets pass 32 bits, read at its end."""
    from self_speculative_sparse_vg_gb300 import vg
    pages, Hkv, d = 150_000, 8, 128
    c = Cache([77], Hkv, d, seed=15)
    kp = torch.zeros(pages, Hkv, PAGE, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    n = c.kp.shape[0]
    kp[-n:], vp[-n:] = c.kp.cuda(), c.vp.cuda()
    table = torch.where(c.table >= 0, c.table + pages - n, -1).int().cuda()
    check_chunk(c, [30], 32, kv=vg.PagedKV(kp, vp, table))


def test_length_shorter_than_the_cache():
    """kv_lens cuts the cache: later slots of the same pages are not seen."""
    c = Cache([250, 90], 2, 128, seed=16)
    check_chunk(c, [20, 33], 8, kv_lens=[131, 33])


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 1, 64), (2, 1, 128)])
def test_long_shares(Hq, Hkv, d):
    """Enough positions that every CTA streams many tiles (its ring goes round
    many times) before the ones that need care: ends of sequences inside a
    tile, the diagonal of a chunk, single tokens beside chunks."""
    lens = [29999, 30001, 23456, 30000, 27777, 31000, 12345, 30123]
    new = [1, 1, 70, 1, 33, 1, 6, 300 // Hq]
    check_chunk(Cache(lens, Hkv, d, seed=17), new, Hq)


def test_short_wait_bound_reports_and_completes():
    """A wait bound that every wait outlasts is reported; the call completes
    with the same results, and the next call reports nothing."""
    from self_speculative_sparse_vg_gb300 import vg
    c = Cache([9000, 400], 2, 128, seed=18)
    kv = c.gpu()
    qd, want, lse = check_chunk(c, [1, 150], 8, kv=kv)
    args = (kv, qd, i32([0, 1, 151]), i32([9000, 400]), 128 ** -0.5)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    l2 = torch.cuda.get_device_properties(0).L2_cache_size
    cold = torch.ones(int(1.5 * l2) // 4, device="cuda")
    vg.set_wait_limit_ns(1)
    try:
        out = torch.zeros_like(want)
        cold.sum()
        vg.chunk_attention(*args, out, error_flag=flag)
        assert int(flag.item()) == vg.DEVERR_TIMEOUT
        assert torch.equal(out, want)
    finally:
        vg.set_wait_limit_ns(0)
    flag.zero_()
    out = torch.zeros_like(want)
    vg.chunk_attention(*args, out, error_flag=flag)
    assert int(flag.item()) == 0 and torch.equal(out, want)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_queries_and_keys_that_are_not_finite_stay_in_their_rows(bad):
    """A bad value in one query row spoils that row alone; one in a key spoils
    the rows that attend it (a key's +-infinity times the query's sign may also
    just take the position out) and no earlier ones."""
    from self_speculative_sparse_vg_gb300 import vg
    c = Cache([180], 1, 64, seed=19)
    g = torch.Generator().manual_seed(5)
    q = torch.randn(120, 4, 64, generator=g).bfloat16()
    _, want, _ = check_chunk(c, [120], 4, q=q)
    q2 = q.clone()
    q2[33, 2, 5] = bad
    out = torch.zeros_like(want)
    vg.chunk_attention(c.gpu(), q2.cuda(), i32([0, 120]), i32([180]), 0.125, out)
    keep = torch.ones(120, 4, dtype=torch.bool, device="cuda")
    keep[33, 2] = False
    assert torch.equal(out[keep], want[keep]) and out[33, 2].isnan().all()
    k = c.k[0].clone()
    k[100, 0, 9] = bad                      # position 100: token 40
    c.write(0, k, c.v[0])
    out = torch.zeros_like(want)
    vg.chunk_attention(c.gpu(), q.cuda(), i32([0, 120]), i32([180]), 0.125, out)
    assert torch.equal(out[:40], want[:40])
    s = q.double()[40:, :, 9] * bad         # the logit's sign at position 100
    spoiled = ~(s == -float("inf"))
    assert torch.equal(out[40:].isnan().all(-1).cpu(), spoiled)
    assert torch.equal(out[40:].isnan().any(-1).cpu(), spoiled)


def test_outputs_on_16_bytes():
    """An output that starts on 16 bytes but not on 32, and odd row strides."""
    from self_speculative_sparse_vg_gb300 import vg
    c = Cache([140, 3], 2, 64, seed=20)
    qd, want, _ = check_chunk(c, [70, 3], 8)
    flat = torch.full((73 * 520 + 8,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = flat[8:].view(73, 520)[:, :512].unflatten(1, (8, 64))
    assert out.data_ptr() % 32 == 16
    vg.chunk_attention(c.gpu(), qd, i32([0, 70, 73]), i32([140, 3]), 0.125, out)
    assert torch.equal(out, want)
    assert (flat[:8] == 9).all() and (flat[8:].view(73, 520)[:, 512:] == 9).all()


def test_largest_batch():
    """4096 sequences, one token each, a few positions; and one token more of
    them is refused."""
    from self_speculative_sparse_vg_gb300 import vg
    rng = np.random.default_rng(1)
    lens = rng.integers(1, 20, 4096)
    check_chunk(Cache(lens.tolist(), 1, 64, seed=21), [1] * 4096, 2)
    kv = Cache([1], 1, 64).gpu()
    big = vg.PagedKV(kv.k_pages, kv.v_pages, kv.page_table.expand(4097, -1).contiguous())
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(vg.VGError) as e:
        vg.chunk_attention(big, q, i32([0] * 4097 + [1]), i32([0] * 4096 + [1]), 0.125, torch.zeros_like(q),
                           workspace=torch.zeros(1 << 26, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 2


def test_two_graphs_with_their_own_workspaces():
    """Two captured calls of different shapes replayed in turn and again."""
    from self_speculative_sparse_vg_gb300 import vg
    runs = []
    for lens, new, seed in (([3000, 50], [3, 50], 22), ([777], [200], 23)):
        c = Cache(lens, 2, 128, seed=seed)
        qd, want, _ = check_chunk(c, new, 8)
        kv, cu, ln = c.gpu(), i32(np.concatenate([[0], np.cumsum(new)])), i32(lens)
        ws = torch.empty(vg.chunk_workspace_bytes(len(new), sum(new), 8, 2, 128), dtype=torch.uint8,
                         device="cuda")
        out = torch.zeros_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            vg.chunk_attention(kv, qd, cu, ln, 128 ** -0.5, out, workspace=ws)
        runs.append((g, out, want, kv, cu, ln, ws, qd))
    for _ in range(3):
        for g, out, want, *_ in runs:
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        for g, out, want, *_ in runs:
            assert torch.equal(out, want)
