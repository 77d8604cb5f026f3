"""The calls for beams and encoder states at their far ends: offsets past 32 bits,
calls at once on two streams, and a workspace that graphs of several shapes share."""
import numpy as np
import pytest
import torch

from tests.beam_util import States, check_beam_tables, check_cross, check_select, cross_bounds, run_beam_tables
from tests.fill_util import PAGE, i32
from oracle import beam_oracle as O

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,V,stride", [(torch.bfloat16, 5001, 400_000_001), (torch.float32, 9000, 200_000_004)])
def test_rows_of_logits_far_apart(dtype, V, stride):
    """12 rows in 9.6 GB."""
    x = torch.empty(12, stride, dtype=dtype, device="cuda")[:, 3:3 + V]
    x.copy_(torch.randn(12, V, generator=torch.Generator().manual_seed(1)))
    check_select(x, np.random.default_rng(1).normal(size=(3, 4)).astype(np.float32), 8)


def test_wide_tables():
    """The last row begins 2.2e9 entries into the table."""
    from self_speculative_sparse_vg_gb300 import vg
    W, width, near = 32, 70_000_000, 300
    rng = np.random.default_rng(3)
    lens = np.full(W, 250 * PAGE + 5)
    owned = np.full(W, 251)
    table = np.full((W, near), -1)
    table[:, :200] = np.arange(200)
    table[:, 200:251] = 200 + np.arange(W * 51).reshape(W, 51)
    pool = 200 + W * 51 + 40
    free = np.concatenate([np.arange(pool - 40, pool), np.full(W * 51, -1)])
    parents = rng.integers(0, W, (1, W))
    want = run_beam_tables(parents, lens, table, pool, owned, free, 40)
    wide = torch.full((W, width), -1, dtype=torch.int32, device="cuda")
    wide[:, :near] = i32(table)
    dev = dict(lens=i32(lens), owned=i32(owned), free=i32(free), count=i32([40]))
    copies = torch.zeros(W, 3, dtype=torch.int32, device="cuda")
    vg.beam_tables(wide, pool, i32(parents), dev["lens"], dev["owned"], dev["free"], dev["count"], copies)
    np.testing.assert_array_equal(wide[:, :near].cpu().numpy(), want["table"])
    assert int(wide[:, near:].max()) == -1
    for k, v in dev.items():
        np.testing.assert_array_equal(v.cpu().numpy().squeeze(), np.squeeze(want[k]), err_msg=k)
    np.testing.assert_array_equal(copies.cpu().numpy(), want["copies"])


def test_copies_far_in_a_large_pool():
    """Pages at 4.6 GB of a pool."""
    from self_speculative_sparse_vg_gb300 import vg
    n, Hkv, d = 140_000, 8, 128
    pools = [torch.empty(n, Hkv, PAGE, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pages = torch.tensor([n - 1, 3, n - 2, 7], device="cuda")
    for p in pools:
        p[pages] = torch.randn(4, Hkv, PAGE, d, device="cuda").bfloat16()
    before = [p[pages].clone() for p in pools]
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    vg.copy_pages(vg.PagedKV(*pools, table), i32([[n - 1, 3, 9], [7, n - 2, 16]]))
    for p, b in zip(pools, before):
        got = p[pages]
        assert torch.equal(got[1, :, :9], b[0, :, :9]) and torch.equal(got[1, :, 9:], b[1, :, 9:])
        assert torch.equal(got[2], b[3]) and torch.equal(got[0], b[0]) and torch.equal(got[3], b[3])


@pytest.mark.parametrize("Hq,Hkv,d", [(32, 8, 128), (66, 66, 64)])
def test_rows_far_in_a_large_query(Hq, Hkv, d):
    """The last rows' outputs lie past 2^31 elements."""
    from self_speculative_sparse_vg_gb300 import vg
    T, S, last = 2 ** 31 // (Hq * d) + 4000, 200, 40
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(S, Hkv, d, generator=g).bfloat16() for _ in range(2))
    q = torch.zeros(T, Hq, d, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(last, Hq, d, generator=g).bfloat16()
    q[T - last:] = tail.cuda()
    out = torch.empty_like(q)
    lse = torch.empty(T, Hq, device="cuda")
    vg.cross_attention(q, k.cuda(), v.cuda(), i32([0, T - last, T]), i32([0, 0]), i32([S, S]), d ** -0.5, out, lse=lse)
    ro, rl, A, X = O.cross_attention(tail.double().numpy(), k.double().numpy(), v.double().numpy(),
                                     np.ones(S, bool), d ** -0.5)
    tol, tol_l = cross_bounds(ro, rl, A, X, S, d, torch.bfloat16, float(v.abs().max()))
    assert (np.abs(out[T - last:].double().cpu().numpy() - ro) <= tol).all()
    assert (np.abs(lse[T - last:].double().cpu().numpy() - rl) <= tol_l).all()
    # rows whose scores are all zero: weights of one, a sum and one rounding (under 2^-7)
    mean = v.double().mean(0).repeat_interleave(Hq // Hkv, 0)
    got = out[T - last - 5:T - last].double().cpu()
    assert ((got - mean).abs() <= 2.0 ** -7 * (mean.abs() + v.double().abs().mean(0).repeat_interleave(Hq // Hkv, 0))).all()


def test_calls_at_once_on_two_streams():
    from self_speculative_sparse_vg_gb300 import vg
    g = torch.Generator().manual_seed(2)
    q = torch.randn(40, 16, 64, generator=g).bfloat16().cuda()
    k, v = (torch.randn(8 * 1500, 16, 64, generator=g).bfloat16().cuda() for _ in range(2))
    cu, starts, lens = i32(np.arange(9) * 5), i32(np.arange(8) * 1500), i32([1500] * 8)
    x = torch.randn(64, 50000, generator=g).bfloat16().cuda()
    s = torch.randn(8, 8, generator=g).cuda()
    new = lambda: [torch.zeros(8, 16, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]  # noqa: E731
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    alone_o, alone = torch.zeros_like(q), new()
    vg.cross_attention(q, k, v, cu, starts, lens, 0.125, alone_o)
    vg.beam_select(x, s, *alone)
    outs, sel = [torch.zeros_like(q) for _ in range(12)], [new() for _ in range(12)]
    torch.cuda.synchronize()
    for i in range(12):                                     # both calls on both streams
        vg.cross_attention(q, k, v, cu, starts, lens, 0.125, outs[i], stream=streams[i % 2])
        vg.beam_select(x, s, *sel[i], stream=streams[(i + 1) % 2])
    torch.cuda.synchronize()
    for o, t in zip(outs, sel):
        assert torch.equal(o, alone_o)
        assert all(torch.equal(a, b) for a, b in zip(t, alone))


def test_two_graphs_share_a_selection_workspace():
    from self_speculative_sparse_vg_gb300 import vg
    shapes = [(3, 4, 9001, 8, torch.bfloat16), (20, 5, 50257, 10, torch.float16), (1, 2, 300, 4, torch.float32)]
    ws = torch.empty(max(vg.beam_select_workspace_bytes(B, W, V, t, K) for B, W, V, K, t in shapes), dtype=torch.uint8,
                     device="cuda")
    graphs, calls = [], []
    for i, (B, W, V, K, t) in enumerate(shapes):
        x, s = torch.zeros(B * W, V, dtype=t, device="cuda"), torch.zeros(B, W, device="cuda")
        out = [torch.zeros(B, K, dtype=u, device="cuda") for u in (torch.float32, torch.int32, torch.int32)]
        calls.append((x, s, out))
        vg.beam_select(x, s, *out, workspace=ws)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            vg.beam_select(x, s, *out, workspace=ws)
    for seed in range(3):
        for x, s, _ in calls:
            x.normal_()
            s.normal_()
        ws.fill_(255)
        for i in (0, 1, 0, 2, 1):
            graphs[i].replay()
        for (x, s, out), (B, W, V, K, t) in zip(calls, shapes):
            want = [torch.zeros_like(o) for o in out]
            vg.beam_select(x, s, *want)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), (seed, B, W)


def test_every_row_asks_for_a_copy_of_one_page():
    """Shared last pages in the most rows that a call takes."""
    W = 32
    B = 4096 // W
    table = np.arange(B)[:, None].repeat(W, 0).reshape(B * W, 1)
    free = np.concatenate([np.arange(B, B + B * W), np.full(9, -1)])
    got = check_beam_tables(np.zeros((B, W), int), np.full(B * W, 7), table, B + B * W, np.ones(B * W, int), free, B * W)
    assert got["count"] == B and len(np.unique(got["table"])) == B * W


def test_the_longest_group_of_heads():
    check_cross(States([300, 77], 1, 64, seed=4), [3, 1], 128)
    check_cross(States([300, 77], 1, 128, seed=5, masked=0.2), [2, 300], 128)


@pytest.mark.parametrize("masked", [0.0, 0.3])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Hq,Hkv", [(16, 16), (6, 2), (10, 2), (48, 4), (66, 2), (128, 2), (80, 80)])
def test_pairs_of_heads_with_full_row_tiles(Hq, Hkv, dtype, masked):
    """Up to 128 rows of a head on average, among many states: single tokens, full
    tiles and sequences of several units in one call."""
    lens = [700, 1, 2500, 128, 0, 129, 1111, 40, 1300]
    gap = 7 * 128 * 160 // Hkv // len(lens)                 # the buffer's states decide
    tile = 128 * Hkv // Hq
    new = [tile, 1, tile // 2 + 1, max(1, tile // 4), tile, 0, tile + tile // 2, 2, 2 * tile + 1]
    new[4] -= max(0, sum(new) - len(lens) * tile)
    assert 0 <= new[4] and sum(new) <= len(lens) * tile
    check_cross(States(lens, Hkv, 64, dtype, seed=Hq, gap=gap, masked=masked, fused=Hkv < 16), new, Hq, rows_after=1,
                strided=dtype == torch.float16)


@pytest.mark.parametrize("Hkv,g,d", [(8, 4, 128), (2, 4, 64), (1, 3, 128)])
@pytest.mark.parametrize("new", [[8, 0, 0, 0, 0, 0, 0, 0], [0, 0, 6, 0, 0, 1, 0, 1], [1] * 8])
def test_the_rows_of_a_padded_batch_are_one_sequences(Hkv, g, d, new):
    """Few rows, whose units have many parts: more rows of one unit than a sequence has
    on average, for both attentions that divide their units."""
    from tests.fill_util import Cache, check_chunk
    lens = [6000, 300, 9000, 40, 0, 2000, 1, 500]
    check_cross(States(lens, Hkv, d, seed=g), new, Hkv * g)
    check_chunk(Cache([n + m for n, m in zip(lens, new)], Hkv, d, seed=g), new, Hkv * g)
