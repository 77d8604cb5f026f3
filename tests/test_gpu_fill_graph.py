"""The three cache-filling calls captured together and replayed as requests
grow, with workspaces that the calls make themselves inside the capture."""
import numpy as np
import pytest
import torch

from tests.fill_util import PAGE, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("room", [40, 1500])
def test_a_captured_step_replayed_as_requests_grow(room):
    """One graph of a whole step; lengths, rows and tables change between
    replays.  Every replay equals the same calls made one by one on copies."""
    from self_speculative_sparse_vg_gb300 import vg
    rng = np.random.default_rng(room)
    g = torch.Generator().manual_seed(room)
    B, Hq, Hkv, d, width = 4, 8, 2, 64, 400
    pages = 600
    freq = (1e4 ** (-torch.arange(d // 2, dtype=torch.float64) * 2 / d)).float().cuda()

    def state():
        table, owned = i32(np.full((B, width), -1)), i32([0] * B)
        pool = torch.zeros(2, pages, Hkv, PAGE, d, dtype=torch.bfloat16, device="cuda")
        rows = torch.zeros(room, (Hq + 2 * Hkv) * d, dtype=torch.bfloat16, device="cuda")
        ints = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        return dict(table=table, owned=owned, free=i32(np.arange(pages)), count=i32([pages]), pool=pool, rows=rows,
                    cached=ints(B), new=ints(B), cu=ints(B + 1), lens=ints(B), pos=ints(room), slots=ints(room),
                    turned=torch.zeros(room, Hq, d, dtype=torch.bfloat16, device="cuda"),
                    out=torch.zeros(room, Hq, d, dtype=torch.bfloat16, device="cuda"),
                    lse=torch.zeros(room, Hq, device="cuda"), flag=ints(1))

    def step(s):
        kv = vg.PagedKV(s["pool"][0], s["pool"][1], s["table"])
        q, k, v = (x.unflatten(1, (-1, d)) for x in s["rows"].split([Hq * d, Hkv * d, Hkv * d], 1))
        vg.step_tables(s["table"], pages, s["cached"], s["new"], s["cu"], s["lens"], s["pos"], s["slots"],
                       owned=s["owned"], free_pages=s["free"], free_count=s["count"], error_flag=s["flag"])
        vg.rope_append(kv, q, k, v, s["slots"], s["turned"], positions=s["pos"], inv_freq=freq, error_flag=s["flag"])
        vg.chunk_attention(kv, s["turned"], s["cu"], s["lens"], d ** -0.5, s["out"], lse=s["lse"],
                           error_flag=s["flag"])

    a, b = state(), state()
    step(b)                                        # nothing new: loads the kernels before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    cached = np.zeros(B, int)
    for i in range(8):
        new = rng.integers(0, min(7, room // B), B)
        new[i % B] += rng.integers(0, room - int(new.sum()) + 1)
        if i == 5:
            cached[2], new[2] = 0, 0               # a finished request
        rows = torch.randn(room, (Hq + 2 * Hkv) * d, generator=g).bfloat16()
        for s in (a, b):
            s["rows"].copy_(rows)
            s["cached"].copy_(i32(cached))
            s["new"].copy_(i32(new))
        graph.replay()
        junk = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
        step(b)
        torch.cuda.synchronize()
        assert int(b["flag"].item()) == 0
        for name in a:
            assert torch.equal(a[name], b[name]), (i, name)
        cached = cached + new
        del junk
    assert int(a["lens"].max()) > 2 * room // B
