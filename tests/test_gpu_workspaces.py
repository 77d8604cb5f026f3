"""Workspaces that a call makes itself, on a stream that is not the current one:
they belong to the call's stream, so that no later work of the current stream
is handed memory that the call still uses."""
import pytest
import torch

from tests.fill_util import Cache, check_chunk, i32

pytestmark = pytest.mark.gpu


def _calls():
    """name -> a call without a workspace, given a stream, and what it writes."""
    from self_speculative_sparse_vg_gb300 import vg
    B, Hq, Hkv, d, L = 2, 8, 2, 64, 5000
    cap = 128 + 4 + 16
    capture = torch.randn(B, Hkv, L, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    rows = torch.randn(vg.all_rows_capture_floats(B, Hq, 3, L), device="cuda",
                       generator=torch.Generator("cuda").manual_seed(2))
    lens = i32([L, 4000])
    index = lambda: (torch.full((B, 1, cap), -1, dtype=torch.int32, device="cuda"), i32([[0], [0]]))  # noqa: E731
    c = Cache([L + 3, 4003], Hkv, d, seed=3, junk=0.0)
    kv = c.gpu()
    q = torch.randn(B * 3, Hq, d, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    cu, kv_lens = i32([0, 3, 6]), i32([L + 3, 4003])
    blocks, counts = i32([[list(range(64))] * 3] * B), i32([[64] * 3] * B)

    def after_inputs(stream):
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        return stream

    def chunk(stream):
        out = torch.zeros_like(q)
        vg.chunk_attention(kv, q, cu, kv_lens, 0.125, out, stream=after_inputs(stream))
        return out,

    def select(stream):
        ix, n = index()
        vg.select_kv(capture, vg.CAPTURE_GROUP_SUM, lens, Hq, Hkv, L, 128, 4, 16, False, ix, n,
                     stream=after_inputs(stream))
        return ix, n

    def weights(stream):
        ix, n = index()
        vg.select_kv_weights(rows, 3, lens, Hq, Hkv, L, 128, 4, 16, False, ix, n,
                     stream=after_inputs(stream))
        return ix, n

    def sparse(stream):
        out = torch.zeros(B, 3, Hq, d, dtype=torch.bfloat16, device="cuda")
        vg.sparse_verify_attention(kv, q.view(B, 3, Hq, d), lens, L, 0.125, blocks, counts, out,
                                   stream=after_inputs(stream))
        return out,
    return dict(chunk_attention=chunk, select_kv=select, select_kv_weights=weights,
                sparse_verify_attention=sparse)


NAMES = ["chunk_attention", "select_kv", "select_kv_weights", "sparse_verify_attention"]


class _Idle:
    """The library, without the launches."""

    def __init__(self, lib):
        self.lib = lib

    def __getattr__(self, name):
        return getattr(self.lib, name) if name.endswith("_bytes") else lambda *a: 0


@pytest.mark.parametrize("name", NAMES)
def test_the_block_goes_back_to_the_calls_stream(name, monkeypatch):
    """Nothing is launched here: whose memory the workspace was is seen from
    what the allocator hands out next."""
    from self_speculative_sparse_vg_gb300 import vg
    call = _calls()[name]
    seen = []
    real_zeros, real_empty = torch.zeros, torch.empty
    note = lambda t: (seen.append((t.data_ptr(), t.numel())) if t.dtype == torch.uint8 else None, t)[1]  # noqa: E731
    monkeypatch.setattr(vg, "_lib", _Idle(vg._lib))
    monkeypatch.setattr(vg, "_binding", _Idle(vg._binding))
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: note(real_zeros(*a, **k)))
    monkeypatch.setattr(torch, "empty", lambda *a, **k: note(real_empty(*a, **k)))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    call(side)
    monkeypatch.undo()
    assert len(seen) == 1 and seen[0][1] > 1, "the call made its own workspace"
    at, n = seen[0]
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(b.data_ptr() + n <= at or at + n <= b.data_ptr() for b in blocks)


@pytest.mark.parametrize("name", NAMES)
def test_results_on_a_stream_of_ones_own(name):
    """The same bits as on the current stream while that one's allocations come
    and go."""
    call = _calls()[name]
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        got = call(side)
        junk = [torch.full((1 << k,), 255, dtype=torch.uint8, device="cuda") for k in range(8, 25)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del junk
