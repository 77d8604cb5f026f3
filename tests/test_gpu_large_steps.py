"""Steps of more sequences than one call of chunk attention takes."""
import numpy as np
import pytest
import torch

from oracle import fill_oracle as F
from tests.fill_util import Cache, chunk_bounds, i32

pytestmark = pytest.mark.gpu


def test_a_step_of_8192_requests_is_attended_in_two_calls():
    """One step of the most requests that block tables take, planned once; its
    rows attended 4096 sequences at a time with one workspace."""
    from self_speculative_sparse_vg_gb300 import vg
    rng = np.random.default_rng(2)
    B, Hq, Hkv, d = 8192, 2, 1, 64
    new = rng.integers(0, 3, B)
    cached = rng.integers(0, 25, B)
    lens = cached + new
    c = Cache(lens.tolist(), Hkv, d, seed=41)
    kv = c.gpu()
    T = int(new.sum())
    cu, kv_lens = (torch.full((m,), -1, dtype=torch.int32, device="cuda") for m in (B + 1, B))
    pos, slots = (torch.empty(T, dtype=torch.int32, device="cuda") for _ in range(2))
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    vg.step_tables(kv.page_table, kv.k_pages.shape[0], i32(cached), i32(new), cu, kv_lens, pos, slots,
                   error_flag=flag)
    g = torch.Generator().manual_seed(5)
    q = torch.randn(T, Hq, d, generator=g).bfloat16()
    out = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    ws = torch.empty(vg.chunk_workspace_bytes(4096, T, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    for a in range(0, B, 4096):
        b = a + 4096
        part = vg.PagedKV(kv.k_pages, kv.v_pages, kv.page_table[a:b])
        vg.chunk_attention(part, q.cuda(), cu[a:b + 1], kv_lens[a:b], d ** -0.5, out, lse=lse, workspace=ws,
                           error_flag=flag)
    assert int(flag.item()) == 0
    got, rows = out.double().cpu().numpy(), np.concatenate([[0], np.cumsum(new)])
    assert cu.tolist() == rows.tolist()
    ls = lse.double().cpu().numpy()
    for b in range(B):
        n, L, r = int(new[b]), int(lens[b]), slice(int(rows[b]), int(rows[b + 1]))
        o, l, A, S = F.chunk_attention(q[r].double().numpy(), c.k[b].double().numpy(), c.v[b].double().numpy(), n,
                                       d ** -0.5)
        tol, tol_l = chunk_bounds(o, l, A, S, (L - n + np.arange(n) + 1)[:, None], d)
        assert (np.abs(got[r] - o) <= tol).all() and (np.abs(ls[r] - l) <= tol_l).all(), b
