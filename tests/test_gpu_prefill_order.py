"""When a prompt may enter the decode stack, and what the stack keeps of it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _stack(**kw):
    from self_speculative_sparse_vg_gb300.stack import DecodeStack
    from self_speculative_sparse_vg_gb300.workloads import small_stack
    spec = small_stack(prefix_lens=(37, 200), iterations=2, prompt=60, top_k=32, n_recent=16, **kw)
    return DecodeStack(spec, "cuda", gen_device="cpu")


def test_no_prompt_once_decoding_has_started():
    """It would be placed over the decoded tokens: refused, and nothing changes."""
    st = _stack()
    x = torch.randn(10, st.spec.hidden, dtype=torch.float64, device="cuda")
    st.prefill(x, [4, 6])
    st.seed_selection()
    for after in (lambda: None, st.step):
        after()
        lens, e, pools = st.lens.clone(), st.e.clone(), [p.clone() for p in st.kp + st.vp]
        for rows, new in ((x, [4, 6]), (x[:0], [0, 0])):
            with pytest.raises(ValueError, match="decoding has started"):
                st.prefill(rows, new)
        assert torch.equal(st.lens, lens) and torch.equal(st.e, e)
        assert all(torch.equal(a, b) for a, b in zip(st.kp + st.vp, pools))
    assert int(st.flag.item()) == 0


def test_what_a_chunk_used_goes_with_it():
    """Chunks of many sizes leave no buffers behind; the decode steps' own, one
    set for each block length, are kept."""
    st = _stack()
    for n in range(1, 9):
        st.prefill(torch.randn(2 * n + 1, st.spec.hidden, dtype=torch.float64, device="cuda"), [n, n + 1])
    assert len(st._places) == 0
    st.run()
    kept = {n: id(p) for n, p in st._places.items()}
    assert set(kept) == {1, st.spec.n_drafts + 1}
    st.draws = st.draws.repeat(2, 1, 1)
    st.step()
    assert {n: id(p) for n, p in st._places.items()} == kept and int(st.flag.item()) == 0


def test_rows_are_written_where_they_were_placed():
    """Rows for positions that were not the last to be placed are refused (they
    would be written over other tokens)."""
    st = _stack()
    s, before = st.spec, st.lens
    k = torch.ones(s.batch, 1, s.num_kv_heads, s.head_dim, dtype=torch.bfloat16, device="cuda")
    st._place(before, 1)
    st._write_kv(0, k, k, before)
    st._place(before + 1, 1)
    pool = st.kp[0].clone()
    with pytest.raises(ValueError, match="other positions"):
        st._write_kv(0, k * 2, k * 2, before)
    assert torch.equal(st.kp[0], pool)
