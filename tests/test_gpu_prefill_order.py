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
