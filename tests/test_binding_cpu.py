"""The native part of the binding: what it refuses before anything is launched,
and that a refusal is a Python exception (no GPU is needed for it)."""
import pytest
import torch

from self_speculative_sparse_vg_gb300 import vg, vg_binding


def _cache():
    p = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    return vg.PagedKV(p, p.clone(), torch.zeros(1, 2, dtype=torch.int32))


@pytest.mark.parametrize("bad", [None, 3, "x", [1, 2], object()])
def test_what_is_no_tensor_is_refused(bad):
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="page_table"):
        vg.step_tables(bad, 2, i, i, i, i, i, i)
    kv = _cache()
    kv.k_pages = bad
    with pytest.raises(ValueError, match="cache"):   # of the host: refused before k and v are looked at
        vg.rope_append(_cache(), None, bad, bad, i)
    with pytest.raises(ValueError, match="k_pages: a tensor"):
        vg.rope_append(kv, None, i, i, i)
    with pytest.raises(ValueError, match="k_pages: a tensor"):
        vg.chunk_attention(kv, i, i, i, 1.0, i, workspace=i)


def test_tensors_of_the_host_are_refused():
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        vg.step_tables(torch.zeros(1, 2, dtype=torch.int32), 2, i, i, torch.zeros(2, dtype=torch.int32), i, i, i)
    r = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="cache"):
        vg.rope_append(_cache(), r, r, r, i)
    with pytest.raises(ValueError):
        vg.chunk_attention(_cache(), r, torch.zeros(2, dtype=torch.int32), i, 1.0, r.clone(),
                           workspace=torch.zeros(64, dtype=torch.uint8))


@pytest.mark.parametrize("name", ["step_tables", "rope_append", "chunk_attention"])
def test_a_wrong_number_of_arguments_is_a_type_error(name):
    with pytest.raises(TypeError):
        getattr(vg_binding, name)(1, 2)
