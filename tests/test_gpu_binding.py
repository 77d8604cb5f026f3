"""What the native binding refuses of tensors on the GPU: one argument of a good
call wrong at a time, refused by its name before anything is launched."""
import pytest
import torch

from tests.fill_util import i32

pytestmark = pytest.mark.gpu

B, T, HQ, HKV, D, PAGES, WIDTH = 3, 7, 8, 2, 64, 9, 4


def _i(*n):
    return torch.zeros(*n, dtype=torch.int32, device="cuda")


def _h(*n):
    return torch.zeros(*n, dtype=torch.bfloat16, device="cuda")


def _wide(t):
    """The same values, every second element of a tensor twice as wide."""
    return torch.stack((t, t), -1).flatten(-2)[..., ::2]


def _refused(call, good, cases):
    """cases: (the name in the refusal, {argument: value})."""
    call(**good)                                   # the good call is one
    torch.cuda.synchronize()
    before = {k: v.clone() for k, v in good.items() if torch.is_tensor(v)}
    for words, change in cases:
        with pytest.raises(ValueError, match=f"^{words}: "):
            call(**{**good, **change})
    torch.cuda.synchronize()
    for k, v in before.items():
        assert torch.equal(good[k], v), k


def test_step_tables():
    from self_speculative_sparse_vg_gb300 import vg
    good = dict(page_table=_i(B, WIDTH), num_pages=PAGES, cached_lens=i32([1, 2, 3]), new_lens=i32([2, 2, 3]),
                cu_tokens=_i(B + 1), kv_lens=_i(B), positions=_i(T), slots=_i(T), owned=_i(B) + 1,
                free_pages=_i(5), free_count=_i(1), error_flag=_i(1))
    sizes = dict(cached_lens=B, new_lens=B, cu_tokens=B + 1, kv_lens=B, slots=T, owned=B, free_count=1)
    cases = [("page_table", dict(page_table=good["page_table"][0])),
             ("page_table", dict(page_table=_wide(_i(B, WIDTH)))),
             ("num_pages", dict(num_pages=-1)), ("num_pages", dict(num_pages=1 << 32)),
             ("num_pages", dict(num_pages=2.5)),
             ("num_pages", dict(num_pages=None)), ("error_flag", dict(error_flag=_i(0))),
             ("slots", dict(positions=_i(T + 1))), ("positions", dict(positions=_i(T).long())),
             ("free_pages", dict(free_pages=_i(10)[::2])),
             ("owned, free_pages and free_count", dict(owned=None)),
             ("owned, free_pages and free_count", dict(free_pages=None)),
             ("owned, free_pages and free_count", dict(free_count=None)),
             ("stream", dict(stream=type("S", (), dict(cuda_stream="x"))()))]
    for name, n in sizes.items():
        cases += [(name, {name: _i(n - 1)}), (name, {name: _i(n + 1)}), (name, {name: _i(n).float()}),
                  (name, {name: _i(n).cpu()}), (name, {name: 3})]
        if n > 1:
            cases.append((name, {name: _i(2 * n)[::2]}))
    _refused(vg.step_tables, good, cases)


def test_rope_append():
    from self_speculative_sparse_vg_gb300 import vg
    cache = lambda: vg.PagedKV(_h(PAGES, HKV, 16, D), _h(PAGES, HKV, 16, D), _i(1, WIDTH))  # noqa: E731
    half = D // 2
    good = dict(kv=cache(), q=_h(T, HQ, D), k=_h(T, HKV, D), v=_h(T, HKV, D), slots=_i(T), q_out=_h(T, HQ, D),
                positions=_i(3, T), inv_freq=torch.ones(half, device="cuda"), freq_axis=_i(half),
                error_flag=_i(1))
    good["slots"].copy_(torch.arange(T))
    bad_kv = cache()
    bad_kv.v_pages = _h(PAGES - 1, HKV, 16, D)
    host_kv = cache()
    host_kv.k_pages = host_kv.k_pages.cpu()
    flat_kv = cache()
    flat_kv.page_table = _i(4)
    cases = [("cache", dict(kv=bad_kv)), ("cache", dict(kv=host_kv)), ("page_table", dict(kv=flat_kv)),
             ("k, v", dict(k=_h(T + 1, HKV, D))), ("k, v", dict(v=_h(T, HKV + 1, D))),
             ("k, v", dict(v=_h(T, HKV, 2 * D))),
             ("k, v", dict(k=_h(T, HKV + 1, D), v=_h(T, HKV + 1, D))),
             ("k, v", dict(k=_h(T, HKV, 32), v=_h(T, HKV, 32))),
             ("q, q_out", dict(q=_h(T + 1, HQ, D))), ("q, q_out", dict(q_out=_h(T - 1, HQ, D))),
             ("q, q_out", dict(q_out=_h(T, HQ + 1, D))), ("q, q_out", dict(q=_h(T, HQ, 128))),
             ("slots", dict(slots=_i(T - 1))), ("slots", dict(slots=_i(T + 1))),
             ("slots", dict(slots=_i(T).long())),
             ("slots", dict(slots=_i(T, 2)[:, 0])), ("positions", dict(positions=_i(T - 1))),
             ("positions", dict(positions=_i(3, T + 1))), ("positions", dict(positions=_i(1, 3, T))),
             ("positions", dict(positions=_i(T, 3).T)), ("positions", dict(positions=_i(T).long())),
             ("positions", dict(positions=None)),
             ("inv_freq", dict(inv_freq=torch.ones(half, device="cuda").double())),
             ("inv_freq", dict(inv_freq=torch.ones(half))),
             ("inv_freq", dict(inv_freq=torch.ones(D, device="cuda")[::2])),
             ("freq_axis", dict(freq_axis=_i(half - 1))), ("freq_axis", dict(freq_axis=_i(half).float())),
             ("error_flag", dict(error_flag=torch.zeros(1, device="cuda")))]
    for name, heads in (("q", HQ), ("k", HKV), ("v", HKV), ("q_out", HQ)):
        cases += [(name, {name: _h(T, heads * D)}), (name, {name: _h(T, heads, D).float()}),
                  (name, {name: _h(T, heads, D).cpu()}), (name, {name: _wide(_h(T, heads, D))}),
                  (name, {name: _h(T, D, heads).transpose(1, 2)}),
                  (name, {name: _h(heads, T, D).transpose(0, 1)}), (name, {name: "x"})]
    _refused(vg.rope_append, good, cases)
    for change in (dict(q=_h(T, HQ, D + 4)[..., :D]), dict(k=_h(1, HKV, D).expand(T, HKV, D)),
                   dict(q_out=_h(T * HQ * D + 1)[1:].view(T, HQ, D)),
                   dict(inv_freq=torch.ones(12, device="cuda"), freq_axis=_i(12)),
                   dict(inv_freq=torch.ones(D, device="cuda"), freq_axis=_i(D))):
        # well formed, but not for the library: odd strides, rows that coincide, odd addresses and widths
        with pytest.raises((ValueError, vg.VGError)):
            vg.rope_append(**{**good, **change})


def test_chunk_attention():
    from self_speculative_sparse_vg_gb300 import vg
    kv = vg.PagedKV(_h(PAGES, HKV, 16, D), _h(PAGES, HKV, 16, D), _i(B, WIDTH))
    ws = torch.zeros(vg.chunk_workspace_bytes(B, T, HQ, HKV, D), dtype=torch.uint8, device="cuda")
    good = dict(kv=kv, q=_h(T, HQ, D), cu_q=i32([0, 2, 4, 7]), kv_lens=i32([3, 4, 6]), softmax_scale=0.125,
                out=_h(T, HQ, D), lse=torch.zeros(T, HQ, device="cuda"), workspace=ws, error_flag=_i(1))
    rows = vg.PagedKV(kv.k_pages, kv.v_pages, _i(B + 1, WIDTH))
    cases = [("out", dict(out=_h(T + 1, HQ, D))), ("out", dict(out=_h(T, HQ + 2, D))),
             ("out", dict(out=_h(T, HQ, 128))),
             ("out", dict(q=_h(T, HQ, 128), out=_h(T, HQ, 128))), ("page_table", dict(kv=rows)),
             ("page_table", dict(kv_lens=_i(B - 1))), ("kv_lens", dict(kv_lens=i32([3, 4, 6]).long())),
             ("kv_lens", dict(kv_lens=_i(2 * B)[::2])), ("cu_q", dict(cu_q=_i(B))),
             ("cu_q", dict(cu_q=_i(B + 2))),
             ("cu_q", dict(cu_q=_i(B + 1).long())), ("cu_q", dict(cu_q=_i(B + 1).cpu())),
             ("lse", dict(lse=torch.zeros(T, HQ - 1, device="cuda"))),
             ("lse", dict(lse=torch.zeros(T, HQ, device="cuda").double())),
             ("lse", dict(lse=torch.zeros(HQ, T, device="cuda").T)), ("lse", dict(lse=torch.zeros(T, HQ))),
             ("softmax_scale", dict(softmax_scale="x")), ("workspace", dict(workspace=ws.cpu())),
             ("workspace", dict(workspace=ws.new_zeros(2 * ws.numel())[::2])),
             ("error_flag", dict(error_flag=_i(0)))]
    for name in ("q", "out"):
        cases += [(name, {name: _h(T, HQ * D)}), (name, {name: _h(T, HQ, D).float()}),
                  (name, {name: _h(T, HQ, D).cpu()}), (name, {name: _wide(_h(T, HQ, D))}),
                  (name, {name: _h(HQ, T, D).transpose(0, 1)}), (name, {name: None})]
    _refused(vg.chunk_attention, good, cases)
    for change, status in ((dict(workspace=ws[:-1]), 3), (dict(softmax_scale=0.0), 1),
                           (dict(softmax_scale=float("nan")), 1),
                           (dict(workspace=torch.zeros(ws.numel() + 8, dtype=torch.uint8, device="cuda")[8:]), 1),
                           (dict(out=_h(1, HQ, D).expand(T, HQ, D)), 1),
                           (dict(q=_h(T * HQ * D + 1)[1:].view(T, HQ, D)), 1)):
        with pytest.raises(vg.VGError) as e:
            vg.chunk_attention(**{**good, **change})
        assert e.value.status == status, change
