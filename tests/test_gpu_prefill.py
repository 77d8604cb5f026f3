"""The three cache-filling calls together, as a user runs them: prompts enter
the decode stack in chunks (block tables, rotary append, chunk attention, layer
by layer), then the seed verify and draft / verify iterations run on that
cache; and a serving loop over a free list admits, grows and finishes requests."""
import dataclasses

import numpy as np
import pytest
import torch

from oracle import fill_oracle as F
from tests.fill_util import PAGE, chunk_bounds, i32

pytestmark = pytest.mark.gpu


def _spec(**kw):
    from self_speculative_sparse_vg_gb300.workloads import small_stack
    return small_stack(prefix_lens=(37, 200), iterations=2, prompt=150, top_k=32, n_recent=16, **kw)


def _rows(pool, table, n):
    """Logical rows [n][Hkv][d] of one sequence, float64."""
    pos = torch.arange(n)
    return pool.cpu()[table.cpu()[pos // PAGE].long(), :, pos % PAGE].double().numpy()


@pytest.mark.parametrize("theta", [0.0, 10000.0])
def test_prompt_in_chunks_then_decode(theta):
    from self_speculative_sparse_vg_gb300.stack import DecodeStack
    spec = _spec(rope_theta=theta)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2, 150, spec.hidden, generator=g, dtype=torch.float64)
    seen = []
    st = DecodeStack(spec, "cuda", gen_device="cpu",
                     record=lambda kind, l, r: seen.append((kind, l, {k: v.clone() for k, v in r.items()
                                                                      if k in ("out", "q")})))
    done = [0, 0]
    for new in ([100, 0], [1, 77], [0, 1], [49, 72]):
        rows = torch.cat([x[b, done[b]:done[b] + new[b]] for b in range(2)]).cuda()
        seen.clear()
        st.prefill(rows, new)
        done = [a + n for a, n in zip(done, new)]
        # every layer's attention against float64 on its own queries and cache
        for kind, l, r in seen:
            assert kind == "chunk"
            at = 0
            for b in range(2):
                n, L = new[b], spec.prefix_lens[b] + done[b]
                if n == 0:
                    continue
                k, v = (_rows(p[l], st.page_table[b], L) for p in (st.kp, st.vp))
                q = r["q"][at:at + n].double().cpu().numpy()
                o, _, A, S = F.chunk_attention(q, k, v, n, spec.softmax_scale)
                tol, _ = chunk_bounds(o, np.zeros(S.shape), A, S, (L - n + np.arange(n) + 1)[:, None],
                                      spec.head_dim)
                assert (np.abs(r["out"][at:at + n].double().cpu().numpy() - o) <= tol).all(), (l, b)
                at += n
    assert st.lens.tolist() == [187, 350] and int(st.flag.item()) == 0
    st.run()
    torch.cuda.synchronize()
    assert int(st.flag.item()) == 0
    assert torch.isfinite(st.e).all()
    assert (st.lens.cpu() >= torch.tensor([187, 350]) + 1 + 2).all()


def test_rotary_keys_in_the_cache():
    """With rotary positions the cache holds turned keys: layer 0 of a prompt,
    whose keys are known from the inputs, against the rotation in float64."""
    from self_speculative_sparse_vg_gb300.stack import DecodeStack
    spec = _spec(rope_theta=10000.0)
    x = torch.randn(60, spec.hidden, generator=torch.Generator().manual_seed(4), dtype=torch.float64).cuda()
    st = DecodeStack(spec, "cuda", gen_device="cpu")
    _, k, v = st._qkv(0, x)
    st.prefill(x, [20, 40])
    f = st.inv_freq.double().cpu().numpy()
    at = 0
    for b, n in enumerate((20, 40)):
        L = spec.prefix_lens[b]
        kk = k[at:at + n].double().cpu().numpy()
        want = F.rope(kk, [np.arange(L, L + n)], f, [0] * len(f), False)
        got = _rows(st.kp[0], st.page_table[b], L + n)[L:]
        h = spec.head_dim // 2
        pair = np.abs(kk[..., :h]) + np.abs(kk[..., h:])
        tol = 2.0 ** -8 * np.abs(want) * 1.001 + 2.0 ** -20 * np.concatenate([pair, pair], -1)
        assert (np.abs(got - want) <= tol).all()
        np.testing.assert_array_equal(_rows(st.vp[0], st.page_table[b], L + n)[L:],
                                      v[at:at + n].double().cpu().numpy())
        at += n


def test_prefill_refusals():
    from self_speculative_sparse_vg_gb300.stack import DecodeStack
    st = DecodeStack(dataclasses.replace(_spec(), prompt=10), "cuda", gen_device="cpu")
    x = torch.randn(11, st.spec.hidden, dtype=torch.float64, device="cuda")
    for rows, new in ((x, [11, 0]), (x, [5, 5]), (x[:5], [5]), (x[:5], [6, -1])):
        with pytest.raises(ValueError):
            st.prefill(rows, new)
    assert st.prefill(x[:0], [0, 0]).shape[0] == 0
    st.prefill(x[:10], [10, 0])
    with pytest.raises(ValueError):
        st.prefill(x[:1], [1, 0])
    st.prefill(x[:1], [0, 1])
    assert int(st.flag.item()) == 0


@pytest.mark.parametrize("pages", [40, 14, 7])
def test_serving_loop_over_a_free_list(pages):
    """Twelve steps of admissions, prompt chunks, single tokens, rejected drafts
    and finished requests over one free list: every step's tables equal the
    oracle's, no page is held twice, and every row's attention equals float64
    on a dense copy of what was written."""
    from self_speculative_sparse_vg_gb300 import vg
    rng = np.random.default_rng(5)
    g = torch.Generator().manual_seed(6)
    B, Hq, Hkv, d, width = 5, 8, 2, 64, 16
    kp = torch.full((pages, Hkv, PAGE, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    table, owned = i32(np.full((B, width), -1)), i32([0] * B)
    free, count = i32(rng.permutation(pages)), i32([pages])
    kv = vg.PagedKV(kp, vp, table)
    room = 130
    cu, lens = (torch.zeros(m, dtype=torch.int32, device="cuda") for m in (B + 1, B))
    pos, slots = (torch.zeros(room, dtype=torch.int32, device="cuda") for _ in range(2))
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros(room, Hq, d, dtype=torch.bfloat16, device="cuda")
    freq = (1e4 ** (-torch.arange(d // 2, dtype=torch.float64) * 2 / d)).float().cuda()
    ws = torch.empty(vg.chunk_workspace_bytes(B, room, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    dense = [(np.zeros((0, Hkv, d)), np.zeros((0, Hkv, d))) for _ in range(B)]
    cached = [0] * B
    refused = 0
    for step in range(12):
        new = []
        for b in range(B):
            if cached[b] and rng.random() < 0.15:             # finished: everything goes back
                cached[b], dense[b] = 0, tuple(x[:0] for x in dense[b])
                new.append(0)
            elif cached[b] == 0:
                new.append(int(rng.integers(0, 60)))          # a prompt, or none
            else:
                if rng.random() < 0.3:                        # rejected drafts
                    back = int(rng.integers(0, min(cached[b], 20)))
                    cached[b] -= back
                    dense[b] = tuple(x[:cached[b]] for x in dense[b])
                new.append(int(rng.integers(0, 7)))
        while sum(new) > room:
            new[int(np.argmax(new))] //= 2
        want = F.step_tables(table.cpu().numpy(), pages, cached, new, room, owned.tolist(),
                             free.tolist(), int(count.item()))
        flag.zero_()
        vg.step_tables(table, pages, i32(cached), i32(new), cu, lens, pos, slots, owned=owned,
                       free_pages=free, free_count=count, error_flag=flag)
        for got, name in ((table, "table"), (owned, "owned"), (free, "free"), (cu, "cu"),
                          (lens, "lens"), (pos, "positions"), (slots, "slots")):
            np.testing.assert_array_equal(got.cpu().numpy(), want[name], err_msg=f"{step} {name}")
        assert int(count.item()) == want["count"] and int(flag.item()) == want["flag"]
        held = [int(p) for b in range(B) for p in table[b, :int(owned[b])].tolist()]
        stack = free[:want["count"]].tolist()
        assert sorted(held + stack) == list(range(pages)), "a page is lost or held twice"
        refused += want["flag"] != 0
        qkv = torch.randn(room, (Hq + 2 * Hkv) * d, generator=g).bfloat16().cuda()
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
        turned = vg.rope_append(kv, q, k, v, slots, torch.empty(room, Hq, d, dtype=torch.bfloat16,
                                                                 device="cuda"),
                                positions=pos, inv_freq=freq, error_flag=flag)
        out.fill_(5.0)
        vg.chunk_attention(kv, turned, cu, lens, d ** -0.5, out, workspace=ws, error_flag=flag)
        torch.cuda.synchronize()
        assert int(flag.item()) == want["flag"]
        rows = np.concatenate([[0], np.cumsum(new)])
        for b in range(B):
            r = slice(int(rows[b]), int(rows[b + 1]))
            o = out[r].double().cpu().numpy()
            if want["lens"][b] == 0:
                assert (o == 0).all()                         # refused: nothing attended
                continue
            s = slots[r].long().cpu()
            fresh = tuple(p.cpu()[s // PAGE, :, s % PAGE].double().numpy() for p in (kp, vp))
            np.testing.assert_array_equal(fresh[1], v[r].double().cpu().numpy())
            dense[b] = tuple(np.concatenate([x, y]) for x, y in zip(dense[b], fresh))
            cached[b] += new[b]
            n, L = new[b], cached[b]
            ro, _, A, S = F.chunk_attention(turned[r].double().cpu().numpy(), *dense[b], n, d ** -0.5)
            tol, _ = chunk_bounds(ro, np.zeros(S.shape), A, S, (L - n + np.arange(n) + 1)[:, None], d)
            assert (np.abs(o - ro) <= tol).all(), (step, b)
        assert (out[int(rows[-1]):] == 5.0).all()
    assert refused or pages > 7, "the small pool never ran out: the loop is too easy"
