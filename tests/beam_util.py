"""Shared pieces of the tests of beams and of cross attention."""
import numpy as np
import torch

from oracle import beam_oracle as O
from tests.fill_util import i32

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


class States:
    """Encoder states of several sequences in one buffer, `gap` rows apart (a
    `room` gives slots of that many rows instead); what no sequence holds is
    `junk`, and so is what the mask leaves out (NaN by default)."""

    def __init__(self, lens, Hkv, d, dtype=torch.bfloat16, seed=0, gap=0, room=0, masked=0.0, junk=float("nan"),
                 fused=False):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.starts, at = list(lens), [], gap
        for n in lens:
            self.starts.append(at)
            at += room if room else n + gap
        total = at
        wide = torch.full((total, 2 * Hkv + 1, d), junk, dtype=dtype)
        keep = torch.ones(total, dtype=torch.bool)
        if masked:
            keep = torch.rand(total, generator=g) >= masked
        self.mask = keep if masked else None
        self.attended = []
        for s, n in zip(self.starts, lens):
            rows = torch.randn(n, 2 * Hkv, d, generator=g).to(dtype)
            rows[~keep[s:s + n]] = junk
            wide[s:s + n, :2 * Hkv] = rows
            self.attended.append(keep[s:s + n].numpy())
        self.k, self.v = wide[:, :Hkv], wide[:, Hkv:2 * Hkv]
        self.fused, self.wide, self.Hkv, self.d, self.dtype, self.gen = fused, wide, Hkv, d, dtype, g

    def gpu(self):
        if self.fused:
            w = self.wide.cuda()
            return w[:, :self.Hkv], w[:, self.Hkv:2 * self.Hkv]
        return self.k.contiguous().cuda(), self.v.contiguous().cuda()


def cross_bounds(out, lse, A, S, attended, d, dtype, vmax):
    """Largest deviations arithmetic allows: the output is rounded once and each
    softmax weight may be (half a step of the type; an fp16 weight below 2^-14 by
    2^-25 of the largest, which is at least one); logits are float32 sums of d
    products (a step of 2^-23 each, S bounds their magnitudes) and shift a weight
    by that much, relatively, above and below the line; `attended` float32
    additions make the sums."""
    rel = 2.0 * (d + 8) * 2.0 ** -23 * (S + 1.0) + 2.0 * attended * 2.0 ** -23 + 2.0 ** -20
    tol = HALF_STEP[dtype] * (np.abs(out) + A) * 1.01 + rel[..., None] * A + 1e-30
    if dtype == torch.float16:
        tol += (attended * vmax + 1.0) * 2.0 ** -25
    tol_lse = rel + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0.0))
    return tol, tol_lse


def check_cross(st, new, Hq, scale=None, seed=5, q=None, lse=True, strided=False, rows_after=0, workspace=None,
                stream=None):
    """vg.cross_attention against the oracle for `new` rows per sequence.
    Returns (q, out, lse) on the GPU."""
    from self_speculative_sparse_vg_gb300 import vg
    d, dtype = st.d, st.dtype
    scale = d ** -0.5 if scale is None else scale
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1]) + rows_after
    if q is None:
        q = torch.randn(T, Hq, d, generator=torch.Generator().manual_seed(seed)).to(dtype)
    if strided:   # rows of a wider projection, outputs into a wider buffer
        wide = torch.full((T, Hq + 3, d), 9.0, dtype=dtype)
        wide[:, 2:2 + Hq] = q
        qd = wide.cuda()[:, 2:2 + Hq]
        buf = torch.full((T, Hq + 1, d), 7.0, dtype=dtype, device="cuda")
        out = buf[:, :Hq]
    else:
        qd = q.cuda()
        buf = out = torch.full((T, Hq, d), 7.0, dtype=dtype, device="cuda")
    ls = torch.full((T, Hq), 7.0, dtype=torch.float32, device="cuda") if lse else None
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = st.gpu()
    mask = None if st.mask is None else st.mask.cuda()
    cu_d, starts, lens = i32(cu), i32(st.starts), i32(st.lens)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    vg.cross_attention(qd, k, v, cu_d, starts, lens, scale, out, mask=mask, lse=ls, workspace=workspace,
                       error_flag=flag, stream=stream)
    torch.cuda.synchronize()
    assert int(flag.item()) == 0
    got = out.double().cpu().numpy()
    gl = ls.double().cpu().numpy() if lse else None
    for e, n in enumerate(new):
        r = slice(int(cu[e]), int(cu[e + 1]))
        s = slice(st.starts[e], st.starts[e] + st.lens[e])
        kk, vv = (torch.nan_to_num(x[s].double()).numpy() for x in (st.k, st.v))
        ro, rl, A, S = O.cross_attention(q[r].double().numpy(), kk, vv, st.attended[e], scale)
        count = int(st.attended[e].sum())
        vmax = float(np.abs(vv).max()) if vv.size else 0.0
        tol, tol_l = cross_bounds(ro, rl, A, S, count, d, dtype, vmax)
        assert np.isfinite(got[r]).all(), f"sequence {e}"
        bad = np.abs(got[r] - ro) > tol
        assert not bad.any(), (f"sequence {e}: {bad.sum()} of {bad.size} values, worst "
                               f"{np.max(np.abs(got[r] - ro) / tol):.2f} times the bound")
        if count == 0:
            assert (got[r] == 0).all()
        if lse:
            dead = np.isneginf(rl)
            assert np.isneginf(gl[r][dead]).all()
            assert (np.abs(gl[r][~dead] - rl[~dead]) <= tol_l[~dead]).all(), f"lse of sequence {e}"
    if rows_after:
        assert (got[int(cu[-1]):] == 7.0).all(), "rows past the last sequence were written"
        assert not lse or (gl[int(cu[-1]):] == 7.0).all()
    if strided:
        assert (buf[:, Hq:] == 7.0).all(), "written outside the output's heads"
    return qd, out, ls


def score_bound(spread, vocab, size, score):
    """How far a score may be from the exact one.  A slice's thread adds at most
    (96 KB / 4 B / 256 threads) words of two logits, 5 + 8 + 5 + 1 sums follow; an
    exponential is off by 2^-22 and by its argument's three roundings, 2^-24 of
    the distance from the maximum each, under the softmax `spread`; expf (2 ulp),
    its sum and the logarithm's parts 2^-22; the result is rounded once."""
    words = min(-(-vocab * size // 4), 24576)
    adds = 2 * -(-words // 256) + 19
    return 2.0 ** -24 * (adds + 4 + 3 * spread + 8 + abs(score)) + 1e-37


def run_select(logits, scores, num_out, ended=None, end_token=-1, with_ended=True, workspace=None, stream=None):
    """vg.beam_select on GPU tensors made of the given ones; host results."""
    from self_speculative_sparse_vg_gb300 import vg
    x = logits if logits.is_cuda else logits.cuda()
    s = torch.as_tensor(scores, dtype=torch.float32).cuda()
    B = s.shape[0]
    new = lambda t, v: torch.full((B, num_out), v, dtype=t, device="cuda")  # noqa: E731
    out = new(torch.float32, 5.0), new(torch.int32, -9), new(torch.int32, -9)
    marks = new(torch.uint8, 9) if with_ended else None
    e = None if ended is None else torch.as_tensor(ended).to(torch.bool).cuda()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    vg.beam_select(x, s, *out, ended=e, end_token=end_token, out_ended=marks, workspace=workspace, error_flag=flag,
                   stream=stream)
    torch.cuda.synchronize()
    got = [t.cpu().numpy() for t in out]
    return got[0].astype(np.float64), got[1], got[2], None if marks is None else marks.cpu().numpy(), int(flag.item())


def check_select(logits, scores, num_out, ended=None, end_token=-1, exactly=False, **kw):
    """Against the oracle.  Candidates of one beam compare as their logits do, so
    their order has to be the oracle's; candidates of different beams whose scores
    lie closer than the bounds may change places.  exactly: nothing may."""
    score, token, parent, marks, flag = run_select(logits, scores, num_out, ended, end_token, **kw)
    x = logits.double().cpu().numpy()
    scores = np.asarray(scores, dtype=np.float64)
    B, W = scores.shape
    size, V = logits.element_size(), x.shape[1]
    want_flag = 0
    for b in range(B):
        e = None if ended is None else np.asarray(ended)[b]
        cand, f, spread = O.beam_candidates(x[b * W:(b + 1) * W], scores[b], e, end_token)
        want_flag |= f
        n = min(num_out, len(cand))
        assert (token[b, n:] == -1).all() and (parent[b, n:] == -1).all() and np.isneginf(score[b, n:]).all(), b
        if marks is not None:
            assert (marks[b, n:] == 0).all(), b
        bound = lambda c: score_bound(spread[c[1]], V, size, c[0])  # noqa: E731
        near = any(cand[i][1] != cand[i + 1][1] and cand[i][0] - cand[i + 1][0] <= bound(cand[i]) + bound(cand[i + 1])
                   for i in range(min(n, len(cand) - 1)))
        if exactly or not near:
            got = list(zip(parent[b, :n].tolist(), token[b, :n].tolist()))
            assert got == [(c[1], c[2]) for c in cand[:n]], (b, got, cand[:n])
        where = {(c[1], c[2]): c for c in cand}
        seen = [(int(p), int(t)) for p, t in zip(parent[b, :n], token[b, :n])]
        assert len(set(seen)) == n
        for w in range(W):   # of one beam: the oracle's first ones, in its order
            mine = [t for p, t in seen if p == w]
            assert mine == [c[2] for c in cand if c[1] == w][:len(mine)], (b, w)
        for i, s in enumerate(seen):
            c = where[s]
            assert abs(score[b, i] - c[0]) <= bound(c), (b, i, score[b, i], c, bound(c))
            assert c[0] >= cand[n - 1][0] - bound(c) - bound(cand[n - 1])
            if marks is not None:
                assert marks[b, i] == int(c[3])
        assert (np.diff(score[b, :n]) <= 0).all()
    assert flag == want_flag
    return score, token, parent


def run_beam_tables(parents, lens, table, num_pages, owned, free, count, stream=None):
    """vg.beam_tables on copies of the given host arrays; host results."""
    from self_speculative_sparse_vg_gb300 import vg
    dev = dict(table=i32(table), lens=i32(lens), owned=i32(owned), free=i32(free), count=i32([count]))
    copies = torch.full((len(lens), 3), -9, dtype=torch.int32, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    par = i32(parents)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    vg.beam_tables(dev["table"], num_pages, par, dev["lens"], dev["owned"], dev["free"], dev["count"], copies,
                   error_flag=flag, stream=stream)
    torch.cuda.synchronize()
    got = {k: v.cpu().numpy() for k, v in dev.items()}
    got["count"], got["copies"], got["flag"] = int(got["count"][0]), copies.cpu().numpy(), int(flag.item())
    return got


def check_beam_tables(parents, lens, table, num_pages, owned, free, count):
    want = O.beam_tables(parents, lens, table, num_pages, owned, free, count)
    got = run_beam_tables(parents, lens, table, num_pages, owned, free, count)
    for k in want:
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)
    return got
