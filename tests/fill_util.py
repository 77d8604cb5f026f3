"""Shared pieces of the tests of the cache-filling calls."""
import numpy as np
import torch

from oracle import fill_oracle as F

PAGE = 16


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def run_tables(table, num_pages, cached, new, max_tokens, owned=None, free=None, count=None,
               stream=None):
    """vg.step_tables on copies of the given host arrays; host results."""
    from self_speculative_sparse_vg_gb300 import vg
    B = len(cached)
    dev = dict(table=i32(table), cached=i32(cached), new=i32(new))
    pool = {} if owned is None else dict(owned=i32(owned), free_pages=i32(free),
                                         free_count=i32([count]))
    cu = torch.full((B + 1,), -9, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    pos = torch.full((max_tokens,), -9, dtype=torch.int32, device="cuda")
    slots = torch.full((max_tokens,), -9, dtype=torch.int32, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    vg.step_tables(dev["table"], num_pages, dev["cached"], dev["new"], cu, lens, pos, slots,
                   error_flag=flag, stream=stream, **pool)
    torch.cuda.synchronize()
    got = dict(table=dev["table"], cu=cu, lens=lens, positions=pos, slots=slots)
    if pool:
        got.update(owned=pool["owned"], free=pool["free_pages"], count=pool["free_count"][0])
    got = {k: v.cpu().numpy() for k, v in got.items()}
    got["flag"] = int(flag.item())
    return got


def check_tables(table, num_pages, cached, new, max_tokens, owned=None, free=None, count=None):
    want = F.step_tables(table, num_pages, cached, new, max_tokens, owned, free, count)
    got = run_tables(table, num_pages, cached, new, max_tokens, owned, free, count)
    for k in got:
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)
    return got


class Cache:
    """A paged cache with random bf16 rows: sequence b holds lens[b] positions
    on shuffled pages; every slot that no sequence holds is filled with
    `junk` (NaN by default), so that a kernel that reads one shows it."""

    def __init__(self, lens, Hkv, d, seed=0, spare=3, extra_width=2, junk=float("nan")):
        g = torch.Generator().manual_seed(seed)
        counts = [(n + PAGE - 1) // PAGE for n in lens]
        pages = sum(counts) + spare
        order = torch.randperm(pages, generator=g).int()
        self.table = torch.full((len(lens), max(counts + [0]) + extra_width), -1, dtype=torch.int32)
        self.kp = torch.full((pages, Hkv, PAGE, d), junk, dtype=torch.bfloat16)
        self.vp = self.kp.clone()
        self.k, self.v, self.lens = [], [], list(lens)
        at = 0
        for b, n in enumerate(lens):
            ids = order[at:at + counts[b]]
            at += counts[b]
            self.table[b, :counts[b]] = ids
            k = torch.randn(n, Hkv, d, generator=g).bfloat16()
            v = torch.randn(n, Hkv, d, generator=g).bfloat16()
            self.k.append(k)
            self.v.append(v)
            self.write(b, k, v)
        self.gen = g

    def write(self, b, k, v):
        pos = torch.arange(k.shape[0])
        page, off = self.table[b, pos // PAGE].long(), pos % PAGE
        self.kp[page, :, off] = k
        self.vp[page, :, off] = v

    def gpu(self):
        from self_speculative_sparse_vg_gb300 import vg
        return vg.PagedKV(self.kp.cuda(), self.vp.cuda(), self.table.cuda())


def chunk_bounds(out, lse, A, S, attended, d):
    """Largest deviations arithmetic allows (bf16 half step 2^-8): the output
    is rounded once; each softmax weight may be rounded to bf16 once; logits
    are float32 sums of d products (a step of 2^-23 each, S bounds their
    magnitudes) and shift a weight by that much, relatively, above and below
    the line; `attended` float32 additions make the sums."""
    rel = 2.0 * (d + 8) * 2.0 ** -23 * (S + 1.0) + 2.0 * attended * 2.0 ** -23 + 2.0 ** -20
    tol = 2.0 ** -8 * (np.abs(out) + A) * 1.01 + rel[..., None] * A + 1e-30
    tol_lse = rel + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0.0))
    return tol, tol_lse


def check_chunk(cache, new, Hq, scale=None, seed=5, q=None, lse=True, strided=False, rows_after=0,
                workspace=None, kv=None, kv_lens=None):
    """vg.chunk_attention against the oracle for `new` tokens per sequence.
    Returns (q, out, lse) on the GPU."""
    from self_speculative_sparse_vg_gb300 import vg
    Hkv, d = cache.kp.shape[1], cache.kp.shape[3]
    lens = cache.lens if kv_lens is None else kv_lens
    scale = d ** -0.5 if scale is None else scale
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1]) + rows_after
    g = torch.Generator().manual_seed(seed)
    if q is None:
        q = torch.randn(T, Hq, d, generator=g).bfloat16()
    if strided:   # rows of a wider projection, outputs into a wider buffer
        wide = torch.randn(T, Hq + 3, d, generator=g).bfloat16()
        wide[:, 2:2 + Hq] = q
        qd = wide.cuda()[:, 2:2 + Hq]
        buf = torch.full((T, Hq + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[:, :Hq]
    else:
        qd = q.cuda()
        buf = out = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ls = torch.full((T, Hq), 7.0, dtype=torch.float32, device="cuda") if lse else None
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    vg.chunk_attention(cache.gpu() if kv is None else kv, qd, i32(cu), i32(lens), scale, out, lse=ls,
                       workspace=workspace, error_flag=flag)
    torch.cuda.synchronize()
    assert int(flag.item()) == 0
    got = out.double().cpu().numpy()
    gl = ls.double().cpu().numpy() if lse else None
    for b, n in enumerate(new):
        r = slice(int(cu[b]), int(cu[b + 1]))
        L = lens[b]
        ro, rl, A, S = F.chunk_attention(q[r].double().numpy(), cache.k[b][:L].double().numpy(),
                                         cache.v[b][:L].double().numpy(), n, scale)
        att = np.maximum(L - n + np.arange(n) + 1, 0)[:, None]
        tol, tol_l = chunk_bounds(ro, rl, A, S, att, d)
        assert np.isfinite(got[r]).all(), f"sequence {b}"
        bad = np.abs(got[r] - ro) > tol
        assert not bad.any(), (f"sequence {b}: {bad.sum()} of {bad.size} values, worst "
                               f"{np.max(np.abs(got[r] - ro) / tol):.2f} times the bound")
        if lse:
            dead = np.isneginf(rl)
            assert np.isneginf(gl[r][dead]).all()
            assert (np.abs(gl[r][~dead] - rl[~dead]) <= tol_l[~dead]).all(), f"lse of sequence {b}"
    if rows_after:
        assert (got[int(cu[-1]):] == 7.0).all(), "rows past the last sequence were written"
    if strided:
        assert (buf[:, Hq:] == 7.0).all(), "written outside the output's heads"
    return qd, out, ls
