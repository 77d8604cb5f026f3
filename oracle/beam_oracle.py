"""Float64 CPU oracle of decoding with beams: cross attention, the selection
over beams and vocabulary, the beams' block tables, copies of pages.

TEST INFRASTRUCTURE ONLY.  Only the test-suite may import it; it shares no
code with the library.
"""
from __future__ import annotations

import numpy as np

PAGE = 16
DEVERR_PAGE, DEVERR_INDEX, DEVERR_LENGTH, DEVERR_POOL, DEVERR_VALUE = 1, 2, 16, 32, 64


def cross_attention(q, k, v, attended, scale):
    """One sequence.  q [n][Hq][d], k and v [S][Hkv][d], attended bool [S].
    Returns out, lse, and A = softmax . |v| and S = max_j scale sum |q||k_j| for
    error bounds."""
    n, Hq, d = q.shape
    Hkv = k.shape[1]
    g = Hq // Hkv
    out, lse = np.zeros((n, Hq, d)), np.full((n, Hq), -np.inf)
    A, S = np.zeros((n, Hq, d)), np.zeros((n, Hq))
    pick = np.flatnonzero(attended)
    if len(pick) == 0:
        return out, lse, A, S
    for h in range(Hq):
        kk, vv = k[pick, h // g], v[pick, h // g]
        s = scale * (q[:, h] @ kk.T)
        top = s.max(axis=1, keepdims=True)
        e = np.exp(s - top)
        z = e.sum(axis=1, keepdims=True)
        out[:, h], A[:, h] = (e / z) @ vv, (e / z) @ np.abs(vv)
        lse[:, h] = (top + np.log(z))[:, 0]
        S[:, h] = scale * (np.abs(q[:, h]) @ np.abs(kk).T).max(axis=1)
    return out, lse, A, S


def beam_candidates(logits, scores, ended, end_token):
    """One request: (score, beam, token, has ended) of every candidate in order,
    the error bits, and for each beam the mean distance of its logits from their
    maximum under the softmax (for error bounds)."""
    found, flag, spread = [], 0, []
    for w, s in enumerate(scores):
        spread.append(0.0)
        if np.isnan(s) or s == np.inf:
            flag |= DEVERR_VALUE
        elif s == -np.inf:
            continue
        elif ended is not None and ended[w]:
            found.append((s, w, end_token, True))
        else:
            x = logits[w]
            if np.isnan(x).any() or (x == np.inf).any():
                flag |= DEVERR_VALUE
                continue
            m = x.max()
            if m == -np.inf:
                continue
            e = np.exp(x - m)
            z = e.sum()
            with np.errstate(invalid="ignore"):
                spread[w] = float(np.where(e > 0, e * (m - x), 0.0).sum() / z)
            y = s + (x - m - np.log(z))
            for t in np.flatnonzero(y > -np.inf):
                found.append((y[t], w, int(t), t == end_token))
    found.sort(key=lambda c: (-c[0], c[1], c[2]))
    return found, flag, spread


def beam_tables(parents, lens, table, num_pages, owned, free_pages, free_count):
    """One request after another, one page after another.  Returns a dict of the
    updated and written arrays and the error bits."""
    parents = np.asarray(parents)
    B, W = parents.shape
    table = np.array(table, dtype=np.int64)
    lens, owned = [int(x) for x in lens], [int(x) for x in owned]
    free, n = [int(x) for x in free_pages], int(free_count)
    width = table.shape[1]
    flag = 0
    good = []
    for b in range(B):
        rows = range(b * W, (b + 1) * W)
        bad = 0
        if any(not -1 <= p < W for p in parents[b]):
            bad |= DEVERR_INDEX
        if any(lens[r] < 0 or not 0 <= owned[r] <= width or -(-lens[r] // PAGE) > owned[r] for r in rows):
            bad |= DEVERR_LENGTH
        flag |= bad
        good.append(not bad)
    back = []
    for b in range(B):
        if not good[b]:
            continue
        rows = range(b * W, (b + 1) * W)
        taken = {int(p) + b * W for p in parents[b] if p >= 0}
        for c in range(max(owned[r] for r in rows)):
            stays = {int(table[r, c]) for r in taken if c < -(-lens[r] // PAGE)}
            for r in rows:
                page = int(table[r, c])
                if c >= owned[r] or page in stays:
                    continue
                stays.add(page)
                if 0 <= page < num_pages:
                    back.append(page)
                else:
                    flag |= DEVERR_PAGE
    copies = np.tile(np.array([-1, -1, 0]), (B * W, 1))
    same = dict(table=table, lens=np.array(lens), owned=np.array(owned), free=np.array(free), count=n, copies=copies)
    if not 0 <= n <= len(free) or n + len(back) > len(free):
        return dict(same, flag=flag | DEVERR_POOL)
    for page in back:
        free[n] = page
        n += 1
    new, new_lens, new_owned = table.copy(), list(lens), list(owned)
    for b in range(B):
        if not good[b]:
            continue
        own_tails = set()
        for j in range(W):
            r, p = b * W + j, int(parents[b, j])
            length = lens[b * W + p] if p >= 0 else 0
            cols = -(-length // PAGE)
            row = [int(x) for x in table[b * W + p, :cols]] if p >= 0 else []
            rest = length % PAGE
            if rest and row[-1] >= 0:
                if (cols, row[-1]) not in own_tails:
                    own_tails.add((cols, row[-1]))
                elif n == 0:
                    flag |= DEVERR_POOL
                    length, cols, row = 0, 0, []
                else:
                    n -= 1
                    page = free[n]
                    if 0 <= page < num_pages:
                        copies[r] = (row[-1], page, rest)
                    else:
                        flag |= DEVERR_PAGE
                        page = -1
                    row[-1] = page
            new[r, :cols] = row
            new[r, cols:max(cols, owned[r])] = -1
            new_lens[r], new_owned[r] = length, cols
    return dict(table=new, lens=np.array(new_lens), owned=np.array(new_owned), free=np.array(free), count=n,
                copies=copies, flag=flag)


def copy_pages(pool, copies):
    """pool [pages][heads][16][d], one pool."""
    out = pool.copy()
    for src, dst, n in copies:
        if n:
            out[dst, :, :n] = pool[src, :, :n]
    return out
