"""Float64 CPU oracle of the calls that fill the paged cache: block tables and
slot maps, rotary positions with the append, attention of a chunk.

TEST INFRASTRUCTURE ONLY.  Only the test-suite may import it; it shares no
code with the library.
"""
from __future__ import annotations

import math

import numpy as np

PAGE = 16
DEVERR_PAGE, DEVERR_INDEX, DEVERR_LENGTH, DEVERR_POOL = 1, 2, 16, 32


def step_tables(table, num_pages, cached, new, max_tokens, owned=None, free_pages=None,
                free_count=None):
    """One request after another, one page after another.  Returns a dict of
    the updated and written arrays and the error bits."""
    table = np.array(table, dtype=np.int64)
    B, width = table.shape
    fixed = owned is None
    flag = 0
    own = [0] * B if fixed else [int(x) for x in owned]
    free = None if fixed else [int(x) for x in free_pages]
    n = 0 if fixed else int(free_count)
    cu = [0]
    for x in new:
        cu.append(cu[-1] + max(int(x), 0))
    served, need = [True] * B, [0] * B
    for b in range(B):
        c, m = int(cached[b]), int(new[b])
        need[b] = -(-(c + m) // PAGE)
        if c < 0 or m < 0 or need[b] > width or cu[b + 1] > max_tokens or not 0 <= own[b] <= width:
            served[b] = False
            flag |= DEVERR_LENGTH
    if not fixed:
        for b in range(B):
            if served[b] and any(not 0 <= table[b, p] < num_pages for p in range(need[b], own[b])):
                served[b] = False
                flag |= DEVERR_PAGE
        returned = sum(max(own[b] - need[b], 0) for b in range(B) if served[b])
        if n < 0 or n + returned > len(free):
            for b in range(B):
                if served[b] and own[b] != need[b]:
                    served[b] = False
                    flag |= DEVERR_POOL
        else:
            for b in range(B):
                for p in range(need[b], own[b]) if served[b] else ():
                    free[n] = int(table[b, p])
                    table[b, p] = -1
                    n += 1
                if served[b] and own[b] > need[b]:
                    own[b] = need[b]
            asked, top = 0, n
            for b in range(B):
                if not served[b]:
                    continue
                more = max(need[b] - own[b], 0)
                asked += more
                if more and asked > top:
                    served[b] = False
                    flag |= DEVERR_POOL
                    continue
                for p in range(own[b], need[b]):
                    n -= 1
                    page = free[n]
                    if not 0 <= page < num_pages:
                        flag |= DEVERR_PAGE
                        page = -1
                    table[b, p] = page
                own[b] = need[b]
    positions, slots = np.zeros(max_tokens, np.int64), np.full(max_tokens, -1, np.int64)
    lens = [0] * B
    for b in range(B):
        if not served[b]:
            continue
        lens[b] = int(cached[b]) + int(new[b])
        for i in range(int(new[b])):
            pos = int(cached[b]) + i
            positions[cu[b] + i] = pos
            page = table[b, pos // PAGE]
            if 0 <= page < num_pages:
                slots[cu[b] + i] = page * PAGE + pos % PAGE
            else:
                flag |= DEVERR_PAGE
    return dict(table=table, owned=None if fixed else np.array(own),
                free=None if fixed else np.array(free), count=n,
                cu=np.array([min(x, max_tokens) for x in cu]), lens=np.array(lens),
                positions=positions, slots=slots, flag=flag)


def rope(x, positions, inv_freq, axes, interleaved):
    """x [T][H][d] float64, positions [A][T], inv_freq float64 [rot/2]: the
    rotation written as 2 x 2 products, pair by pair."""
    y = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    for t in range(x.shape[0]):
        for i in range(half):
            a = float(positions[axes[i]][t]) * float(inv_freq[i])
            u, w = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            m = np.array([[math.cos(a), -math.sin(a)], [math.sin(a), math.cos(a)]])
            y[t, :, [u, w]] = m @ np.stack([x[t, :, u], x[t, :, w]])
    return y


def chunk_attention(q, k, v, q_rows, scale):
    """One sequence.  q [n][Hq][d], k and v [len][Hkv][d] (logical order),
    q_rows = n: row i attends positions <= len - n + i.  Returns out, lse, and
    A = softmax . |v| and S = max_j scale sum |q||k_j| for error bounds."""
    n, Hq, d = q.shape
    L, Hkv, _ = k.shape
    g = Hq // Hkv
    out, lse = np.zeros((n, Hq, d)), np.full((n, Hq), -np.inf)
    A, S = np.zeros((n, Hq, d)), np.zeros((n, Hq))
    for i in range(n):
        m = L - q_rows + i + 1
        if m <= 0:
            continue
        for h in range(Hkv):
            qq = q[i, h * g:(h + 1) * g]
            s = scale * (qq @ k[:m, h].T)
            top = s.max(axis=1, keepdims=True)
            e = np.exp(s - top)
            z = e.sum(axis=1, keepdims=True)
            out[i, h * g:(h + 1) * g] = (e / z) @ v[:m, h]
            A[i, h * g:(h + 1) * g] = (e / z) @ np.abs(v[:m, h])
            lse[i, h * g:(h + 1) * g] = (top + np.log(z))[:, 0]
            S[i, h * g:(h + 1) * g] = scale * (np.abs(qq) @ np.abs(k[:m, h]).T).max(axis=1)
    return out, lse, A, S
