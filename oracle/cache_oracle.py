"""Plain CPU oracle for the calls around the decode step: chunk append, chunk attention, window
decode with accumulated weights, eviction.

TEST INFRASTRUCTURE, NOT PART OF THE PRODUCT.  numpy float64 on exact copies of the inputs, one
function per call, by the definitions in include/sas.h; it shares no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np

PAGE = 64


def slot(page_table, b, pos):
    """Cache coordinates (first axis, third axis) of positions `pos` of sequence b."""
    pos = np.asarray(pos, np.int64)
    if page_table is None:
        return np.full_like(pos, b), pos
    return np.asarray(page_table[b], np.int64)[pos // PAGE], pos % PAGE


def visible(p, n, window, sinks):
    """Boolean mask over 0..n-1 of what the token at position p sees."""
    j = np.arange(n)
    m = j <= p
    if window > 0:
        m &= (j > p - window) | (j < sinks)
    return m


def chunk_errors(q_start, seqlens, n_new, cap):
    """Why each sequence of a chunk batch is skipped: 0 (taken), 1 (its length), 6 (its rows)."""
    why, top = [], None
    for b, n in enumerate(seqlens):
        s0, s1 = int(q_start[b]), int(q_start[b + 1])
        top = s0 if top is None else max(top, s0)
        if not 0 <= n <= cap:
            why.append(1)
        else:
            why.append(0 if 0 <= s0 and top == s0 <= s1 <= n_new and s1 - s0 <= n else 6)
    return why


def append_chunk(K, V, K_new, V_new, q_start, seqlens, page_table):
    """K, V updated copies: rows N_b - T_b .. N_b - 1 of every (b, h) from the chunk."""
    K, V = K.copy(), V.copy()
    for b in range(len(seqlens)):
        s0, s1, n = int(q_start[b]), int(q_start[b + 1]), int(seqlens[b])
        i1, i3 = slot(page_table, b, np.arange(n - (s1 - s0), n))
        for h in range(K.shape[1]):
            K[i1, h, i3] = K_new[s0:s1, h]
            V[i1, h, i3] = V_new[s0:s1, h]
    return K, V


def attend_row(q, k, v, sigma):
    """q [G][d] over rows k, v [n][d]: out [G][d], lse [G], weights [G][n]; n = 0 gives zeros, -inf."""
    if k.shape[0] == 0:
        return np.zeros_like(q), np.full(q.shape[0], -np.inf), np.zeros((q.shape[0], 0))
    z = sigma * (q @ k.T)
    top = z.max(axis=1, keepdims=True)
    e = np.exp(z - top)
    s = e.sum(axis=1, keepdims=True)
    w = e / s
    return w @ v, (top + np.log(s))[:, 0], w


def evict_positions(weights, n, keep, sinks, recent):
    """Kept positions of one (b, h), ascending: sinks, then the newest, then the largest weights."""
    keep = max(0, min(int(keep), n))
    forced = list(range(min(sinks, n)))
    forced += [j for j in range(n - 1, n - 1 - min(recent, n), -1) if j >= sinks]
    seen = set(forced)
    w = np.where(np.isnan(weights[:n]), -np.inf, weights[:n].astype(np.float64))
    # NaN sorts below -inf: a second key
    rest = [j for j in np.lexsort((np.arange(n), -w, np.isnan(weights[:n]))) if j not in seen]
    return np.sort(np.array((forced + rest)[:keep], dtype=np.int64))
