"""Paged-cache operators in float64, plain loops over positions and keys.

Test infrastructure: the append of rotated keys and values to a paged cache,
and the attention of new positions over a shared prefix and their sequences'
pages.  Pools are float64 arrays [n_pages, page_size, n_heads, D].
"""
from __future__ import annotations

import numpy as np


def rotate(x, positions, inv_freq, axis=None, interleaved=False):
    """x [heads, D] of one new position; positions [n_axes]; pair f turns by
    positions[axis[f]] * inv_freq[f]."""
    y = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    for f in range(half):
        a, b = (2 * f, 2 * f + 1) if interleaved else (f, f + half)
        t = float(positions[axis[f] if axis is not None else 0]) * float(inv_freq[f])
        y[:, a] = x[:, a] * np.cos(t) - x[:, b] * np.sin(t)
        y[:, b] = x[:, a] * np.sin(t) + x[:, b] * np.cos(t)
    return y


def entry_of(q_len, kv_len, i):
    """The cache entry of a sequence's new position i."""
    return kv_len - q_len + i


def kv_append(k_pages, v_pages, q, k, v, q_indptr, block_table, kv_len, inv_freq, positions=None, axis=None,
              interleaved=False, position_base=0):
    """Returns q rotated and the pools after the append (copies)."""
    k_pages, v_pages = k_pages.copy(), v_pages.copy()
    q_out = np.array(q, dtype=np.float64)
    page_size = k_pages.shape[1]
    for b in range(len(kv_len)):
        first, end = int(q_indptr[b]), int(q_indptr[b + 1])
        for n in range(first, end):
            t = entry_of(end - first, int(kv_len[b]), n - first)
            pos = [position_base + t] if positions is None else positions[:, n]
            q_out[n] = rotate(q[n], pos, inv_freq, axis, interleaved)
            page = int(block_table[b, t // page_size])
            k_pages[page, t % page_size] = rotate(k[n], pos, inv_freq, axis, interleaved)
            v_pages[page, t % page_size] = v[n]
    return q_out, k_pages, v_pages


def sees(i, j, mask_word=None):
    """Whether new position i sees new entry j: a chain, or a 64-bit mask."""
    if mask_word is None:
        return j <= i
    return j < 64 and (int(mask_word) >> j) & 1 == 1


def prefix_attention(k_pages, v_pages, q, q_indptr, block_table, kv_len, prefix_table=None, prefix_len=0,
                     draft_mask=None, scale=None):
    """Returns out and lse, and per output the sum of weights times |v| and the
    largest scaled |q||k| sum of its row (for error bounds)."""
    N, Hq, D = q.shape
    page_size, Hk = k_pages.shape[1:3]
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.zeros((N, Hq, D)), np.full((N, Hq), -np.inf)
    absv, absqk, keys_seen = np.zeros((N, Hq, D)), np.zeros((N, Hq)), np.zeros(N, dtype=int)
    for b in range(len(kv_len)):
        first, end = int(q_indptr[b]), int(q_indptr[b + 1])
        q_len, kv = end - first, int(kv_len[b])
        where = [(int(prefix_table[t // page_size]), t % page_size) for t in range(prefix_len)]
        where += [(int(block_table[b, t // page_size]), t % page_size) for t in range(kv)]
        if not where:
            continue
        pages, slots = np.array(where).T
        K, V = k_pages[pages, slots], v_pages[pages, slots]  # [keys, Hk, D]
        for n in range(first, end):
            word = None if draft_mask is None else draft_mask[n]
            old = prefix_len + kv - q_len
            seen = np.array([t < old or sees(n - first, t - old, word) for t in range(prefix_len + kv)])
            keys_seen[n] = seen.sum()
            if not seen.any():
                continue
            for h in range(Hq):
                Kh, Vh = K[seen, h // (Hq // Hk)], V[seen, h // (Hq // Hk)]
                s = scale * (Kh @ q[n, h])
                w = np.exp(s - s.max())
                lse[n, h] = np.log(w.sum()) + s.max()
                w /= w.sum()
                out[n, h] = w @ Vh
                absv[n, h] = w @ np.abs(Vh)
                absqk[n, h] = scale * (np.abs(Kh) @ np.abs(q[n, h])).max()
    return out, lse, absv, absqk, keys_seen
