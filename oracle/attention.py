"""Cache append and attention in float64: the plain definitions, token by token.

Caches are numpy arrays [pages, kv_heads, page_size, head_dim]; a slot is
page * page_size + row.
"""

import numpy as np


def turn_heads(x, positions, inv_freq, pair_axis=None, interleaved=False, norm=None, eps=1e-6):
    """x [T, heads, D] float64 -> head norm (norm given) and rotation.
    positions [axes, T]; pair i turns by positions[pair_axis[i]][t] * inv_freq[i]."""
    x = np.array(x, np.float64)
    T, heads, D = x.shape
    for t in range(T):
        for h in range(heads):
            v = x[t, h]
            if norm is not None:
                v = v / np.sqrt(np.mean(v * v) + eps) * np.asarray(norm, np.float64)
            out = v.copy()
            n = len(inv_freq)
            for i in range(n):
                p = float(positions[0 if pair_axis is None else pair_axis[i]][t]) * float(inv_freq[i])
                ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
                out[ia] = v[ia] * np.cos(p) - v[ib] * np.sin(p)
                out[ib] = v[ib] * np.cos(p) + v[ia] * np.sin(p)
            x[t, h] = out
    return x


def append(cache, rows, slots):
    """Writes rows [T, kv_heads, D] to the cache rows `slots` (-1: not stored), in place."""
    page = cache.shape[2]
    for t, s in enumerate(slots):
        if 0 <= s < cache.shape[0] * page:
            cache[s // page, :, s % page] = rows[t]


def prefix_attention(k_cache, v_cache, q, prefix_pages, prefix_len, page_table, suffix_len, scale, row_seq=None):
    """out [T, q_heads, D], lse [T, q_heads] and, per output element, sum of weight * |v|
    over the softmax (what an error of the weights is relative to)."""
    T, hq, D = q.shape
    hk, page = k_cache.shape[1], k_cache.shape[2]
    out, lse, mag = np.zeros((T, hq, D)), np.full((T, hq), -np.inf), np.zeros((T, hq, D))
    for t in range(T):
        seq = t if row_seq is None else row_seq[t]
        at = [(prefix_pages[j // page], j % page) for j in range(prefix_len)]
        at += [(page_table[seq][j // page], j % page) for j in range(suffix_len[t])]
        if not at:
            continue
        pg, of = np.array([a[0] for a in at]), np.array([a[1] for a in at])
        for h in range(hq):
            kh = h // (hq // hk)
            k, v = k_cache[pg, kh, of], v_cache[pg, kh, of]
            s = scale * (k @ q[t, h])
            m = s.max()
            w = np.exp(s - m)
            out[t, h] = w @ v / w.sum()
            mag[t, h] = w @ np.abs(v) / w.sum()
            lse[t, h] = m + np.log(w.sum())
    return out, lse, mag
