"""Rotary positions of appended tokens and tree nodes (oracle; test infrastructure only).

A token at position pos turns the pair number j of the leading ``rot`` elements of
every query and key head by the angle pos * freq[j]; the pairs are elements
(j, j + rot / 2), or (2j, 2j + 1) when interleaved.  Values are not turned.  New
token i of sequence b is at position base + prefix_len[b] + i and lands in cache
row prefix_len[b] + i; tree node i at base + prefix_len[b] + depth[i], the place
it has on its own path.

Everything in float64 and unrounded: callers compare with their own rounding.
"""

import numpy as np


def rotate(x, pos, freq, interleaved):
    """x [..., D] float64 turned as position pos (a number)."""
    x = np.array(x, dtype=np.float64)
    freq = np.asarray(freq, dtype=np.float64)
    half = len(freq)
    first = np.arange(half) * 2 if interleaved else np.arange(half)
    second = first + 1 if interleaved else first + half
    phi = float(pos) * freq
    a, b = x[..., first].copy(), x[..., second].copy()
    x[..., first] = a * np.cos(phi) - b * np.sin(phi)
    x[..., second] = a * np.sin(phi) + b * np.cos(phi)
    return x


def kv_append(q, k, v, seq_start, prefix_len, k_cache, v_cache, freq, interleaved=False, base=0, table=None):
    """Return (q', k_cache', v_cache', written [rows of q]) in float64.

    q [N, Hq, D], k, v [N, Hkv, D]; caches [B, Hkv, Lmax, D], or pools
    [num_blocks, Hkv, block_size, D] with table [B, max_blocks].  A sequence whose
    tokens do not fit, whose prefix_len is negative or whose offsets leave 0 .. N, and a
    token whose block lies outside the pool are left out; rows of no sequence are not
    written.
    """
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    out = q.copy()
    kc, vc = np.array(k_cache, dtype=np.float64), np.array(v_cache, dtype=np.float64)
    rows = kc.shape[2]
    cap = rows if table is None else table.shape[1] * rows
    written = np.zeros(len(q), dtype=bool)
    for b in range(len(prefix_len)):
        L, s0, s1 = int(prefix_len[b]), int(seq_start[b]), int(seq_start[b + 1])
        if L < 0 or L + s1 - s0 > cap or s0 < 0 or s1 > len(q):
            continue
        for n in range(s0, s1):
            at = L + n - s0
            blk = b if table is None else int(table[b, at // rows])
            if table is not None and not 0 <= blk < len(kc):
                continue
            kc[blk, :, at % rows] = rotate(k[n], base + at, freq, interleaved)
            vc[blk, :, at % rows] = v[n]
            out[n] = rotate(q[n], base + at, freq, interleaved)
            written[n] = True
    return out, kc, vc, written


def tree_rope(q, k, v, prefix_len, depth, freq, interleaved=False, base=0):
    """q [B, T, Hq, D], k, v [B, T, Hkv, D] -> q [B, Hq, T, D], k_tree, v_tree [B, Hkv, T, D], float64."""
    q, k, v = (np.moveaxis(np.array(t, dtype=np.float64), 1, 2).copy() for t in (q, k, v))
    for b in range(q.shape[0]):
        for i in range(q.shape[2]):
            pos = base + int(prefix_len[b]) + int(depth[i])
            q[b, :, i] = rotate(q[b, :, i], pos, freq, interleaved)
            k[b, :, i] = rotate(k[b, :, i], pos, freq, interleaved)
    return q, k, v
