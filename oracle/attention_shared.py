"""Tree attention behind a shared prefix and with transformed scores (oracle; test infrastructure only).

Sequence b's keys in order: the shared ones (positions 0 ..), its own cached ones,
its tree's nodes (position shared + own + depth).  Node i sees every shared and
cached key and, of the tree, its ancestors and itself; with a window only keys less
than `window` positions back.  The score of a key `far` positions back is

    x = scale q.k;  x = softcap tanh(x / softcap);  x = x - slope[h] far

and the output softmax(x) . values.  Full rows, float64, nothing blocked or fused.
"""

import numpy as np

from .tree import tree_mask


def attention(q, k_cache, v_cache, prefix_len, k_tree, v_tree, tree, k_shared=None, v_shared=None, scale=None, softcap=0.0,
              window=0, slopes=None):
    """q [B, Hq, T, D], caches [B, Hkv, Lmax, D], tree K/V [B, Hkv, T, D], shared [Hkv, Ls, D] or None, all float64.

    Returns a dict: out [B, Hq, T, D], lse [B, Hq, T], and what error bounds need: weight
    (softmax(x) . |values|), size (the largest scale * sum |q_i k_i| of a row), keys (its longest row).
    """
    B, Hq, T, D = q.shape
    Hkv = k_cache.shape[1]
    g = Hq // Hkv
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    ancestors = tree_mask(tree) == 0
    depth = np.asarray(tree["depth"])
    Ls = 0 if k_shared is None else k_shared.shape[1]
    r = {"out": np.zeros((B, Hq, T, D)), "lse": np.zeros((B, Hq, T)), "weight": np.zeros((B, Hq, T, D)),
         "size": np.zeros((B, Hq, T)), "keys": 0}
    for b in range(B):
        n = Ls + int(prefix_len[b])
        far = (n + depth)[:, None] - np.concatenate([np.arange(n), n + depth])[None]
        seen = np.concatenate([np.ones((T, n), dtype=bool), ancestors], axis=1)
        if window:
            seen &= far < window
        r["keys"] = max(r["keys"], n + T)
        for h in range(Hq):
            kv = h // g
            own = int(prefix_len[b])
            K = np.concatenate(([k_shared[kv]] if Ls else []) + [k_cache[b, kv, :own], k_tree[b, kv]])
            V = np.concatenate(([v_shared[kv]] if Ls else []) + [v_cache[b, kv, :own], v_tree[b, kv]])
            x = scale * (q[b, h] @ K.T)
            r["size"][b, h] = (scale * (np.abs(q[b, h]) @ np.abs(K).T) * seen).max(axis=1)
            if softcap:
                x = softcap * np.tanh(x / softcap)
            if slopes is not None:
                x = x - float(slopes[h]) * far
            x = np.where(seen, x, -np.inf)
            m = x.max(axis=1, keepdims=True)
            e = np.exp(x - m)
            total = e.sum(axis=1, keepdims=True)
            r["out"][b, h] = (e / total) @ V
            r["weight"][b, h] = (e / total) @ np.abs(V)
            r["lse"][b, h] = (m + np.log(total))[:, 0]
    return r
