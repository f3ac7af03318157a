"""Accumulated attention weight of cached keys and eviction by it (oracle; test infrastructure only).

Weighing: the last ``count`` tokens of a sequence of n cached keys are rows; row i of them sees
keys 0 .. n - count + i and gives each exp(scale q . k - lse).  A key's acc grows by what the rows of
its KV head's query heads give it; the rows' own keys start at zero, the others at
decay * acc.

Eviction: a KV head of more than ``budget`` keys keeps the budget best of them by (position
protected, acc, lower place), NaN last.  Kept keys below the budget keep their places; the free
places take the kept keys from behind it, both in ascending order.

Everything in float64, one key and head at a time.
"""

import numpy as np


def _line(k, b, h, n, table):
    """The first n keys of one sequence and head."""
    if table is None:
        return k[b, h, :n]
    rows = k.shape[2]
    return np.array([k[table[b, j // rows], h, j % rows] for j in range(n)]).reshape(n, k.shape[3])


def kv_weigh(q, lse, k, prefix_len, acc, pos, seen=None, n_rows=None, path=None, decay=1.0, scale=None, table=None):
    """q [B, Hq, T, D], lse [B, Hq, T], k [B, Hkv, Lmax, D] (or a pool with table), acc and pos [B, Hkv, Lmax];
    path: a list of node lists.  Returns (acc', pos', size), size [B, Hkv, Lmax] the sum of weights times (the sum of
    |q k| in them, scaled, plus |lse|), for the tolerance."""
    q, lse, k = (np.asarray(t, dtype=np.float64) for t in (q, lse, k))
    acc, pos = np.array(acc, dtype=np.float64), np.array(pos)
    size = np.zeros_like(acc)
    B, Hq, T, D = q.shape
    Hkv = acc.shape[1]
    scale = D ** -0.5 if scale is None else scale
    for b in range(B):
        n = int(prefix_len[b])
        rows = list(path[b]) if path is not None else list(range(T if n_rows is None else int(n_rows[b])))
        first = n - len(rows)
        for h in range(Hkv):
            K = _line(k, b, h, n, table)
            new = np.zeros(n)
            for hq in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                for i, node in enumerate(rows):
                    if not np.isfinite(lse[b, hq, node]):
                        continue
                    see = first + i + 1
                    w = np.exp(scale * (K[:see] @ q[b, hq, node]) - lse[b, hq, node])
                    new[:see] += w
                    size[b, h, :see] += w * (scale * (np.abs(K[:see]) @ np.abs(q[b, hq, node])) + abs(lse[b, hq, node]))
            old = np.zeros(n)
            if decay:
                old[:first] = decay * acc[b, h, :first]
            acc[b, h, :n] = old + new
            for j in range(first, n):
                pos[b, h, j] = (n if seen is None else int(seen[b])) - n + j
    return acc, pos, size


def kept_places(acc, pos, n, budget, sink, recent, seen):
    """For each place below min(n, budget), the place its key comes from (one head)."""
    if n <= budget:
        return list(range(n))
    safe = [pos[j] < sink or pos[j] >= seen - recent for j in range(n)]
    weight = [-np.inf if np.isnan(acc[j]) else acc[j] for j in range(n)]
    last = [bool(np.isnan(acc[j])) for j in range(n)]
    kept = sorted(sorted(range(n), key=lambda j: (not safe[j], last[j], -weight[j], j))[:budget])
    late = [j for j in kept if j >= budget]
    front = set(kept)
    return [j if j in front else late.pop(0) for j in range(budget)]


def kv_evict(k, v, acc, pos, prefix_len, budget, seen=None, sink=0, recent=0, table=None, out=None, out_table=None):
    """Returns (k', v', acc', pos', len') of the cache gone to: the same, or copies of out = (k, v, acc, pos) [B, Hkv, Lout, ..]
    (paged: (k, v) are pools and out = (acc, pos), with out_table)."""
    ko, vo, ao, po = (np.array(t) for t in ((k, v, acc, pos) if out is None else (k, v, *out) if table is not None else out))
    to = table if out is None else out_table
    for b in range(len(prefix_len)):
        n = int(prefix_len[b])
        for h in range(acc.shape[1]):
            places = kept_places(acc[b, h], pos[b, h], n, budget, sink, recent, n if seen is None else int(seen[b]))
            for p, j in enumerate(places):
                src, dst = (b, h, j), (b, h, p)
                if table is not None:
                    rows = k.shape[2]
                    src, dst = (table[b, j // rows], h, j % rows), (to[b, p // rows], h, p % rows)
                ko[dst], vo[dst] = k[src], v[src]
                ao[b, h, p], po[b, h, p] = acc[b, h, j], pos[b, h, j]
    return ko, vo, ao, po, np.minimum(prefix_len, budget)
