"""Selection of a beam search and the reordering that follows it (oracle; test infrastructure only).

A live beam w offers every token t at  scores[w] + log_softmax(x[w])[t]  with one more token of
length; an ended one offers itself (token eos, score and length unchanged); one whose score
is not finite, or none of whose logits is (or one of whose is +inf), offers nothing.  NaN logits count as -inf and -inf
is never chosen.  The K best by score / max(length, 1)^alpha are taken, equal ones by the lower
beam, then the lower token.

Everything in float64 and sorted whole.
"""

import numpy as np


def beam_select(logits, scores, K, eos=-1, ended=None, length=None, alpha=0.0):
    """logits [B, W, V], scores [B, W] -> dict of token, parent, score, ended, length, rank, each [B, K] (-1, -1, -inf, 1, 0 and
    -inf where there is no pair)."""
    x = np.array(logits, dtype=np.float64)
    x[np.isnan(x)] = -np.inf
    B, W, _ = x.shape
    out = {"token": np.full((B, K), -1), "parent": np.full((B, K), -1), "score": np.full((B, K), -np.inf),
           "ended": np.ones((B, K), dtype=int), "length": np.zeros((B, K), dtype=int), "rank": np.full((B, K), -np.inf)}
    for b in range(B):
        pairs = []      # (-rank, beam, token, score, ended, length)
        for w in range(W):
            base = float(scores[b, w])
            n = 0 if length is None else int(length[b, w])
            if not np.isfinite(base):
                continue
            if ended is not None and ended[b, w]:
                pairs.append((-base / max(n, 1) ** alpha, w, eos, base, 1, n))
                continue
            top = x[b, w].max()
            if not np.isfinite(top):
                continue
            score = base + (x[b, w] - (top + np.log(np.exp(x[b, w] - top).sum())))
            for t in np.lexsort((np.arange(len(score)), -score))[:K]:
                if score[t] > -np.inf:
                    pairs.append((-score[t] / max(n + 1, 1) ** alpha, w, int(t), score[t], int(t == eos), n + 1))
        for r, e in enumerate(sorted(pairs)[:K]):
            out["rank"][b, r] = -e[0]
            for name, v in zip(("parent", "token", "score", "ended", "length"), e[1:]):
                out[name][b, r] = v
    return out


def reorder(state, parent):
    """state [B, W, ...]: row w becomes what row parent[b, w] was; parents outside 0 .. W - 1 leave their row."""
    out = np.array(state)
    for b in range(parent.shape[0]):
        for w, p in enumerate(parent[b]):
            if 0 <= p < parent.shape[1]:
                out[b, w] = state[b, p]
    return out


def kv_reorder(cache, parent, start, end, table=None):
    """Positions start[b] .. end[b] - 1 of cache [B * W, Hkv, Lmax, D], or of a pool [blocks, Hkv, bs, D] with table [B * W, max_blocks]."""
    out = np.array(cache)
    B, W = parent.shape
    rows = cache.shape[2]
    cap = rows if table is None else table.shape[1] * rows
    for b in range(B):
        if not 0 <= start[b] <= end[b] <= cap:
            continue
        for w in range(W):
            p = int(parent[b, w])
            if not 0 <= p < W:
                continue
            for j in range(int(start[b]), int(end[b])):
                to, src = b * W + w, b * W + p
                if table is not None:
                    to, src = int(table[to, j // rows]), int(table[src, j // rows])
                    if not (0 <= to < len(cache) and 0 <= src < len(cache)):
                        continue
                out[to, :, j % rows] = cache[src, :, j % rows]
    return out
