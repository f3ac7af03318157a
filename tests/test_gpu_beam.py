"""Selection of a beam search and reordering of beams: CUDA path vs the oracle (GPU).

Tokens, parents, ended flags and lengths are exact: where the ranks of pairs of different beams are nearer than the kernel's
error, the case says so by its margin, which is checked on the oracle's side first.  The error of a score is that
of the row's log-sum plus one rounding of the output: exponentials within 2^-22, the argument's rounding below
2^-24 |a| e^-|a| each (below 2^-25), sums of at most V / 1024 + 16 terms in a row, 2^-24 each; so
(4 + 0.5 + V / 1024 + 16) 2^-24 + 2^-24 |score|.  Reorders are copies and exact.
"""

import numpy as np
import pytest

from gpu_util import lib
from oracle import beam

pytestmark = pytest.mark.gpu


def _dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a))
    return t.to(dtype).cuda() if dtype is not None else t.cuda()


def _f(dtype):
    import torch
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _check(st, x, scores, K, ties=False, ws=None, **kw):
    """x a CUDA tensor [B, W, V]; the oracle gets the values it holds."""
    dev = {k: (_dev(v.astype(np.int32)) if k in ("ended", "length") and v is not None else v) for k, v in kw.items()}
    got = st.beam_select(x, _dev(scores.astype(np.float32)), K, ws=ws, **dev)
    want = beam.beam_select(x.double().cpu().numpy(), scores.astype(np.float32), K + 1, **kw)
    tol = (20.5 + x.shape[2] / 1024) * 2.0 ** -24
    token, parent, score, ended, length = (t.cpu().numpy() for t in got)
    rank = want["rank"]
    with np.errstate(invalid="ignore"):
        gap = np.where(np.isfinite(rank[:, 1:]), rank[:, :-1] - rank[:, 1:], np.inf)
    near = gap < 8 * tol + 1e-12 * np.abs(np.where(np.isfinite(rank[:, 1:]), rank[:, 1:], 0))
    same = want["parent"][:, :-1] == want["parent"][:, 1:]
    assert ties or not (near & ~same).any(), "the case's ranks are too near to each other to be told apart"
    np.testing.assert_array_equal(parent, want["parent"][:, :K])
    np.testing.assert_array_equal(token, want["token"][:, :K])
    np.testing.assert_array_equal(ended, want["ended"][:, :K])
    np.testing.assert_array_equal(length, want["length"][:, :K])
    ref = want["score"][:, :K]
    some = np.isfinite(ref)
    np.testing.assert_array_equal(score[~some], ref[~some])
    assert (np.abs(score - ref)[some] <= tol + 2.0 ** -24 * np.abs(ref[some])).all()
    return got


SELECTS = [
    # dtype, B, W, K, V, padding of the rows, alpha, share of ended beams
    ("f32", 1, 8, 8, 32000, 0, 0.0, 0.0),
    ("bf16", 3, 4, 4, 32000, 0, 0.0, 0.3),
    ("bf16", 4, 5, 7, 50257, 47, 0.6, 0.3),
    ("bf16", 2, 3, 5, 1001, 0, 1.0, 0.0),        # rows that start anywhere
    ("f32", 2, 7, 3, 4099, 2, 0.0, 0.2),
    ("bf16", 1, 1, 64, 131073, 0, 0.0, 0.0),     # one beam, many out
    ("f32", 2, 64, 64, 777, 0, 0.7, 0.1),        # the most beams
    ("bf16", 70, 2, 2, 300, 0, 0.0, 0.0),
    ("f32", 1, 1, 1, 2, 0, 0.0, 0.0),            # the smallest
    ("bf16", 1, 2, 64, 20, 3, 0.0, 0.0),         # fewer pairs than asked for
    ("bf16", 200, 8, 8, 2500, 0, 0.0, 0.0),      # one slice a row
]


@pytest.mark.parametrize("c", SELECTS, ids=lambda c: "-".join(map(str, c)))
def test_selections(c):
    import torch
    dtype, B, W, K, V, pad, alpha, share = c
    st = lib()
    rng = np.random.default_rng(B * 1000 + V)
    x = _dev((2.5 * rng.standard_normal((B, W, V + pad))).astype(np.float32), _f(dtype))[..., :V]
    scores = -rng.random((B, W)) * 5 - 3
    ended = (rng.random((B, W)) < share).astype(int)
    _check(st, x, scores, K, eos=min(1, V - 1), ended=ended, length=np.where(ended, rng.integers(0, 9, (B, W)), 9), alpha=alpha)
    ws = torch.empty(st.beam_select_workspace_size(B, W, V, K), dtype=torch.uint8, device="cuda").fill_(255)
    _check(st, x, scores, K, ws=ws)
    assert st.spec_read_device_status(ws) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "steps", "one", "last"])
@pytest.mark.parametrize("K", [1, 8, 64])
def test_logits_that_many_threads_find_good(dtype, kind, K):
    """More candidates than a slice's list holds, and orders that raise the threshold with every element."""
    import torch
    V = 70001
    t = torch.arange(V, device="cuda")
    x = {"equal": torch.zeros(V, device="cuda"), "rising": t / 1024.0, "falling": -t / 1024.0, "steps": (t // 9000) * 0.5,
         "one": (t == 33333).float(), "last": (t >= V - 3).float()}[kind]
    x = torch.stack([x, x - 0.25, x.flip(0)]).to(_f(dtype))[None].contiguous()
    _check(lib(), x, np.array([[-1.0, -1.8125, -2.4375]]), K, ties=True)


def test_equal_ranks_in_all_beams():
    """More equal pairs than the join's list holds: taken one after the other."""
    import torch
    x = torch.zeros(2, 64, 4096, device="cuda")
    token, parent, score, _, _ = lib().beam_select(x, torch.full((2, 64), -1.0, device="cuda"), 64)
    assert token.tolist() == [list(range(64))] * 2 and not parent.any()
    x = torch.full((1, 64, 4096), -float("inf"), device="cuda")
    x[0, :, 7] = 1.0
    token, parent, score, _, _ = lib().beam_select(x, torch.full((1, 64), -1.0, device="cuda"), 64)
    assert (token == 7).all() and parent.tolist() == [list(range(64))] and (score == -1.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dead_ended_and_masked_beams(dtype):
    import torch
    st = lib()
    rng = np.random.default_rng(4)
    B, W, V, K = 4, 6, 5000, 6
    x = _dev(rng.standard_normal((B, W, V)).astype(np.float32), _f(dtype))
    scores = -rng.random((B, W)) - 1
    scores[0, 1:] = -np.inf                          # a first step: one beam
    scores[1, 2], scores[1, 3] = np.nan, np.inf
    x[1, 0] = -float("inf")                          # nothing to choose
    x[1, 1, 3:] = float("nan")                       # three tokens left
    x[2, :, 1::2] = -float("inf")                    # a masked vocabulary
    x[2, 3, 2::4] = float("nan")
    x[3, :, 9] = 60.0                                # almost certain
    x[1, 4:], scores[1, 4:] = float("nan"), -1.0
    ended = np.zeros((B, W), dtype=int)
    ended[2, 1] = ended[3, 5] = 1
    _check(st, x, scores, K, eos=9, ended=ended, length=np.full((B, W), 3), alpha=0.5)
    x[0, 0, 17] = float("inf")
    ws = torch.empty(st.beam_select_workspace_size(B, W, V, K), dtype=torch.uint8, device="cuda")
    got = _check(st, x, scores, K, ws=ws)
    assert st.spec_read_device_status(ws) == 1 and (got[0][0] == -1).all()
    x[0, 0, 17] = 0.0
    _check(st, x, scores, K, ws=ws)
    assert st.spec_read_device_status(ws) == 0


def test_outputs_over_their_inputs_and_a_captured_search():
    """Ten steps, state in place, captured once: the beams' tokens equal the oracle's step by step."""
    import torch
    st = lib()
    rng = np.random.default_rng(5)
    B, W, V, n = 3, 4, 700, 10
    table = _dev((2 * rng.standard_normal((V, V))).astype(np.float32))     # logits by the last token
    scores = torch.full((B, W), -float("inf"), device="cuda")
    scores[:, 0] = 0.0
    ended, length = torch.zeros(B, W, dtype=torch.int32, device="cuda"), torch.zeros(B, W, dtype=torch.int32, device="cuda")
    history = torch.full((B, W, n + 1), -1, dtype=torch.int32, device="cuda")
    history[:, :, 0] = _dev(rng.integers(0, V, (B, 1)).astype(np.int32))
    token, parent, x = history[:, :, 0].clone(), torch.zeros(B, W, dtype=torch.int32, device="cuda"), torch.empty(B, W, V, device="cuda")
    ws, ws2 = torch.empty(st.beam_select_workspace_size(B, W, V, W), dtype=torch.uint8, device="cuda"), torch.empty(256, dtype=torch.uint8, device="cuda")
    at = torch.zeros(1, dtype=torch.long, device="cuda")

    def step():
        torch.index_select(table, 0, token.clamp(min=0).view(-1), out=x.view(B * W, V))
        st.beam_select(x, scores, W, eos=3, ended=ended, length=length, alpha=0.6, token=token, parent=parent, score=scores, ended_out=ended,
                       length_out=length, ws=ws)
        st.beam_reorder(history, parent, ws=ws2)
        at.add_(1)
        history.index_copy_(2, at, token.unsqueeze(2))
    start = [t.clone() for t in (scores, ended, length, history, token, parent, at)]
    step()
    for t, s in zip((scores, ended, length, history, token, parent, at), start):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    sc, en, le, hi = (t.cpu().numpy().astype(np.float64 if i == 0 else np.int64) for i, t in enumerate((scores, ended, length, history)))
    tab = table.double().cpu().numpy()
    for i in range(1, n + 1):
        graph.replay()
        r = beam.beam_select(tab[np.maximum(hi[:, :, i - 1], 0)], sc, W, eos=3, ended=en, length=le, alpha=0.6)
        hi = beam.reorder(hi, r["parent"])
        hi[:, :, i] = r["token"]
        sc, en, le = r["score"].astype(np.float32).astype(np.float64), r["ended"], r["length"]
        np.testing.assert_array_equal(history.cpu().numpy(), hi)
        np.testing.assert_array_equal(length.cpu().numpy(), le)
        # each step's error joins the one before it
        assert np.abs(scores.cpu().numpy() - sc).max() <= i * (21.5 * 2.0 ** -24 + 2.0 ** -24 * np.abs(sc).max())
    assert st.spec_read_device_status(ws) == st.spec_read_device_status(ws2) == 0


@pytest.mark.parametrize("row,dtype", [(1, "int32"), (2, "int32"), (3, "int32"), (4, "float32"), (1000, "bfloat16"), (4098, "bfloat16"), (6, "int64")])
@pytest.mark.parametrize("W", [1, 2, 4, 7, 8, 13, 16, 17, 32, 33, 64])
def test_states(W, row, dtype):
    import torch
    st = lib()
    rng = np.random.default_rng(W * 100 + row)
    B = 3
    x = torch.arange(B * W * row, device="cuda").view(B, W, row).to(getattr(torch, dtype))
    parent = rng.integers(0, W, (B, W)).astype(np.int32)
    parent[0] = np.roll(np.arange(W), 1)             # one cycle
    parent[1, rng.random(W) < 0.3] = -1
    want = beam.reorder(x.view(torch.int16 if dtype == "bfloat16" else x.dtype).cpu().numpy(), parent)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda").fill_(255)
    assert st.beam_reorder(x, _dev(parent), ws=ws) is x
    np.testing.assert_array_equal(x.view(torch.int16 if dtype == "bfloat16" else x.dtype).cpu().numpy(), want)
    assert st.spec_read_device_status(ws) == 0


def test_parents_that_do_not_exist():
    import torch
    st = lib()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    x = torch.arange(12, device="cuda", dtype=torch.float32).view(1, 3, 4).contiguous()
    st.beam_reorder(x, _dev(np.array([[1, 3, -2]], dtype=np.int32)), ws=ws)
    assert st.spec_read_device_status(ws) == 1 and x[0, :, 0].tolist() == [4.0, 4.0, 8.0]


CACHES = [
    # dtype, B, W, Hkv, D, block (0: contiguous), start, end
    ("bf16", 2, 4, 2, 128, 0, (3, 0), (40, 1)),
    ("bf16", 3, 8, 3, 64, 16, (0, 17, 30), (50, 17, 33)),       # one with nothing to move
    ("f32", 1, 13, 1, 20, 7, (5,), (40,)),
    ("f32", 2, 20, 2, 8, 0, (0, 2), (11, 9)),
    ("bf16", 1, 64, 2, 8, 5, (4,), (21,)),
    ("bf16", 2, 2, 8, 128, 64, (100, 63), (700, 65)),
]


@pytest.mark.parametrize("c", CACHES, ids=lambda c: "-".join(map(str, c[:6])))
def test_caches(c):
    import torch
    st = lib()
    dtype, B, W, H, D, block, start, end = c
    rng = np.random.default_rng(B * W * D)
    parent = rng.integers(0, W, (B, W)).astype(np.int32)
    parent[0] = rng.permutation(W)
    n = max(end) + 3
    rows = B * W
    table = None
    shape = (rows, H, n, D)
    if block:
        width = -(-n // block)
        table = rng.permutation(rows * width + 2)[:rows * width].reshape(rows, width).astype(np.int32)
        shape = (rows * width + 2, H, block, D)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda").fill_(255)
    k, v = (torch.randn(shape, device="cuda").to(_f(dtype)) for _ in range(2))
    want = [beam.kv_reorder(t.float().cpu().numpy(), parent, start, end, table) for t in (k, v)]
    args = _dev(parent), _dev(np.array(start, dtype=np.int32)), _dev(np.array(end, dtype=np.int32))
    if block:
        st.kv_reorder_paged(k, v, _dev(table), *args, ws=ws)
    else:
        st.kv_reorder(k, v, *args, ws=ws)
    assert st.spec_read_device_status(ws) == 0
    for t, w in zip((k, v), want):
        np.testing.assert_array_equal(t.float().cpu().numpy(), w)


def test_ranges_and_blocks_that_do_not_exist():
    import torch
    st = lib()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    parent = np.array([[1, 0]] * 4, dtype=np.int32)
    k, v = torch.randn(8, 1, 6, 8, device="cuda"), torch.randn(8, 1, 6, 8, device="cuda")
    start, end = np.array([-1, 4, 0, 2], dtype=np.int32), np.array([3, 3, 7, 6], dtype=np.int32)
    want = [beam.kv_reorder(t.cpu().numpy(), parent, start, end) for t in (k, v)]
    st.kv_reorder(k, v, _dev(parent), _dev(start), _dev(end), ws=ws)
    assert st.spec_read_device_status(ws) == 1
    np.testing.assert_array_equal(k.cpu().numpy(), want[0])
    np.testing.assert_array_equal(v.cpu().numpy(), want[1])
    np.testing.assert_array_equal(want[0][:6], k[:6].cpu().numpy())
    table = np.array([[0, 1], [2, 8], [3, -1], [4, 5], [6, 7], [6, 7], [0, 1], [0, 1]], dtype=np.int32)
    start, end = np.array([0, 1, 2, 3], dtype=np.int32), np.array([12, 11, 2, 3], dtype=np.int32)
    want = [beam.kv_reorder(t.cpu().numpy(), parent, start, end, table) for t in (k, v)]
    st.kv_reorder_paged(k, v, _dev(table), _dev(parent), _dev(start), _dev(end), ws=ws)
    assert st.spec_read_device_status(ws) == 1
    np.testing.assert_array_equal(k.cpu().numpy(), want[0])
    np.testing.assert_array_equal(v.cpu().numpy(), want[1])


def test_beams_as_a_tree_of_candidates():
    """A search of four steps, each beam with a cache of its own that kv_reorder and kv_append carry along; its pairs as one candidate tree.
    Tree attention's rows of the last level are the attention of the beams over their caches."""
    import torch
    st = lib()
    g = torch.Generator().manual_seed(11)
    rand = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    W, V, Hq, Hkv, D, n0, steps = 3, 50, 4, 2, 64, 20, 4
    table, ek, ev, eq = 2 * rand(V, V), rand(V, Hkv, D), rand(V, Hkv, D), rand(V, Hq, D)
    kc, vc = rand(1, Hkv, n0 + steps + 1, D).repeat(W, 1, 1, 1), rand(1, Hkv, n0 + steps + 1, D).repeat(W, 1, 1, 1)
    prefix = kc[:1, :, :n0].clone(), vc[:1, :, :n0].clone()
    token = torch.tensor([[7] * W], dtype=torch.int32, device="cuda")
    scores = torch.tensor([[0.0] + [-float("inf")] * (W - 1)], device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    parent, node, nodes = [-1], [0] * W, [7]           # the tree so far, each beam's node in it, the nodes' tokens
    for s in range(steps + 1):
        t = token[0].clamp(min=0).long()
        st.kv_append(None, ek[t], ev[t], i32(list(range(W + 1))), i32([n0 + s] * W), kc, vc)
        if s == steps:
            break
        token, p, scores, _, _ = st.beam_select(table[t][None].contiguous(), scores, W)
        st.kv_reorder(kc, vc, p, i32([n0]), i32([n0 + s + 1]))
        parent += [node[w] for w in p[0].tolist()]
        nodes += token[0].tolist()
        node = list(range(len(parent) - W, len(parent)))
    tree = st.spec_tree_build(parent)
    at = torch.tensor(nodes, device="cuda")
    heads = lambda e: e[at].transpose(0, 1)[None].contiguous()  # noqa: E731
    out, lse = st.tree_attention(heads(eq), prefix[0].contiguous(), prefix[1].contiguous(), i32([n0]), heads(ek), heads(ev), tree)
    for w in range(W):
        for h in range(Hq):
            x = kc[w, h // 2].double() @ eq[at[node[w]], h].double() / 8.0
            ref = torch.softmax(x, 0) @ vc[w, h // 2].double()
            assert (out[0, h, node[w]] - ref).abs().max() < 1e-5
            assert abs(lse[0, h, node[w]] - torch.logsumexp(x, 0)) < 1e-5


@pytest.mark.parametrize("alpha", [0.0, 2.0])
def test_scores_and_logits_near_the_largest_numbers(alpha):
    """A score less its row's logits may pass 32 bits on the way: the pair is there all the same."""
    import torch
    x = torch.full((1, 3, 900), -3e38, device="cuda")
    x[0, 0, 5], x[0, 1, 600], x[0, 2, 7] = 3e38, 3.2e38, 1.0
    # ranks as far apart as their sizes, of one token a beam
    _check(lib(), x, np.array([[-3e38, -1e38, -2e38]]), 3, length=np.array([[1, 1, 1]]), alpha=alpha)
