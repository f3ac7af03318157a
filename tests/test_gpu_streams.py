"""Calls on a stream of the caller's that leave their outputs and workspace to the binding (GPU).

That memory has to come from the given stream's: memory of the current stream may still be read or written by work
pending there, which the call does not wait for.  What the caller gets back must not be handed out again while work that
the current stream has queued on it is pending.
"""

import numpy as np
import pytest

import spec_workloads as wl
from gpu_util import lib

pytestmark = pytest.mark.gpu


def _i32(a):
    import torch
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _serving(st):
    """{name: call(**kw) -> its tensors}: every serving call, ready to be made."""
    import torch
    g = torch.Generator().manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    B, Hq, Hkv, D, T, Lmax, bs, Ls = 4, 16, 4, 64, 40, 128, 16, 96
    parent = [int(p) for p in wl.random_tree(np.random.default_rng(3), T, max_depth=14, max_children=6)[0]]
    tree = st.spec_tree_build(parent)
    q, kt, vt = rand(B, Hq, T, D), rand(B, Hkv, T, D), rand(B, Hkv, T, D)
    kc, vc, ks, vs = rand(B, Hkv, Lmax, D), rand(B, Hkv, Lmax, D), rand(Hkv, Ls, D), rand(Hkv, Ls, D)
    kp, vp = rand(40, Hkv, bs, D), rand(40, Hkv, bs, D)
    kc2, vc2, kp2, vp2 = (t.clone() for t in (kc, vc, kp, vp))
    L, sl = _i32([100, 0, 17, 64]), _i32([90])
    table, stable = _i32(np.arange(32).reshape(4, 8)), _i32(np.arange(32, 38))
    x, y = rand(30, Hq + 2 * Hkv, D), rand(B, T, Hq + 2 * Hkv, D)
    rows = lambda z: (z[..., :Hq, :], z[..., Hq:Hq + Hkv, :], z[..., Hq + Hkv:, :])  # noqa: E731
    start, freq = _i32([0, 9, 9, 20, 30]), torch.tensor(10000.0 ** (-np.arange(32) / 32), device="cuda")
    return {
        "tree_attention_shared": lambda **kw: st.tree_attention_shared(q, ks, vs, sl, kc, vc, L, kt, vt, tree, **kw),
        "tree_attention_shared_paged": lambda **kw: st.tree_attention_shared_paged(q, kp, vp, stable, sl, table, L, kt, vt, tree, **kw),
        "tree_attention_scored": lambda **kw: st.tree_attention_scored(q, kc, vc, L, kt, vt, tree, softcap=20.0, **kw),
        "tree_attention_scored_paged": lambda **kw: st.tree_attention_scored_paged(q, kp, vp, table, L, kt, vt, tree, window=50, **kw),
        "kv_append": lambda **kw: st.kv_append(*rows(x), start, L, kc2, vc2, freq=freq, **kw),
        "kv_append_paged": lambda **kw: st.kv_append_paged(*rows(x), start, L, kp2, vp2, table, freq=freq, **kw),
        "tree_rope": lambda **kw: st.tree_rope(*rows(y), L, tree, freq=freq, **kw),
    }


def _verifying(st):
    """The same of the calls of a verification step."""
    import torch
    g = torch.Generator().manual_seed(6)
    rand = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    B, T, V, d, Hq, Hkv, D, Lmax = 2, 6, 300, 64, 4, 2, 64, 128
    parent = [-1, 0, 0, 1, 1, 3]
    tree = st.spec_tree_build(parent)
    h, emb, root = rand(B, d), rand(V, d), _i32([3, 5])
    W1, W2, folds = [rand(d, 2 * d) * 0.1 for _ in range(3)], [rand(V, d) for _ in range(3)], rand(d, 2 * d)
    heads = [dict(cond=1, topk=4, W1=a, W2=b) for a, b in zip(W1, W2)]
    q, kt, vt = rand(B, Hq, T, D), rand(B, Hkv, T, D), rand(B, Hkv, T, D)
    kc, vc, kp, vp = rand(B, Hkv, Lmax, D), rand(B, Hkv, Lmax, D), rand(4, Hkv, 64, D), rand(4, Hkv, 64, D)
    L, table = _i32([100, 17]), _i32([[0, 1], [2, 3]])
    L0, L1 = _i32([0, 0]), _i32([0, 0])
    logits, tok = rand(B, T, V), _i32(np.arange(B * T).reshape(B, T))
    alen, path = _i32([1, 0]), _i32([[0, 1, -1, -1], [0, -1, -1, -1]])
    one = lambda x: (x,)  # noqa: E731
    return {
        "spec_tree_build": lambda **kw: one(st.spec_tree_build(parent, **kw).buf),
        "hydra_fold_embedding": lambda **kw: one(st.hydra_fold_embedding(folds, emb, **kw)),
        "hydra_draft": lambda **kw: st.hydra_draft(h, emb, W1, None, W2, [1] * 3, [4] * 3, root, tree, **kw),
        "hydra_draft_heads": lambda **kw: st.hydra_draft_heads(h, emb, heads, root, tree, **kw),
        "tree_attention": lambda **kw: st.tree_attention(q, kc, vc, L, kt, vt, tree, **kw),
        "tree_attention_paged": lambda **kw: st.tree_attention_paged(q, kp, vp, table, L, kt, vt, tree, **kw),
        "tree_attention_noalloc": lambda **kw: st.tree_attention_noalloc(q, kc, vc, L, kt, vt, tree, **kw),
        "tree_accept": lambda **kw: st.tree_accept(0, logits, None, tok, tree, **kw),
        "tree_accept_typical": lambda **kw: st.tree_accept_typical(logits, tok, tree, **kw),
        "tree_kv_commit": lambda **kw: one(st.tree_kv_commit(kt, vt, kc, vc, L0, alen, path, tree, **kw)),
        "tree_kv_commit_paged": lambda **kw: one(st.tree_kv_commit_paged(kt, vt, kp, vp, table, 64, L1, alen, path, tree, **kw)),
        "spec_philox_uniform": lambda **kw: st.spec_philox_uniform(1, 2, B, T, **kw),
    }


def _calls(st):
    return {**_serving(st), **_verifying(st)}


SERVING = ["tree_attention_shared", "tree_attention_shared_paged", "tree_attention_scored", "tree_attention_scored_paged", "kv_append",
           "kv_append_paged", "tree_rope"]
ALL = SERVING + ["spec_tree_build", "hydra_fold_embedding", "hydra_draft", "hydra_draft_heads", "tree_attention", "tree_attention_paged",
                 "tree_attention_noalloc", "tree_accept", "tree_accept_typical", "tree_kv_commit", "tree_kv_commit_paged",
                 "spec_philox_uniform"]


def _stream_of(t):
    """The stream whose memory a tensor's is."""
    import torch
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's memory")


@pytest.mark.parametrize("name", ALL)
def test_memory_comes_from_the_given_stream(name):
    import torch
    call = _calls(lib())[name]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(stream=side)
    torch.cuda.synchronize()
    assert [_stream_of(t) for t in got] == [side.cuda_stream] * len(got)
    named = type("Named", (), {"cuda_stream": side.cuda_stream})()      # what is only the name of a stream will do
    assert [_stream_of(t) for t in call(stream=named)] == [side.cuda_stream] * len(got)
    here = call()
    torch.cuda.synchronize()
    assert [_stream_of(t) for t in here] == [torch.cuda.current_stream().cuda_stream] * len(here)


@pytest.mark.parametrize("name", ALL)
def test_work_pending_on_the_current_stream_does_not_reach_the_call(name):
    """Temporaries of the results' sizes and of workspaces', freed with a write to them still to come."""
    import torch
    call = _calls(lib())[name]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)
    for n in [t.nbytes for t in want] + [1 << k for k in range(12, 26)]:
        temporary = torch.empty(n, dtype=torch.uint8, device="cuda")
        temporary.fill_(255)
        del temporary
    got = call(stream=side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert a.dtype == torch.uint8 or torch.equal(a, b)      # (a returned workspace says no more than its status)


@pytest.mark.parametrize("name", ALL)
def test_results_are_not_handed_out_again_while_the_current_stream_reads_them(name):
    import torch
    call = _calls(lib())[name]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(20_000_000)
    seen = [t.clone() for t in got]                             # queued behind the sleep
    sizes = [t.nbytes for t in got]
    del got
    with torch.cuda.stream(side):
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    for a, b in zip(seen, want):
        assert a.dtype == torch.uint8 or torch.equal(a, b)


@pytest.mark.parametrize("name", SERVING)
def test_captured_on_the_given_stream(name):
    """A capture in which the call allocates for itself, replayed."""
    import torch
    call = _calls(lib())[name]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side = torch.cuda.current_stream()
        got = call(stream=side)
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert a.dtype == torch.uint8 or torch.equal(a, b)


@pytest.mark.parametrize("name", SERVING)
def test_captured_on_a_stream_that_joins_the_capture(name):
    """Two calls on a side stream inside a capture, the first one's results dropped at once, replayed twice."""
    import torch
    call = _calls(lib())[name]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        call(stream=side)
        got = call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert a.dtype == torch.uint8 or torch.equal(a, b)
