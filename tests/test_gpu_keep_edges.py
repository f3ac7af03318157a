"""Calls of the beam and eviction operators that lie between the others' cases (GPU)."""

import numpy as np
import pytest

from gpu_util import lib
from oracle import beam, evict

pytestmark = pytest.mark.gpu


def _i32(a):
    import torch
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def test_a_workspace_of_the_largest_batch_serves_every_smaller_one():
    """Of exactly the size that the largest call asks for, with what lies behind it left alone; results are those with a workspace of
    the call's own."""
    import torch
    st = lib()
    W, K, V, Hq, Hkv, D, L, T, most = 4, 4, 32000, 8, 2, 64, 517, 100, 40
    g = torch.Generator().manual_seed(21)
    sizes = (st.beam_select_workspace_size(most, W, V, K), st.kv_weigh_workspace_size(most, Hq, Hkv, T, 0, L, D, 0),
             st.kv_evict_workspace_size(most, Hkv, L, 200))
    room = [torch.full((n + 4096,), 171, dtype=torch.uint8, device="cuda") for n in sizes]
    for B in (most, 37, 24, 18, 16, 8, 4, 2, 1):
        ws = [r[:n] for r, n in zip(room, sizes)]
        x, scores = torch.randn(B, W, V, generator=g).cuda(), -torch.rand(B, W, generator=g).cuda()
        got, want = st.beam_select(x, scores, K, ws=ws[0]), st.beam_select(x, scores, K)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), B
        k, q = torch.randn(B, Hkv, L, D, generator=g).cuda(), torch.randn(B, Hq, T, D, generator=g).cuda()
        lse, n = torch.full((B, Hq, T), 4.0, device="cuda"), _i32(np.linspace(T, L, B).astype(int))
        acc = [torch.ones(B, Hkv, L, device="cuda") for _ in range(2)]
        pos = _i32(np.tile(np.arange(L), (B, Hkv, 1)))
        for a, w in zip(acc, (ws[1], None)):
            st.kv_weigh(q, lse, k, n, a, ws=w)
        assert torch.equal(*acc), B
        v = k.flip(2).contiguous()
        two = [(k, v, acc[0], pos), tuple(t.clone() for t in (k, v, acc[0], pos))]
        for c, w in zip(two, (ws[2], None)):
            st.kv_evict(c[0], c[1], n, c[2], c[3], 200, ws=w)
        assert all(torch.equal(a, b) for a, b in zip(*two)), B
        assert [st.spec_read_device_status(w) for w in ws] == [0, 0, 0]
    for r, n in zip(room, sizes):
        assert (r[n:] == 171).all()


def _two(st, seed):
    """{name: (call(**kw) -> outputs of its own, the tensors it works on)} of inputs and lengths that go by the seed."""
    import torch
    g, r = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    rand = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    B, W, V, Hq, Hkv, D, L, T = 2, 4, 30000, 8, 2, 64, 700, 150
    x, scores = rand(B, W, V), -torch.rand(B, W, generator=g).cuda()
    k, n = rand(B, Hkv, L, D), _i32(r.integers(T, L, B))
    q, q2, kf, qf = rand(B, Hq, 1, D), rand(B, Hq, T, D), rand(B, Hkv, L, D).float(), rand(B, Hq, T, D).float()
    lse, lse2 = torch.full((B, Hq, 1), 3.0, device="cuda"), torch.full((B, Hq, T), 3.0, device="cuda")
    led = lambda: (torch.rand(B, Hkv, L, generator=g).cuda(), _i32(np.tile(r.permutation(L), (B, Hkv, 1))))  # noqa: E731
    one, many, f32, step, half = led(), led(), led(), led(), led()
    cache, cache2, beams = (rand(B, Hkv, L, D), rand(B, Hkv, L, D)), (rand(B, Hkv, L, D), rand(B, Hkv, L, D)), (rand(B * W, Hkv, L, D), rand(B * W, Hkv, L, D))
    hist, parent = torch.randint(0, 999, (B, W, 50), generator=g).cuda(), _i32(np.stack([r.permutation(W) for _ in range(B)]))
    a, z = _i32(r.integers(0, 100, B)), _i32(r.integers(400, L, B))
    full = _i32(r.integers(L - 9, L, B))
    return {
        "beam_select": (lambda **kw: st.beam_select(x, scores, 4, alpha=0.5, **kw), ()),
        "beam_reorder": (lambda **kw: st.beam_reorder(hist, parent, **kw), (hist,)),
        "kv_reorder": (lambda **kw: st.kv_reorder(*beams, parent, a, z, **kw), beams),
        "kv_weigh": (lambda **kw: st.kv_weigh(q, lse, k, n, one[0], pos=one[1], decay=0.5, **kw), one),
        "kv_weigh prompts": (lambda **kw: st.kv_weigh(q2, lse2, k, n, many[0], pos=many[1], decay=0.5, **kw), many),
        "kv_weigh f32": (lambda **kw: st.kv_weigh(qf, lse2, kf, n, f32[0], pos=f32[1], decay=0.5, **kw), f32),
        "kv_evict step": (lambda **kw: st.kv_evict(*cache, full, *step, L - 20, **kw), (*cache, *step)),
        "kv_evict": (lambda **kw: st.kv_evict(*cache2, n, *half, 70, sink=2, recent=5, **kw), (*cache2, *half)),
    }


KEEP = ["beam_select", "beam_reorder", "kv_reorder", "kv_weigh", "kv_weigh prompts", "kv_weigh f32", "kv_evict step", "kv_evict"]


@pytest.mark.parametrize("name", KEEP)
def test_two_calls_at_once_keep_to_their_own(name):
    """Two streams, inputs that differ, every state put back in front of each pair of calls: memory that the two shared would hold the
    other's numbers."""
    import torch
    st = lib()
    sides = [(torch.cuda.Stream(), *_two(st, seed)[name]) for seed in (31, 32)]
    first = [[t.clone() for t in state] for _, _, state in sides]
    want = []
    for _, call, state in sides:
        got = call()
        want.append([t.clone() for t in (*state, *(got if name == "beam_select" else ()))])
    torch.cuda.synchronize()
    assert not any(torch.equal(x, y) for x, y in zip(*want) if x.is_floating_point())
    for _ in range(20):
        for (_, _, state), s in zip(sides, first):
            for t, x in zip(state, s):
                t.copy_(x)
        torch.cuda.synchronize()
        got = [call(stream=stream) for stream, call, _ in sides]
        torch.cuda.synchronize()
        for (_, _, state), r, w in zip(sides, got, want):
            assert all(torch.equal(x, y) for x, y in zip((*state, *(r if name == "beam_select" else ())), w))


@pytest.mark.parametrize("name", KEEP)
def test_workspaces_too_are_the_given_stream_s_memory(name, monkeypatch):
    """Everything that the binding allocates for a call, what the caller never sees too: on a given stream of that stream's memory, else
    of the current stream's."""
    import torch
    st = lib()
    from tree_speculative_decoding_spec_gb300 import _binding
    call, _ = _two(st, 33)[name]
    side, made, raw = torch.cuda.Stream(), [], []

    def stream_of(t):
        at = t.data_ptr()
        return next(s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"])

    def new(*args, plain=_binding._new, **kw):
        made.append(plain(*args, **kw))
        return made[-1]

    def raw_alloc(n, stream, plain=_binding._raw_alloc):
        raw.append((n, stream))
        return plain(n, stream)

    monkeypatch.setattr(_binding, "_new", new)
    monkeypatch.setattr(_binding, "_raw_alloc", raw_alloc)
    torch.cuda.synchronize()
    call(stream=side)
    torch.cuda.synchronize()
    assert made and not raw and {stream_of(t) for t in made} == {side.cuda_stream}
    assert any(t.dtype is torch.uint8 and t.numel() >= 256 for t in made)          # the workspace among them
    made.clear()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    assert {stream_of(t) for t in made} <= {side.cuda_stream} and {s for _, s in raw} <= {side.cuda_stream}
    assert [n for n, _ in raw if n >= 256] or [t for t in made if t.dtype is torch.uint8]


def _weighed(dtype, Hq, Hkv, T, D, block, n, scale, seed):
    """A case of test_gpu_evict whose lse is that of `scale`, run and compared with the oracle within its bound."""
    import torch
    from test_gpu_evict import _case, _run
    st = lib()
    t = _case((dtype, len(n), Hq, Hkv, T, D, block, n, None, 0.75), seed=seed)
    q, k = t["q"].double().cpu().numpy(), t["k"].double().cpu().numpy()
    c = D ** -0.5 if scale is None else scale
    for b, m in enumerate(n):
        for hq in range(Hq):
            K = evict._line(k, b, hq // (Hq // Hkv), m, t["table"])
            for i in range(T):
                s = K[:m - T + i + 1] @ q[b, hq, i] * c
                t["lse"][b, hq, i] = s.max() + np.log(np.exp(s - s.max()).sum())
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda").fill_(255)
    acc, pos = _run(st, t, ws, scale=scale)
    assert st.spec_read_device_status(ws) == 0
    want, wpos, size = evict.kv_weigh(q, t["lse"], k, t["n"], t["acc"], t["pos"], seen=t["seen"], decay=t["decay"], scale=scale, table=t["table"])
    # the bound at the head of test_gpu_evict: D + 4 roundings of scale |q||k| + |lse| a weight, its exponential, the sum's roundings
    tol = (D + 4) * 2.0 ** -24 * size + (2.0 ** -20 + (Hq // Hkv * T + 4) * 2.0 ** -24) * (np.abs(want) + np.abs(t["acc"]))
    assert (np.abs(acc.cpu().numpy() - want) <= tol).all()
    np.testing.assert_array_equal(pos.cpu().numpy(), wpos)


@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 1), (9, 1), (24, 3)])
def test_single_tokens_in_fp32_at_head_dim_128(Hq, Hkv, block):
    """One row a thread up to eight rows of a KV head, four from nine on."""
    _weighed("f32", Hq, Hkv, 1, 128, block, (130, 64, 1, 333), None, 41)


@pytest.mark.parametrize("dtype,T,D,n", [("f32", 3, 64, (100, 40)), ("f32", 30, 128, (150, 64)), ("bf16", 2, 128, (300, 129)), ("bf16", 5, 64, (140, 77)),
                                         ("bf16", 150, 64, (400, 150)), ("bf16", 140, 128, (300, 256))])
@pytest.mark.parametrize("scale", [0.21, 0.03])
def test_scales_of_the_caller_s_own(dtype, T, D, n, scale):
    _weighed(dtype, 8, 2, T, D, 0, n, scale, 42)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("alpha", [0.0, 0.7])
@pytest.mark.parametrize("W,K", [(1, 4), (2, 5), (3, 64), (64, 64)])
def test_sequences_whose_beams_have_all_ended(W, K, alpha, dtype):
    """Each ended beam offers itself and nothing else: what is missing from K is token -1, parent -1, score -inf, ended, of length 0."""
    import torch
    from test_gpu_beam import _check
    rng = np.random.default_rng(W + K)
    B, V = 5, 900
    ended = np.ones((B, W), dtype=int)
    ended[1, -1] = 0                                 # one of the last sequences still has a live beam
    ended[3] = rng.integers(0, 2, W)
    x = torch.from_numpy((2.5 * rng.standard_normal((B, W, V))).astype(np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    scores = -rng.random((B, W)) * 5 - 8
    scores[4, 0] = -np.inf                           # an ended beam that is no more
    _check(lib(), x, scores, K, eos=2, ended=ended, length=np.where(ended, rng.integers(1, 12, (B, W)), 12), alpha=alpha)


@pytest.mark.parametrize("dtype,V", [("bf16", 60001), ("f32", 50000)])
def test_scores_of_long_rows_in_one_slice(dtype, V):
    """As many rows as keep every SM busy with whole ones.  A thread sums V / (1024 E) chunks of 4 E elements, E of them 16 bytes: in each 2 E
    additions a chain, 2 to join the chains and a rescaling, whose factor is off by four roundings; then 5 + 8 additions of threads and warps and the
    logarithm.  An exponential is off by four roundings and by what its argument x - max is: two roundings of it."""
    import torch
    B, W, K, E = 60, 16, 16, 8 if dtype == "bf16" else 4
    g = torch.Generator().manual_seed(51)
    x = (2.5 * torch.randn(B, W, V, generator=g)).cuda().to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    scores = -torch.rand(B, W, generator=g).cuda() - 3
    token, parent, score, _, length = lib().beam_select(x, scores, K)
    d = x.double()
    a = d - d.amax(-1, keepdim=True)
    w = torch.exp(a)
    rel = 2 * float((-a * w).sum(-1).div(w.sum(-1)).max()) + 4 + -(-V // (1024 * E)) * (2 * E + 2 + 1 + 4) + 13 + 2
    ranks = (scores.double()[..., None] + torch.log_softmax(d, -1)).view(B, W * V)
    want, at = torch.topk(ranks, K + 1, -1)
    tol = rel * 2.0 ** -24
    got = ranks.gather(1, parent.long() * V + token.long())
    assert ((score.double() - got).abs() <= tol + 2.0 ** -24 * got.abs()).all()
    # pairs in another order are nearer to each other than the log-sums can be off; equal logits of a row go to the lower token
    assert ((got - want[:, :K]).abs() <= 2 * tol).all() and (length == 1).all()
    flat = parent.long() * V + token.long()
    assert all(len(set(r)) == K for r in flat.tolist())
    tie = (got[:, 1:] == got[:, :-1]) & (parent[:, 1:] == parent[:, :-1])
    assert (token[:, 1:] > token[:, :-1])[tie].all()


@pytest.mark.parametrize("name", KEEP)
def test_calls_behind_a_fork_a_copy_and_a_join_of_a_capture(name):
    """Captured on a side stream that waits for two others' work and for a copy, and joined again: replays give what a single call gives."""
    import torch
    st = lib()
    call, state = _two(st, 34)[name]
    first = [t.clone() for t in state]
    outs = lambda got: [t.clone() for t in (*state, *(got if name == "beam_select" else ()))]  # noqa: E731
    want = outs(call())
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    x, y = torch.zeros(1 << 20, device="cuda"), torch.zeros(1 << 20, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        other.wait_stream(main)
        with torch.cuda.stream(other):
            x.add_(1.0)
        with torch.cuda.stream(side):
            y.add_(1.0)
            for t, s in zip(state, first):
                t.copy_(s)                           # the last node in front of the call, where it has a state
        side.wait_stream(other)
        got = call(stream=side)
        with torch.cuda.stream(side):
            y.add_(x)
        main.wait_stream(side)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs(got), want))
    assert (x == 3.0).all() and (y == 9.0).all()
