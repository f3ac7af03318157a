"""The beam and eviction calls on streams of the caller's, side by side, in graphs and far into large buffers (GPU).

What the binding allocates for a call with a stream is that stream's memory: memory of the current one may still be in
use by work pending there.  Results on a side stream, of two calls at once and of replays are those of single calls, to the last bit.
"""

import numpy as np
import pytest

from gpu_util import lib
from oracle import beam, evict

pytestmark = pytest.mark.gpu


def _i32(a):
    import torch
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _calls(st):
    """{name: (call(**kw) -> tensors the binding may have allocated, the tensors that hold the result)}."""
    import torch
    g = torch.Generator().manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    B, W, V, Hq, Hkv, D, L, bs = 2, 4, 3000, 8, 2, 64, 192, 16
    x, scores = rand(B, W, V), -torch.rand(B, W, generator=g).cuda()
    parent, start, end = _i32([[1, 1, 0, 3], [3, 2, 1, 0]]), _i32([5, 0]), _i32([100, 192])
    hist = torch.arange(B * W * 6, device="cuda", dtype=torch.int32).view(B, W, 6)
    kb, vb, kp, vp = rand(B * W, Hkv, L, D), rand(B * W, Hkv, L, D), rand(B * W * 12, Hkv, bs, D), rand(B * W * 12, Hkv, bs, D)
    beams = _i32(np.arange(B * W * 12).reshape(B * W, 12))
    k, v, table = kb[:B].clone(), vb[:B].clone(), _i32(np.arange(24).reshape(2, 12))
    k2, v2 = kp[:24].clone(), vp[:24].clone()
    q, lse, q2, lse2 = rand(B, Hq, 1, D), torch.full((B, Hq, 1), 3.0, device="cuda"), rand(B, Hq, 150, D), torch.full((B, Hq, 150), 3.0, device="cuda")
    n = _i32([192, 150])
    led = lambda: (torch.rand(B, Hkv, L, generator=g).cuda(), _i32(np.tile(np.arange(L), (B, Hkv, 1))))  # noqa: E731
    l1, l2, l3, l4, l5 = led(), led(), led(), led(), led()
    return {
        "beam_select": (lambda **kw: st.beam_select(x, scores, 5, alpha=0.5, **kw), ()),
        "beam_reorder": (lambda **kw: (st.beam_reorder(hist, parent, **kw),)[1:], (hist,)),
        "kv_reorder": (lambda **kw: (st.kv_reorder(kb, vb, parent, start, end, **kw),), (kb, vb)),
        "kv_reorder_paged": (lambda **kw: (st.kv_reorder_paged(kp, vp, beams, parent, start, end, **kw),), (kp, vp)),
        "kv_weigh": (lambda **kw: (st.kv_weigh(q, lse, k, n, l1[0], pos=l1[1], decay=0.0, **kw),)[1:], l1),
        "kv_weigh prompts": (lambda **kw: (st.kv_weigh(q2, lse2, k, n, l2[0], decay=0.0, **kw),)[1:], l2),
        "kv_weigh_paged": (lambda **kw: (st.kv_weigh_paged(q, lse, k2, table, n, l3[0], decay=0.0, **kw),)[1:], l3),
        "kv_evict": (lambda **kw: (st.kv_evict(k, v, n, *l4, 180, **kw),), (k, v, *l4)),
        "kv_evict_paged": (lambda **kw: (st.kv_evict_paged(k2, v2, table, n, *l5, 40, sink=2, recent=5, **kw),), (k2, v2, *l5)),
    }


NAMES = ["beam_select", "beam_reorder", "kv_reorder", "kv_reorder_paged", "kv_weigh", "kv_weigh prompts", "kv_weigh_paged", "kv_evict", "kv_evict_paged"]


def _stream_of(t):
    import torch
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's memory")


@pytest.mark.parametrize("name", NAMES)
def test_memory_comes_from_the_given_stream(name):
    import torch
    call, _ = _calls(lib())[name]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(stream=side)
    torch.cuda.synchronize()
    assert [_stream_of(t) for t in got] == [side.cuda_stream] * len(got)


@pytest.mark.parametrize("name", NAMES)
def test_side_streams_and_replays_give_what_a_single_call_gives(name):
    import torch
    st = lib()
    call, state = _calls(st)[name]
    first = [t.clone() for t in state]

    def back():
        for t, s in zip(state, first):
            t.copy_(s)
        torch.cuda.synchronize()

    def result(got):
        torch.cuda.synchronize()
        return [t.clone() for t in state] + ([t.clone() for t in got] if name == "beam_select" else [])

    want = result(call())
    back()
    side = torch.cuda.Stream()
    same = lambda a: all(torch.equal(x, y) for x, y in zip(a, want))  # noqa: E731
    assert same(result(call(stream=side)))
    back()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(2):
        back()
        graph.replay()
        assert same(result(got))


def test_two_at_once():
    """Different sequences' calls on two streams, workspaces of their own, many times over."""
    import torch
    st = lib()
    a, b = _calls(st), _calls(st)
    want = {n: [t.clone() for t in (c()[:5] if n == "beam_select" else (c(), s)[1])] for n, (c, s) in a.items() if n.startswith(("beam_sel", "kv_weigh"))}
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    got = {}
    for _ in range(20):
        for n in want:
            for side, calls in ((one, a), (two, b)):
                r = calls[n][0](stream=side)
                got[n, side] = r if n == "beam_select" else calls[n][1]
    torch.cuda.synchronize()
    for n in want:
        for side in (one, two):
            assert all(torch.equal(x, y) for x, y in zip(got[n, side], want[n])), n


def test_far_into_large_buffers():
    """Rows whose element offsets pass 32 bits."""
    import torch
    st = lib()
    B, H, L, D = 2, 8, (1 << 21) + 64, 128                   # 2^32 elements and some
    k, v = (torch.empty(B, H, L, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = 70
    small = torch.randn(2, H, n, D).bfloat16()
    k[1, :, :n], v[1, :, :n] = small[0].cuda(), small[1].cuda()
    acc, pos = torch.rand(B, H, L, device="cuda"), torch.zeros(B, H, L, dtype=torch.int32, device="cuda")
    pos[1, :, :n] = torch.arange(n, device="cuda", dtype=torch.int32)
    q = torch.randn(B, H, 1, D).bfloat16().cuda()
    lse = torch.full((B, H, 1), 2.0, device="cuda")
    old = acc[1, :, :n].cpu().numpy()
    st.kv_weigh(q, lse, k, _i32([0, n]), acc, pos=pos, n_rows=_i32([0, 1]))
    want, _, _ = evict.kv_weigh(q[1:].double().cpu().numpy(), lse[1:].cpu().numpy(), small[:1].double().numpy(), [n], old[None], np.zeros((1, H, n), dtype=int))
    got = acc[1, :, :n].cpu().numpy()
    np.testing.assert_allclose(got, want[0], rtol=1e-5)
    m = st.kv_evict(k, v, _i32([0, n]), acc, pos, 40, recent=4)
    want = evict.kv_evict(small[:1].float().numpy(), small[1:].float().numpy(), got[None], np.tile(np.arange(n), (1, H, 1)), np.array([n]), 40, recent=4)
    assert m.tolist() == [0, 40]
    np.testing.assert_array_equal(k[1, :, :40].float().cpu().numpy(), want[0][0, :, :40])
    np.testing.assert_array_equal(v[1, :, :40].float().cpu().numpy(), want[1][0, :, :40])
    # the same buffers as one sequence of two beams
    before = k[1, :, :40].clone()
    k[0, :, :40] = torch.randn(H, 40, D).bfloat16().cuda()
    other = k[0, :, :40].clone()
    st.kv_reorder(k, v, _i32([[1, 0]]), _i32([0]), _i32([40]))
    assert torch.equal(k[0, :, :40], before) and torch.equal(k[1, :, :40], other)
    # logits of rows 2^32 elements behind the first
    x = torch.empty(1, 3, 1 << 31, dtype=torch.bfloat16, device="cuda")[..., :5000]
    x.copy_(torch.randn(1, 3, 5000))
    r = st.beam_select(x, torch.tensor([[-1.0, -1.5, -0.5]], device="cuda"), 4)
    w = beam.beam_select(x.double().cpu().numpy(), np.array([[-1.0, -1.5, -0.5]]), 4)
    assert r[0].tolist() == w["token"].tolist() and r[1].tolist() == w["parent"].tolist()


def test_calls_in_a_row_see_what_the_ones_before_them_wrote():
    """Every call's first kernel may start while the last one's still runs: a chain in place, each step on the results of the one
    before, gives the same bits with and without a pause between the calls."""
    import torch
    st = lib()
    g = torch.Generator().manual_seed(9)
    B, W, V, Hq, Hkv, D, L = 3, 6, 40000, 8, 2, 64, 640
    x = [torch.randn(B, W, V, generator=g).mul_(2).cuda() for _ in range(2)]
    q, q2 = torch.randn(B, Hq, 1, D, generator=g).bfloat16().cuda(), torch.randn(B, Hq, 200, D, generator=g).bfloat16().cuda()
    lse, lse2 = torch.full((B, Hq, 1), 4.0, device="cuda"), torch.full((B, Hq, 200), 4.0, device="cuda")
    kv = [torch.randn(B * W, Hkv, L, D, generator=g).bfloat16().cuda() for _ in range(2)]
    start, end, n = _i32([0, 7, 300]), _i32([640, 600, 301]), _i32([640, 630, 500])

    def chain(pause):
        scores, ended, length = torch.zeros(B, W, device="cuda"), torch.zeros(B, W, dtype=torch.int32, device="cuda"), torch.zeros(B, W, dtype=torch.int32, device="cuda")
        hist = torch.arange(B * W * 40, device="cuda").view(B, W, 40)
        k, v = kv[0].clone(), kv[1].clone()
        acc, pos = torch.zeros(B, Hkv, L, device="cuda"), _i32(np.tile(np.arange(L), (B, Hkv, 1)))
        out = []
        for i in range(12):
            token, parent, *_ = st.beam_select(x[i & 1], scores, W, eos=3, ended=ended, length=length, alpha=0.5, token=torch.empty_like(ended),
                                               parent=torch.empty_like(ended), score=scores, ended_out=ended, length_out=length)
            pause()
            st.beam_reorder(hist, parent)
            pause()
            hist[:, :, i] = token
            st.kv_reorder(k, v, parent, start, end)
            pause()
            st.kv_weigh(q2, lse2, k[:B], n, acc, pos=pos, decay=0.9)
            pause()
            st.kv_weigh(q, lse, k[:B], n, acc, pos=pos)
            pause()
            out.append(st.kv_evict(k[:B], v[:B], n, acc, pos, 600 - 20 * i))
            pause()
        torch.cuda.synchronize()
        return [scores, ended, length, hist, k, v, acc, pos, *out]

    want = chain(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(chain(lambda: None), want))
