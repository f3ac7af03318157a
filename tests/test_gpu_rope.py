"""Rotated appends to the cache and the rotation of tree projections: CUDA path vs the oracle (GPU).

Tolerance of a rotated value: half a step of the output type, plus the 32-bit
arithmetic.  There the angle's rest is rounded once (at most half a turn, so pi
2^-24 radians), sine and cosine are within 2 units of 2^-23, and the two products
and their sum round three times 2^-24: (pi + 4 + 3) 2^-24 (|x| + |y|) for the pair
(x, y), taken as 11 2^-24.  Copies are exact.
"""

import numpy as np
import pytest

import spec_workloads as wl
from gpu_util import lib
from oracle import rope

pytestmark = pytest.mark.gpu

STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _torch(dtype):
    import torch
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _rand(g, dtype, *shape):
    import torch
    return torch.randn(*shape, generator=g, dtype=torch.float32).to(_torch(dtype)).cuda()


def _np(t):
    return t.detach().double().cpu().numpy()


def _assert_rotated(got, ref, x, freq, interleaved, dtype, what):
    """got against ref [..., D]; x [..., D] holds the same rows before the rotation."""
    half = len(freq)
    x = np.abs(x)
    size = np.zeros_like(x)
    if interleaved:
        size[..., 0:2 * half:2] = size[..., 1:2 * half:2] = x[..., 0:2 * half:2] + x[..., 1:2 * half:2]
    else:
        size[..., :half] = size[..., half:2 * half] = x[..., :half] + x[..., half:2 * half]
    near = 11 * 2.0 ** -24 * size
    tol = near + STEP[dtype] * (np.abs(ref) + near)
    tol[..., 2 * half:] = 0.0
    bad = np.abs(got - ref) > tol
    assert not bad.any(), f"{what}: {bad.sum()} values out of tolerance, worst {np.abs(got - ref).max():.3e}"


APPENDS = [
    # dtype, Hq, Hkv, D, rot, interleaved, block (0: contiguous), new tokens, prefix lengths, base
    ("bf16", 8, 2, 128, 128, False, 64, (1, 1, 1), (0, 63, 64), 0),           # one token each, page borders
    ("bf16", 7, 1, 128, 64, False, 16, (40, 0, 17, 1), (5, 3, 31, 0), 1000),  # an empty sequence, partial rotation
    ("f32", 4, 2, 64, 32, True, 0, (9, 30), (11, 0), 0),
    ("bf16", 3, 3, 80, 20, False, 7, (5, 6), (2, 20), 3),                     # pairs that do not fill 16-byte chunks
    ("f32", 2, 1, 12, 6, True, 5, (3, 4), (0, 1), 0),
    ("bf16", 2, 2, 64, 0, False, 32, (4, 4), (10, 30), 7),                    # no rotation
    ("f32", 1, 1, 8, 8, False, 0, (1,), (0,), 0),                             # the smallest
    ("bf16", 64, 8, 128, 128, True, 64, (300, 1, 77), (100, 4000, 0), 123),
]


def _case(c, seed=0, tail=3, lead=0):
    import torch
    dtype, Hq, Hkv, D, rot, inter, block, new, L, base = c
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    N, B = lead + sum(new) + tail, len(new)
    x = _rand(g, dtype, N, Hq + 2 * Hkv, D)
    start = lead + np.concatenate([[0], np.cumsum(new)])
    total = [a + b for a, b in zip(L, new)]
    t = dict(q=x[:, :Hq], k=x[:, Hq:Hq + Hkv], v=x[:, Hq + Hkv:], start=start, L=np.array(L), table=None)
    if block:
        width = max(1, max(-(-n // block) for n in total))
        t["table"] = rng.permutation(B * width + 2)[:B * width].reshape(B, width)
        shape = (B * width + 2, Hkv, block, D)
    else:
        shape = (B, Hkv, max(total) + 2, D)
    t["kc"], t["vc"] = _rand(g, dtype, *shape), _rand(g, dtype, *shape)
    t["freq"] = 10000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))
    return t


def _dev32(a):
    import torch
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _append(st, c, t, q_out=None, **kw):
    import torch
    base = _dev32([c[9]])
    freq = torch.tensor(t["freq"], dtype=torch.float64, device="cuda") if len(t["freq"]) else None
    a = (t["q"], t["k"], t["v"], _dev32(t["start"]), _dev32(t["L"]), t["kc"], t["vc"])
    if t["table"] is not None:
        a += (_dev32(t["table"]),)
    f = st.kv_append if t["table"] is None else st.kv_append_paged
    return f(*a, freq=freq, interleaved=c[5], pos_base=base, q_out=q_out, **kw)


def _check(c, t, kc0, vc0, q_out, q0, status, want_status=0):
    freq, inter, dtype = t["freq"], c[5], c[0]
    qr, kr, vr, written = rope.kv_append(_np(t["q"]), _np(t["k"]), _np(t["v"]), t["start"], t["L"], kc0, vc0, freq, inter,
                                         c[9], t["table"])
    # the rows before the rotation, laid out like the results
    none = np.zeros_like(freq)
    qx, kx, _, _ = rope.kv_append(_np(t["q"]), _np(t["k"]), _np(t["v"]), t["start"], t["L"], kc0, vc0, none, inter, 0,
                                  t["table"])
    got_q, got_k = _np(q_out), _np(t["kc"])
    np.testing.assert_array_equal(got_q[~written], q0[~written])
    _assert_rotated(got_q[written], qr[written], qx[written], freq, inter, dtype, "q")
    untouched = kr == kc0
    np.testing.assert_array_equal(got_k[untouched & (kx == kc0)], kc0[untouched & (kx == kc0)])
    _assert_rotated(got_k, kr, kx, freq, inter, dtype, "k")
    np.testing.assert_array_equal(_np(t["vc"]), vr)
    assert status == want_status


@pytest.mark.parametrize("c", APPENDS, ids=[f"{c[0]}-D{c[3]}-rot{c[4]}-{'pairs' if c[5] else 'halves'}-b{c[6]}" for c in APPENDS])
@pytest.mark.parametrize("lead", [0, 5])
def test_append_matches_oracle(c, lead):
    import torch
    st = lib()
    t = _case(c, seed=len(c[7]) + c[3], lead=lead)
    kc0, vc0 = _np(t["kc"]), _np(t["vc"])
    q_out = torch.full(t["q"].shape, 7.0, dtype=t["q"].dtype, device="cuda")
    q0 = _np(q_out)
    out, ws = _append(st, c, t, q_out=q_out)
    assert out is q_out
    _check(c, t, kc0, vc0, out, q0, st.spec_read_device_status(ws))


def test_append_without_queries_and_without_rows():
    st = lib()
    c = APPENDS[1]
    t = _case(c, seed=3)
    ref = {k: t[k].clone() for k in ("kc", "vc")}
    _append(st, c, {**t, **ref})
    none, _ = _append(st, c, {**t, "q": None})
    assert none is None
    assert (t["kc"] == ref["kc"]).all() and (t["vc"] == ref["vc"]).all()
    empty = {**t, **{k: t[k][:0] for k in "qkv"}, "start": np.zeros(len(c[7]) + 1, dtype=int)}
    before = t["kc"].clone()
    q, ws = _append(st, c, empty)
    assert q.shape[0] == 0 and st.spec_read_device_status(ws) == 0 and (t["kc"] == before).all()


def test_far_positions_keep_their_angle():
    """At position 2^22 the angle's product needs more than 32 bits."""
    st = lib()
    c = ("f32", 2, 1, 64, 64, False, 64, (2,), (0,), 1 << 30)
    t = _case(c, tail=0)
    t["L"] = np.array([(1 << 22) - 2])
    width = (1 << 22) // 64
    t["table"] = np.zeros((1, width), dtype=int)
    t["table"][0, -1] = 1
    t["kc"], t["vc"] = t["kc"][:2].clone(), t["vc"][:2].clone()
    kc0, vc0 = _np(t["kc"]), _np(t["vc"])
    q, ws = _append(st, c, t)
    _check(c, t, kc0, vc0, q, _np(q), st.spec_read_device_status(ws))


def test_sequences_that_do_not_fit_are_left_out_and_reported():
    import torch
    st = lib()
    c = ("bf16", 4, 2, 64, 64, False, 16, (4, 3, 20, 2), (0, 0, 3, 0), 0)
    t = _case(c, seed=9)
    width = t["table"].shape[1]
    t["L"] = np.array([width * 16 - 3, -1, 3, 0])    # past the end, negative, one bad page, fine
    t["table"][2, 1] = len(t["kc"])
    kc0, vc0 = _np(t["kc"]), _np(t["vc"])
    q_out = torch.full(t["q"].shape, 7.0, dtype=t["q"].dtype, device="cuda")
    q0 = _np(q_out)
    _, ws = _append(st, c, t, q_out=q_out)
    _check(c, t, kc0, vc0, q_out, q0, st.spec_read_device_status(ws), want_status=1)
    t["L"], t["table"] = np.zeros(4, dtype=int), np.arange(4 * width).reshape(4, width) % len(t["kc"])
    _, ws = _append(st, c, t, q_out=q_out, ws=ws)    # the next call clears the word
    assert st.spec_read_device_status(ws) == 0


def test_offsets_outside_the_rows_are_reported():
    st = lib()
    c = APPENDS[0]
    t = _case(c, tail=0)
    t["start"] = np.array([0, 1, 2, 9])
    _, ws = _append(st, c, t)
    assert st.spec_read_device_status(ws) == 1
    t["start"] = np.array([0, 2, 1, 3])
    _, ws = _append(st, c, t)
    assert st.spec_read_device_status(ws) == 1


def test_many_sequences_are_found():
    st = lib()
    B = 2500
    rng = np.random.default_rng(2)
    new = rng.integers(0, 4, size=B)
    c = ("f32", 1, 1, 8, 8, False, 0, tuple(int(n) for n in new), tuple(int(n) for n in rng.integers(0, 5, size=B)), 0)
    t = _case(c, seed=4)
    kc0, vc0 = _np(t["kc"]), _np(t["vc"])
    q, ws = _append(st, c, t)
    written = np.zeros(len(t["q"]), dtype=bool)
    written[:int(new.sum())] = True
    q0 = _np(q)
    _check(c, t, kc0, vc0, q, q0, st.spec_read_device_status(ws))


TREES = [
    # dtype, B, T, Hq, Hkv, D, rot, interleaved, base
    ("bf16", 1, 64, 32, 32, 128, 128, False, None),
    ("bf16", 5, 1, 8, 2, 128, 128, True, 100),     # single tokens
    ("f32", 3, 17, 6, 2, 64, 32, False, 0),
    ("bf16", 2, 130, 4, 1, 80, 20, True, 9),
    ("f32", 2, 5, 2, 1, 4, 2, False, None),
]


@pytest.mark.parametrize("c", TREES, ids=[f"{c[0]}-B{c[1]}-T{c[2]}-D{c[5]}-rot{c[6]}" for c in TREES])
def test_tree_rope_matches_oracle(c):
    import torch
    st = lib()
    dtype, B, T, Hq, Hkv, D, rot, inter, base = c
    rng = np.random.default_rng(T)
    g = torch.Generator().manual_seed(T)
    parent, rank = wl.random_tree(rng, T, max_children=3) if T > 1 else ([-1], [0])
    depth = wl.tree_depths(parent)
    tree = st.spec_tree_build(list(parent), list(rank))
    x = _rand(g, dtype, B, T, Hq + 2 * Hkv, D)
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    L = rng.integers(0, 5000, size=B)
    freq = 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    got = st.tree_rope(q, k, v, _dev32(L), tree, freq=torch.tensor(freq, device="cuda"), interleaved=inter,
                       pos_base=None if base is None else _dev32([base]))
    ref = rope.tree_rope(_np(q), _np(k), _np(v), L, depth, freq, inter, base or 0)
    for name, a, b, r in zip("qk", got, ref, (q, k)):
        _assert_rotated(_np(a), b, np.moveaxis(_np(r), 1, 2), freq, inter, dtype, name)
    np.testing.assert_array_equal(_np(got[2]), ref[2])


def test_replays_follow_the_lengths_and_another_stream_gives_the_same():
    import torch
    st = lib()
    c = APPENDS[7]
    t = _case(c, seed=12)
    q_out = torch.empty(t["q"].shape, dtype=t["q"].dtype, device="cuda")
    ws = torch.empty(st.kv_append_workspace_size(), dtype=torch.uint8, device="cuda")
    L, start, table = _dev32(t["L"]), _dev32(t["start"]), _dev32(t["table"])
    freq = torch.tensor(t["freq"], device="cuda")
    kc, vc = t["kc"].clone(), t["vc"].clone()

    def call(kc, vc, stream=None):
        return st.kv_append_paged(t["q"], t["k"], t["v"], start, L, kc, vc, table, freq=freq, interleaved=True, q_out=q_out,
                                  ws=ws, stream=stream)
    call(kc, vc)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(kc, vc)
    for step in (0, 1):
        L.copy_(_dev32(np.maximum(t["L"] - step, 0)))
        kc.copy_(t["kc"])
        vc.copy_(t["vc"])
        g.replay()
        torch.cuda.synchronize()
        got = (kc.clone(), vc.clone(), q_out.clone())
        k2, v2 = t["kc"].clone(), t["vc"].clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        call(k2, v2, stream=side)
        side.synchronize()
        for a, b in zip(got, (k2, v2, q_out)):
            assert torch.equal(a, b)
        assert st.spec_read_device_status(ws) == 0


def test_binding_refuses():
    import torch
    st = lib()
    c = APPENDS[1]
    t = _case(c)
    z = torch.zeros
    with pytest.raises(ValueError, match="dense"):
        _append(st, c, {**t, "k": t["k"].transpose(1, 2).contiguous().transpose(1, 2)} if t["k"].shape[1] > 1 else
                {**t, "q": z(t["q"].shape[0], 128, 7, device="cuda", dtype=torch.bfloat16).transpose(1, 2)})
    with pytest.raises(ValueError, match="seq_start"):
        _append(st, c, {**t, "start": t["start"][:-1]})
    with pytest.raises(TypeError):
        _append(st, c, {**t, "v": t["v"].float()})
    with pytest.raises(ValueError, match="evenly spaced"):
        x = z(3, 4, 2, 64, device="cuda")[:, :3]
        st.tree_rope(x, x, x, _dev32([0, 0, 0]), st.spec_tree_build([-1, 0, 0]))
    with pytest.raises(st.SpecError, match="overlaps"):
        x = z(6, 2, 64, device="cuda")
        kc = z(1, 2, 9, 64, device="cuda")
        st.kv_append(x, x, x, _dev32([0, 6]), _dev32([0]), kc, kc.clone(), q_out=x)


def test_single_rows_and_odd_strides():
    """One token of one sequence, tokens far apart, and a batch without tokens in front of one that has them."""
    import torch
    st = lib()
    g = torch.Generator().manual_seed(1)
    for dtype in ("bf16", "f32"):
        wide = _rand(g, dtype, 9, 40, 64)                      # tokens 40 heads apart
        q, k, v = wide[::4, :6], wide[::4, 6:8], wide[::4, 8:10]   # three tokens, every fourth row
        freq = 100.0 ** (-np.arange(16) / 16)
        kc, vc = _rand(g, dtype, 4, 2, 8, 64), _rand(g, dtype, 4, 2, 8, 64)
        k0, v0 = _np(kc), _np(vc)
        start, L = _dev32([0, 0, 1, 1, 3]), _dev32([3, 7, 8, 5])
        q_out, ws = st.kv_append(q, k, v, start, L, kc, vc, freq=torch.tensor(freq, device="cuda"), interleaved=True)
        assert st.spec_read_device_status(ws) == 0
        ref_q, ref_k, ref_v, _ = rope.kv_append(_np(q), _np(k), _np(v), [0, 0, 1, 1, 3], [3, 7, 8, 5], k0, v0, freq, interleaved=True)
        _assert_rotated(_np(q_out), ref_q, _np(q), freq, True, dtype, "q")
        untouched = np.ones(k0.shape[:1] + k0.shape[2:3], dtype=bool)
        untouched[1, 7] = untouched[3, 5] = untouched[3, 6] = False
        for got, ref, old in ((_np(kc), ref_k, k0), (_np(vc), ref_v, v0)):
            assert (got.transpose(0, 2, 1, 3)[untouched] == old.transpose(0, 2, 1, 3)[untouched]).all()
        _assert_rotated(_np(kc)[1, :, 7], ref_k[1, :, 7], _np(k)[0], freq, True, dtype, "k")
        _assert_rotated(_np(kc)[3, :, 5:7].transpose(1, 0, 2), ref_k[3, :, 5:7].transpose(1, 0, 2), _np(k)[1:], freq, True, dtype, "k")
        assert (_np(vc)[3, :, 5:7] == ref_v[3, :, 5:7]).all()


@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("start", [(0, 1, 2, 9), (0, 1, 2, 4), (-5, 1, 2, 3), (-1, 0, 3, 3), (0, 3, 3, 10), (-2, 12)],
                         ids=lambda s: "_".join(map(str, s)))
def test_sequences_with_offsets_outside_the_rows_are_left_alone(start, block):
    """Their caches and queries keep their bits, though their tokens would fit and some of their rows are there."""
    import torch
    st = lib()
    new = tuple(b - a for a, b in zip(start, start[1:]))
    c = ("bf16", 4, 2, 64, 64, False, block, new, (3, 14, 7)[:len(new)], 5)
    t = _case(c, seed=6)
    t.update({n: t[n][:3] for n in "qkv"}, start=np.array(start))
    kc0, vc0 = _np(t["kc"]), _np(t["vc"])
    q_out = torch.full(t["q"].shape, 7.0, dtype=t["q"].dtype, device="cuda")
    q0 = _np(q_out)
    out, ws = _append(st, c, t, q_out=q_out)
    _check(c, t, kc0, vc0, out, q0, st.spec_read_device_status(ws), want_status=1)


@pytest.mark.parametrize("block", [0, 16])
def test_decreasing_offsets_write_no_row_but_the_sequences_own(block):
    """Rows 1 of three belongs to two sequences: either may get it, in its own place, and nothing else changes."""
    st = lib()
    c = ("f32", 2, 1, 16, 0, False, block, (2, 0, 2), (3, 14, 7), 0)
    t = _case(c, seed=7)
    t.update({n: t[n][:3] for n in "qkv"}, start=np.array([0, 2, 1, 3]))
    before = {"kc": _np(t["kc"]), "vc": _np(t["vc"])}
    _, ws = _append(st, c, t)
    assert st.spec_read_device_status(ws) == 1
    for name, x in (("kc", _np(t["k"])), ("vc", _np(t["v"]))):
        got, mine = _np(t[name]), {}
        for b, at, n in ((0, 3, 0), (0, 4, 1), (2, 7, 1), (2, 8, 2)):
            mine[(b, at) if not block else (int(t["table"][b, at // block]), at % block)] = x[n]
        for i in range(got.shape[0]):
            for j in range(got.shape[2]):
                if (got[i, :, j] != before[name][i, :, j]).any():
                    np.testing.assert_array_equal(got[i, :, j], mine[i, j])
