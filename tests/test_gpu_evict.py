"""Attention weight of cached keys and eviction by it: CUDA path vs the oracle (GPU).

Tolerance of a key's weight, for the sum over rows of w = exp(scale q.k - lse): the product's D terms are exact
and summed in 32 bits (D 2^-24 scale |q||k| at most), scaled, subtracted and brought to base 2 (4 roundings of 2^-24 of
scale |q||k| + |lse|), exp2 and its argument's rounding within 2^-20, and the sum's roundings, 2^-24 times the rows in a row of
one thread (at most all).  The oracle gives the sum of w (scale |q||k| + |lse|).  Evictions are copies and exact.
"""

import numpy as np
import pytest

from gpu_util import lib
from oracle import evict

pytestmark = pytest.mark.gpu


def _dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _i32(a):
    return _dev(np.asarray(a, dtype=np.int32))


def _f(dtype):
    import torch
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _pages(rng, B, width, spare=2):
    return rng.permutation(B * width + spare)[:B * width].reshape(B, width).astype(np.int32)


WEIGHS = [
    # dtype, B, Hq, Hkv, T, D, block (0: contiguous), lengths, rows (n_rows, or "path"), decay
    ("bf16", 3, 16, 2, 1, 128, 64, (1, 64, 300), None, 1.0),                 # one token each
    ("bf16", 2, 8, 8, 1, 64, 0, (129, 5), None, 0.9),
    ("f32", 2, 4, 2, 1, 64, 16, (33, 100), None, 1.0),
    ("bf16", 4, 16, 2, 40, 128, 0, (700, 17, 4, 128), "path", 0.98),
    ("f32", 2, 6, 2, 20, 128, 48, (150, 9), "path", 0.5),
    ("bf16", 2, 8, 1, 200, 128, 16, (256, 200), (200, 0), 1.0),              # a prompt and a sequence without rows
    ("bf16", 3, 4, 4, 130, 64, 0, (130, 400, 129), (130, 129, 1), 0.0),      # forgetting what was there
    ("f32", 2, 4, 2, 70, 64, 0, (100, 70), (33, 70), 1.0),
    ("bf16", 1, 71, 1, 1, 64, 0, (1000,), None, 1.0),                        # one KV head for many
    ("bf16", 1, 3, 3, 513, 128, 0, (777,), (500,), 1.0),
    ("bf16", 1, 64, 2, 17, 128, 128, (333,), "path", 1.0),                   # 32 heads times a deep path
    ("f32", 1, 1, 1, 1, 64, 0, (1,), None, 1.0),                             # the smallest
    ("bf16", 2, 7, 7, 33, 128, 80, (320, 161), (33, 20), 1.0),               # blocks that are no power of two
]


def _case(c, seed=0):
    import torch
    dtype, B, Hq, Hkv, T, D, block, n, rows, decay = c
    rng = np.random.default_rng(seed + B * 1000 + T)
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g).to(_f(dtype)).cuda()  # noqa: E731
    Lmax = max(n) + 5
    table = None
    t = {"dtype": dtype, "n": np.array(n), "decay": decay}
    if block:
        width = -(-Lmax // block)
        table = _pages(rng, B, width)
        Lmax = width * block
        t["k"] = rand(B * width + 2, Hkv, block, D)
    else:
        t["k"] = rand(B, Hkv, Lmax, D)
    t["q"], t["table"] = rand(B, Hq, T, D), table
    t["path"], t["n_rows"] = None, None
    if rows == "path":
        P = min(T, 17)
        m = [min(int(x), int(rng.integers(1, P + 1))) for x in n]
        m[0] = min(P, n[0])
        t["path"] = [sorted(rng.choice(T, x, replace=False).tolist()) for x in m]
        t["accept_len"] = _i32([x - 1 for x in m])
        t["accept_path"] = _i32([p + [-1] * (P - len(p)) for p in t["path"]])
    elif rows is not None:
        t["n_rows"] = np.array(rows)
    t["acc"] = rng.random((B, Hkv, Lmax)).astype(np.float32)
    t["pos"] = rng.integers(0, 99, (B, Hkv, Lmax)).astype(np.int32)
    t["seen"] = t["n"] + 7
    # lse as the attention leaves it: of what each row sees, for those that count
    lse = np.full((B, Hq, T), np.nan, dtype=np.float32)
    q, k = t["q"].double().cpu().numpy(), t["k"].double().cpu().numpy()
    for b in range(B):
        which = t["path"][b] if t["path"] is not None else list(range(T if rows is None else rows[b]))
        first = n[b] - len(which)
        for h in range(Hkv):
            K = evict._line(k, b, h, n[b], table)
            for hq in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                for i, node in enumerate(which):
                    s = K[:first + i + 1] @ q[b, hq, node] * D ** -0.5
                    lse[b, hq, node] = s.max() + np.log(np.exp(s - s.max()).sum())
    t["lse"] = lse
    return t


def _run(st, t, ws=None, lse=None, acc=None, pos=None, **kw):
    acc, pos = _dev(t["acc"]) if acc is None else acc, _dev(t["pos"]) if pos is None else pos
    more = dict(pos=pos, seen=_i32(t["seen"]), decay=t["decay"], ws=ws, **kw)
    if t["path"] is not None:
        more |= dict(accept_len=t["accept_len"], accept_path=t["accept_path"])
    elif t["n_rows"] is not None:
        more |= dict(n_rows=_i32(t["n_rows"]))
    lse = _dev(t["lse"]) if lse is None else lse
    if t["table"] is not None:
        st.kv_weigh_paged(t["q"], lse, t["k"], _i32(t["table"]), _i32(t["n"]), acc, **more)
    else:
        st.kv_weigh(t["q"], lse, t["k"], _i32(t["n"]), acc, **more)
    return acc, pos


def _assert_weighed(t, acc, pos, lse=None):
    q, k = t["q"].double().cpu().numpy(), t["k"].double().cpu().numpy()
    want, wpos, size = evict.kv_weigh(q, t["lse"] if lse is None else lse, k, t["n"], t["acc"], t["pos"], seen=t["seen"], n_rows=t["n_rows"],
                                      path=t["path"], decay=t["decay"], table=t["table"])
    D, rows = q.shape[3], q.shape[1] // t["acc"].shape[1] * q.shape[2]
    new = np.abs(want) + np.abs(t["acc"])
    tol = (D + 4) * 2.0 ** -24 * size + (2.0 ** -20 + (rows + 4) * 2.0 ** -24) * new
    got = acc.cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.nanmax(np.abs(got - want)):.3e}"
    np.testing.assert_array_equal(pos.cpu().numpy(), wpos)
    for b in range(len(t["n"])):
        np.testing.assert_array_equal(got[b, :, t["n"][b]:], t["acc"][b, :, t["n"][b]:])


@pytest.mark.parametrize("c", WEIGHS, ids=lambda c: "-".join(map(str, c[:7])))
def test_weights(c):
    import torch
    st = lib()
    t = _case(c)
    dtype, B, Hq, Hkv, T, D = c[:6]
    cap = t["acc"].shape[2]
    P = 0 if t["path"] is None else t["accept_path"].shape[1]
    ws = torch.empty(st.kv_weigh_workspace_size(B, Hq, Hkv, T, P, cap, D, 1 if dtype == "bf16" else 0), dtype=torch.uint8, device="cuda").fill_(255)
    acc, pos = _run(st, t, ws)
    assert st.spec_read_device_status(ws) == 0
    _assert_weighed(t, acc, pos)
    again, _ = _run(st, t, ws)
    assert torch.equal(again, acc)                   # the same to the last bit


@pytest.mark.parametrize("c", [WEIGHS[0], WEIGHS[3], WEIGHS[5], WEIGHS[7]], ids=lambda c: "-".join(map(str, c[:7])))
def test_what_no_row_sees_does_not_count(c):
    """Keys behind the lengths and rows that do not count hold NaN and infinities; rows that saw nothing have no lse."""
    import torch
    st = lib()
    t = _case(c, seed=1)
    B, T = t["q"].shape[0], t["q"].shape[2]
    k, q = t["k"], t["q"]
    for b in range(B):
        for j in range(int(t["n"][b]), t["acc"].shape[2]):
            row = k[b, :, j] if t["table"] is None else k[t["table"][b, j // k.shape[2]], :, j % k.shape[2]]
            row.fill_(float("nan") if j % 2 else float("inf"))
        which = t["path"][b] if t["path"] is not None else range(T if t["n_rows"] is None else t["n_rows"][b])
        for i in set(range(T)) - set(which):
            q[b, :, i] = float("nan")
    if c[3] > 1:
        t["lse"][0, ::2] = -np.inf                   # every other head of the first sequence saw nothing
    t["acc"][:, :, -1] = np.nan
    acc, pos = _run(st, t)
    q2 = torch.nan_to_num(q)
    t["q"] = q2
    t["k"] = torch.nan_to_num(k, nan=0.0, posinf=0.0)
    got = acc.cpu().numpy()
    assert np.isnan(got[:, :, -1]).all()
    t["acc"][:, :, -1] = got[:, :, -1] = 0.0
    _assert_weighed(t, _dev(got), pos)


@pytest.mark.parametrize("c", [("bf16", 2, 16, 2, 1, 128, 64, (400, 129), None, 1.0), ("bf16", 2, 4, 2, 300, 64, 0, (900, 300), (300, 257), 0.5),
                               ("bf16", 2, 24, 1, 20, 128, 0, (500, 50), "path", 1.0), ("f32", 2, 4, 2, 40, 64, 16, (100, 70), None, 1.0)],
                         ids=lambda c: "-".join(map(str, c[:7])))
def test_rows_without_an_lse_may_hold_anything(c):
    """Rows among those that count, but whose lse is not finite: NaN and infinities in them weigh nothing."""
    st = lib()
    t = _case(c, seed=7)
    B, Hq, T = c[1], c[2], c[4]
    rng = np.random.default_rng(8)
    q = t["q"].clone()
    for b in range(B):
        for h in range(Hq):
            for i in {0, T - 1, *rng.integers(0, T, 3).tolist()} if h % 3 == 0 else {int(rng.integers(0, T))} if T > 1 else ():
                t["lse"][b, h, i] = (-np.inf, np.inf, np.nan)[(h + i) % 3]
                q[b, h, i] = float("nan") if i % 2 else float("inf")
    acc, pos = _run(st, {**t, "q": q})
    _assert_weighed(t, acc, pos)


@pytest.mark.parametrize("dtype,T", [("bf16", 1), ("bf16", 200), ("f32", 30)])
def test_a_sequence_without_rows_fades(dtype, T):
    st = lib()
    t = _case((dtype, 2, 8, 2, T, 64, 16, (300, 250), (0, T), 0.5), seed=5)
    acc, pos = _run(st, t)
    _assert_weighed(t, acc, pos)
    np.testing.assert_array_equal(acc[0].cpu().numpy()[:, :300], 0.5 * t["acc"][0, :, :300])


@pytest.mark.parametrize("T,Hq,Hkv", [(95, 8, 2), (96, 8, 2), (129, 5, 1), (64, 24, 3), (385, 2, 1)])
@pytest.mark.parametrize("n", [(1000, 400, 500), (385, 513, 640)])
def test_both_ways_through_and_their_borders(T, Hq, Hkv, n):
    """Short prompts side by side and long ones in chunks, lengths around the tiles' borders, rows cut over many CTAs."""
    st = lib()
    t = _case(("bf16", 3, Hq, Hkv, T, 128, 0, n, (T, max(1, T - 37), min(T, 3)), 0.9), seed=6)
    ws = _ws(t)
    acc, pos = _run(st, t, ws)
    assert st.spec_read_device_status(ws) == 0
    _assert_weighed(t, acc, pos)


@pytest.mark.parametrize("T,Hq,Hkv", [(47, 12, 2), (48, 12, 2), (48, 5, 1), (79, 3, 1), (80, 3, 1), (63, 32, 1)])
@pytest.mark.parametrize("n", [(300, 80, 129), (80, 1200, 513)])
def test_short_prompts_on_both_sides_of_the_choice(T, Hq, Hkv, n):
    st = lib()
    t = _case(("bf16", 3, Hq, Hkv, T, 64, 0, n, (T, min(T, 50), 0), 0.5), seed=9)
    ws = _ws(t)
    acc, pos = _run(st, t, ws)
    assert st.spec_read_device_status(ws) == 0
    _assert_weighed(t, acc, pos)


def _ws(t):
    import torch
    return torch.empty(1 << 20, dtype=torch.uint8, device="cuda").fill_(255)


def test_sequences_and_blocks_that_make_no_sense():
    import torch
    st = lib()
    c = ("bf16", 6, 4, 2, 20, 64, 16, (30, 30, 30, 30, 30, 30), "path", 0.5)
    t = _case(c, seed=2)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    keep = t["n"].copy()
    t["n"] = np.array([30, -1, 5000, 30, 2, 30])
    al, ap = t["accept_len"].cpu().numpy(), t["accept_path"].cpu().numpy()
    al[3], al[4] = 17, 5
    ap[4, :6] = range(6)
    ap[5, 0] = 20
    t["accept_len"], t["accept_path"] = _i32(al), _i32(ap)
    acc, pos = _run(st, t, ws)
    assert st.spec_read_device_status(ws) == 1
    np.testing.assert_array_equal(acc[1:].cpu().numpy(), t["acc"][1:])
    np.testing.assert_array_equal(pos[1:].cpu().numpy(), t["pos"][1:])
    one = {**t, "n": keep[:1], "path": t["path"][:1], "q": t["q"][:1], "lse": t["lse"][:1], "acc": t["acc"][:1], "pos": t["pos"][:1],
           "table": t["table"][:1], "seen": t["seen"][:1]}
    one["seen"] = t["seen"][:1]
    _assert_weighed(one, acc[:1], pos[:1])
    # a block outside the pool: its keys keep what they have
    t = _case(("bf16", 2, 4, 2, 1, 64, 16, (100, 100), None, 0.5), seed=3)
    good, _ = _run(st, t, ws)
    assert st.spec_read_device_status(ws) == 0
    table = t["table"].copy()
    table[0, 2], table[1, 0] = -1, t["k"].shape[0]
    acc, pos = _run(st, {**t, "table": table}, ws)
    assert st.spec_read_device_status(ws) == 1
    want = good.cpu().numpy()
    want[0, :, 32:48], want[1, :, :16] = t["acc"][0, :, 32:48], t["acc"][1, :, :16]
    np.testing.assert_array_equal(acc.cpu().numpy(), want)


def test_prompts_weigh_the_same_in_one_piece_or_two():
    import torch
    st = lib()
    t = _case(("bf16", 1, 8, 2, 300, 128, 0, (300,), None, 1.0), seed=4)
    whole, pos = _run(st, t)
    acc, pos2 = _dev(t["acc"]), _dev(t["pos"])
    lse = _dev(t["lse"])
    for a, z in ((0, 111), (111, 300)):
        st.kv_weigh(t["q"][:, :, a:z].contiguous(), lse[:, :, a:z].contiguous(), t["k"], _i32([z]), acc, pos=pos2, seen=_i32([z + 7]))
    assert torch.equal(pos2, pos)
    np.testing.assert_allclose(acc[:, :, :300].cpu().numpy(), whole[:, :, :300].cpu().numpy(), rtol=2.0 ** -20 + 600 * 2.0 ** -24)


EVICTS = [
    # dtype, B, Hkv, D, block (0: contiguous), lengths, budget, sink, recent
    ("bf16", 3, 2, 128, 0, (40, 33, 20), 32, 4, 8),                   # one below the budget
    ("bf16", 2, 3, 64, 16, (2065, 2050), 2048, 4, 64),                # a step of a full cache
    ("f32", 2, 2, 20, 7, (500, 133), 60, 0, 0),
    ("bf16", 1, 2, 128, 64, (30000,), 1000, 4, 100),
    ("f32", 2, 1, 4, 0, (70000, 69), 40001, 3, 50),                   # more keys than ranks fit shared memory
    ("bf16", 1, 1, 8, 0, (300,), 64, 0, 64),                          # nothing but the last keys
    ("f32", 1, 1, 4, 0, (1,), 1, 0, 0),                               # the smallest
    ("bf16", 2, 1, 8, 0, (700, 0), 1, 0, 1),
    ("bf16", 2, 2, 16, 0, (900, 513), 512, 100, 412),                 # protected keys fill the budget
    ("f32", 1, 2, 8, 0, (5000,), 4900, 1, 3),
]


def _cache(c, seed, ties):
    import torch
    dtype, B, H, D, block, n, budget, sink, recent = c
    rng = np.random.default_rng(seed + budget)
    Lmax = max(n) + 2
    table = None
    if block:
        width = -(-Lmax // block)
        table, Lmax = _pages(rng, B, width), width * block
        shape = (B * width + 2, H, block, D)
    else:
        shape = (B, H, Lmax, D)
    k, v = (torch.randn(shape, device="cuda").to(_f(dtype)) for _ in range(2))
    acc = rng.exponential(1.0, (B, H, Lmax)).astype(np.float32)
    if ties == "few":
        acc = np.round(acc)
    elif ties == "all":
        acc[:] = 0.0
    elif ties == "odd":
        acc *= rng.choice([-1.0, 1.0, 0.0, np.inf, np.nan], acc.shape).astype(np.float32)
    pos = np.argsort(rng.random((B, H, Lmax)), -1).astype(np.int32)
    return k, v, acc, pos, table, np.array(n, dtype=np.int32)


@pytest.mark.parametrize("into", [False, True])
@pytest.mark.parametrize("ties", ["none", "few", "all", "odd"])
@pytest.mark.parametrize("c", EVICTS, ids=lambda c: "-".join(map(str, c[:5] + c[6:7])))
def test_evictions(c, ties, into):
    import torch
    st = lib()
    dtype, B, H, D, block, _, budget, sink, recent = c
    k, v, acc, pos, table, n = _cache(c, 0, ties)
    seen = n + 3
    Lmax = acc.shape[2]
    ws = torch.empty(st.kv_evict_workspace_size(B, H, Lmax, budget), dtype=torch.uint8, device="cuda").fill_(255)
    more = dict(seen=_i32(seen), sink=sink, recent=recent, ws=ws)
    args = dict(seen=seen, sink=sink, recent=recent)
    num = lambda t: t.float().cpu().numpy()  # noqa: E731
    da, dp, dn = _dev(acc), _dev(pos), _dev(n)
    if not into:
        want = evict.kv_evict(num(k), num(v), acc, pos, n, budget, table=table, **args)
        m = st.kv_evict_paged(k, v, _dev(table), dn, da, dp, budget, **more) if block else st.kv_evict(k, v, dn, da, dp, budget, **more)
        got = (k, v, da, dp)
    elif block:
        width = -(-budget // block)
        first = k.shape[0]
        k, v = (torch.cat([t, torch.full((B * width, *t.shape[1:]), 7.0, device="cuda", dtype=t.dtype)]) for t in (k, v))
        out_table = first + np.random.default_rng(1).permutation(B * width).reshape(B, width).astype(np.int32)
        oa, op = np.full((B, H, width * block), 5.0, dtype=np.float32), np.full((B, H, width * block), -9, dtype=np.int32)
        want = evict.kv_evict(num(k), num(v), acc, pos, n, budget, table=table, out=(oa, op), out_table=out_table, **args)
        oa, op = _dev(oa), _dev(op)
        m = st.kv_evict_paged(k, v, _dev(table), dn, da, dp, budget, out_table=_dev(out_table.astype(np.int32)), acc_out=oa, pos_out=op, **more)
        got = (k, v, oa, op)
    else:
        out = budget + 3
        ko, vo = (torch.full((B, H, out, D), 7.0, device="cuda", dtype=k.dtype) for _ in range(2))
        oa, op = np.full((B, H, out), 5.0, dtype=np.float32), np.full((B, H, out), -9, dtype=np.int32)
        want = evict.kv_evict(num(k), num(v), acc, pos, n, budget, out=(num(ko), num(vo), oa, op), **args)
        oa, op = _dev(oa), _dev(op)
        before = k.clone()
        m = st.kv_evict(k, v, dn, da, dp, budget, k_out=ko, v_out=vo, acc_out=oa, pos_out=op, **more)
        assert torch.equal(k, before) and np.array_equal(da.cpu().numpy(), acc, equal_nan=True)
        got = (ko, vo, oa, op)
    assert st.spec_read_device_status(ws) == 0
    for g, w, name in zip((*got, m), want, ("k", "v", "acc", "pos", "len")):
        np.testing.assert_array_equal(num(g) if name in "kv" else g.cpu().numpy(), w, err_msg=name)


def test_lengths_and_blocks_that_make_no_sense():
    import torch
    st = lib()
    c = ("bf16", 4, 2, 64, 16, (100, 100, 100, 100), 30, 0, 0)
    k, v, acc, pos, table, n = _cache(c, 1, "none")
    n[1], n[2] = -4, acc.shape[2] + 1
    table[3, 5] = k.shape[0]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    safe = table.copy()
    safe[3] = 0
    want = evict.kv_evict(k.float().cpu().numpy(), v.float().cpu().numpy(), acc[:1], pos[:1], n[:1], 30, table=safe[:1])
    da, dp = _dev(acc), _dev(pos)
    m = st.kv_evict_paged(k, v, _dev(table), _dev(n), da, dp, 30, ws=ws)
    assert st.spec_read_device_status(ws) == 1 and m.tolist() == [30, -4, acc.shape[2] + 1, 100]
    np.testing.assert_array_equal(k.float().cpu().numpy(), want[0])
    np.testing.assert_array_equal(v.float().cpu().numpy(), want[1])
    np.testing.assert_array_equal(da.cpu().numpy(), np.concatenate([want[2], acc[1:]]))
    np.testing.assert_array_equal(dp.cpu().numpy(), np.concatenate([want[3], pos[1:]]))


def test_steps_of_a_bounded_cache():
    """Verification steps whose accepted nodes are committed, weighed and evicted, captured in a graph: lse, cache, weights and
    positions are the oracle's at every step."""
    import torch
    st = lib()
    B, Hq, Hkv, D, budget, steps = 2, 8, 2, 64, 40, 6
    parent = [-1, 0, 0, 1, 1, 3]
    T, P = len(parent), 4
    tree = st.spec_tree_build(parent)
    cap = budget + P
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    k, v = (torch.randn(B, Hkv, cap, D, device="cuda") for _ in range(2))
    acc, pos = torch.rand(B, Hkv, cap, device="cuda"), torch.arange(cap, device="cuda", dtype=torch.int32).expand(B, Hkv, cap).contiguous()
    n, seen = _i32([budget - 2, 17]), _i32([budget + 5, 17])
    q, kt, vt = f(B, Hq, T, D), f(B, Hkv, T, D), f(B, Hkv, T, D)
    alen, path = _i32([0, 0]), _i32([[0, -1, -1, -1]] * B)
    out, lse = f(B, Hq, T, D), f(B, Hq, T)
    wss = [torch.empty(1 << 22, dtype=torch.uint8, device="cuda") for _ in range(4)]
    m = _i32([0, 0])

    def step():
        st.tree_attention(q, k, v, n, kt, vt, tree, out=out, lse=lse, ws=wss[0])
        st.tree_kv_commit(kt, vt, k, v, n, alen, path, tree, ws=wss[1])
        seen.add_(alen + 1)
        st.kv_weigh(q, lse, k, n, acc, pos=pos, seen=seen, accept_len=alen, accept_path=path, decay=0.9, ws=wss[2])
        st.kv_evict(k, v, n, acc, pos, budget, seen=seen, sink=2, recent=8, len_out=m, ws=wss[3])
        n.copy_(m)
    state = (k, v, acc, pos, n, seen)
    start = [t.clone() for t in state]
    step()
    for t, s in zip(state, start):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    num = lambda t: t.cpu().numpy().copy()  # noqa: E731
    for i in range(steps):
        for t in (q, kt, vt):
            t.copy_(torch.randn(t.shape))
        paths = [[0, 1, 3, 5], [0, 2]] if i % 2 else [[0], [0, 1, 4]]
        alen.copy_(_i32([len(p) - 1 for p in paths]))
        path.copy_(_i32([p + [-1] * (P - len(p)) for p in paths]))
        K, V, A, X, N, S = (num(t) for t in state)
        graph.replay()
        torch.cuda.synchronize()
        assert [st.spec_read_device_status(w) for w in wss] == [0] * 4
        # by hand: attention's lse, the commit, the weights, the eviction
        L = num(lse)
        for b, p in enumerate(paths):
            for j, node in enumerate(p):
                K[b, :, N[b] + j], V[b, :, N[b] + j] = num(kt)[b, :, node], num(vt)[b, :, node]
            for hq in range(Hq):
                for j, node in enumerate(p):
                    s = K[b, hq // 4, :N[b] + j + 1].astype(np.float64) @ num(q)[b, hq, node].astype(np.float64) / 8.0
                    assert abs(s.max() + np.log(np.exp(s - s.max()).sum()) - L[b, hq, node]) < 1e-5
            N[b] += len(p)
            S[b] += len(p)
        A2, X2, _ = evict.kv_weigh(num(q), L, K, N, A, X, seen=S, path=paths, decay=0.9)
        got = num(acc)
        K2, V2, A3, X3, N2 = evict.kv_evict(K, V, A2, X2, N, budget, seen=S, sink=2, recent=8)
        np.testing.assert_array_equal(num(n), N2)
        np.testing.assert_array_equal(num(seen), S)
        for b in range(B):
            np.testing.assert_array_equal(num(pos)[b, :, :N2[b]], X3[b, :, :N2[b]])
            np.testing.assert_array_equal(num(k)[b, :, :N2[b]], K2[b, :, :N2[b]])
            np.testing.assert_array_equal(num(v)[b, :, :N2[b]], V2[b, :, :N2[b]])
            np.testing.assert_allclose(got[b, :, :N2[b]], A3[b, :, :N2[b]], rtol=1e-4)
    assert num(n)[0] == budget
