"""Shared-prefix and scored tree attention: CUDA paths vs the oracle in 64 bits (GPU).

Tolerances, from the arithmetic.  A score is a sum of D products in 32 bits (u = 2^-23
a step, truncation allowed for), so it is off by at most dx = D u size, size = scale sum
|q_i k_i|; the cap adds 8 u cap, the bias 4 u slope far, the base-2 exponential, its
argument's rounding and the rescaling of partial sums 16 u (1 + |x|) with |x| <= size.
Weights then are off by a factor exp(+-2 dx) (their sum as well), sums of n keys by n u.
bf16 rounds every weight once more, by half a step 2^-8, and the output once:
    |out - ref| <= weight (2 dx + n u + [2^-8]) + half step of the output (|ref| + that)
with weight = softmax . |values|; lse: dx + n u + 4 u |lse|.
"""

import itertools

import numpy as np
import pytest

import oracle
import spec_workloads as wl
from gpu_util import lib
from oracle import attention_shared as osh

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _np(t):
    return t.detach().double().cpu().numpy()


def _i32(a):
    import torch
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Case:
    """Inputs on the device, and the calls on them."""

    def __init__(self, dtype, B, Hq, Hkv, D, T, lens, Lmax, Ls=0, block=0, softcap=0.0, window=0, slopes=False, shared_len=None,
                 seed=0, tree="random", gain=1.0):
        import torch
        self.st = lib()
        rng = np.random.default_rng([seed, B, Hq, D, T, Lmax, Ls])
        g = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        rand = lambda *s: torch.randn(*s, generator=g).to(dt).cuda()  # noqa: E731
        if T == 1:
            self.parent = [-1]
        elif tree == "random":
            self.parent = [int(p) for p in wl.random_tree(rng, T, max_depth=14, max_children=6)[0]]
        else:
            self.parent = list(range(-1, T - 1))
        self.tree, self.tree_o = self.st.spec_tree_build(self.parent), oracle.tree_encode(self.parent, None)
        self.dtype, self.B, self.Hkv, self.D, self.Lmax, self.Ls, self.block = dtype, B, Hkv, D, Lmax, Ls, block
        self.lens, self.shared_len = np.array(lens), Ls if shared_len is None else shared_len
        self.q = rand(B, Hq, T, D) * gain
        self.kt, self.vt = rand(B, Hkv, T, D), rand(B, Hkv, T, D)
        self.kc, self.vc = rand(B, Hkv, Lmax, D), rand(B, Hkv, Lmax, D)
        self.ks, self.vs = (rand(Hkv, Ls, D), rand(Hkv, Ls, D)) if Ls else (None, None)
        self.score = {"softcap": softcap, "window": window,
                      "slopes": torch.tensor(rng.uniform(-0.02, 0.5, Hq), dtype=torch.float32).cuda() if slopes else None}
        if block:
            self._page(rng, rand)

    def _page(self, rng, rand):
        import torch
        bs, B = self.block, self.B
        nb, ns = -(-self.Lmax // bs), -(-self.Ls // bs)
        ids = rng.permutation(B * nb + ns + 3)
        self.table, self.stable = ids[:B * nb].reshape(B, nb), ids[B * nb:B * nb + ns]
        self.kp, self.vp = rand(len(ids), self.Hkv, bs, self.D), rand(len(ids), self.Hkv, bs, self.D)
        pad = lambda x, n: torch.nn.functional.pad(x, (0, 0, 0, n - x.shape[-2]))  # noqa: E731
        for pool, own, sh in ((self.kp, self.kc, self.ks), (self.vp, self.vc, self.vs)):
            own = pad(own, nb * bs)
            for b, j in itertools.product(range(B), range(nb)):
                pool[int(self.table[b, j])] = own[b, :, j * bs:(j + 1) * bs]
            if self.Ls:
                sh = pad(sh, ns * bs)
                for j in range(ns):
                    pool[int(self.stable[j])] = sh[:, j * bs:(j + 1) * bs]

    def call(self, **kw):
        """The entry point for this case: (out, lse)."""
        st, L, tree = self.st, kw.pop("L", None), (self.kt, self.vt, self.tree)
        L = _i32(self.lens) if L is None else L
        kw = {**self.score, **kw}
        if self.Ls and self.block:
            return st.tree_attention_shared_paged(self.q, self.kp, self.vp, _i32(self.stable), _i32([self.shared_len]),
                                                  _i32(self.table), L, *tree, **kw)
        if self.Ls:
            return st.tree_attention_shared(self.q, self.ks, self.vs, _i32([self.shared_len]), self.kc, self.vc, L, *tree, **kw)
        if self.block:
            return st.tree_attention_scored_paged(self.q, self.kp, self.vp, _i32(self.table), L, *tree, **kw)
        return st.tree_attention_scored(self.q, self.kc, self.vc, L, *tree, **kw)

    def workspace(self):
        import torch
        st, dt = self.st, 1 if self.dtype == "bf16" else 0
        up = (lambda n: -(-n // self.block) * self.block) if self.block else (lambda n: n)
        a = (self.B, self.q.shape[1], self.Hkv)
        n = st.tree_attention_shared_workspace_size(self.tree, *a, up(self.Ls), up(self.Lmax), self.D, dt) if self.Ls else \
            st.tree_attention_scored_workspace_size(self.tree, *a, up(self.Lmax), self.D, dt)
        return torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda")   # garbage: no call may count on its contents

    def reference(self, scale=None):
        Ls = min(max(self.shared_len, 0), self.Ls)
        sl = self.score["slopes"]
        cut = lambda x: None if not Ls else _np(x)[:, :Ls]  # noqa: E731
        return osh.attention(_np(self.q), _np(self.kc), _np(self.vc), np.clip(self.lens, 0, self.Lmax), _np(self.kt), _np(self.vt),
                             self.tree_o, cut(self.ks), cut(self.vs), scale, self.score["softcap"], self.score["window"],
                             None if sl is None else _np(sl))

    def check(self, out, lse, ref=None):
        ref = self.reference() if ref is None else ref
        far = 0.0 if self.score["slopes"] is None else float(self.score["slopes"].abs().max()) * ref["keys"]
        dx = U * (self.D * ref["size"] + 8 * self.score["softcap"] + 4 * far + 16 * (1 + ref["size"]))
        n = U * ref["keys"]
        near = ref["weight"] * (2 * dx + n + (STEP["bf16"] if self.dtype == "bf16" else 0.0))[..., None]
        tol = near + STEP[self.dtype] * (np.abs(ref["out"]) + near)
        got = _np(out)
        assert np.isfinite(got).all(), "non-finite output"
        bad = np.abs(got - ref["out"]) > tol
        assert not bad.any(), f"out: {bad.sum()} values out of tolerance, worst {np.abs(got - ref['out']).max():.3e}"
        if lse is not None:
            off = np.abs(_np(lse) - ref["lse"])
            assert (off <= dx + n + 4 * U * np.abs(ref["lse"])).all(), f"lse: off by {off.max():.3e}"


CASES = {
    # single tokens, grouped heads, lengths from none to a tile's border and past it
    "tokens": dict(B=5, Hq=8, Hkv=1, D=128, T=1, lens=(0, 1, 127, 128, 300), Lmax=300, Ls=260),
    "tokens-paged-16": dict(B=6, Hq=16, Hkv=2, D=128, T=1, lens=(0, 15, 16, 17, 200, 64), Lmax=200, Ls=130, block=16),
    "tokens-mha": dict(B=3, Hq=4, Hkv=4, D=64, T=1, lens=(5, 64, 65), Lmax=70, Ls=64),
    # more sequences than fit one block of rows, and one that ends inside a block
    "many": dict(B=37, Hq=14, Hkv=2, D=64, T=3, lens=[(7 * i) % 90 for i in range(37)], Lmax=90, Ls=33, block=64),
    # trees
    "tree": dict(B=2, Hq=8, Hkv=2, D=128, T=64, lens=(100, 513), Lmax=600, Ls=700),
    "tree-paged": dict(B=3, Hq=8, Hkv=1, D=128, T=40, lens=(3, 0, 257), Lmax=320, Ls=200, block=64),
    "tree-odd": dict(B=2, Hq=3, Hkv=3, D=128, T=131, lens=(40, 129), Lmax=131, Ls=5),
    "tree-wide": dict(B=1, Hq=2, Hkv=1, D=64, T=300, lens=(77,), Lmax=77, Ls=129, block=16),
    "chain": dict(B=2, Hq=4, Hkv=2, D=64, T=15, lens=(9, 30), Lmax=64, tree="chain", window=4, slopes=True),
    # nothing of the shared part is used, or less than its room
    "shared-none": dict(B=2, Hq=4, Hkv=2, D=128, T=5, lens=(9, 200), Lmax=200, Ls=128, shared_len=0),
    "shared-part": dict(B=2, Hq=4, Hkv=2, D=128, T=5, lens=(9, 200), Lmax=200, Ls=300, shared_len=129, block=64),
    # scores
    "cap": dict(B=2, Hq=8, Hkv=2, D=128, T=9, lens=(300, 17), Lmax=300, softcap=5.0),
    "cap-binding": dict(B=1, Hq=8, Hkv=2, D=128, T=9, lens=(150,), Lmax=160, softcap=2.0, gain=8.0),
    "cap-shared": dict(B=3, Hq=8, Hkv=4, D=64, T=21, lens=(50, 17, 0), Lmax=64, Ls=140, softcap=30.0),
    "window": dict(B=3, Hq=4, Hkv=1, D=128, T=20, lens=(1000, 300, 6), Lmax=1024, window=200, block=16),
    "window-one": dict(B=2, Hq=4, Hkv=2, D=128, T=20, lens=(300, 6), Lmax=300, window=1, Ls=130),
    "window-shared": dict(B=3, Hq=4, Hkv=2, D=128, T=12, lens=(500, 30, 3), Lmax=500, window=100, Ls=300),
    "window-in-shared": dict(B=2, Hq=4, Hkv=2, D=64, T=12, lens=(3, 30), Lmax=64, window=130, Ls=700, block=64),
    "bias": dict(B=2, Hq=8, Hkv=2, D=128, T=33, lens=(511, 40), Lmax=512, slopes=True),
    "bias-shared-paged": dict(B=2, Hq=8, Hkv=2, D=64, T=6, lens=(100, 40), Lmax=128, Ls=200, slopes=True, block=32),
    "everything": dict(B=3, Hq=6, Hkv=2, D=128, T=70, lens=(257, 0, 90), Lmax=260, Ls=150, softcap=10.0, window=300, slopes=True),
    "large-scores": dict(B=2, Hq=4, Hkv=2, D=128, T=8, lens=(400, 129), Lmax=400, gain=12.0),
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(CASES))
def test_matches_oracle(name, dtype):
    c = Case(dtype, **CASES[name])
    ws = c.workspace()
    out, lse = c.call(ws=ws)
    c.check(out, lse)
    assert c.st.spec_read_device_status(ws) == 0
    again, _ = c.call(want_lse=False, ws=ws)       # the same bits from a used workspace
    assert (again == out).all()


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(seed):
    r = np.random.default_rng(1000 + seed)
    Hkv, B, T = int(r.integers(1, 5)), int(r.integers(1, 9)), int(np.exp(r.uniform(0, np.log(200))))
    Lmax = int(r.integers(1, 700))
    Ls = int(r.integers(1, 700)) if r.random() < 0.6 else 0
    c = Case("bf16" if r.random() < 0.75 else "f32", B=B, Hq=Hkv * int(r.integers(1, 9)), Hkv=Hkv, D=int(r.choice([64, 128])), T=T,
             lens=r.integers(0, Lmax + 1, size=B), Lmax=Lmax, Ls=Ls, block=int(r.choice([0, 16, 48, 64, 128])),
             softcap=float(r.choice([0.0, 8.0])), window=int(r.choice([0, 1, 50, 400])), slopes=bool(r.random() < 0.4),
             shared_len=int(r.integers(0, Ls + 1)) if Ls else None, seed=seed)
    c.check(*c.call())


def test_lengths_outside_the_room_are_clamped():
    c = Case("bf16", B=3, Hq=4, Hkv=2, D=128, T=4, lens=(-5, 400, 90), Lmax=200, Ls=100, shared_len=4000)
    c.check(*c.call())


def test_what_is_not_seen_does_not_matter():
    """NaN and infinities behind the lengths, in unused pages and in keys no one sees."""
    import torch
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda")
    for block in (0, 16):
        for dtype in ("bf16", "f32"):
            c = Case(dtype, B=3, Hq=8, Hkv=2, D=128, T=7, lens=(0, 130, 37), Lmax=256, Ls=200, shared_len=150, block=block)
            ref = c.reference()
            if block:
                used = {int(c.table[b, j]) for b in range(3) for j in range(-(-int(c.lens[b]) // block))}
                used |= {int(c.stable[j]) for j in range(-(-150 // block))}
                for t in (c.kp, c.vp):
                    for i in range(len(t)):
                        if i not in used:
                            t[i] = bad[i % 3]
                    for b in range(3):
                        if c.lens[b] % block:
                            t[int(c.table[b, int(c.lens[b]) // block]), :, int(c.lens[b]) % block:] = bad[b]
                    t[int(c.stable[150 // block]), :, 150 % block:] = bad[0]
            else:
                for t in (c.kc, c.vc):
                    for b in range(3):
                        t[b, :, int(c.lens[b]):] = bad[b]
                for t in (c.ks, c.vs):
                    t[:, 150:] = bad[1]
            c.check(*c.call(), ref)


def test_non_finite_trees_stay_in_their_sequence():
    c = Case("bf16", B=3, Hq=8, Hkv=2, D=128, T=7, lens=(30, 130, 37), Lmax=256, Ls=200)
    ref = c.reference()
    c.kt[1], c.vt[1] = float("nan"), float("inf")
    out, lse = c.call()
    assert not np.isfinite(_np(out[1])).any()
    c.lens = c.lens[[0, 2]]
    pick = lambda a: a[[0, 2]] if isinstance(a, np.ndarray) else a  # noqa: E731
    c.check(out[[0, 2]], lse[[0, 2]], {k: pick(v) for k, v in ref.items()})


def test_pages_outside_the_pool_are_reported():
    for dtype in ("bf16", "f32"):
        for where in ("own", "shared"):
            c = Case(dtype, B=2, Hq=4, Hkv=2, D=64, T=3, lens=(40, 33), Lmax=64, Ls=64, block=16)
            good, _ = c.call()
            if where == "own":
                c.table[0, 1] = len(c.kp)
            else:
                c.stable[2] = -1
            ws = c.workspace()
            out, _ = c.call(ws=ws)
            assert c.st.spec_read_device_status(ws) == 1
            if where == "own":
                assert (out[1] == good[1]).all()
            c.table[0, 1], c.stable[2] = 0, 0
            c.call(ws=ws)
            assert c.st.spec_read_device_status(ws) == 0


def test_single_tokens_are_the_one_node_tree():
    """A chain's nodes one at a time, each after its parent entered the cache, equal the chain at once."""
    c = Case("f32", B=2, Hq=4, Hkv=2, D=64, T=6, lens=(10, 41), Lmax=64, Ls=70, tree="chain", window=60, slopes=True)
    ref = c.reference()
    c.check(*c.call(), ref)
    one = c.st.spec_tree_build([-1])
    q, kt, vt = c.q.clone(), c.kt.clone(), c.vt.clone()
    kc, vc, L = c.kc.clone(), c.vc.clone(), c.lens.copy()
    for i in range(6):
        c.q, c.kt, c.vt, c.tree = q[:, :, i:i + 1].contiguous(), kt[:, :, i:i + 1].contiguous(), vt[:, :, i:i + 1].contiguous(), one
        c.kc, c.vc, c.lens = kc, vc, L
        out, lse = c.call()
        c.check(out, lse, {k: v if k == "keys" else v[:, :, i:i + 1] for k, v in ref.items()})
        for b in range(2):
            kc[b, :, L[b]], vc[b, :, L[b]] = kt[b, :, i], vt[b, :, i]
        L = L + 1


def test_plain_scores_are_tree_attention():
    c = Case("bf16", B=2, Hq=8, Hkv=2, D=128, T=64, lens=(300, 1000), Lmax=1024)
    out, lse = c.call()
    ref_out, ref_lse = c.st.tree_attention(c.q, c.kc, c.vc, _i32(c.lens), c.kt, c.vt, c.tree)
    r = c.reference()
    c.check(ref_out.to(out.dtype), ref_lse, r)
    c.check(out, lse, r)


@pytest.mark.parametrize("name", ["tree-paged", "tokens", "everything"])
def test_replays_and_other_streams(name):
    """Two graphs on one workspace, replayed in turn with new lengths, and an eager call on a side stream."""
    import torch
    c = Case("bf16", **CASES[name])
    d = Case("bf16", **{**CASES[name], "seed": 5})
    ws = c.workspace()
    L = _i32(c.lens)
    fixed = {}
    for case in (c, d):
        fixed[case] = dict(out=torch.empty_like(case.q), lse=torch.empty(case.q.shape[:3], device="cuda"), ws=ws, L=L)
    # the tables' device copies live as long as the graphs
    keep = {case: [_i32(getattr(case, n, [0])) for n in ("table", "stable")] + [_i32([case.shared_len])] for case in (c, d)}

    def call(case, stream=None, **kw):
        st, k, tree = case.st, keep[case], (case.kt, case.vt, case.tree)
        a = {**case.score, "stream": stream, "out": kw["out"], "lse": kw["lse"], "ws": kw["ws"]}
        if case.block:
            return st.tree_attention_shared_paged(case.q, case.kp, case.vp, k[1], k[2], k[0], kw["L"], *tree, **a)
        return st.tree_attention_shared(case.q, case.ks, case.vs, k[2], case.kc, case.vc, kw["L"], *tree, **a)
    call(c, **fixed[c])
    torch.cuda.synchronize()
    graphs = {}
    for case in (c, d):
        graphs[case] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[case]):
            call(case, **fixed[case])
    for shift in (0, 1, 0):
        lens = np.maximum(np.array(CASES[name]["lens"]) - shift, 0)
        L.copy_(_i32(lens))
        for case in (c, d):
            fixed[case]["out"].fill_(7.0)
            graphs[case].replay()
        torch.cuda.synchronize()
        for case in (c, d):
            case.lens = lens
            case.check(fixed[case]["out"], fixed[case]["lse"])
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            mine = dict(out=torch.empty_like(case.q), lse=torch.empty_like(fixed[case]["lse"]), ws=case.workspace(), L=L)
            side.wait_stream(torch.cuda.current_stream())
            call(case, stream=side, **mine)
            side.synchronize()
            assert torch.equal(mine["out"], fixed[case]["out"]) and torch.equal(mine["lse"], fixed[case]["lse"])


def test_prompt_tree_and_commit_together():
    """The path of a served batch: rotated appends of a shared prompt and of each sequence's own, the tree's rotation,
    shared attention, the commit of a path, and the next step's single tokens -- against the oracles run in a row."""
    import torch
    from oracle import rope
    st = lib()
    B, Hq, Hkv, D, bs, Ls = 2, 8, 2, 64, 16, 50
    g = torch.Generator().manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    freq = 10000.0 ** (-np.arange(D // 2) / (D // 2))
    tfreq = torch.tensor(freq, device="cuda")
    pool_k, pool_v = torch.zeros(16, Hkv, bs, D, device="cuda"), torch.zeros(16, Hkv, bs, D, device="cuda")
    shared_table, table = _i32([3, 9, 1, 14]), _i32([[0, 2, 4, 5], [6, 7, 8, 10]])
    sl, L = _i32([Ls]), _i32([0, 0])
    # the shared prompt goes into its own blocks as one sequence
    x = rand(Ls, 2 * Hkv, D)
    st.kv_append_paged(None, x[:, :Hkv], x[:, Hkv:], _i32([0, Ls]), _i32([0]), pool_k, pool_v, shared_table[None], freq=tfreq)
    own = [20, 33]
    y = rand(sum(own), 2 * Hkv, D)
    st.kv_append_paged(None, y[:, :Hkv], y[:, Hkv:], _i32([0, 20, 53]), L, pool_k, pool_v, table, freq=tfreq, pos_base=sl)
    L += _i32(own)
    parent = [-1, 0, 0, 1, 1, 3]
    tree, tree_o = st.spec_tree_build(parent), oracle.tree_encode(parent, None)
    z = rand(B, 6, Hq + 2 * Hkv, D)
    q, kt, vt = st.tree_rope(z[:, :, :Hq], z[:, :, Hq:Hq + Hkv], z[:, :, Hq + Hkv:], L, tree, freq=tfreq, pos_base=sl)
    out, _ = st.tree_attention_shared_paged(q, pool_k, pool_v, shared_table, sl, table, L, kt, vt, tree)
    path = _i32([[0, 1, 3, 5], [0, 2, -1, -1]])
    st.tree_kv_commit_paged(kt, vt, pool_k, pool_v, table, bs, L, _i32([3, 1]), path, tree)
    one, one_o = st.spec_tree_build([-1]), oracle.tree_encode([-1], None)
    w = rand(B, 1, Hq + 2 * Hkv, D)
    q1, kt1, vt1 = st.tree_rope(w[:, :, :Hq], w[:, :, Hq:Hq + Hkv], w[:, :, Hq + Hkv:], L, one, freq=tfreq, pos_base=sl)
    out1, _ = st.tree_attention_shared_paged(q1, pool_k, pool_v, shared_table, sl, table, L, kt1, vt1, one, softcap=20.0)

    zero = lambda *s: np.zeros(s)  # noqa: E731
    x, y, z, w = (_np(t) for t in (x, y, z, w))
    none = zero(Ls, 1, D)
    _, ks, vs, _ = rope.kv_append(none, x[:, :Hkv], x[:, Hkv:], [0, Ls], [0], zero(1, Hkv, Ls, D), zero(1, Hkv, Ls, D), freq)
    _, kc, vc, _ = rope.kv_append(zero(53, 1, D), y[:, :Hkv], y[:, Hkv:], [0, 20, 53], [0, 0], zero(B, Hkv, 64, D), zero(B, Hkv, 64, D),
                                  freq, base=Ls)
    qo, ko, vo = rope.tree_rope(z[:, :, :Hq], z[:, :, Hq:Hq + Hkv], z[:, :, Hq + Hkv:], own, tree_o["depth"], freq, base=Ls)
    ref = osh.attention(qo, kc, vc, own, ko, vo, tree_o, ks[0], vs[0])
    # the rotations' 32-bit rounding moves every score by at most 22 2^-24 of its size (11 for each side)
    tol = lambda r: r["weight"] * (2 * (D * U + 30 * U) * r["size"] + 1e-5)[..., None]  # noqa: E731
    assert (np.abs(_np(out) - ref["out"]) <= tol(ref)).all()
    for b, nodes in enumerate(([0, 1, 3, 5], [0, 2])):
        for n in nodes:
            kc[b, :, own[b]], vc[b, :, own[b]] = ko[b, :, n], vo[b, :, n]
            own[b] += 1
    assert L.tolist() == own
    q1, k1, v1 = rope.tree_rope(w[:, :, :Hq], w[:, :, Hq:Hq + Hkv], w[:, :, Hq + Hkv:], own, one_o["depth"], freq, base=Ls)
    ref = osh.attention(q1, kc, vc, own, k1, v1, one_o, ks[0], vs[0], softcap=20.0)
    assert (np.abs(_np(out1) - ref["out"]) <= tol(ref)).all()


def test_binding_refuses():
    c = Case("bf16", B=2, Hq=4, Hkv=2, D=64, T=3, lens=(4, 3), Lmax=16, Ls=16, block=16)
    for kw, err in (({"slopes": c.q[0, 0, 0].float()}, ValueError), ({"window": -1}, c.st.SpecError),
                    ({"softcap": -1.0}, c.st.SpecError), ({"softcap": float("nan")}, c.st.SpecError),
                    ({"out": c.q.float()}, TypeError), ({"scale": -1.0}, c.st.SpecError),
                    ({"ws": c.workspace()[:64]}, c.st.SpecError)):
        with pytest.raises(err):
            c.call(**kw)
    c.block, c.kp, c.vp = 8, c.kp[:, :, :8].contiguous(), c.vp[:, :, :8].contiguous()
    with pytest.raises(c.st.SpecError, match="multiple of 16"):
        c.call()


RISING = {
    # 256 rows against 128 keys at a time, 128 rows and fewer against 64, few rows
    "rows-256": dict(B=1, Hq=4, Hkv=1, D=128, T=64, lens=(700,), Lmax=700),
    "rows-128": dict(B=2, Hq=4, Hkv=2, D=64, T=40, lens=(500, 130), Lmax=500, Ls=300),
    "few-rows": dict(B=3, Hq=4, Hkv=2, D=128, T=2, lens=(400, 64, 9), Lmax=400, Ls=200),
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", [dict(), dict(softcap=300.0), dict(slopes=True)], ids=["plain", "cap", "bias"])
@pytest.mark.parametrize("name", list(RISING))
def test_maxima_that_keep_rising(name, score, dtype):
    """Keys that grow along the line: the running maximum moves in every tile, also between a tile's halves."""
    import torch
    c = Case(dtype, **RISING[name], **score, gain=4.0)
    n = c.Ls + c.Lmax
    ramp = torch.linspace(0.1, 30.0, n, device="cuda")[:, None]
    c.kc.mul_(ramp[c.Ls:])
    if c.Ls:
        c.ks.mul_(ramp[:c.Ls])
    ws = c.workspace()
    c.check(*c.call(ws=ws))
    assert c.st.spec_read_device_status(ws) == 0


@pytest.mark.parametrize("T", [64, 9, 1])
@pytest.mark.parametrize("cap", [500.0, 50.0, 10.0, 3.0, 0.5])
def test_caps_near_and_far_from_the_scores(cap, T):
    """Whole tiles whose scores are small, middling and large beside the cap."""
    for dtype in ("bf16", "f32"):
        c = Case(dtype, B=2, Hq=8, Hkv=2, D=128, T=T, lens=(640, 200), Lmax=640, Ls=256, softcap=cap)
        c.check(*c.call())


def test_calls_in_a_row_wait_for_each_other():
    """Inputs written just before a call and overwritten just after it, one workspace, nothing waited for in between."""
    import torch
    cases = [Case("bf16", B=4, Hq=8, Hkv=2, D=128, T=T, lens=(300, 17, 90, 0), Lmax=320, Ls=200, seed=i)
             for i, T in enumerate((1, 9, 64, 3))]
    alone = [c.call() for c in cases]
    ws = max((c.workspace() for c in cases), key=len)
    args = [(_i32([c.shared_len]), _i32(c.lens)) for c in cases]
    names = ("q", "ks", "vs", "kc", "vc", "kt", "vt")
    room = [{n: torch.empty_like(getattr(c, n)) for n in names} for c in cases]
    torch.cuda.synchronize()
    got = []
    for i in range(24):
        c, x, (sl, L) = cases[i % 4], room[i % 4], args[i % 4]
        for n in names:
            x[n].copy_(getattr(c, n))
        got.append(c.st.tree_attention_shared(x["q"], x["ks"], x["vs"], sl, x["kc"], x["vc"], L, x["kt"], x["vt"], c.tree, ws=ws))
        for n in names:
            x[n].fill_(float("nan"))
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, alone[i % 4][0]) and torch.equal(lse, alone[i % 4][1])


def test_binding_names_what_is_wrong():
    import torch
    c = Case("bf16", B=2, Hq=4, Hkv=2, D=64, T=3, lens=(4, 3), Lmax=16, Ls=16)
    st, L, sl = c.st, _i32(c.lens), _i32([16])
    good = dict(q=c.q, k_shared=c.ks, v_shared=c.vs, shared_len=sl, k_cache=c.kc, v_cache=c.vc, prefix_len=L, k_tree=c.kt, v_tree=c.vt,
                tree=c.tree)
    st.tree_attention_shared(**good)
    for wrong, err, text in (({"q": c.q.cpu()}, ValueError, "q must be a CUDA tensor"), ({"q": [1]}, TypeError, "q must be a torch.Tensor"),
                             ({"q": c.q.half()}, TypeError, "float32 or bfloat16"), ({"q": c.q[0]}, ValueError, "4 dimensions"),
                             ({"k_tree": c.kt.float()}, TypeError, "k_tree must be"), ({"v_tree": c.vt[:, :1]}, ValueError, "v_tree"),
                             ({"k_cache": c.kc.transpose(1, 2)}, ValueError, "k_cache"), ({"v_cache": c.vc.cpu()}, ValueError, "v_cache"),
                             ({"k_shared": c.ks[0]}, ValueError, "k_shared"), ({"shared_len": _i32([1, 2])}, ValueError, "one value"),
                             ({"shared_len": sl.long()}, TypeError, "shared_len"), ({"prefix_len": _i32([1])}, ValueError, "prefix_len"),
                             ({"tree": st.spec_tree_build([-1])}, ValueError, "the tree 1"), ({"out": c.q}, st.SpecError, "overlaps"),
                             ({"ws": torch.empty(64, dtype=torch.uint8)}, ValueError, "ws must be a CUDA tensor")):
        with pytest.raises(err, match=text):
            st.tree_attention_shared(**{**good, **wrong})


@pytest.mark.parametrize("T", [64, 20, 2])
def test_the_largest_cap(T):
    """Whole and partial tiles, windows and a bias at the largest cap taken; beyond it the call is refused."""
    for dtype in ("bf16", "f32"):
        c = Case(dtype, B=2, Hq=8, Hkv=2, D=128, T=T, lens=(330, 77), Lmax=340, softcap=4096.0)
        c.check(*c.call())
        c.score["window"] = 300
        c.check(*c.call())
        d = Case(dtype, B=2, Hq=8, Hkv=2, D=128, T=T, lens=(330, 77), Lmax=340, softcap=4096.0, slopes=True, gain=20.0)
        d.check(*d.call())
        with pytest.raises(c.st.SpecError, match="softcap"):
            c.call(softcap=5000.0)


def test_the_largest_tree():
    for name, kw in (("f32", dict(D=64, Hq=2, Hkv=1)), ("bf16", dict(D=128, Hq=2, Hkv=2))):
        c = Case(name, B=1, T=1024, lens=(100,), Lmax=128, Ls=70, **kw)
        c.check(*c.call())
        c.score["softcap"], c.score["window"] = 20.0, 90
        c.check(*c.call())


def test_far_into_a_long_cache():
    """Keys some millions of positions into the cache, seen through a window: rows past 2^31 bytes of it."""
    import torch
    n = 1 << 22
    for dtype, Hkv in (("bf16", 5), ("f32", 3)):
        c = Case(dtype, B=1, Hq=Hkv, Hkv=Hkv, D=64, T=5, lens=(300,), Lmax=300, window=257, slopes=True)
        kc = torch.zeros(1, Hkv, n, 64, dtype=c.kc.dtype, device="cuda")
        vc = torch.zeros_like(kc)
        L = n - 3
        kc[:, :, L - 300:L], vc[:, :, L - 300:L] = c.kc, c.vc
        ref = c.reference()       # positions are seen through their differences only
        c.kc, c.vc = kc, vc
        c.check(*c.call(L=_i32([L])), ref)
        del c, kc, vc
        torch.cuda.empty_cache()


def test_two_streams_at_once():
    import torch
    a = Case("bf16", B=4, Hq=16, Hkv=2, D=128, T=30, lens=(900, 1, 300, 77), Lmax=1000, Ls=2000)
    b = Case("bf16", B=5, Hq=8, Hkv=4, D=64, T=1, lens=(500, 400, 3, 77, 0), Lmax=500, block=16, softcap=30.0)
    want = [a.call(), b.call()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    rooms = [c.workspace() for c in (a, b)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(12):
        for i, c in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(c.call(ws=rooms[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


JUMPS = {
    # blocks of 256 rows and a smaller one in turn, several of each in a CTA: the first tile is the tree's, or cut out of the prefix
    "tree": dict(B=6, Hq=192, Hkv=64, D=64, T=100, lens=(0, 3, 200, 0, 70, 130), Lmax=200),
    "prefix": dict(B=2, Hq=64, Hkv=64, D=64, T=341, lens=(700, 620), Lmax=700),
}


@pytest.mark.parametrize("score", [dict(softcap=50.0), dict(slopes=True), dict(window=300)], ids=["cap", "bias", "window"])
@pytest.mark.parametrize("name", list(JUMPS))
def test_a_maximum_that_jumps_in_an_items_first_tile(name, score):
    """Every second 64 keys by far exceed the first: a group that rescales in an item's first tile, ahead of the
    other, must leave the other's reading of the item before alone."""
    c = Case("bf16", **JUMPS[name], **score)
    for keys in (c.kc, c.kt):
        for j in range(64, keys.shape[2], 128):
            keys[:, :, j:j + 64] *= 32.0
    ws = c.workspace()
    out, lse = c.call(ws=ws)
    c.check(out, lse)
    assert c.st.spec_read_device_status(ws) == 0
    for _ in range(40):
        again, lse2 = c.call(ws=ws)
        assert (again == out).all() and (lse2 == lse).all()


def test_a_window_that_does_not_fit_is_refused():
    for Ls, block in ((0, 0), (16, 0), (0, 16), (16, 16)):
        c = Case("bf16", B=2, Hq=4, Hkv=2, D=64, T=3, lens=(4, 3), Lmax=16, Ls=Ls, block=block)
        for window in (1 << 31, (1 << 32) + 5, 2.5):
            with pytest.raises(ValueError, match="window"):
                c.call(window=window)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 20, 100])
def test_the_largest_windows_hide_nothing(T, dtype):
    """Up to the largest number the field holds, over partial tiles of shared and own keys."""
    for window in ((1 << 24) - 1, 1 << 24, (1 << 31) - 100, (1 << 31) - 1):
        c = Case(dtype, B=2, Hq=6, Hkv=2, D=64, T=T, lens=(65, 200), Lmax=200, Ls=70, window=window)
        out, lse = c.call()
        ref = {**c.score, "window": 0}
        c.score = ref
        c.check(out, lse)
