"""Cases of the serving operators around tree attention: rotated appends to the KV cache, the rotation of
a tree's projections, tree attention over a prefix that the batch shares, and tree attention with capped,
biased and windowed scores.

`run` computes a case in elementary torch operations in 32 bits (angles in 64), or, where `own` is true, by the
package's calls."""

import math
import random

import numpy as np
import torch

own = False

# Head layouts: "70b" 64 query and 8 key/value heads of 128, "7b" 32 and 32 of 128.
_70B = {"Hq": 64, "Hkv": 8, "D": 128}
_7B = {"Hq": 32, "Hkv": 32, "D": 128}
_SMALL = {"Hq": 8, "Hkv": 2, "D": 64}


def _append(name, **kw):
    c = {"name": name, "op": "append", "dtype": "bf16", "block": 64, "interleaved": False, "rot": kw["D"], "base": 0}
    return {**c, **kw}


def _rope(name, **kw):
    c = {"name": name, "op": "rope", "dtype": "bf16", "interleaved": False, "rot": kw["D"], "base": 0}
    return {**c, **kw}


def _attn(name, **kw):
    c = {"name": name, "op": "attn", "dtype": "bf16", "Ls": 0, "lo": 0, "block": 0, "softcap": 0.0, "window": 0, "slopes": False}
    return {**c, **kw}


def listed():
    return [
        # one generated token for each of 64 sequences goes into the paged cache: latency
        _append("append-tokens-70b-b64", B=64, lo=1, hi=1, prefix=4096, **_70B),
        # a chunk of prompts of unequal lengths, 6569 tokens in all: bandwidth
        _append("append-prompts-70b", B=8, lo=300, hi=1748, prefix=1024, **_70B),
        # a small model that rotates a part of each head in neighbouring pairs, fp32, contiguous cache
        _append("append-partial-f32", B=3, lo=90, hi=517, prefix=37, block=0, dtype="f32", **{**_SMALL, "rot": 32, "interleaved": True}),
        # the 64 nodes of one sequence's candidate tree, once per layer and step
        _rope("rope-tree-7b", B=1, T=64, prefix=1024, **_7B),
        # the trees of a served batch behind a shared prefix
        _rope("rope-trees-70b-b32", B=32, T=64, prefix=4096, **{**_70B, "base": 8192}),
        # plain decoding of 64 sequences behind one system prompt of 8192 tokens, paged
        _attn("shared-tokens-70b-b64", B=64, T=1, Ls=8192, lo=1, Lmax=1024, block=64, **_70B),
        # candidate trees of 8 sequences over a shared document of 16384 tokens
        _attn("shared-trees-70b-b8", B=8, T=64, Ls=16384, lo=512, Lmax=2048, block=64, **_70B),
        # four samples of one prompt, contiguous caches
        _attn("shared-samples-7b-b4", B=4, T=64, Ls=1000, lo=17, Lmax=256, **_7B),
        # a layer with a sliding window and capped scores, paged with short pages
        _attn("window-trees-70b-b8", B=8, T=64, lo=2048, Lmax=8192, block=16, softcap=50.0, window=4096, **_70B),
        # a full-attention layer with capped scores: the dense 341-node tree over a 32K prefix
        _attn("capped-tree-7b-32k", B=1, T=341, lo=32768, Lmax=32768, softcap=50.0, **_7B),
        # single tokens with a bias by distance
        _attn("biased-tokens-7b-b16", B=16, T=1, lo=100, Lmax=4096, slopes=True, **_7B),
        # a small fp32 model with everything on
        _attn("scored-small-f32", B=2, T=9, lo=37, Lmax=200, dtype="f32", softcap=20.0, window=150, slopes=True, **_SMALL),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "rope", "attn", "attn"])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    heads = {"Hq": Hkv * rng.choice([1, 2, 4, 7, 8]), "Hkv": Hkv, "D": D, "dtype": dtype}
    rot = {"rot": rng.choice([D, D // 2]), "interleaved": rng.random() < 0.3, "base": rng.choice([0, 1000])}
    if op == "append":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, 8192 // B)
        return _append("", B=B, lo=rng.randint(1, hi), hi=hi, prefix=_log(rng, 1, 4096),
                       **{**heads, **rot, "block": rng.choice([0, 16, 64, 128])}) | {"name": "drawn-append"}
    if op == "rope":
        return _rope("", B=_log(rng, 1, 32), T=_log(rng, 1, 128), prefix=_log(rng, 1, 8192), **{**heads, **rot}) | {"name": "drawn-rope"}
    shared = rng.random() < 0.5
    B, T = _log(rng, 1, 64), _log(rng, 1, 341)
    rows = B * T * heads["Hq"]
    # at most a quarter of the largest listed case's scores, and a tenth of that in fp32
    most = max(64, min(16384, (8 * 64 * 64 * 18432 // (40 if dtype == "f32" else 4)) // rows))
    Ls = _log(rng, 1, most) if shared else 0
    Lmax = _log(rng, 64, max(64, min(8192, most // (2 if shared else 1))))
    block = rng.choice([0, 16, 64, 128])
    if block:
        Lmax = -(-Lmax // block) * block
    return _attn("", B=B, T=T, Ls=Ls, Lmax=Lmax, block=block, softcap=rng.choice([0.0, 0.0, 30.0]),
                 window=rng.choice([0, 0, _log(rng, 1, 2 * Lmax)]), slopes=rng.random() < 0.3,
                 **{**heads, "lo": rng.randint(0, Lmax)}) | {"name": "drawn-attn"}


def _tree(T):
    """Parents and depths of a tree of T nodes, 14 deep at most, bushy near the root."""
    r = random.Random(T)
    parent, depth = [-1], [0]
    while len(parent) < T:
        p = min(r.randrange(len(parent)), r.randrange(len(parent)))
        if depth[p] < 14:
            parent.append(p)
            depth.append(depth[p] + 1)
    return parent, depth


def _lengths(case):
    """Prefix lengths [B] and, for appends, new tokens [B]: part of the case, not of the seed."""
    r = random.Random(case["B"] * 7919 + case.get("T", 1))
    if case["op"] == "append":
        new = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
        return [r.randint(0, case["prefix"]) for _ in range(case["B"])], new
    if case["op"] == "rope":
        return [r.randint(0, case["prefix"]) for _ in range(case["B"])], None
    return [r.randint(case["lo"], case["Lmax"]) for _ in range(case["B"])], None


def _pages(r, lengths, block, spare):
    """A block table [B][max_blocks] of distinct pool blocks in random order, and the pool's size."""
    most = max(-(-max(n, 1) // block) for n in lengths)
    used = [-(-n // block) for n in lengths]
    ids = list(range(sum(used) + spare))
    r.shuffle(ids)
    table, at = [], 0
    for n in used:
        table.append(ids[at:at + n] + [0] * (most - n))
        at += n
    return table, len(ids)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    r = random.Random(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    lengths, new = _lengths(case)
    s = {"case": case, "prefix_len": ints(lengths), "max_len": max(lengths)}
    if case["op"] in ("append", "rope"):
        half = case["rot"] // 2
        s["freq"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        s["base"] = ints([case["base"]])
    if case["op"] == "append":
        N = sum(new)
        x = normal(N, Hq + 2 * Hkv, D)          # the projection's rows: queries, keys and values side by side
        s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        start = [0]
        for n in new:
            start.append(start[-1] + n)
        s["seq_start"] = ints(start)
        s["N"] = N
        total = [a + b for a, b in zip(lengths, new)]
        if case["block"]:
            table, blocks = _pages(r, total, case["block"], 3)
            s["table"] = ints(table)
            s["k_cache"], s["v_cache"] = normal(blocks, Hkv, case["block"], D), normal(blocks, Hkv, case["block"], D)
        else:
            s["k_cache"], s["v_cache"] = normal(B, Hkv, max(total), D), normal(B, Hkv, max(total), D)
        if own:
            import tree_speculative_decoding_spec_gb300 as st
            s["st"] = st
            s["q_out"] = torch.empty(N, Hq, D, dtype=dt, device=dev)
            s["ws"] = torch.empty(st.kv_append_workspace_size(), dtype=torch.uint8, device=dev)
        return s
    T = case["T"]
    parent, depth = _tree(T)
    s["depth"] = ints(depth)
    if own:
        import tree_speculative_decoding_spec_gb300 as st
        s["st"] = st
        s["tree"] = st.spec_tree_build(parent)
    if case["op"] == "rope":
        x = normal(B, T, Hq + 2 * Hkv, D)
        s["q"], s["k"], s["v"] = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
        if own:
            s["outs"] = {"q_out": torch.empty(B, Hq, T, D, dtype=dt, device=dev), "k_out": torch.empty(B, Hkv, T, D, dtype=dt, device=dev),
                         "v_out": torch.empty(B, Hkv, T, D, dtype=dt, device=dev)}
        return s
    seen = [[False] * T for _ in range(T)]
    for i in range(T):
        j = i
        while j >= 0:
            seen[i][j] = True
            j = parent[j]
    s["seen"] = torch.tensor(seen, device=dev)
    s["q"] = normal(B, Hq, T, D)
    s["k_tree"], s["v_tree"] = normal(B, Hkv, T, D), normal(B, Hkv, T, D)
    Ls, Lmax, block = case["Ls"], case["Lmax"], case["block"]
    if block:
        lists = lengths + ([Ls] if Ls else [])
        table, blocks = _pages(r, lists, block, 3)
        s["k_cache"], s["v_cache"] = normal(blocks, Hkv, block, D), normal(blocks, Hkv, block, D)
        width = Lmax // block
        s["table"] = ints([(t + [0] * width)[:width] for t in table[:B]])
        if Ls:
            s["shared_table"] = ints(table[B][:-(-Ls // block)])
    else:
        s["k_cache"], s["v_cache"] = normal(B, Hkv, Lmax, D), normal(B, Hkv, Lmax, D)
        if Ls:
            s["k_shared"], s["v_shared"] = normal(Hkv, Ls, D), normal(Hkv, Ls, D)
    s["shared_len"] = ints([Ls])
    s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], dtype=torch.float32, device=dev) if case["slopes"] else None
    if own:
        code = 1 if dt == torch.bfloat16 else 0
        n = st.tree_attention_shared_workspace_size(s["tree"], B, Hq, Hkv, Ls, Lmax, D, code) if Ls else \
            st.tree_attention_scored_workspace_size(s["tree"], B, Hq, Hkv, Lmax, D, code)
        s["outs"] = {"out": torch.empty(B, Hq, T, D, dtype=dt, device=dev), "lse": torch.empty(B, Hq, T, dtype=torch.float32, device=dev),
                     "ws": torch.empty(n, dtype=torch.uint8, device=dev)}
    return s


def _rotated(x, pos, s):
    """x [..., heads, D] rotated at pos [...] (in 32 bits; the angles in 64)."""
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    phi = pos.double()[..., None] * s["freq"]
    cos, sin = phi.cos().float()[..., None, :], phi.sin().float()[..., None, :]
    x = x.float()
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _run_append(s):
    c = s["case"]
    dt = s["q"].dtype
    n = torch.arange(s["N"], device=s["q"].device)
    b = torch.searchsorted(s["seq_start"][1:].long(), n, right=True)
    at = n - s["seq_start"].long()[b] + s["prefix_len"].long()[b]
    pos = at + s["base"].long()
    q, k, v = _rotated(s["q"], pos, s).to(dt), _rotated(s["k"], pos, s).to(dt), s["v"]
    if c["block"]:
        page = s["table"].long()[b, at // c["block"]]
        s["k_cache"][page, :, at % c["block"]] = k
        s["v_cache"][page, :, at % c["block"]] = v
    else:
        s["k_cache"][b, :, at] = k
        s["v_cache"][b, :, at] = v
    return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}


def _run_rope(s):
    dt = s["q"].dtype
    pos = (s["base"] + s["prefix_len"])[:, None].long() + s["depth"].long()

    def turned(x):
        return _rotated(x, pos, s).to(dt).transpose(1, 2).contiguous()
    return {"q": turned(s["q"]), "k": turned(s["k"]), "v": s["v"].transpose(1, 2).contiguous()}


def _keys(s, name):
    """The own keys (or values) [B, Hkv, L, D] and the shared ones [Hkv, Ls, D] or None, in 32 bits."""
    c, x = s["case"], s[name + "_cache"]
    if not c["block"]:
        return x[:, :, :s["max_len"]].float(), s[name + "_shared"].float() if c["Ls"] else None
    n = -(-s["max_len"] // c["block"])
    mine = x[s["table"][:, :n].long()].transpose(1, 2).flatten(2, 3)[:, :, :s["max_len"]].float()
    if not c["Ls"]:
        return mine, None
    return mine, x[s["shared_table"].long()].transpose(0, 1).flatten(1, 2)[:, :c["Ls"]].float()


def _run_attn(s):
    c, q = s["case"], s["q"]
    B, Hq, T, D = q.shape
    Hkv, Ls = c["Hkv"], c["Ls"]
    x = q.float().view(B, Hkv, Hq // Hkv, T, D) / math.sqrt(D)
    (k, ks), (v, vs) = _keys(s, "k"), _keys(s, "v")
    L = k.shape[2]
    kt, vt = s["k_tree"].float(), s["v_tree"].float()
    scores = [torch.einsum("bhgtd,bhld->bhgtl", x, k), torch.einsum("bhgtd,bhld->bhgtl", x, kt)]
    if Ls:
        scores.insert(0, torch.einsum("bhgtd,hld->bhgtl", x, ks))
    scores = torch.cat(scores, -1)
    here = s["prefix_len"].long()[:, None]
    i = torch.arange(Ls + L, device=q.device)
    kpos = torch.cat([i.expand(B, Ls + L), Ls + here + s["depth"].long()], 1)      # [B, Ls + L + T]
    qpos = Ls + here + s["depth"].long()                                           # [B, T]
    seen = torch.cat([(i < Ls + here)[:, None].expand(B, T, Ls + L), s["seen"].expand(B, T, T)], 2)
    far = qpos[:, :, None] - kpos[:, None, :]
    if c["window"]:
        seen = seen & (far < c["window"])
    if c["softcap"]:
        scores = c["softcap"] * torch.tanh(scores / c["softcap"])
    if s["slopes"] is not None:
        scores = scores - s["slopes"].view(1, Hkv, -1, 1, 1) * far[:, None, None].float()
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgtl,bhld->bhgtd", p[..., Ls:Ls + L], v) + torch.einsum("bhgtl,bhld->bhgtd", p[..., Ls + L:], vt)
    if Ls:
        o = o + torch.einsum("bhgtl,hld->bhgtd", p[..., :Ls], vs)
    return {"out": (o / total).view(B, Hq, T, D).to(q.dtype), "lse": (top + total.log()).view(B, Hq, T)}


def _own(s):
    c, st = s["case"], s["st"]
    if c["op"] == "append":
        more = {"freq": s["freq"], "interleaved": c["interleaved"], "pos_base": s["base"], "q_out": s["q_out"], "ws": s["ws"]}
        if c["block"]:
            q, _ = st.kv_append_paged(s["q"], s["k"], s["v"], s["seq_start"], s["prefix_len"], s["k_cache"], s["v_cache"], s["table"], **more)
        else:
            q, _ = st.kv_append(s["q"], s["k"], s["v"], s["seq_start"], s["prefix_len"], s["k_cache"], s["v_cache"], **more)
        return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}
    if c["op"] == "rope":
        q, k, v = st.tree_rope(s["q"], s["k"], s["v"], s["prefix_len"], s["tree"], freq=s["freq"], interleaved=c["interleaved"],
                               pos_base=s["base"], **s["outs"])
        return {"q": q, "k": k, "v": v}
    more = {"softcap": c["softcap"], "window": c["window"], "slopes": s["slopes"], **s["outs"]}
    tree = (s["k_tree"], s["v_tree"], s["tree"])
    if c["Ls"] and c["block"]:
        out, lse = st.tree_attention_shared_paged(s["q"], s["k_cache"], s["v_cache"], s["shared_table"], s["shared_len"], s["table"],
                                                  s["prefix_len"], *tree, **more)
    elif c["Ls"]:
        out, lse = st.tree_attention_shared(s["q"], s["k_shared"], s["v_shared"], s["shared_len"], s["k_cache"], s["v_cache"],
                                            s["prefix_len"], *tree, **more)
    elif c["block"]:
        out, lse = st.tree_attention_scored_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["prefix_len"], *tree, **more)
    else:
        out, lse = st.tree_attention_scored(s["q"], s["k_cache"], s["v_cache"], s["prefix_len"], *tree, **more)
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"append": _run_append, "rope": _run_rope, "attn": _run_attn}[state["case"]["op"]](state)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    Hq, Hkv, D, B = case["Hq"], case["Hkv"], case["D"], case["B"]
    lengths, new = _lengths(case)
    if case["op"] == "append":
        values = sum(new) * (Hq + 2 * Hkv) * D
        return {"bytes": 2 * values * es, "flops": 3 * sum(new) * (Hq + Hkv) * case["rot"]}
    T = case["T"]
    if case["op"] == "rope":
        return {"bytes": 2 * B * T * (Hq + 2 * Hkv) * D * es, "flops": 3 * B * T * (Hq + Hkv) * case["rot"]}
    depth = _tree(T)[1]
    window, Ls = case["window"] or 1 << 40, case["Ls"]
    # keys that a node of depth d sees: of its path d + 1, then the own prefix, then the shared one
    pairs = sum(min(d + 1, window) + min(n, max(0, window - 1 - d)) + min(Ls, max(0, window - 1 - d - n)) for n in lengths for d in depth)
    mine = sum(min(n, window - 1) for n in lengths)
    shared = min(Ls, max(0, window - 1 - min(lengths)))
    rows = B * Hq * T
    return {"bytes": 2 * (mine + shared + B * T) * Hkv * D * es + 2 * rows * D * es + 4 * rows, "flops": 4 * Hq * D * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "attn":
        return _exact_rotation(s)
    return _exact_attn(s)


def _exact_turn(row, pos, s):
    """One token's heads [H, D] in 64 bits, rotated as complex numbers."""
    rot = s["case"]["rot"]
    x = row.double()
    turn = torch.polar(torch.ones_like(s["freq"]), float(pos) * s["freq"])
    y = x.clone()
    if s["case"]["interleaved"]:
        z = torch.complex(x[:, 0:rot:2], x[:, 1:rot:2]) * turn
        y[:, 0:rot:2], y[:, 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(x[:, :rot // 2], x[:, rot // 2:rot]) * turn
        y[:, :rot // 2], y[:, rot // 2:rot] = z.real, z.imag
    return y


def _exact_rotation(s):
    c = s["case"]
    lengths, new = _lengths(c)
    if c["op"] == "rope":
        depth = _tree(c["T"])[1]
        q, k = s["q"].double().transpose(1, 2).clone(), s["k"].double().transpose(1, 2).clone()
        for b in range(c["B"]):
            for i in range(c["T"]):
                pos = c["base"] + lengths[b] + depth[i]
                q[b, :, i] = _exact_turn(s["q"][b, i], pos, s)
                k[b, :, i] = _exact_turn(s["k"][b, i], pos, s)
        return {"q": q, "k": k, "v": s["v"].double().transpose(1, 2).contiguous()}
    q, k, v = s["q"].double().clone(), s["k_cache"].double(), s["v_cache"].double()
    table = s["table"].cpu().numpy() if c["block"] else None
    n = 0
    for b in range(c["B"]):
        for i in range(new[b]):
            at = lengths[b] + i
            where = (b, slice(None), at) if table is None else (int(table[b, at // c["block"]]), slice(None), at % c["block"])
            q[n] = _exact_turn(s["q"][n], c["base"] + at, s)
            k[where] = _exact_turn(s["k"][n], c["base"] + at, s)
            v[where] = s["v"][n].double()
            n += 1
    return {"q": q, "k": k, "v": v}


def _exact_attn(s):
    c = s["case"]
    B, Hq, T, D = s["q"].shape
    g, Ls, block = Hq // c["Hkv"], c["Ls"], c["block"]
    lengths = _lengths(c)[0]
    depth = np.array(_tree(T)[1])
    out = torch.empty(B, Hq, T, D, dtype=torch.float64, device=s["q"].device)
    lse = torch.empty(B, Hq, T, dtype=torch.float64, device=s["q"].device)

    def rows(b, h, name):
        """Every key (or value) of sequence b and head h in order: shared, own, tree."""
        x, parts = s[name + "_cache"], []
        if Ls:
            parts.append(s[name + "_shared"][h] if not block else x[s["shared_table"].long(), h].reshape(-1, D)[:Ls])
        parts.append(x[b, h, :lengths[b]] if not block else x[s["table"][b, :-(-lengths[b] // block)].long(), h].reshape(-1, D)[:lengths[b]])
        return torch.cat(parts + [s[name + "_tree"][b, h]]).double()

    for b in range(B):
        n = Ls + lengths[b]
        far = (n + depth)[:, None] - np.concatenate([np.arange(n), n + depth])[None, :]
        ok = np.concatenate([np.ones((T, n), dtype=bool), s["seen"].cpu().numpy()], 1)
        if c["window"]:
            ok &= far < c["window"]
        far, hidden = torch.from_numpy(far).to(out.device).double(), torch.from_numpy(~ok).to(out.device)
        for h in range(c["Hkv"]):
            K, V = rows(b, h, "k"), rows(b, h, "v")
            x = s["q"][b, h * g:(h + 1) * g].double() @ K.T * D ** -0.5
            if c["softcap"]:
                x = torch.tanh(x / c["softcap"]) * c["softcap"]
            if c["slopes"]:
                x = x - s["slopes"][h * g:(h + 1) * g].double()[:, None, None] * far
            x = x.masked_fill(hidden, -math.inf)
            z = torch.logsumexp(x, -1)
            out[b, h * g:(h + 1) * g] = torch.exp(x - z[..., None]) @ V
            lse[b, h * g:(h + 1) * g] = z
    return {"out": out, "lse": lse}
