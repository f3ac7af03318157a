"""Cases of the operators that decide what a sequence keeps: the selection of a beam search over beams and vocabulary,
the reordering of the beams' states and caches, the attention weight that cached keys receive, and the eviction
of the keys that received least.

`run` computes a case in elementary torch operations in 32 bits (final scores of beams in 64, where ties are decided), or,
where `own` is true, by the package's calls."""

import math
import random

import torch

own = False

# Head layouts: "70b" 64 query and 8 key/value heads of 128, "7b" 32 and 32 of 128.
_70B = {"Hq": 64, "Hkv": 8, "D": 128}
_7B = {"Hq": 32, "Hkv": 32, "D": 128}
_SMALL = {"Hq": 8, "Hkv": 2, "D": 64}


def _select(name, **kw):
    return {"name": name, "op": "select", "dtype": "bf16", "pad": 0, "alpha": 0.0, "done": 0.0, **kw}


def _states(name, **kw):
    return {"name": name, "op": "states", "dtype": "bf16", **kw}


def _cache(name, **kw):
    return {"name": name, "op": "cache", "dtype": "bf16", "block": 0, **kw}


def _weigh(name, **kw):
    return {"name": name, "op": "weigh", "dtype": "bf16", "block": 0, "path": 0, "decay": 1.0, **kw}


def _evict(name, **kw):
    return {"name": name, "op": "evict", "dtype": "bf16", "block": 0, "sink": 4, "into": False, **kw}


def listed():
    return [
        # one sequence's draft of eight beams: latency
        _select("select-draft-b1", B=1, W=8, K=8, V=32000, dtype="f32"),
        # a served batch over the same vocabulary
        _select("select-batch-b32", B=32, W=4, K=4, V=32000),
        # an odd vocabulary in rows padded to 64, some beams ended, scores weighed by length, more beams out than in
        _select("select-ended-b6", B=6, W=5, K=7, V=50257, pad=47, alpha=0.6, done=0.3),
        # many beams over a large vocabulary: bandwidth
        _select("select-wide-b48", B=48, W=16, K=16, V=131072),
        # hidden states of a recurrent draft head
        _states("states-b32", B=32, W=8, row=4096),
        # paged caches behind a common prompt that stays where it is
        _cache("cache-70b-b16", B=16, W=8, prompt=1000, lo=32, hi=512, block=64, **_70B),
        # one generated token for each of 64 sequences
        _weigh("weigh-tokens-70b-b64", B=64, T=1, lo=512, Lmax=4096, block=64, **_70B),
        # the accepted paths of 64-node trees behind long prefixes, older weights fading
        _weigh("weigh-paths-70b-b8", B=8, T=64, path=5, lo=4096, Lmax=16384, decay=0.98, **_70B),
        # whole prompts
        _weigh("weigh-prompts-70b-b2", B=2, T=4096, lo=2500, Lmax=4096, **_70B),
        # a small fp32 model's prompt
        _weigh("weigh-small-f32", B=2, T=100, lo=150, Lmax=517, dtype="f32", **_SMALL),
        # a full budget after a verification step: a few rows too many in every sequence, in place
        _evict("evict-step-70b-b64", B=64, budget=2048, recent=64, lo=2049, Lmax=2065, **_70B),
        # prompts brought down to the budget, into the cache that serves them
        _evict("evict-prompts-7b-b4", B=4, budget=2048, recent=256, lo=3000, Lmax=16384, into=True, **_7B),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "select", "states", "cache", "weigh", "weigh", "weigh", "evict"])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    if op == "select":
        W, V = _log(rng, 1, 32), _log(rng, 500, 131072)
        B = _log(rng, 1, max(1, min(64, (48 * 16 * 131072) // (W * V * (2 if dtype == "f32" else 1)))))
        return _select("drawn-select", B=B, W=W, K=min(32, max(1, W + rng.choice([0, 0, -1, 3]))), V=V, pad=rng.choice([0, 0, 1, 13]),
                       alpha=rng.choice([0.0, 0.0, 0.7]), done=rng.choice([0.0, 0.2]), dtype=dtype)
    if op == "states":
        return _states("drawn-states", B=_log(rng, 1, 64), W=_log(rng, 2, 32), row=4 * _log(rng, 1, 4096), dtype=dtype)
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    heads = {"Hq": Hkv * rng.choice([1, 2, 4, 7, 8]), "Hkv": Hkv, "D": D, "dtype": dtype}
    block = rng.choice([0, 0, 16, 64, 128])
    if op == "cache":
        B, W = _log(rng, 1, 16), _log(rng, 2, 16)
        hi = _log(rng, 1, 8 * 16 * 8 * 256 // (B * W * Hkv) + 1)
        return _cache("drawn-cache", B=B, W=W, prompt=rng.randint(0, 300), lo=rng.randint(0, hi), hi=hi, block=block, **heads)
    if op == "evict":
        B = _log(rng, 1, 16)
        budget = _log(rng, 16, 2048)
        Lmax = budget + _log(rng, 1, 4096)
        return _evict("drawn-evict", B=B, budget=budget, recent=rng.randint(0, budget // 2), sink=rng.randint(0, 4),
                      lo=rng.randint(1, Lmax), Lmax=-(-Lmax // block) * block if block else Lmax, into=rng.random() < 0.5,
                      block=block, **heads)
    # at most a fifth of the largest listed case's pairs of rows and keys, and its keys, in fp32 a twentieth
    T = rng.choice([1, 1, 64, _log(rng, 2, 2048)])
    path = rng.randint(1, 17) if T >= 17 and rng.random() < 0.4 else 0
    rows = path or T
    most = max(2 * rows, min(131072, 2 * 64 * 4096 * 800 // (rows * heads["Hq"])) // (4 if dtype == "f32" else 1))
    Lmax = _log(rng, rows, min(most, 16384))
    B = _log(rng, 1, max(1, min(64, most // Lmax)))
    Lmax = -(-Lmax // block) * block if block else Lmax
    return _weigh("drawn-weigh", B=B, T=T, path=path, lo=rng.randint(rows, Lmax), Lmax=Lmax, block=block,
                  decay=rng.choice([1.0, 0.95]), **heads)


# ---- what belongs to a case, not to the seed

def _lengths(case):
    """Keys in each cache [B], the new rows with them."""
    r = random.Random(case["B"] * 7919 + case.get("T", case.get("budget", 1)))
    if case["op"] == "cache":
        start = [r.randint(0, case["prompt"]) for _ in range(case["B"])]
        return start, [a + r.randint(case["lo"], case["hi"]) for a in start]
    return [r.randint(case["lo"], case["Lmax"]) for _ in range(case["B"])]


def _rows(case):
    """Rows that count of each sequence [B]: of its accepted path, or the first of its T."""
    r = random.Random(case["B"] * 104729 + case["T"])
    if case["path"]:
        return [r.randint(1, case["path"]) for _ in range(case["B"])]
    return [min(n, case["T"] if r.random() < 0.5 else r.randint(1, case["T"])) for n in _lengths(case)]


def _parents(case):
    """Each beam's parent [B][W]: good beams have several children."""
    r = random.Random(case["B"] * 31 + case["W"])
    return [[min(r.randrange(case["W"]), r.randrange(case["W"])) for _ in range(case["W"])] for _ in range(case["B"])]


def _pages(r, lengths, block, width):
    """A block table [len(lengths)][width] of distinct pool blocks in random order, and the pool's size."""
    used = [-(-n // block) for n in lengths]
    ids = list(range(sum(used) + 2))
    r.shuffle(ids)
    table, at = [], 0
    for n in used:
        table.append(ids[at:at + n] + [0] * (width - n))
        at += n
    return table, len(ids)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    r = random.Random(seed)
    dt, B = _dtype(case), case["B"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    s = {"case": case}
    if case["op"] == "select":
        W, V = case["W"], case["V"]
        s["logits"] = (2.5 * normal(B, W, V + case["pad"])).to(dt)[..., :V]
        s["scores"] = torch.sort(-3.0 * torch.rand(B, W, generator=g, device=dev) - 8.0, descending=True).values
        s["eos"] = 2
        s["ended"] = (torch.rand(B, W, generator=g, device=dev) < case["done"]).int()
        s["length"] = torch.where(s["ended"] > 0, torch.randint(1, 12, (B, W), generator=g, device=dev), 12).int()
        return s
    if case["op"] == "states":
        s["state"] = normal(B, case["W"], case["row"]).to(dt)
        s["parent"] = ints(_parents(case))
        return s
    Hkv, D, block = case["Hkv"], case["D"], case["block"]
    if case["op"] == "cache":
        start, end = _lengths(case)
        W = case["W"]
        s["parent"], s["start"], s["end"] = ints(_parents(case)), ints(start), ints(end)
        s["max_end"] = max(end)
        lens = [n for n in end for _ in range(W)]
        Lmax = max(max(end), 1)
    else:
        lens = _lengths(case)
        Lmax = case["Lmax"]
        s["len"], s["max_len"] = ints(lens), max(lens)
    rows = len(lens)
    if block:
        width = -(-Lmax // block)
        table, blocks = _pages(r, lens, block, width)
        s["table"] = ints(table)
        s["k"], s["v"] = normal(blocks, Hkv, block, D).to(dt), normal(blocks, Hkv, block, D).to(dt)
    else:
        s["k"], s["v"] = normal(rows, Hkv, Lmax, D).to(dt), normal(rows, Hkv, Lmax, D).to(dt)
    if case["op"] == "cache":
        return s
    s["acc"] = 0.01 * torch.exp(1.5 * normal(B, Hkv, Lmax))
    if case["op"] == "evict":
        # what is left of some more positions, in the order that earlier evictions left; the last ones as they came
        steady = torch.rand(B, Hkv, Lmax, generator=g, device=dev)
        steady[:, :, case["budget"]:] = 2.0 + torch.arange(Lmax - case["budget"], device=dev)
        s["pos"] = torch.argsort(torch.argsort(steady, -1), -1).int()
        s["seen"] = s["len"].clone()
        if case["into"]:
            n = case["budget"]
            if block:
                out, blocks = _pages(r, [n] * B, block, -(-n // block))
                first = s["k"].shape[0]
                s["out_table"] = ints([[first + b for b in row] for row in out])
                s["k"], s["v"] = (torch.cat([x, torch.zeros(blocks, *x.shape[1:], dtype=dt, device=dev)]) for x in (s["k"], s["v"]))
            else:
                s["k_out"], s["v_out"] = torch.zeros(B, Hkv, n, D, dtype=dt, device=dev), torch.zeros(B, Hkv, n, D, dtype=dt, device=dev)
            n = -(-n // block) * block if block else n
            s["acc_out"], s["pos_out"] = torch.zeros(B, Hkv, n, device=dev), torch.zeros(B, Hkv, n, dtype=torch.int32, device=dev)
        return s
    T = case["T"]
    s["q"] = (1.5 * normal(B, case["Hq"], T, D)).to(dt)
    s["pos"] = torch.full((B, Hkv, Lmax), -1, dtype=torch.int32, device=dev)
    s["seen"] = s["len"] + 100
    n = _rows(case)
    if case["path"]:
        s["accept_len"] = ints([m - 1 for m in n])
        s["accept_path"] = ints([[0] + sorted(r.sample(range(1, T), m - 1)) + [-1] * (case["path"] - m) for m in n])
    else:
        s["n_rows"] = ints(n)
    # the attention's own log of sums, of the rows that count; the others' are what an unused row leaves
    s["lse"] = torch.full((B, case["Hq"], T), -math.inf, device=dev)
    x, seen, rows, _ = _scores(s)
    lse = torch.logsumexp(x.masked_fill_(~seen, -math.inf), -1).reshape(B, case["Hq"], -1)
    lse = lse.masked_fill((torch.arange(rows.shape[1], device=dev) >= ints(n)[:, None])[:, None], -math.inf)
    s["lse"] = s["lse"].scatter_reduce(2, rows[:, None].expand_as(lse), lse, "amax")
    return s


# ---- plain forms

def _run_select(s):
    c = s["case"]
    B, W, V = s["logits"].shape
    K = c["K"]
    x = s["logits"].float()
    top = x.amax(-1, keepdim=True)
    total = torch.exp(x - top).sum(-1, keepdim=True)
    score = s["scores"].double()[..., None] + (x.double() - (top.double() + total.double().log()))
    ended = s["ended"][..., None] > 0
    token = torch.arange(V, device=x.device)
    score = torch.where(ended, torch.where(token == s["eos"], s["scores"].double()[..., None], -math.inf), score)
    length = s["length"][..., None] + (~ended).int()
    key = score / length.clamp(min=1).double() ** c["alpha"] if c["alpha"] else score
    key = key.reshape(B, W * V)
    # the K largest, of equal ones those of the lowest beam and token: all above the K-th value, then the first of its equals
    kth = torch.topk(key, K, -1).values[:, -1:]
    flat = torch.arange(W * V, device=x.device)
    at = torch.topk(torch.where(key > kth, 2 * W * V, torch.where(key == kth, W * V - flat, -1)), K, -1).indices
    at = at.sort(-1).values
    at = at.gather(1, torch.sort(key.gather(1, at), dim=-1, descending=True, stable=True).indices)
    parent, token = at // V, at % V
    got = score.reshape(B, W * V).gather(1, at)
    was = s["ended"].gather(1, parent)
    none = got == -math.inf                             # fewer pairs than K: ended beams offer one each
    return {"token": token.masked_fill(none, -1).int(), "parent": parent.masked_fill(none, -1).int(), "score": got.float(),
            "ended": ((was > 0) | (token == s["eos"]) | none).int(), "length": length[..., 0].gather(1, parent).masked_fill(none, 0).int()}


def _run_states(s):
    x = s["state"]
    b = torch.arange(x.shape[0], device=x.device)[:, None]
    x.copy_(x[b, s["parent"].long()])
    return x


def _run_cache(s):
    c, block = s["case"], s["case"]["block"]
    B, W, n = c["B"], c["W"], s["max_end"]
    dev = s["k"].device
    i = torch.arange(n, device=dev)
    moved = ((i >= s["start"][:, None]) & (i < s["end"][:, None])).repeat_interleave(W, 0)             # [B W, n]
    source = (torch.arange(B, device=dev)[:, None] * W + s["parent"].long()).reshape(-1, 1)            # [B W, 1]
    if block:
        table = s["table"].long()
        page, line = table[:, i // block], (i % block).expand(B * W, n)
        from_page = table[source, (i // block)[None]]
        spare = s["k"].shape[0]
        for x in (s["k"], s["v"]):
            more = torch.cat([x, x[:1]])                                # a row that is not moved goes to a spare block
            more[torch.where(moved, page, spare), :, line] = x[from_page, :, line]
            x.copy_(more[:spare])
    else:
        for x in (s["k"], s["v"]):
            y = x[source[:, 0], :, :n]
            x[:, :, :n] = torch.where(moved[:, None, :, None], y, x[:, :, :n])
    return {"k": s["k"], "v": s["v"]}


def _all_keys(s, name, n):
    """The first n keys (or values) of each sequence [B, Hkv, n, D], as they are stored."""
    x, block = s[name], s["case"]["block"]
    if not block:
        return x[:, :, :n]
    return x[s["table"][:, :-(-n // block)].long()].transpose(1, 2).flatten(2, 3)[:, :, :n]


def _scores(s):
    """Scores [B, Hkv, g, R, n] of the rows that count, which keys each of them sees, the rows [B, R], how many [B]."""
    c, q = s["case"], s["q"]
    B, Hq, T, D = q.shape
    n = s["max_len"]
    if c["path"]:
        rows, count = s["accept_path"].long().clamp(min=0), s["accept_len"].long() + 1
    else:
        rows, count = torch.arange(T, device=q.device).expand(B, T), s["n_rows"].long()
    R = rows.shape[1]
    x = q.gather(2, rows[:, None, :, None].expand(B, Hq, R, D)).float().view(B, c["Hkv"], -1, D) / math.sqrt(D)
    x = torch.matmul(x, _all_keys(s, "k", n).float().transpose(2, 3)).view(B, c["Hkv"], Hq // c["Hkv"], R, n)
    r = torch.arange(R, device=q.device)
    last = (s["len"].long() - count)[:, None] + r                                                     # the last key that row r sees
    seen = (torch.arange(n, device=q.device) <= last[..., None]) & (r < count[:, None])[..., None]    # [B, R, n]
    return x, seen[:, None, None], rows, count


def _run_weigh(s):
    c, n = s["case"], s["max_len"]
    x, seen, rows, count = _scores(s)
    B, Hkv, g, R, _ = x.shape
    lse = s["lse"].gather(2, rows[:, None].expand(B, Hkv * g, R)).view(B, Hkv, g, R, 1)
    w = torch.exp(x - lse).masked_fill(~(seen & torch.isfinite(lse)), 0.0).sum((2, 3))
    i = torch.arange(n, device=x.device)
    end = s["len"].long()[:, None]
    fresh = ((i >= end - count[:, None]) & (i < end))[:, None]
    inside = (i < end)[:, None]
    old = s["acc"][:, :, :n]
    s["acc"][:, :, :n] = torch.where(inside, w + torch.where(fresh, 0.0, c["decay"] * old), old)
    at = (s["seen"].long()[:, None] - end + i)[:, None]
    s["pos"][:, :, :n] = torch.where(fresh, at.int(), s["pos"][:, :, :n])
    return {"acc": s["acc"], "pos": s["pos"]}


def _run_evict(s):
    c = s["case"]
    n, m, block = s["max_len"], c["budget"], c["block"]
    acc, pos = s["acc"][:, :, :n], s["pos"][:, :, :n]
    B, Hkv, _ = acc.shape
    dev = acc.device
    i = torch.arange(n, device=dev)
    end = s["len"].long()[:, None, None]
    safe = (pos < c["sink"]) | (pos >= s["seen"][:, None, None] - c["recent"])
    # ranks by (inside the length, safe, weight), of equal ones the lowest index first
    order = torch.sort(acc, dim=-1, descending=True, stable=True).indices
    grade = (2 * (i < end).int() + safe.int()).gather(2, order)
    order = order.gather(2, torch.sort(grade, dim=-1, descending=True, stable=True).indices)
    kept = torch.empty_like(order).scatter_(2, order, i.expand_as(order)) < torch.minimum(end, torch.full_like(end, m))
    # place p < m holds key p where that is kept, else the next kept key from behind m
    p = torch.arange(min(m, n), device=dev)
    hole = ~kept[:, :, :m] & (p < end)
    late = kept & (i >= m)
    late_at = torch.sort((~late).int(), dim=-1, stable=True).indices                     # kept keys behind m, in order
    source = torch.where(hole, late_at.gather(2, (hole.int().cumsum(-1) - 1).clamp(min=0)), p)
    there = p < end
    k, v = ((_all_keys(s, x, n).gather(2, source[..., None].expand(B, Hkv, len(p), c["D"]))) for x in ("k", "v"))
    to_acc, to_pos = (s["acc_out"], s["pos_out"]) if c["into"] else (s["acc"], s["pos"])
    new_acc, new_pos = acc.gather(2, source), pos.gather(2, source)
    to_acc[:, :, :len(p)] = torch.where(there, new_acc, to_acc[:, :, :len(p)])
    to_pos[:, :, :len(p)] = torch.where(there, new_pos, to_pos[:, :, :len(p)])
    if block:
        table = (s["out_table"] if c["into"] else s["table"]).long()
        page, spare = table[:, p // block], s["k"].shape[0]
        where = torch.where(there[:, 0], page, spare)
        for x, y in ((s["k"], k), (s["v"], v)):
            more = torch.cat([x, x[:1]])
            more[where, :, (p % block).expand_as(where)] = y.transpose(1, 2)
            x.copy_(more[:spare])
        to_k, to_v = s["k"], s["v"]
    else:
        to_k, to_v = (s["k_out"], s["v_out"]) if c["into"] else (s["k"], s["v"])
        for x, y in ((to_k, k), (to_v, v)):
            x[:, :, :len(p)] = torch.where(there[..., None], y, x[:, :, :len(p)])
    return {"k": to_k, "v": to_v, "acc": to_acc, "pos": to_pos, "len": s["len"].clamp(max=m)}


# ---- the package's calls

def _own(s):
    import tree_speculative_decoding_spec_gb300 as st
    c = s["case"]
    if c["op"] == "select":
        token, parent, score, ended, length = st.beam_select(s["logits"], s["scores"], c["K"], eos=s["eos"], ended=s["ended"],
                                                             length=s["length"], alpha=c["alpha"])
        return {"token": token, "parent": parent, "score": score, "ended": ended, "length": length}
    if c["op"] == "states":
        return st.beam_reorder(s["state"], s["parent"])
    if c["op"] == "cache":
        if c["block"]:
            st.kv_reorder_paged(s["k"], s["v"], s["table"], s["parent"], s["start"], s["end"])
        else:
            st.kv_reorder(s["k"], s["v"], s["parent"], s["start"], s["end"])
        return {"k": s["k"], "v": s["v"]}
    if c["op"] == "weigh":
        rows = {"accept_len": s["accept_len"], "accept_path": s["accept_path"]} if c["path"] else {"n_rows": s["n_rows"]}
        more = {"pos": s["pos"], "seen": s["seen"], "decay": c["decay"], **rows}
        if c["block"]:
            st.kv_weigh_paged(s["q"], s["lse"], s["k"], s["table"], s["len"], s["acc"], **more)
        else:
            st.kv_weigh(s["q"], s["lse"], s["k"], s["len"], s["acc"], **more)
        return {"acc": s["acc"], "pos": s["pos"]}
    more = {"seen": s["seen"], "sink": c["sink"], "recent": c["recent"]}
    if c["block"]:
        into = {"out_table": s["out_table"], "acc_out": s["acc_out"], "pos_out": s["pos_out"]} if c["into"] else {}
        n = st.kv_evict_paged(s["k"], s["v"], s["table"], s["len"], s["acc"], s["pos"], c["budget"], **more, **into)
        k, v = s["k"], s["v"]
    else:
        into = {"k_out": s["k_out"], "v_out": s["v_out"], "acc_out": s["acc_out"], "pos_out": s["pos_out"]} if c["into"] else {}
        n = st.kv_evict(s["k"], s["v"], s["len"], s["acc"], s["pos"], c["budget"], **more, **into)
        k, v = (s["k_out"], s["v_out"]) if c["into"] else (s["k"], s["v"])
    acc, pos = (s["acc_out"], s["pos_out"]) if c["into"] else (s["acc"], s["pos"])
    return {"k": k, "v": v, "acc": acc, "pos": pos, "len": n}


def run(state):
    if own:
        return _own(state)
    return {"select": _run_select, "states": _run_states, "cache": _run_cache, "weigh": _run_weigh, "evict": _run_evict}[state["case"]["op"]](state)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    B = case["B"]
    if case["op"] == "select":
        live = B * case["W"] * (1.0 - case["done"])
        return {"bytes": int(live * case["V"] * es) + 12 * B * case["W"] + 20 * B * case["K"], "flops": int(3 * live * case["V"])}
    if case["op"] in ("states", "cache"):
        # every beam that takes another's rows is written, every beam that others take from is read
        lines = [len([1 for w, p in enumerate(row) if p != w]) + len({p for w, p in enumerate(row) if p != w}) for row in _parents(case)]
        if case["op"] == "states":
            return {"bytes": sum(lines) * case["row"] * es + 4 * B * case["W"], "flops": 0}
        start, end = _lengths(case)
        return {"bytes": 2 * sum(x * (b - a) for x, a, b in zip(lines, start, end)) * case["Hkv"] * case["D"] * es + 4 * B * case["W"] + 8 * B, "flops": 0}
    lens, Hkv, D = _lengths(case), case["Hkv"], case["D"]
    if case["op"] == "weigh":
        rows = _rows(case)
        pairs = sum(r * (n - r) + r * (r + 1) // 2 for n, r in zip(lens, rows))
        bytes = sum(lens) * Hkv * (D * es + 4) + sum(n - r for n, r in zip(lens, rows)) * Hkv * 4
        return {"bytes": bytes + sum(rows) * (case["Hq"] * (D * es + 4) + Hkv * 4), "flops": 2 * case["Hq"] * D * pairs}
    m = case["budget"]
    # the weights and positions are looked at; all that is kept goes to another cache, or what is behind the budget into it
    moved = sum(min(n, m) if case["into"] else max(0, min(n - m, m)) for n in lens) * Hkv
    return {"bytes": sum(8 * n for n in lens if n > m or case["into"]) * Hkv + moved * (4 * D * es + 8), "flops": 0}


# ---- from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"select": _exact_select, "states": _exact_states, "cache": _exact_cache, "weigh": _exact_weigh, "evict": _exact_evict}[case["op"]](s)


def _exact_select(s):
    c = s["case"]
    B, W, V = s["logits"].shape
    out = {k: [] for k in ("token", "parent", "score", "ended", "length")}
    for b in range(B):
        best = []                                       # (rank, parent, token, score, ended, length)
        for w in range(W):
            base, n = float(s["scores"][b, w]), int(s["length"][b, w])
            if int(s["ended"][b, w]):
                best.append((base / max(n, 1) ** c["alpha"], w, s["eos"], base, 1, n))
                continue
            p = torch.log_softmax(s["logits"][b, w].double(), 0)
            value, token = torch.sort(p, dim=0, descending=True, stable=True)
            for x, t in zip(value[:c["K"]].tolist(), token[:c["K"]].tolist()):
                best.append(((base + x) / max(n + 1, 1) ** c["alpha"], w, t, base + x, int(t == s["eos"]), n + 1))
        best.sort(key=lambda e: (-e[0], e[1], e[2]))
        best += [(-math.inf, -1, -1, -math.inf, 1, 0)] * (c["K"] - len(best))         # where fewer pairs exist
        for name, k in (("parent", 1), ("token", 2), ("score", 3), ("ended", 4), ("length", 5)):
            out[name].append([e[k] for e in best[:c["K"]]])
    return {k: torch.tensor(v, dtype=torch.float64 if k == "score" else torch.int32) for k, v in out.items()}


def _exact_states(s):
    x = s["state"].double()
    return torch.stack([torch.stack([x[b, p] for p in row]) for b, row in enumerate(_parents(s["case"]))])


def _exact_cache(s):
    c, block = s["case"], s["case"]["block"]
    start, end = _lengths(c)
    table = s["table"].tolist() if block else None
    out = {}
    for name in ("k", "v"):
        x = s[name].double()
        y = x.clone()
        for b, row in enumerate(_parents(c)):
            for w, p in enumerate(row):
                to, frm = b * c["W"] + w, b * c["W"] + p
                if not block:
                    y[to, :, start[b]:end[b]] = x[frm, :, start[b]:end[b]]
                    continue
                for j in range(start[b] // block, -(-end[b] // block)):
                    a, z = max(start[b] - j * block, 0), min(end[b] - j * block, block)
                    if a < z:
                        y[table[to][j], :, a:z] = x[table[frm][j], :, a:z]
        out[name] = y
    return out


def _exact_line(s, name, b, h, n):
    """The first n keys (or values) of one sequence and head."""
    x, block = s[name], s["case"]["block"]
    if not block:
        return x[b, h, :n]
    return x[s["table"][b, :-(-n // block)].long(), h].reshape(-1, x.shape[-1])[:n]


def _exact_weigh(s):
    c = s["case"]
    lens, rows = _lengths(c), _rows(c)
    g = c["Hq"] // c["Hkv"]
    acc, pos = s["acc"].double(), s["pos"].clone()
    for b, (n, r) in enumerate(zip(lens, rows)):
        which = s["accept_path"][b, :r].long() if c["path"] else slice(0, r)
        before = n - r
        hidden = torch.ones(r, n, dtype=torch.bool, device=acc.device).triu(before + 1)
        pos[b, :, before:n] = torch.arange(before, n, device=acc.device, dtype=torch.int32) + (int(s["seen"][b]) - n)
        for h in range(c["Hkv"]):
            K = _exact_line(s, "k", b, h, n).double()
            total = torch.zeros(n, dtype=torch.float64, device=acc.device)
            for j in range(h * g, (h + 1) * g):
                x = s["q"][b, j, which].double() @ K.T * c["D"] ** -0.5 - s["lse"][b, j, which].double()[:, None]
                total += torch.exp(x.masked_fill_(hidden, -math.inf)).sum(0)
            acc[b, h, :before] *= c["decay"]
            acc[b, h, before:n] = 0.0
            acc[b, h, :n] += total
    return {"acc": acc, "pos": pos}


def _exact_evict(s):
    c, block, m = s["case"], s["case"]["block"], s["case"]["budget"]
    lens = _lengths(c)
    into = c["into"]
    k, v = (s["k_out"], s["v_out"]) if into and not block else (s["k"], s["v"])
    k, v = k.double(), v.double()
    acc, pos = (s["acc_out"].double(), s["pos_out"].clone()) if into else (s["acc"].double(), s["pos"].clone())
    weight, place = s["acc"].cpu().numpy(), s["pos"].cpu().numpy()
    for b, n in enumerate(lens):
        table = (s["out_table"] if into else s["table"])[b].long() if block else None
        for h in range(c["Hkv"]):
            w, at = weight[b, h, :n], place[b, h, :n]
            safe = (at < c["sink"]) | (at >= n - c["recent"])
            best = sorted(range(n), key=lambda j: (not safe[j], -w[j], j))[:m] if n > m else list(range(n))
            here, late = {j for j in best if j < m}, sorted(j for j in best if j >= m)
            source = torch.tensor([p if p in here else late.pop(0) for p in range(min(m, n))], device=k.device)
            p = torch.arange(len(source), device=k.device)
            for to, name in ((k, "k"), (v, "v")):
                line = _exact_line(s, name, b, h, n).double()[source]
                if block:
                    to[table[p // block], h, p % block] = line
                else:
                    to[b, h, :len(p)] = line
            acc[b, h, :len(p)], pos[b, h, :len(p)] = s["acc"][b, h, source].double(), s["pos"][b, h, source]
    return {"k": k, "v": v, "acc": acc, "pos": pos, "len": torch.tensor([min(n, m) for n in lens], dtype=torch.int32)}
