"""Cases of the cache operators of a decode step: attention for a tree of
drafted tokens over a slot's cache, the commit of the tree's accepted path, and
eviction from the cache by accumulated attention weight.

Each case is run in a plain form (elementary torch operations, fp32 arithmetic)
or, where ``own`` is true, through the calls that a user makes.
"""
import random

import torch

own = False

D = 128
PAGE = 128
BLOCK = 512


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one plain decode token of a small model with a short cache: the call's latency
        {"name": "tree one token", "op": "tree", "q_heads": 8, "kv_heads": 2, "nodes": 1, "lens": "17",
         "tree": 0, "paged": False, "scores": False},
        # four slots verifying small draft trees at the serving benchmark's context
        {"name": "tree 4x4 serving", "op": "tree", "q_heads": 40, "kv_heads": 8, "nodes": 4,
         "lens": "2047,2051,1999,2040", "tree": 1, "paged": False, "scores": False},
        # one slot with the widest tree, its scores kept for the weights that eviction goes by
        {"name": "tree 16 with scores", "op": "tree", "q_heads": 40, "kv_heads": 8, "nodes": 16, "lens": "2035",
         "tree": 2, "paged": False, "scores": True},
        # long contexts in pages, lengths that end inside a page
        {"name": "tree 4x3 long paged", "op": "tree", "q_heads": 32, "kv_heads": 8, "nodes": 3,
         "lens": "32757,16385,27000,20011", "tree": 3, "paged": True, "scores": False},
        # the longest cache one call takes, with the widest tree
        {"name": "tree 16 longest", "op": "tree", "q_heads": 40, "kv_heads": 8, "nodes": 16, "lens": "130800",
         "tree": 4, "paged": False, "scores": False},
        # no weights kept: the accepted path's rows move together, all layers of the 64-layer stack
        {"name": "commit rows", "op": "commit", "q_heads": 40, "kv_heads": 8, "layers": 64, "nodes": 4, "accepted": 3,
         "lens": "100,17,513,1000", "tree": 5, "weights": False},
        # one layer of a small model, one token accepted
        {"name": "commit one token", "op": "commit", "q_heads": 8, "kv_heads": 2, "layers": 1, "nodes": 1, "accepted": 1,
         "lens": "513", "tree": 0, "weights": True},
        # a verified tree of 16 over a few layers at the serving context
        {"name": "commit 16 layers weights", "op": "commit", "q_heads": 40, "kv_heads": 8, "layers": 16, "nodes": 16,
         "accepted": 5, "lens": "2051", "tree": 2, "weights": True},
        # a long cache: the weights of four slots' plain decode tokens
        {"name": "commit 4 slots long", "op": "commit", "q_heads": 32, "kv_heads": 8, "layers": 8, "nodes": 2,
         "accepted": 2, "lens": "32757,16385,27000,20011", "tree": 6, "weights": True},
        # the steady state of serving: one step's tokens over the budget, in every layer of four slots
        {"name": "evict steady", "op": "evict", "kv_heads": 8, "layers": 16, "slots": 4, "len": 2051, "budget": 2048,
         "sinks": 4, "recent": 256},
        # a small cache of one layer
        {"name": "evict small", "op": "evict", "kv_heads": 2, "layers": 1, "slots": 1, "len": 100, "budget": 67,
         "sinks": 1, "recent": 17},
        # a long prompt cut to a budget
        {"name": "evict prompt", "op": "evict", "kv_heads": 8, "layers": 8, "slots": 1, "len": 32757, "budget": 4096,
         "sinks": 4, "recent": 513},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    case = _draw(rng)
    most = 480e6  # bytes: no more than the largest listed case
    while work(case)["bytes"] > most or work(case)["flops"] > 40e9:
        case["lens"] = ",".join(str(v // 2) for v in _lens(case))
    return case


def _draw(rng):
    kv = rng.choice([1, 2, 4, 8])
    group = rng.randint(1, 8)
    op = rng.choice(["tree", "tree", "commit", "evict"])
    if op == "evict":
        layers, slots = rng.randint(1, 8), rng.randint(1, 4)
        n = _log(rng, 2, 32757 // slots)
        budget = max(1, min(n - 1, int(n * rng.random()) if rng.random() < 0.5 else n - rng.randint(1, 16)))
        sinks = rng.randint(0, min(4, budget))
        return {"op": op, "kv_heads": kv, "layers": layers, "slots": slots, "len": n, "budget": budget, "sinks": sinks,
                "recent": rng.randint(0, budget - sinks)}
    slots = rng.randint(1, 4)
    nodes = rng.randint(1, 16 // slots)
    top = (130000 if op == "tree" else 16385) // slots
    lens = ",".join(str(_log(rng, 1, top)) for _ in range(slots))
    case = {"op": op, "q_heads": kv * group, "kv_heads": kv, "nodes": nodes, "lens": lens, "tree": rng.randint(0, 1 << 20)}
    if op == "tree":
        case.update(paged=rng.random() < 0.5, scores=rng.random() < 0.3)
    else:
        case.update(layers=rng.randint(1, 8), accepted=rng.randint(1, nodes), weights=rng.random() < 0.8)
    return case


def _lens(case):
    return [int(v) for v in case["lens"].split(",")]


def _parents(case):
    """Per slot, the parent of each drafted node: tree 0 is a chain, others grow at random (node 0 is the first)."""
    rng = random.Random(case["tree"])
    n = case["nodes"]
    if case["tree"] == 0:
        return [list(range(-1, n - 1)) for _ in _lens(case)]
    return [[-1] + [rng.randrange(0, j) for j in range(1, n)] for _ in _lens(case)]


def _paths(case):
    """Per slot, the accepted nodes (ascending)."""
    rng = random.Random(case["tree"] + 1)
    return [sorted([0] + rng.sample(range(1, case["nodes"]), case["accepted"] - 1)) for _ in _lens(case)]


def work(case):
    if case["op"] == "tree":
        hq, hkv, n, lens = case["q_heads"], case["kv_heads"], case["nodes"], _lens(case)
        keys = sum(v + n for v in lens)
        rows = n * len(lens)
        b = keys * hkv * 2 * D * 2 + 2 * rows * hq * D * 4
        if case["scores"]:
            b += keys * n * hq * 4 + rows * hq * 8
        return {"bytes": b, "flops": 4 * D * hq * n * keys}
    if case["op"] == "commit":
        hq, hkv, L, a, lens = case["q_heads"], case["kv_heads"], case["layers"], case["accepted"], _lens(case)
        moved = sum(sum(1 for i, p in enumerate(path) if p != i) for path in _paths(case))
        b = moved * L * hkv * 2 * 2 * D * 2 + len(lens) * a * L * hkv * 4
        f = 0
        if case["weights"]:
            keys = sum(v + a for v in lens)
            b += keys * L * (hq * a * 4 + hkv * 8)
            f = keys * L * hq * a * 4
        return {"bytes": max(b, 1), "flops": f}
    heads, n, budget = case["kv_heads"] * case["layers"] * case["slots"], case["len"], case["budget"]
    free = max(1, n - case["sinks"] - case["recent"])
    moved = (n - budget) * max(0, budget - case["sinks"] - case["recent"] * budget / n) / free  # expected holes
    return {"bytes": heads * (n * 8 + budget * 8 + moved * 2 * 2 * D * 2), "flops": heads * n * 4}


# ------------------------------------------------------------------ inputs

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"tree": _prepare_tree, "commit": _prepare_commit, "evict": _prepare_evict}[case["op"]](case, g)


def _prepare_tree(case, g):
    hq, hkv, n, lens, parents = case["q_heads"], case["kv_heads"], case["nodes"], _lens(case), _parents(case)
    S, top = len(lens), max(_lens(case)) + n
    T = S * n
    anc = torch.zeros(S, n, n, dtype=torch.bool)
    for s, par in enumerate(parents):
        for j, p in enumerate(par):
            if p >= 0:
                anc[s, j] = anc[s, p]
            anc[s, j, j] = True
    st = {"case": case, "q": _normal(g, T, hq, D), "anc": anc.cuda(), "lens": torch.tensor(lens, device="cuda"), "top": top,
          "scores": None, "stats": None}
    if case["paged"]:
        per = [-(-(v + n) // PAGE) for v in lens]
        width, pages = max(per), sum(per)
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        st["k"] = _normal(g, pages, hkv, PAGE, D).half()
        st["v"] = _normal(g, pages, hkv, PAGE, D).half()
        table = torch.zeros(S, width, dtype=torch.int32, device="cuda")
        at = 0
        for s, c in enumerate(per):
            table[s, :c] = order[at:at + c]
            at += c
        st["table"] = table
    else:
        st["k"] = _normal(g, S, hkv, top, D).half()
        st["v"] = _normal(g, S, hkv, top, D).half()
    if case["scores"]:
        ld = -(-top // 4) * 4
        st["scores"] = torch.zeros(T, hq, ld, device="cuda")
        st["stats"] = torch.zeros(T, hq, 2, device="cuda")
    if own:
        import invariant_sequence_decode_gb300 as luce
        if case["paged"]:
            views = [luce.PagedTreeView(st["k"], st["v"], st["table"][s], lens[s], parents[s], s * n) for s in range(S)]
        else:
            views = [luce.TreeView(st["k"][s], st["v"][s], lens[s], parents[s], s * n) for s in range(S)]
        st["call"] = luce.TreeAttention(st["q"], views, hkv, D ** -0.5, scores=st["scores"], stats=st["stats"])
    return st


def _prepare_commit(case, g):
    hq, hkv, L, n, lens, paths = (case["q_heads"], case["kv_heads"], case["layers"], case["nodes"], _lens(case),
                                  _paths(case))
    S, top = len(lens), max(_lens(case)) + n
    st = {"case": case, "k": _normal(g, S, L, hkv, top, D).half(), "v": _normal(g, S, L, hkv, top, D).half(),
          "lens": torch.tensor(lens, device="cuda"), "paths": torch.tensor(paths, device="cuda"), "acc": None, "pos": None,
          "scores": None, "stats": None}
    if case["weights"]:
        T, ld = S * n, -(-top // 4) * 4
        st["acc"] = torch.rand(S, L, hkv, top, generator=g, device="cuda").square()
        st["pos"] = torch.arange(top, device="cuda", dtype=torch.int32).repeat(S, L, hkv, 1)
        sc = 2 * _normal(g, L, T, hq, ld)
        seen = torch.arange(ld, device="cuda") < (st["lens"] + n).repeat_interleave(n)[:, None]
        sc.masked_fill_(~seen[None, :, None, :], float("-inf"))
        m = sc.amax(-1)
        st["scores"], st["stats"] = sc, torch.stack([m, (sc - m[..., None]).exp().sum(-1)], -1)
    if own:
        import invariant_sequence_decode_gb300 as luce
        pick = lambda name, s: None if st[name] is None else st[name][s]  # noqa: E731
        slots = [luce.CommitSlot(st["k"][s], st["v"][s], lens[s], paths[s], row0=s * n, acc=pick("acc", s),
                                 pos=pick("pos", s), pos0=lens[s]) for s in range(S)]
        st["call"] = luce.TreeCommit(slots, hq, scores=st["scores"], stats=st["stats"])
    return st


def _prepare_evict(case, g):
    hkv, L, S, n = case["kv_heads"], case["layers"], case["slots"], case["len"]
    # accumulated weights: a few keys hold most of the weight, many hold none at all
    acc = torch.rand(S, L, hkv, n, generator=g, device="cuda").pow(8) * 4
    acc.masked_fill_(torch.rand(S, L, hkv, n, generator=g, device="cuda") < 0.05, 0.0)
    # earlier evictions left the keys in no order of their positions
    pos = torch.rand(S, L, hkv, n, generator=g, device="cuda").argsort(-1).to(torch.int32)
    st = {"case": case, "k": _normal(g, S, L, hkv, n, D).half(), "v": _normal(g, S, L, hkv, n, D).half(), "acc": acc,
          "pos": pos, "acc_out": torch.zeros_like(acc), "pos_out": torch.zeros_like(pos)}
    if own:
        import invariant_sequence_decode_gb300 as luce
        slots = [luce.EvictSlot(st["k"][s], st["v"][s], acc[s], pos[s], n, case["budget"], sinks=case["sinks"],
                                recent=case["recent"], next_pos=n, acc_out=st["acc_out"][s], pos_out=st["pos_out"][s])
                 for s in range(S)]
        st["call"] = luce.KvEvict(slots)
    return st


# ------------------------------------------------------------------ the operators

def run(st):
    op = st["case"]["op"]
    if own:
        st["call"]()
        if op == "tree":
            out = {"out": st["call"].out, "scores": st["scores"], "stats": st["stats"]}
        elif op == "commit":
            out = {"k": st["k"], "v": st["v"], "acc": st["acc"], "pos": st["pos"]}
        else:
            out = {"k": st["k"], "v": st["v"], "acc": st["acc_out"], "pos": st["pos_out"]}
        return {k: v for k, v in out.items() if v is not None}
    return {"tree": _plain_tree, "commit": _plain_commit, "evict": _plain_evict}[op](st)


def _seen(st, dtype=None):
    """[S, nodes, keys]: the cache positions that each node sees."""
    n, col = st["case"]["nodes"], torch.arange(st["top"], device="cuda")
    j = col - st["lens"][:, None]                                             # index in the tree
    tree = st["anc"].gather(2, j.clamp(0, n - 1)[:, None, :].expand(-1, n, -1)) & ((j >= 0) & (j < n))[:, None, :]
    return (j < 0)[:, None, :] | tree


def _flat(st, x):
    """The caches as [S, kv_heads, keys, D]."""
    if not st["case"]["paged"]:
        return x
    t = st["table"].long()
    return x[t].permute(0, 2, 1, 3, 4).reshape(t.shape[0], x.shape[1], t.shape[1] * PAGE, D)[:, :, :st["top"]]


def _plain_tree(st):
    c = st["case"]
    hq, hkv, n = c["q_heads"], c["kv_heads"], c["nodes"]
    S, G = st["lens"].shape[0], hq // hkv
    q = st["q"].view(S, n, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(S, hkv, n * G, D)
    s = (q @ _flat(st, st["k"]).float().transpose(2, 3)) * D ** -0.5
    s = s.view(S, hkv, n, G, -1).masked_fill(~_seen(st)[:, None, :, None, :], float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = (s - m).exp()
    l = p.sum(-1, keepdim=True)
    # summed in blocks of keys: one long 32-bit sum would lose digits that the result needs
    short = -st["top"] % BLOCK
    p = torch.nn.functional.pad(p, (0, short)).view(S, hkv, n * G, -1, BLOCK).transpose(2, 3)
    v = torch.nn.functional.pad(_flat(st, st["v"]).float(), (0, 0, 0, short)).view(S, hkv, -1, BLOCK, D)
    o = (p @ v).sum(2).view(S, hkv, n, G, D) / l
    rows = lambda x: x.permute(0, 2, 1, 3, 4).reshape(S * n, hq, -1)  # noqa: E731
    out = {"out": rows(o)}
    if c["scores"]:
        buf = st["scores"].clone()
        own_cols = torch.arange(st["top"], device="cuda") < (st["lens"] + n).repeat_interleave(n)[:, None, None]
        buf[:, :, :st["top"]] = torch.where(own_cols, rows(s), buf[:, :, :st["top"]])
        out["scores"] = buf
        out["stats"] = torch.cat([rows(m), rows(l)], -1)
    return out


def _plain_commit(st):
    c = st["case"]
    lens, paths, k, v = st["lens"], st["paths"], st["k"], st["v"]
    S, A = paths.shape
    slot = torch.arange(S, device="cuda")[:, None]
    new = lens[:, None] + torch.arange(A, device="cuda")
    old = lens[:, None] + paths
    k[slot, :, :, new] = k[slot, :, :, old]
    v[slot, :, :, new] = v[slot, :, :, old]
    if not c["weights"]:
        return {"k": k, "v": v}
    L, hkv, top = c["layers"], c["kv_heads"], st["acc"].shape[-1]
    rows = slot * c["nodes"] + paths                                           # the accepted rows
    w = (st["scores"][:, rows, :, :top] - st["stats"][:, rows, :, 0, None]).exp() / st["stats"][:, rows, :, 1, None]
    w = w.view(L, S, A, hkv, -1, top).sum((2, 4)).transpose(0, 1)              # [S, L, kv_heads, keys]
    col = torch.arange(top, device="cuda")
    st["acc"].add_(torch.where((col < lens[:, None])[:, None, None, :], w, torch.zeros_like(w)))
    st["acc"][slot, :, :, new] = w[slot, :, :, old]
    st["pos"][slot, :, :, new] = new.to(torch.int32)[:, :, None, None]
    return {"k": k, "v": v, "acc": st["acc"], "pos": st["pos"]}


def _plain_evict(st):
    c = st["case"]
    n, budget = c["len"], c["budget"]
    acc, pos = st["acc"].view(-1, n), st["pos"].view(-1, n)
    k, v = st["k"].view(-1, n, D), st["v"].view(-1, n, D)
    kept = (pos < c["sinks"]) | (pos >= n - c["recent"])
    key = torch.where(kept, torch.full_like(acc, float("inf")), torch.where(acc.isnan(), torch.full_like(acc, -float("inf")), acc))
    # ascending; of equal keys the one with the highest index leaves first
    leave = n - 1 - key.flip(-1).sort(dim=-1, stable=True).indices[:, :n - budget]
    out = torch.zeros_like(kept).scatter_(1, leave, True)
    col = torch.arange(n, device="cuda")
    most = min(budget, n - budget)
    last = torch.full_like(leave, n - 1)
    hole = torch.where(out & (col < budget), col, n).sort(dim=-1).values[:, :most]
    come = torch.where(~out & (col >= budget), col, n).sort(dim=-1).values[:, :most]
    # where there are fewer holes than that, the last key is copied onto itself
    hole, come = torch.where(hole < n, hole, last[:, :most]), torch.where(come < n, come, last[:, :most])
    head = torch.arange(acc.shape[0], device="cuda")[:, None]
    k[head, hole] = k[head, come]
    v[head, hole] = v[head, come]
    a, p = acc.scatter(1, hole, acc.gather(1, come)), pos.scatter(1, hole, pos.gather(1, come))
    st["acc_out"].view(-1, n)[:, :budget] = a[:, :budget]
    st["pos_out"].view(-1, n)[:, :budget] = p[:, :budget]
    return {"k": st["k"], "v": st["v"], "acc": st["acc_out"], "pos": st["pos_out"]}


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"tree": _exact_tree, "commit": _exact_commit, "evict": _exact_evict}[case["op"]](case, st)


def _exact_tree(case, st):
    hq, hkv, n, lens, parents = case["q_heads"], case["kv_heads"], case["nodes"], _lens(case), _parents(case)
    G = hq // hkv
    out = torch.empty(len(lens) * n, hq, D, dtype=torch.float64, device="cuda")
    scores = None if st["scores"] is None else st["scores"].double()
    stats = None if st["stats"] is None else st["stats"].double()
    for s, cached in enumerate(lens):
        if case["paged"]:
            pages = st["table"][s, :-(-(cached + n) // PAGE)].long()
            k, v = (x[pages].transpose(0, 1).reshape(hkv, -1, D) for x in (st["k"], st["v"]))
        else:
            k, v = st["k"][s], st["v"][s]
        for j in range(n):
            path, at = [], j
            while at >= 0:
                path.insert(0, cached + at)
                at = parents[s][at]
            keys = torch.cat([torch.arange(cached), torch.tensor(path)]).cuda()
            for g in range(hkv):
                q = st["q"][s * n + j, g * G:(g + 1) * G].double()
                x = torch.einsum("hd,kd->hk", q, k[g, keys].double()) / D ** 0.5
                w = torch.softmax(x, 1)
                out[s * n + j, g * G:(g + 1) * G] = torch.einsum("hk,kd->hd", w, v[g, keys].double())
                if scores is not None:
                    scores[s * n + j, g * G:(g + 1) * G, :cached + n] = float("-inf")
                    scores[s * n + j, g * G:(g + 1) * G, keys] = x
                    top = x.max(1).values
                    stats[s * n + j, g * G:(g + 1) * G, 0] = top
                    stats[s * n + j, g * G:(g + 1) * G, 1] = torch.exp(torch.logsumexp(x, 1) - top)
    return {"out": out} if scores is None else {"out": out, "scores": scores, "stats": stats}


def _exact_commit(case, st):
    lens, paths, hkv, n = _lens(case), _paths(case), case["kv_heads"], case["nodes"]
    k, v = st["k"].clone(), st["v"].clone()
    for s, cached in enumerate(lens):
        for i, a in enumerate(paths[s]):
            k[s, :, :, cached + i] = st["k"][s, :, :, cached + a]
            v[s, :, :, cached + i] = st["v"][s, :, :, cached + a]
    if not case["weights"]:
        return {"k": k, "v": v}
    acc, pos = st["acc"].double(), st["pos"].clone()
    for s, cached in enumerate(lens):
        for layer in range(case["layers"]):
            w = torch.zeros(hkv, acc.shape[-1], dtype=torch.float64, device="cuda")
            for a in paths[s]:
                x = st["scores"][layer, s * n + a, :, :acc.shape[-1]].double()
                m, l = st["stats"][layer, s * n + a].double().unbind(-1)
                w += (torch.exp(x - m[:, None]) / l[:, None]).view(hkv, -1, acc.shape[-1]).sum(1)
            acc[s, layer, :, :cached] += w[:, :cached]
            for i, a in enumerate(paths[s]):
                acc[s, layer, :, cached + i] = w[:, cached + a]
        for i in range(len(paths[s])):
            pos[s, :, :, cached + i] = cached + i
    return {"k": k, "v": v, "acc": acc, "pos": pos}


def _exact_evict(case, st):
    import numpy as np
    n, budget = case["len"], case["budget"]
    acc, pos = st["acc"].double().cpu().numpy().reshape(-1, n), st["pos"].cpu().numpy().reshape(-1, n)
    acc_out, pos_out = np.zeros_like(acc), np.zeros_like(pos)
    k, v = st["k"].view(-1, n, D), st["v"].view(-1, n, D)
    for h in range(acc.shape[0]):
        held = (pos[h] < case["sinks"]) | (pos[h] >= n - case["recent"])
        leave = np.lexsort((-np.arange(n), acc[h], held))[:n - budget]
        stays = np.ones(n, dtype=bool)
        stays[leave] = False
        hole, come = np.flatnonzero(~stays[:budget]), budget + np.flatnonzero(stays[budget:])
        at = np.arange(budget)
        at[hole] = come
        acc_out[h, :budget], pos_out[h, :budget] = acc[h, at], pos[h, at]
        if len(hole):
            to, frm = torch.from_numpy(hole).cuda(), torch.from_numpy(come).cuda()
            k[h, to], v[h, to] = k[h, frm], v[h, frm]
    shape = st["acc"].shape
    return {"k": st["k"], "v": st["v"], "acc": torch.from_numpy(acc_out).view(shape), "pos": torch.from_numpy(pos_out).view(shape)}
