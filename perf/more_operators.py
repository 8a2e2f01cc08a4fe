"""Cases of the operators of a slot's cache in 8 bits: the pass that norms, rotates
and appends a projection's rows, the sealing of whole blocks of tokens into
8-bit codes, and attention over sealed blocks, the tail behind them and a
draft tree, with or without a sliding window.

Each case is run in a plain form (elementary torch operations, fp32 arithmetic)
or, where ``own`` is true, through the calls that a user makes.
"""
import random

import torch

own = False

D = 128
PAGE = 128   # tokens of a page
BLOCK = 32   # tokens that share a scale
LONG = 512   # keys of a partial sum
THETA = 1e6
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one plain decode token of a small model with a short cache, nothing sealed yet: the call's latency
        {"name": "attend one token", "op": "attend", "q_heads": 8, "kv_heads": 2, "nodes": 1, "lens": "17", "tree": 0,
         "paged": False, "window": 0, "sinks": 0},
        # plain decode of four slots at the serving benchmark's context
        {"name": "attend 4x1 serving", "op": "attend", "q_heads": 40, "kv_heads": 8, "nodes": 1, "lens": "2047,2051,1999,2040",
         "tree": 0, "paged": False, "window": 0, "sinks": 0},
        # the same slots verifying small draft trees
        {"name": "attend 4x4 serving", "op": "attend", "q_heads": 40, "kv_heads": 8, "nodes": 4, "lens": "2047,2051,1999,2040",
         "tree": 1, "paged": False, "window": 0, "sinks": 0},
        # long contexts in pages, lengths that end inside a page and a block
        {"name": "attend 4x1 long paged", "op": "attend", "q_heads": 32, "kv_heads": 8, "nodes": 1,
         "lens": "32757,16385,27000,20011", "tree": 0, "paged": True, "window": 0, "sinks": 0},
        # the longest cache one call takes, with the widest tree
        {"name": "attend 16 longest", "op": "attend", "q_heads": 40, "kv_heads": 8, "nodes": 16, "lens": "130800", "tree": 2,
         "paged": False, "window": 0, "sinks": 0},
        # a layer that attends to a window and the first tokens, trees over long contexts
        {"name": "attend 4x4 window", "op": "attend", "q_heads": 40, "kv_heads": 8, "nodes": 4,
         "lens": "32757,16385,27000,20011", "tree": 3, "paged": True, "window": 4096, "sinks": 4},
        # a small cache's first block of one layer
        {"name": "seal one block", "op": "seal", "kv_heads": 2, "layers": 1, "lens": "33", "sealed": 0, "paged": False},
        # steady serving: the block that each of four slots has filled, in every layer
        {"name": "seal steady", "op": "seal", "kv_heads": 8, "layers": 64, "lens": "32,35,33,47", "sealed": 2016, "paged": True},
        # a long prompt's cache after its prefill
        {"name": "seal prompt", "op": "seal", "kv_heads": 8, "layers": 4, "lens": "32757", "sealed": 0, "paged": False},
        # one decode token of a small model
        {"name": "project one row", "op": "project", "q_heads": 8, "kv_heads": 2, "rows": "1", "axes": 1, "norm": True},
        # the widest verify step: four slots with four rows each
        {"name": "project 4x4 rows", "op": "project", "q_heads": 40, "kv_heads": 8, "rows": "4,4,4,4", "axes": 1, "norm": True},
        # a prompt with images: positions in time, height and width
        {"name": "project prompt", "op": "project", "q_heads": 40, "kv_heads": 8, "rows": "8192", "axes": 3, "norm": True},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    case = _draw(rng)
    while work(case)["bytes"] > 800e6 or work(case)["flops"] > 43e9:  # no more than the largest listed case
        case["lens"] = ",".join(str(v // 2) for v in _list(case["lens"]))
    return case


def _draw(rng):
    kv = rng.choice([1, 2, 4, 8])
    group = rng.randint(1, 8)
    op = rng.choice(["attend", "attend", "seal", "project"])
    slots = rng.randint(1, 4)
    if op == "attend":
        nodes = rng.randint(1, 16 // slots)
        lens = ",".join(str(_log(rng, 1, 130000 // slots)) for _ in range(slots))
        window = 0 if rng.random() < 0.6 else _log(rng, 1, 20000)
        return {"op": op, "q_heads": kv * group, "kv_heads": kv, "nodes": nodes, "lens": lens, "tree": rng.randint(0, 1 << 20),
                "paged": rng.random() < 0.5, "window": window, "sinks": rng.randint(0, 200) if window else 0}
    if op == "seal":
        lens = ",".join(str(_log(rng, BLOCK, 16000 // slots)) for _ in range(slots))
        return {"op": op, "kv_heads": kv, "layers": rng.randint(1, 8), "lens": lens, "sealed": BLOCK * rng.randint(0, 20),
                "paged": rng.random() < 0.5}
    rows = ",".join(str(_log(rng, 1, 8000 // slots)) for _ in range(slots))
    return {"op": op, "q_heads": kv * group, "kv_heads": kv, "rows": rows, "axes": rng.choice([1, 2, 3]), "norm": rng.random() < 0.8}


def _list(text):
    return [int(v) for v in text.split(",")]


def _split(case):
    """Per slot, the keys in sealed blocks and those in the tail."""
    return [(v // BLOCK * BLOCK, v % BLOCK) for v in _list(case["lens"])]


def _parents(case):
    """Per slot, the parent of each drafted node: tree 0 is a chain, others grow at random (node 0 is the first)."""
    rng = random.Random(case["tree"])
    n = case["nodes"]
    if case["tree"] == 0:
        return [list(range(-1, n - 1)) for _ in _list(case["lens"])]
    return [[-1] + [rng.randrange(0, j) for j in range(1, n)] for _ in _list(case["lens"])]


def _pair_axis(axes):
    """The axis of each of the 64 pairs: half of the slow ones for time where there are several, as sections in a row."""
    return {1: [0] * 64, 2: [0] * 32 + [1] * 32, 3: [0] * 16 + [1] * 24 + [2] * 24}[axes]


def work(case):
    if case["op"] == "attend":
        hq, hkv, n = case["q_heads"], case["kv_heads"], case["nodes"]
        sealed = tail = 0
        for s, t in _split(case):
            if case["window"]:
                first = max(0, s + t + 1 - case["window"])
                seen = min(s, case["sinks"]) + max(0, s - max(first, case["sinks"]))
            else:
                seen = s
            sealed, tail = sealed + seen, tail + t + n
        rows = n * len(_split(case))
        b = sealed * hkv * (2 * D + 8 / BLOCK) + tail * hkv * 2 * D * 2 + 2 * rows * hq * D * 4
        return {"bytes": b, "flops": 4 * D * hq * n * (sealed + tail)}
    if case["op"] == "seal":
        heads = case["layers"] * case["kv_heads"]
        whole = sum(v // BLOCK * BLOCK for v in _list(case["lens"]))
        rest = sum(v % BLOCK for v in _list(case["lens"]) if v >= BLOCK)
        return {"bytes": max(1, heads * 2 * (whole * (2 * D + D + 4 / BLOCK) + rest * 4 * D)), "flops": heads * 4 * D * whole}
    hq, hkv, rows = case["q_heads"], case["kv_heads"], sum(_list(case["rows"]))
    return {"bytes": rows * ((hq + 2 * hkv) * D * 4 + hq * D * 4 + 2 * hkv * D * 2 + 4 * case["axes"]),
            "flops": rows * (hq + hkv) * D * (7 if case["norm"] else 3)}


# ------------------------------------------------------------------ inputs

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"attend": _prepare_attend, "seal": _prepare_seal, "project": _prepare_project}[case["op"]](case, g)


def _codes(x, dims):
    """x [..] in codes with one scale over the given dims."""
    scale = x.abs().amax(dims, keepdim=True) / 127
    return (x / scale).round().clamp(-127, 127).to(torch.int8), scale


def _pages(case, per, g):
    """The table of each slot's pages, and their number: in a row, or shuffled."""
    total = max(1, sum(per))
    order = torch.randperm(total, generator=g, device="cuda") if case["paged"] else torch.arange(total, device="cuda")
    table = torch.zeros(len(per), max(1, max(per)), dtype=torch.int32, device="cuda")
    at = 0
    for s, c in enumerate(per):
        table[s, :c] = order[at:at + c].to(torch.int32)
        at += c
    return table, total


def _prepare_attend(case, g):
    hq, hkv, n, split, parents = case["q_heads"], case["kv_heads"], case["nodes"], _split(case), _parents(case)
    S = len(split)
    per = [-(-s // PAGE) for s, _ in split]
    table, total = _pages(case, per, g)
    anc = torch.zeros(S, n, n, dtype=torch.bool)
    for s, par in enumerate(parents):
        for j, p in enumerate(par):
            if p >= 0:
                anc[s, j] = anc[s, p]
            anc[s, j, j] = True
    st = {"case": case, "q": _normal(g, S * n, hq, D), "table": table, "anc": anc.cuda(), "depth": anc.sum(-1).cuda() - 1,
          "sealed": torch.tensor([s for s, _ in split], device="cuda"), "tail": torch.tensor([t for _, t in split], device="cuda")}
    # keys: some dims are larger than others, as behind a projection; blocks differ in size
    k = _normal(g, total, hkv, 4, BLOCK, D) * (0.5 + torch.rand(D, generator=g, device="cuda"))
    k *= 0.5 + torch.rand(total, hkv, 4, 1, 1, generator=g, device="cuda")
    kc, ks = _codes(k, (3, 4))
    del k
    vc, vs = _codes(_normal(g, total, hkv, D, 4, BLOCK) * (0.2 + 2 * torch.rand(total, hkv, 1, 4, 1, generator=g, device="cuda")), (2, 4))
    st["k_codes"], st["v_codes"] = kc.view(total, hkv, PAGE, D), vc.view(total, hkv, D, PAGE)
    st["scales"] = torch.stack([ks.view(total, hkv, 4), vs.view(total, hkv, 4)], 2)
    cap = BLOCK + n
    st["k"], st["v"] = _normal(g, S, hkv, cap, D).half(), _normal(g, S, hkv, cap, D).half()
    if own:
        import invariant_sequence_decode_gb300 as luce
        views, at = [], 0
        for s, (sealed, tail) in enumerate(split):
            pools = [st[x] if case["paged"] else st[x][at:at + per[s]] for x in ("k_codes", "v_codes", "scales")]
            views.append(luce.Q8View(*pools, sealed, st["k"][s], st["v"][s], tail, parents[s], s * n,
                                     table=st["table"][s] if case["paged"] else None, window=case["window"], sinks=case["sinks"]))
            at += per[s]
        st["call"] = luce.Q8Attention(st["q"], views, hkv, D ** -0.5)
    return st


def _prepare_seal(case, g):
    hkv, L, lens, sealed = case["kv_heads"], case["layers"], _list(case["lens"]), case["sealed"]
    S, cap = len(lens), max(lens) + 1
    per = [-(-(sealed + v) // PAGE) for v in lens]
    table, total = _pages(case, per, g)
    st = {"case": case, "table": table, "k": _normal(g, S, L, hkv, cap, D).half(), "v": _normal(g, S, L, hkv, cap, D).half(),
          "k_codes": torch.zeros(total, L, hkv, PAGE, D, dtype=torch.int8, device="cuda"),
          "v_codes": torch.zeros(total, L, hkv, D, PAGE, dtype=torch.int8, device="cuda"),
          "scales": torch.zeros(total, L, hkv, 2, 4, device="cuda")}
    # the slots' whole blocks, one after the other: slot, first row of the tail, page, block of the page
    whole = [(s, b) for s, v in enumerate(lens) for b in range(v // BLOCK)]
    st["slot"] = torch.tensor([s for s, _ in whole], dtype=torch.int64, device="cuda")
    at = torch.tensor([b for _, b in whole], dtype=torch.int64, device="cuda")
    st["row"] = at * BLOCK
    key = sealed // BLOCK + at
    st["page"], st["quarter"] = st["table"][st["slot"], key // 4].long(), key % 4
    # the rows behind them, which move to the front
    rest = [(s, j, v // BLOCK * BLOCK + j) for s, v in enumerate(lens) if v >= BLOCK for j in range(v % BLOCK)]
    st["rest"] = [torch.tensor([r[i] for r in rest], dtype=torch.int64, device="cuda") for i in range(3)]
    if own:
        import invariant_sequence_decode_gb300 as luce
        slots, at = [], 0
        for s, v in enumerate(lens):
            pools = [st[x] if case["paged"] else st[x][at:at + per[s]] for x in ("k_codes", "v_codes", "scales")]
            slots.append(luce.Q8Slot(st["k"][s], st["v"][s], v, *pools, sealed, table=st["table"][s] if case["paged"] else None))
            at += per[s]
        st["call"] = luce.Q8Seal(slots)
    return st


def _prepare_project(case, g):
    hq, hkv, rows, axes = case["q_heads"], case["kv_heads"], _list(case["rows"]), case["axes"]
    S, T, cap = len(rows), sum(rows), max(rows) + 5
    st = {"case": case, "qkv": _normal(g, T, (hq + 2 * hkv) * D) * 3, "q_gamma": None, "k_gamma": None,
          "k": torch.zeros(S, hkv, cap, D, dtype=torch.float16, device="cuda"),
          "v": torch.zeros(S, hkv, cap, D, dtype=torch.float16, device="cuda"),
          "pos": torch.randint(0, 32768, (axes, T), generator=g, device="cuda", dtype=torch.int32),
          "slot": torch.repeat_interleave(torch.arange(S), torch.tensor(rows)).cuda(),
          "at": torch.cat([torch.arange(5, 5 + r) for r in rows]).cuda(), "pair_axis": torch.tensor(_pair_axis(axes), device="cuda")}
    if case["norm"]:
        st["q_gamma"], st["k_gamma"] = 1 + 0.2 * _normal(g, D), 1 + 0.2 * _normal(g, D)
    if own:
        import invariant_sequence_decode_gb300 as luce
        views, row = [], 0
        for s, r in enumerate(rows):
            views.append(luce.SeqView(st["k"][s], st["v"][s], 5 + r, r, row))
            row += r
        st["call"] = luce.QkNormRope(st["qkv"], views, hq, st["pos"], THETA, q_gamma=st["q_gamma"], k_gamma=st["k_gamma"], eps=EPS,
                                     pair_axis=_pair_axis(axes))
    return st


# ------------------------------------------------------------------ the operators

def run(st):
    op = st["case"]["op"]
    if own:
        st["call"]()
        if op == "attend":
            return {"out": st["call"].out}
        if op == "seal":
            return {x: st[x] for x in ("k_codes", "v_codes", "scales", "k", "v")}
        return {"q": st["call"].out, "k": st["k"], "v": st["v"]}
    return {"attend": _plain_attend, "seal": _plain_seal, "project": _plain_project}[op](st)


def _plain_attend(st):
    c = st["case"]
    hq, hkv, n = c["q_heads"], c["kv_heads"], c["nodes"]
    S, G, W = st["sealed"].shape[0], hq // hkv, st["table"].shape[1] * PAGE
    t = st["table"].long()
    ks, vs = st["scales"][t].repeat_interleave(BLOCK, -1).permute(3, 0, 2, 1, 4)        # [S, kv_heads, pages, keys]
    k = st["k_codes"][t].permute(0, 2, 1, 3, 4).float() * ks[..., None]
    v = st["v_codes"][t].permute(0, 2, 1, 4, 3).float() * vs[..., None]
    k = torch.cat([k.reshape(S, hkv, W, D), st["k"].float()], 2)
    v = torch.cat([v.reshape(S, hkv, W, D), st["v"].float()], 2)
    # each key's position, and whether a node sees it
    col, j = torch.arange(W, device="cuda").expand(S, W), torch.arange(st["k"].shape[2], device="cuda").expand(S, -1)
    node = j - st["tail"][:, None]                                                     # index in the tree
    inside = (node >= 0) & (node < n)
    path = st["anc"].gather(2, node.clamp(0, n - 1)[:, None, :].expand(-1, n, -1)) & inside[:, None, :]
    seen = torch.cat([(col < st["sealed"][:, None])[:, None, :].expand(-1, n, -1), (node < 0)[:, None, :] | path], 2)
    total = (st["sealed"] + st["tail"])[:, None]
    pos = torch.cat([col, torch.where(inside, total + st["depth"].gather(1, node.clamp(0, n - 1)), st["sealed"][:, None] + j)], 1)
    if c["window"]:
        seen &= (pos < c["sinks"])[:, None, :] | ((total + st["depth"])[:, :, None] - pos[:, None, :] < c["window"])
    q = st["q"].view(S, n, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(S, hkv, n * G, D)
    s = (q @ k.transpose(2, 3)) * D ** -0.5
    s = s.view(S, hkv, n, G, -1).masked_fill(~seen[:, None, :, None, :], float("-inf"))
    p = (s - s.amax(-1, keepdim=True)).exp()
    l = p.sum(-1, keepdim=True)
    # summed in blocks of keys: one long 32-bit sum would lose digits that the result needs
    short = -p.shape[-1] % LONG
    p = torch.nn.functional.pad(p, (0, short)).view(S, hkv, n * G, -1, LONG).transpose(2, 3)
    v = torch.nn.functional.pad(v, (0, 0, 0, short)).view(S, hkv, -1, LONG, D)
    o = (p @ v).sum(2).view(S, hkv, n, G, D) / l
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(S * n, hq, D)}


def _plain_seal(st):
    L, hkv = st["k"].shape[1:3]
    k_scale, k_codes = _plain_blocks(st, st["k"])
    v_scale, v_codes = _plain_blocks(st, st["v"])
    st["scales"][st["page"], :, :, 0, st["quarter"]] = k_scale
    st["scales"][st["page"], :, :, 1, st["quarter"]] = v_scale
    st["k_codes"].view(-1, L, hkv, 4, BLOCK, D)[st["page"], :, :, st["quarter"]] = k_codes.permute(0, 2, 3, 1, 4)
    st["v_codes"].view(-1, L, hkv, D, 4, BLOCK)[st["page"], :, :, :, st["quarter"]] = v_codes.permute(0, 2, 3, 4, 1)
    s, to, frm = st["rest"]
    st["k"][s, :, :, to] = st["k"][s, :, :, frm]
    st["v"][s, :, :, to] = st["v"][s, :, :, frm]
    return {x: st[x] for x in ("k_codes", "v_codes", "scales", "k", "v")}


def _plain_blocks(st, x):
    """The scales [blocks, L, kv_heads] and codes [blocks, BLOCK, L, kv_heads, D] of the tails' whole blocks."""
    row = st["row"][:, None] + torch.arange(BLOCK, device="cuda")
    b = x[st["slot"][:, None], :, :, row].float()
    top = b.abs().amax((1, 4))
    d = top / torch.full_like(top, 127)  # a division: by a number, torch multiplies by its reciprocal
    f = torch.where(d[:, None, :, :, None] > 0, b / d[:, None, :, :, None], torch.zeros_like(b))
    # halves away from zero; the sum in 64 bits, as one in 32 could round up to the next code
    return d, ((f.abs().double() + 0.5).floor().clamp(max=127) * f.sign()).to(torch.int8)


def _plain_project(st):
    c = st["case"]
    hq, hkv = c["q_heads"], c["kv_heads"]
    x = st["qkv"].view(-1, hq + 2 * hkv, D)
    i = torch.arange(64, device="cuda", dtype=torch.float64)
    angle = st["pos"][st["pair_axis"]].t().double() * THETA ** (-i / 64)               # [T, 64]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(h, gamma):
        if gamma is not None:
            h = h / (h.square().mean(-1, keepdim=True) + EPS).sqrt() * gamma
        a, b = h[..., :64], h[..., 64:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)

    q = turned(x[:, :hq], st["q_gamma"])
    st["k"][st["slot"], :, st["at"]] = turned(x[:, hq:hq + hkv], st["k_gamma"]).half()
    st["v"][st["slot"], :, st["at"]] = x[:, hq + hkv:].half()
    return {"q": q, "k": st["k"], "v": st["v"]}


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"attend": _exact_attend, "seal": _exact_seal, "project": _exact_project}[case["op"]](case, st)


def _exact_attend(case, st):
    hq, hkv, n, parents = case["q_heads"], case["kv_heads"], case["nodes"], _parents(case)
    G = hq // hkv
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    for s, (sealed, tail) in enumerate(_split(case)):
        total = sealed + tail
        pages = st["table"][s, :-(-sealed // PAGE)].long()
        for g in range(hkv):
            scale = st["scales"][pages, g].double()
            k = st["k_codes"][pages, g].double().view(-1, 4, BLOCK, D) * scale[:, 0, :, None, None]
            v = st["v_codes"][pages, g].double().view(-1, D, 4, BLOCK) * scale[:, 1, None, :, None]
            k = torch.cat([k.view(-1, D)[:sealed], st["k"][s, g].double()])
            v = torch.cat([v.permute(0, 2, 3, 1).reshape(-1, D)[:sealed], st["v"][s, g].double()])
            for j in range(n):
                path, at = [], j
                while at >= 0:
                    path.insert(0, at)
                    at = parents[s][at]
                where = torch.cat([torch.arange(total), total + torch.tensor(path)])
                place = torch.arange(total + len(path))
                if case["window"]:
                    keep = (place < case["sinks"]) | (place > total + len(path) - 1 - case["window"])
                    where = where[keep]
                keys = where.cuda()
                x = st["q"][s * n + j, g * G:(g + 1) * G].double() @ k[keys].t() / D ** 0.5
                out[s * n + j, g * G:(g + 1) * G] = torch.softmax(x, 1) @ v[keys]
    return {"out": out}


def _exact_seal(case, st):
    lens, L = _list(case["lens"]), case["layers"]
    got = {x: st[x].clone() for x in ("k_codes", "v_codes", "k", "v")}
    got["scales"] = st["scales"].double()
    for s, v in enumerate(lens):
        nb = v // BLOCK
        if nb == 0:
            continue
        for layer in range(L):
            for which, x in enumerate("kv"):
                rows = st[x][s, layer, :, :nb * BLOCK].double().view(-1, nb, BLOCK * D)
                scale = (rows.abs().max(2).values / 127.0).float().double()
                # the quotient is a 32-bit one by definition: 64 bits hold it to be rounded once more
                quo = (rows / scale[:, :, None]).nan_to_num(0.0).float().double()
                code = torch.copysign(torch.floor(quo.abs() + 0.5), quo).to(torch.int8).view(-1, nb, BLOCK, D)
                key = case["sealed"] // BLOCK + torch.arange(nb)
                for quarter in range(4):
                    pick = (key % 4 == quarter).nonzero()[:, 0].cuda()
                    page = st["table"][s].long()[key[pick.cpu()].cuda() // 4]
                    got["scales"][page, layer, :, which, quarter] = scale[:, pick].t()
                    span = slice(quarter * BLOCK, (quarter + 1) * BLOCK)
                    part = code[:, pick].transpose(0, 1)
                    if which == 0:
                        got["k_codes"][page, layer, :, span] = part
                    else:
                        got["v_codes"][page, layer, :, :, span] = part.transpose(2, 3)
                got[x][s, layer, :, :v - nb * BLOCK] = st[x][s, layer, :, nb * BLOCK:v]
    return got


def _exact_project(case, st):
    hq, hkv, rows = case["q_heads"], case["kv_heads"], _list(case["rows"])
    axis = _pair_axis(case["axes"])
    q = torch.empty(sum(rows), hq, D, dtype=torch.float64, device="cuda")
    k, v = st["k"].double(), st["v"].double()
    pos = st["pos"].double()
    turn = torch.stack([torch.polar(torch.ones_like(pos[0]), pos[axis[i]] * THETA ** (-2 * i / D)) for i in range(64)], 1)
    row = 0
    for s, r in enumerate(rows):
        part = slice(row, row + r)
        row += r
        for h in range(hq + 2 * hkv):
            x = st["qkv"][part, h * D:(h + 1) * D].double()
            if h >= hq + hkv:
                v[s, h - hq - hkv, 5:5 + r] = x
                continue
            gamma = st["q_gamma"] if h < hq else st["k_gamma"]
            if gamma is not None:
                x = x * gamma.double() * (x.pow(2).sum(1, keepdim=True) / D + EPS).rsqrt()
            z = torch.complex(x[:, :64].contiguous(), x[:, 64:].contiguous()) * turn[part]
            y = torch.cat([z.real, z.imag], 1)
            if h < hq:
                q[part, h] = y
            else:
                k[s, h - hq, 5:5 + r] = y
    return {"q": q, "k": k, "v": v}
