"""The decode step over draft trees: a node's hidden state, logits and K/V rows
are the bits of a step over its own path; chains agree with the plain step; and
the step, the commit and eviction run together as a decode loop."""
import numpy as np
import pytest

import cache_reference as ref
from invariant_sequence_decode_gb300 import workloads as wl

torch = pytest.importorskip("torch")
import invariant_sequence_decode_gb300 as luce  # noqa: E402

pytestmark = pytest.mark.gpu
FIELDS = ["attn_norm", "wqkv_q", "wqkv_d", "wo_q", "wo_d", "ffn_norm", "wgu_q", "wgu_d", "wdown_q", "wdown_d"]
VOCAB, LAYERS = 256, 2


@pytest.fixture(scope="module", autouse=True)
def lib():
    from invariant_sequence_decode_gb300 import build
    build.build()
    return luce.load_library()


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bits(t):
    return t.contiguous().view(torch.int32).cpu().numpy()


@pytest.fixture(scope="module")
def model():
    d = wl.TINY_LAYER
    layers = [luce.LayerTensors(*[cuda(getattr(wl.layer_host(3, l, d), f)) for f in FIELDS]) for l in range(LAYERS)]
    fn, hq, hd = wl.head_host(3, d, VOCAB)
    return luce.Model(layers, d.hidden, d.n_q_heads, d.n_kv_heads, d.ffn, final_norm=cuda(fn), head_q=cuda(hq),
                      head_d=cuda(hd))


def cache(seed, length, cap):
    """fp16 [LAYERS][Hkv][cap][128] K and V; positions behind the prefix hold NaN."""
    d = wl.TINY_LAYER
    out = []
    for layer in range(LAYERS):
        out.append([x.copy() for x in wl.cache_host(3, seed, layer, d, cap, length)])
    k, v = (np.stack([o[i] for o in out]) for i in (0, 1))
    k[:, :, length:], v[:, :, length:] = np.nan, np.nan
    return k, v


def step(model, slots, x, scores=None, stats=None):
    T = x.shape[0]
    logits = torch.empty(T, VOCAB, device="cuda")
    am = torch.empty(T, dtype=torch.int32, device="cuda")
    ws = model.tree_workspace(T, max(s.len for s in slots))
    luce.luce_decode_step_tree(model, slots, x, ws, logits, am, scores, stats)
    torch.cuda.synchronize()
    assert luce.wait_timeouts() == 0
    return x, logits, am


@pytest.mark.parametrize("lens,trees,pos0", [
    ([0], [[-1, 0, 0, 1, 1, 2, 5, -1]], [0]), ([130], [[-1, 0, 1, 1, 3, 0]], [500]),
    ([17, 300, 2, 129], [[-1], [-1, 0, 0], [-1, -1, 1, 0, 3], [-1, 0, 1, 2, 2, 4, 0]], [17, 300, 40, 129]),
])
def test_a_node_gives_the_bits_of_its_path_alone(model, lens, trees, pos0):
    cap = max(lens) + 20
    host = [cache(s, n, cap) for s, n in enumerate(lens)]
    T = sum(len(t) for t in trees)
    xh = wl.acts(3, T, wl.TINY_LAYER.hidden, sub=4)
    slots = [luce.TreeSlot(cuda(k), cuda(v), n, t, p) for (k, v), n, t, p in zip(host, lens, trees, pos0)]
    scores = torch.full((LAYERS, T, 4, -(-cap // 4) * 4), 5.0, device="cuda")
    stats = torch.zeros(LAYERS, T, 4, 2, device="cuda")
    x, logits, am = step(model, slots, cuda(xh), scores, stats)
    row0 = 0
    for s, (tree, n) in enumerate(zip(trees, lens)):
        for j in range(len(tree)):
            path = ref.ancestors(tree, j)
            one = luce.TreeSlot(cuda(host[s][0]), cuda(host[s][1]), n, len(path), pos0[s])
            xs, ls, ams = step(model, [one], cuda(xh[row0 + np.array(path)]))
            assert np.array_equal(bits(xs[-1]), bits(x[row0 + j])) and np.array_equal(bits(ls[-1]), bits(logits[row0 + j]))
            assert int(ams[-1]) == int(am[row0 + j])
            for a, b in ((slots[s].k, one.k), (slots[s].v, one.v)):
                assert torch.equal(a[:, :, n + j].view(torch.int16), b[:, :, n + len(path) - 1].view(torch.int16))
        for a, h in zip((slots[s].k, slots[s].v), host[s]):            # the rest of the cache is left as it was
            b = cuda(h)
            assert torch.equal(a[:, :, :n].view(torch.int16), b[:, :, :n].view(torch.int16))
            assert torch.equal(a[:, :, n + len(tree):].view(torch.int16), b[:, :, n + len(tree):].view(torch.int16))
        end = n + len(tree)
        rows = scores[:, row0:row0 + len(tree)]
        assert (rows[..., end:] == 5).all() and not torch.isnan(rows[..., :end]).any()
        w = (rows[..., :end].double() - stats[:, row0:row0 + len(tree), :, :1]).exp() / stats[:, row0:row0 + len(tree), :, 1:]
        assert (w.sum(-1) - 1).abs().max().item() <= 2.0 ** -23 * (end + 100)   # end roundings of scores, m and l
        row0 += len(tree)


@pytest.mark.parametrize("length", [0, 130, 700])
def test_repeated_steps_give_the_same_bits(model, length):
    """Kernels of a step overlap at their ends; none may read ahead of what it waits for."""
    k, v = cache(0, length, length + 20)
    xh = wl.acts(3, 8, wl.TINY_LAYER.hidden, sub=6)
    ws, first = model.tree_workspace(8, length), None
    for it in range(60):
        ws.fill_(255 * (it & 1))
        sl = luce.TreeSlot(cuda(k), cuda(v), length, [-1, 0, 0, 1, 1, 2, 5, -1])
        x, logits, am = cuda(xh), torch.empty(8, VOCAB, device="cuda"), torch.empty(8, dtype=torch.int32, device="cuda")
        luce.luce_decode_step_tree(model, [sl], x, ws, logits, am)
        torch.cuda.synchronize()
        got = [bits(x), bits(logits), sl.k.view(torch.int16).cpu().numpy(), sl.v.view(torch.int16).cpu().numpy()]
        first = first or got
        assert all(np.array_equal(a, b) for a, b in zip(got, first))


def test_chains_agree_with_the_plain_step(model):
    lens, rows, cap = [3, 40, 200, 255], [1, 2, 3, 4], 300
    host = [cache(s, n, cap) for s, n in enumerate(lens)]
    xh = wl.acts(3, sum(rows), wl.TINY_LAYER.hidden, sub=5)
    x, logits, _ = step(model, [luce.TreeSlot(cuda(k), cuda(v), n, r) for (k, v), n, r in zip(host, lens, rows)], cuda(xh))
    plain = cuda(xh)
    want = torch.empty_like(logits)
    luce.luce_decode_step(model, [luce.Slot(cuda(k), cuda(v), n) for (k, v), n in zip(host, lens)], rows, plain,
                          model.workspace(sum(rows), cap), want, torch.empty(sum(rows), dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    # an attention output in another order can move an int8 code by one: the
    # tolerance of the plain step's own end-to-end parity
    for a, b in ((x, plain), (logits, want)):
        err = (a - b).abs().amax(1) / b.norm(dim=1)
        assert err.max().item() <= 2e-3


def test_pages_give_the_bits_of_flat_caches(model):
    lens, trees, pos0 = [120, 0, 300], [[-1, 0, 0, 1, 3, 4, 0, 2, 1], [-1, 0], [-1, 0, 1]], [200, 0, 300]
    rng = np.random.default_rng(3)
    xh = wl.acts(3, sum(len(t) for t in trees), wl.TINY_LAYER.hidden, sub=7)
    flat, paged = [], []
    for s, (n, tree, p0) in enumerate(zip(lens, trees, pos0)):
        k, v = cache(s, n, n + len(tree))
        flat.append(luce.TreeSlot(cuda(k), cuda(v), n, tree, p0))
        per = -(-(n + len(tree)) // 128)
        table, pools = rng.permutation(per + 2)[:per], []
        for x in (k, v):
            pool = np.full((per + 2, LAYERS, x.shape[1], 128, 128), np.nan, dtype=np.float16)
            for i, p in enumerate(table):
                part = x[:, :, 128 * i:128 * (i + 1)]
                pool[p, :, :, :part.shape[2]] = part
            pools.append(cuda(pool))
        paged.append(luce.PagedTreeSlot(*pools, table, n, tree, p0))
    sc = [torch.zeros(LAYERS, xh.shape[0], 4, 320, device="cuda") for _ in range(2)]
    st = [torch.zeros(LAYERS, xh.shape[0], 4, 2, device="cuda") for _ in range(2)]
    a, b = step(model, flat, cuda(xh), sc[0], st[0]), step(model, paged, cuda(xh), sc[1], st[1])
    for x, y in zip((*a, sc[0], st[0]), (*b, sc[1], st[1])):
        assert np.array_equal(bits(x), bits(y))
    for f, p in zip(flat, paged):
        for j in range(f.len, f.len + len(f.parent)):
            for x, y in ((f.k, p.k_pool), (f.v, p.v_pool)):
                assert torch.equal(x[:, :, j].view(torch.int16), y[p.table[j // 128], :, :, j % 128].view(torch.int16))


def test_decode_loop(model):
    """Two slots decode with trees of 8; keys past 48 are evicted.  What the loop
    keeps is checked against its own inputs: the accepted rows' K/V, the
    positions, the sum of the weights added in each step."""
    d, cap, budget, S, n = wl.TINY_LAYER, 80, 48, 2, 8
    G = d.n_q_heads // d.n_kv_heads
    shape = (LAYERS, d.n_kv_heads, cap)
    slots, state = [], []
    for s in range(S):
        k, v = cache(s, 10, cap)
        slots.append(luce.TreeSlot(cuda(k), cuda(v), 10, n, 10))
        pos = np.zeros(shape, dtype=np.int32)
        pos[..., :10] = np.arange(10)
        state.append((torch.zeros(shape, device="cuda"), cuda(pos)))
    rng = np.random.default_rng(1)
    scores, stats = torch.zeros(LAYERS, S * n, 4, cap, device="cuda"), torch.zeros(LAYERS, S * n, 4, 2, device="cuda")
    for it in range(20):
        for sl in slots:
            sl.parent = [-1] + [int(rng.integers(0, j)) for j in range(1, n)]
        step(model, slots, cuda(wl.acts(100 + it, S * n, d.hidden)), scores, stats)
        paths = [ref.ancestors(sl.parent, int(rng.integers(0, n))) for sl in slots]
        rows = [sl.k[:, :, [sl.len + a for a in p]].clone() for sl, p in zip(slots, paths)]
        before = [a.sum(-1) for a, _ in state]
        keep = [a.clone() for a, _ in state]
        luce.luce_tree_commit([luce.CommitSlot(sl.k, sl.v, sl.len, p, s * n, a, q, sl.pos0)
                               for s, (sl, p, (a, q)) in enumerate(zip(slots, paths, state))], d.n_q_heads, scores, stats)
        for s, (sl, p, (a, q)) in enumerate(zip(slots, paths, state)):
            end = sl.len + len(p)
            assert torch.equal(sl.k[:, :, sl.len:end], rows[s])
            assert torch.equal(q[:, :, sl.len:end], torch.arange(sl.pos0, sl.pos0 + len(p), device="cuda", dtype=torch.int32)
                               .expand(LAYERS, d.n_kv_heads, -1))
            added = a[..., :end].sum(-1) - keep[s][..., :sl.len].sum(-1)
            # every weight of an accepted row is on a key that stays
            assert (added - G * len(p)).abs().max().item() <= 2.0 ** -23 * cap * (G * len(p) + float(before[s].max()) + 100)
            sl.len, sl.pos0 = end, sl.pos0 + len(p)
        luce.luce_kv_evict([luce.EvictSlot(sl.k, sl.v, a, q, sl.len, budget, 2, 8, sl.pos0)
                            for sl, (a, q) in zip(slots, state)])
        torch.cuda.synchronize()
        for sl, (a, q) in zip(slots, state):
            sl.len = min(sl.len, budget)
            kept = q[:, :, :sl.len].sort(-1).values
            assert (kept[..., 1:] > kept[..., :-1]).all()               # no position twice
            assert (kept[..., :2] == torch.arange(2, device="cuda")).all()
            assert (kept[..., -8:] == torch.arange(sl.pos0 - 8, sl.pos0, device="cuda")).all()
    assert all(sl.pos0 > budget and sl.len == budget for sl in slots)


def test_python_refusals(model):
    k, v = (cuda(x) for x in cache(0, 10, 30))
    x, ws = cuda(wl.acts(3, 2, wl.TINY_LAYER.hidden)), model.tree_workspace(2, 20)
    with pytest.raises(ValueError):
        luce.luce_decode_step_tree(model, [luce.TreeSlot(k, v, 10, 3)], x, ws)
    with pytest.raises(ValueError):
        luce.luce_decode_step_tree(model, [luce.TreeSlot(k[:1], v[:1], 10, 2)], x, ws)
    with pytest.raises(TypeError):
        luce.luce_decode_step_tree(model, [luce.TreeSlot(k.float(), v.float(), 10, 2)], x, ws)
    with pytest.raises(ValueError):
        luce.luce_decode_step_tree(model, [luce.TreeSlot(k, v, 10, 2)], x, ws, scores=torch.zeros(1, 2, 4, 16, device="cuda"))
    with pytest.raises(luce.LuceError):
        luce.luce_decode_step_tree(model, [luce.TreeSlot(k, v, 10, 2)], x, ws[:1024])
    with pytest.raises(luce.LuceError):
        luce.luce_decode_step_tree(model, [luce.TreeSlot(k, v, 10, [-1, 1])], x, ws)
