"""Attention of draft trees over a slot's cache against a plain 64-bit form, and
the bits that a node's outputs keep whatever else is in the call."""
import random

import numpy as np
import pytest

import cache_reference as ref

torch = pytest.importorskip("torch")
import invariant_sequence_decode_gb300 as luce  # noqa: E402

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def lib():
    from invariant_sequence_decode_gb300 import build
    build.build()
    return luce.load_library()


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bits(t):
    return t.contiguous().view(torch.int32).cpu().numpy()


def tree_of(kind, n, seed=0):
    rng = random.Random(seed)
    if kind == "chain":
        return ref.chain(n)
    if kind == "star":
        return [-1] + [0] * (n - 1)
    if kind == "forest":
        return [-1] * n
    return [-1] + [rng.randrange(-1, j) for j in range(1, n)]


class Slot:
    """A slot's cache on the host; positions behind the tree hold NaN."""

    def __init__(self, rng, Hq, Hkv, length, parent, slack=5):
        n = len(parent)
        self.len, self.parent, self.cap = length, parent, length + n + slack
        self.k = rng.standard_normal((Hkv, self.cap, 128)).astype(np.float16)
        self.v = rng.standard_normal((Hkv, self.cap, 128)).astype(np.float16)
        self.k[:, length + n:] = np.nan
        self.v[:, length + n:] = np.nan
        self.q = rng.standard_normal((n, Hq, 128)).astype(np.float32)

    def flat(self, row0):
        return luce.TreeView(cuda(self.k), cuda(self.v), self.len, self.parent, row0)

    def paged(self, row0, rng, extra=3):
        Hkv, n = self.k.shape[0], self.len + len(self.parent)
        per = -(-n // 128)
        order = rng.permutation(per + extra)[:per].astype(np.int32)
        pools = []
        for x in (self.k, self.v):
            pool = np.full((per + extra, Hkv, 128, 128), np.nan, dtype=np.float16)
            for i, p in enumerate(order):
                part = x[:, 128 * i:min(128 * (i + 1), n)]
                pool[p, :, :part.shape[1]] = part
            pools.append(cuda(pool))
        return luce.PagedTreeView(*pools, cuda(order), self.len, self.parent, row0)


def run(slots, views, Hkv, scores=False, fill=0.0):
    q = cuda(np.concatenate([s.q for s in slots]))
    T, Hq = q.shape[:2]
    lds = -(-max(s.len + len(s.parent) for s in slots) // 4) * 4 + 8
    sc = torch.full((T, Hq, lds), fill, device="cuda") if scores else None
    st = torch.full((T, Hq, 2), fill, device="cuda") if scores else None
    fn = luce.luce_tree_attn_paged if isinstance(views[0], luce.PagedTreeView) else luce.luce_tree_attn
    out = torch.full_like(q, float("nan"))
    fn(q, views, Hkv, SCALE, out=out, scores=sc, stats=st)
    torch.cuda.synchronize()
    assert luce.wait_timeouts() == 0
    return out, sc, st


def check(slots, out, sc, st, Hkv, fill=0.0):
    r0 = 0
    for s in slots:
        n = len(s.parent)
        o, x, ml = ref.tree_attention(s.q, s.k, s.v, s.len, s.parent, SCALE)
        ds, do, dl = ref.tree_tolerance(s.q, s.k, s.v, s.len, n, SCALE, 128)
        got = out[r0:r0 + n].cpu().numpy().astype(np.float64)
        assert np.abs(got - o).max() <= do
        assert np.linalg.norm(got - o) <= 2e-5 * np.linalg.norm(o)
        if sc is not None:
            g = sc[r0:r0 + n].cpu().numpy().astype(np.float64)
            seen = np.isfinite(x)
            assert np.array_equal(np.isneginf(g[:, :, :s.len + n]), ~seen)
            assert np.abs(g[:, :, :s.len + n][seen] - x[seen]).max() <= ds
            assert (g[:, :, s.len + n:] == fill).all()      # later columns are left as they were
            m = st[r0:r0 + n].cpu().numpy().astype(np.float64)
            assert np.abs(m[..., 0] - ml[..., 0]).max() <= ds
            assert np.abs(m[..., 1] - ml[..., 1]).max() <= dl
        r0 += n


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("Hq,Hkv,length,kind,n", [
    (8, 2, 0, "chain", 1), (8, 2, 0, "random", 9), (8, 2, 1, "star", 2), (4, 4, 2, "chain", 3), (40, 8, 127, "random", 16),
    (40, 8, 128, "random", 5), (8, 1, 129, "forest", 16), (7, 1, 255, "random", 7), (6, 2, 256, "chain", 4),
    (5, 1, 1000, "random", 13), (16, 2, 1001, "star", 16), (2, 2, 4097, "random", 3), (3, 1, 8191, "random", 11),
    (70, 70, 300, "random", 3), (200, 200, 1300, "chain", 2), (8, 2, 8192, "chain", 2), (8, 2, 8193, "random", 16), (4, 2, 16500, "random", 6), (2, 1, 40003, "random", 4),
])
def test_one_slot(Hq, Hkv, length, kind, n, paged):
    rng = np.random.default_rng(length * 31 + n)
    s = Slot(rng, Hq, Hkv, length, tree_of(kind, n, length))
    views = [s.paged(0, rng) if paged else s.flat(0)]
    check([s], *run([s], views, Hkv, scores=True, fill=7.0), Hkv, 7.0)


@pytest.mark.parametrize("paged", [False, True])
def test_longest(paged):
    rng = np.random.default_rng(5)
    s = Slot(rng, 8, 1, 130816 - 16, tree_of("random", 16, 3), slack=0)
    out, sc, st = run([s], [s.paged(0, rng) if paged else s.flat(0)], 1, scores=True)
    check([s], out, sc, st, 1)


@pytest.mark.parametrize("lens,nodes,Hq,Hkv", [([0, 17, 513, 1000], [1, 2, 3, 4], 8, 2), ([2051, 1, 130], [16 - 9, 8, 1], 40, 8),
                                               ([128, 9000], [1, 15], 12, 4), ([2047, 2051, 1999, 2040], [4] * 4, 40, 8)])
def test_several_slots(lens, nodes, Hq, Hkv):
    rng = np.random.default_rng(sum(lens))
    slots = [Slot(rng, Hq, Hkv, L, tree_of("random", n, L)) for L, n in zip(lens, nodes)]
    rows = np.cumsum([0] + nodes)
    flat = run(slots, [s.flat(int(r)) for s, r in zip(slots, rows)], Hkv, scores=True)
    check(slots, *flat, Hkv)
    paged = run(slots, [s.paged(int(r), rng) for s, r in zip(slots, rows)], Hkv, scores=True)
    for a, b in zip(flat, paged):
        assert np.array_equal(bits(a), bits(b))                # a paged cache gives a flat one's bits
    for s, r in zip(slots, rows):                              # a slot alone gives the bits it gives with others
        alone, _, st = run([s], [s.flat(0)], Hkv, scores=True)
        n = len(s.parent)
        assert np.array_equal(bits(alone), bits(flat[0][r:r + n]))
        assert np.array_equal(bits(st), bits(flat[2][r:r + n]))
    order = list(range(len(slots)))[::-1]                      # and with the views given in another order
    q = cuda(np.concatenate([s.q for s in slots]))
    out = luce.luce_tree_attn(q, [slots[i].flat(int(rows[i])) for i in order], Hkv, SCALE)
    assert np.array_equal(bits(out), bits(flat[0]))


@pytest.mark.parametrize("length", [0, 5, 200, 2051, 9000])
@pytest.mark.parametrize("Hq,Hkv", [(40, 8), (3, 1)])
def test_a_node_gives_the_bits_of_its_path_alone(length, Hq, Hkv):
    rng = np.random.default_rng(length)
    s = Slot(rng, Hq, Hkv, length, tree_of("random", 16, length))
    out, _, _ = run([s], [s.flat(0)], Hkv)
    for j in (0, 3, 7, 15):
        path = ref.ancestors(s.parent, j)
        t = Slot(rng, Hq, Hkv, length, ref.chain(len(path)))
        for new, old in ((t.k, s.k), (t.v, s.v)):
            new[:, :length] = old[:, :length]
            for i, a in enumerate(path):
                new[:, length + i] = old[:, length + a]
        t.q[:] = s.q[path]
        alone, _, _ = run([t], [t.flat(0)], Hkv)
        assert np.array_equal(bits(alone[-1]), bits(out[j]))


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_other_branches_do_not_reach_a_node(bad):
    rng = np.random.default_rng(8)
    s = Slot(rng, 8, 2, 300, [-1, 0, 0, 1, 1, 2, 5, -1])
    clean, csc, cst = run([s], [s.flat(0)], 2, scores=True)
    s.k[:, 302], s.v[:, 302] = bad, bad                         # node 2: seen by itself and by nodes 5 and 6
    out, sc, st = run([s], [s.flat(0)], 2, scores=True)
    rest = [0, 1, 3, 4, 7]
    assert np.array_equal(bits(out[rest]), bits(clean[rest]))
    assert np.array_equal(bits(sc[rest]), bits(csc[rest])) and np.array_equal(bits(st[rest]), bits(cst[rest]))
    assert not torch.isfinite(out[[2, 5, 6]]).all()


def test_strided_cache_gives_the_same_bits():
    rng = np.random.default_rng(9)
    s = Slot(rng, 8, 2, 700, tree_of("random", 6, 1))
    ref_out, _, _ = run([s], [s.flat(0)], 2)
    wide = torch.full((2, 2, s.cap + 3, 136 + 128), float("nan"), dtype=torch.float16, device="cuda")
    k, v = wide[0, :, :s.cap, 8:136], wide[1, :, :s.cap, 8:136]
    k.copy_(cuda(s.k))
    v.copy_(cuda(s.v))
    out, _, _ = run([s], [luce.TreeView(k, v, s.len, s.parent, 0)], 2)
    assert np.array_equal(bits(out), bits(ref_out))


def test_one_kv_head_of_many():
    rng = np.random.default_rng(10)
    s = Slot(rng, 4, 1, 300, ref.chain(2))
    ref_out, _, _ = run([s], [s.flat(0)], 1)
    big_k, big_v = (torch.randn(3, s.cap, 128, device="cuda").half() for _ in range(2))
    big_k[1], big_v[1] = cuda(s.k)[0], cuda(s.v)[0]
    out, _, _ = run([s], [luce.TreeView(big_k[1:2], big_v[1:2], s.len, s.parent, 0)], 1)
    assert np.array_equal(bits(out), bits(ref_out))


@pytest.mark.parametrize("lens", [[17, 100, 513, 1000], [2051] * 4, [20000, 1, 128, 16384]])
def test_chains_agree_with_decode_attention(lens):
    rng = np.random.default_rng(lens[0])
    nodes = [1, 2, 3, 4]
    slots = [Slot(rng, 40, 8, L, ref.chain(n)) for L, n in zip(lens, nodes)]
    rows = np.cumsum([0] + nodes)
    out, _, _ = run(slots, [luce.TreeView(cuda(s.k), cuda(s.v), s.len, n, int(r)) for s, n, r in zip(slots, nodes, rows)], 8)
    q = cuda(np.concatenate([s.q for s in slots]))
    old = luce.luce_decode_attn_multiseq(
        q, [luce.SeqView(cuda(s.k), cuda(s.v), s.len + n, n, int(r)) for s, n, r in zip(slots, nodes, rows)], 8, SCALE)
    tol = max(ref.tree_tolerance(s.q, s.k, s.v, s.len, 4, SCALE, 128)[1] for s in slots)
    assert (out - old).abs().max().item() <= 2 * tol


def test_pages_outside_the_pool_count_as_zero():
    rng = np.random.default_rng(12)
    s = Slot(rng, 8, 2, 500, tree_of("random", 4, 2), slack=0)
    for bad in (-1, 7, 2 ** 31 - 1, -2 ** 31):
        view = s.paged(0, np.random.default_rng(1))
        view.table[1] = bad
        t = Slot(rng, 8, 2, 500, s.parent, slack=0)
        t.k[:], t.v[:], t.q[:] = s.k, s.v, s.q
        t.k[:, 128:256], t.v[:, 128:256] = 0, 0
        out, sc, st = run([s], [view], 2, scores=True)
        check([t], out, sc, st, 2)
    view = s.paged(0, np.random.default_rng(1))
    view.table[3] = 7                                           # the page of the tree's own rows, and the prefix's last
    t.k[:], t.v[:] = s.k, s.v
    t.k[:, 384:], t.v[:, 384:] = 0, 0
    check([t], *run([s], [view], 2, scores=True), 2)


def test_large_scores_and_a_dominant_key():
    rng = np.random.default_rng(13)
    s = Slot(rng, 8, 2, 600, tree_of("random", 5, 2))
    s.q *= 40                                                   # scores in the hundreds: one key takes all the weight
    out, sc, st = run([s], [s.flat(0)], 2, scores=True)
    assert torch.isfinite(out).all()
    o, x, ml = ref.tree_attention(s.q, s.k, s.v, s.len, s.parent, SCALE)
    ds, do, _ = ref.tree_tolerance(s.q, s.k, s.v, s.len, 5, SCALE, 128)
    assert np.abs(out.cpu().numpy() - o).max() <= do


@pytest.mark.parametrize("scale", [-0.09, 0.0, 1e-30, 1.0, 3.0])
def test_scales(scale):
    rng = np.random.default_rng(16)
    s = Slot(rng, 8, 2, 700, tree_of("random", 5, 2))
    q = cuda(s.q)
    sc, st = torch.zeros(5, 8, 720, device="cuda"), torch.zeros(5, 8, 2, device="cuda")
    out = luce.luce_tree_attn(q, [s.flat(0)], 2, scale, scores=sc, stats=st)
    o, x, ml = ref.tree_attention(s.q, s.k, s.v, s.len, s.parent, scale)
    ds, do, dl = ref.tree_tolerance(s.q, s.k, s.v, s.len, 5, scale, 128)
    assert np.abs(out.cpu().numpy() - o).max() <= do
    got, seen = sc[:, :, :705].cpu().numpy(), np.isfinite(x)
    assert np.array_equal(np.isneginf(got), ~seen) and np.abs(got[seen] - x[seen]).max() <= ds
    assert np.abs(st[..., 0].cpu().numpy() - ml[..., 0]).max() <= ds
    # a weight from the scores and statistics is the weight of the definition
    w = np.exp(got.astype(np.float64) - st[..., :1].cpu().numpy()) / st[..., 1:].cpu().numpy()
    want = np.exp(x - ml[..., :1]) / ml[..., 1:]
    assert np.abs(w - want)[seen].max() <= (4 * ds + 2.0 ** -23 * (700 + 300 + 88)) * want.max()


def test_prepared_call_follows_len_streams_and_graphs():
    rng = np.random.default_rng(14)
    s = Slot(rng, 8, 2, 300, ref.chain(2), slack=40)
    s.k[np.isnan(s.k)], s.v[np.isnan(s.v)] = 0.5, 0.25
    view = s.flat(0)
    q = cuda(s.q)
    call = luce.TreeAttention(q, [view], 2, SCALE)
    for length in (300, 310, 0, 338):
        view.len = length
        got = call().clone()
        want = luce.luce_tree_attn(q, [luce.TreeView(view.k, view.v, length, 2, 0)], 2, SCALE)
        assert np.array_equal(bits(got), bits(want))
    view.len = 339 + 2
    with pytest.raises(ValueError):
        call()
    view.len = 200
    want = bits(call())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call().clone()
    side.synchronize()
    assert np.array_equal(bits(got), want)
    on = luce.luce_tree_attn(q, [view], 2, SCALE, stream=side)
    side.synchronize()
    assert np.array_equal(bits(on), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    call.out.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(bits(call.out), want)
    q.mul_(0.5)                                                 # replayed on new inputs
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(bits(call.out), bits(luce.luce_tree_attn(q, [view], 2, SCALE)))


def test_calls_behind_one_another_share_a_workspace():
    rng = np.random.default_rng(15)
    slots = [Slot(rng, 40, 8, L, tree_of("random", 8, L)) for L in (2051, 900)]
    views = [s.flat(0) for s in slots]
    want = [bits(luce.luce_tree_attn(cuda(s.q), [v], 8, SCALE)) for s, v in zip(slots, views)]
    ws = torch.full((luce.luce_tree_attn_workspace_size(8, 40, 8, 128, 2100),), 255, dtype=torch.uint8, device="cuda")
    calls = [luce.TreeAttention(cuda(s.q), [v], 8, SCALE, ws=ws) for s, v in zip(slots, views)]
    for _ in range(20):
        for c in calls:
            c()
    torch.cuda.synchronize()
    assert all(np.array_equal(bits(c.out), w) for c, w in zip(calls, want))


def test_python_refusals():
    q = torch.zeros(2, 8, 128, device="cuda")
    k = torch.zeros(2, 64, 128, dtype=torch.float16, device="cuda")
    ok = luce.TreeView(k, k.clone(), 10, 2)
    with pytest.raises(TypeError):
        luce.luce_tree_attn(q.half(), [ok], 2, SCALE)
    with pytest.raises(TypeError):
        luce.luce_tree_attn(q, [luce.TreeView(k.float(), k, 10, 2)], 2, SCALE)
    with pytest.raises(TypeError):
        luce.luce_tree_attn(q.cpu(), [ok], 2, SCALE)
    for bad in (luce.TreeView(k[:, :, :64], k[:, :, :64], 10, 2), luce.TreeView(k, k[:, :32], 10, 2),
                luce.TreeView(k, k, 10, 3), luce.TreeView(k, k, 63, 2), luce.TreeView(k[:1], k[:1], 10, 2)):
        with pytest.raises(ValueError):
            luce.luce_tree_attn(q, [bad], 2, SCALE)
    with pytest.raises(ValueError):
        luce.luce_tree_attn(q, [], 2, SCALE)
    with pytest.raises(ValueError):
        luce.luce_tree_attn(q, [ok], 2, SCALE, scores=torch.zeros(2, 4, 16, device="cuda"))
    with pytest.raises(luce.LuceError):
        luce.luce_tree_attn(q, [ok], 2, SCALE, scores=torch.zeros(2, 8, 13, device="cuda"))
    with pytest.raises(luce.LuceError):
        luce.luce_tree_attn(q, [luce.TreeView(k, k.clone(), 10, [0, 0])], 2, SCALE)
