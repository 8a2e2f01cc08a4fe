"""The commit of a verified tree's accepted path and eviction by accumulated
attention weight, against plain 64-bit forms; and both with tree attention in
a decode loop."""
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


def same(t, a):
    return np.array_equal(t.cpu().numpy().view(np.uint8), np.ascontiguousarray(a).view(np.uint8))


def caches(rng, L, Hkv, cap):
    return tuple(rng.standard_normal((L, Hkv, cap, 128)).astype(np.float16) for _ in range(2))


# ------------------------------------------------------------------ commit

def weight_tolerance(acc, group, n):
    """acc is one sum of its old value and n * group weights, each at most 1 and
    off by e^x's argument (|x| <= 88 units of 2^-24), exp, 1 / l and the product."""
    u = 2.0 ** -24
    return u * (np.abs(acc).max() + group * n) * (group * n + 1) + group * n * u * (88 + 8)


@pytest.mark.parametrize("L,Hq,Hkv,lens,paths,slack", [
    (1, 8, 2, [0], [[0]], 0), (1, 8, 2, [1], [[]], 3), (2, 4, 4, [5], [[1]], 0), (3, 40, 8, [127], [[0, 2, 5, 15]], 1),
    (2, 8, 1, [1025], [list(range(16))], 0), (1, 7, 1, [1000, 3], [[0, 1], [2, 3]], 9),
    (4, 6, 2, [17, 100, 513, 2051], [[3], [0, 1, 2], [1, 2], []], 2), (2, 2, 2, [4099], [[0, 7, 9]], 0),
])
def test_commit(L, Hq, Hkv, lens, paths, slack):
    rng = np.random.default_rng(sum(lens) + L)
    per, n = 16 // len(lens), len(lens)
    lds = -(-(max(lens) + 16) // 4) * 4
    T = n * per
    scores = (2 * rng.standard_normal((L, T, Hq, lds))).astype(np.float32)
    scores[rng.random(scores.shape) < 0.05] = -np.inf
    stats = np.zeros((L, T, Hq, 2), dtype=np.float32)
    for s in range(n):
        seen = scores[:, s * per:(s + 1) * per, :, :lens[s] + per].astype(np.float64)
        m = seen.max(-1)
        m[np.isneginf(m)] = 0
        stats[:, s * per:(s + 1) * per, :, 0] = m
        stats[:, s * per:(s + 1) * per, :, 1] = np.exp(seen - m[..., None]).sum(-1)
        scores[:, s * per:(s + 1) * per, :, lens[s] + 16:] = np.nan    # never read
    slots, want = [], []
    for s, (length, path) in enumerate(zip(lens, paths)):
        cap = length + 16 + slack
        k, v = caches(rng, L, Hkv, cap)
        acc = rng.random((L, Hkv, cap)).astype(np.float32)
        pos = rng.integers(0, 1 << 20, (L, Hkv, cap)).astype(np.int32)
        slots.append(luce.CommitSlot(cuda(k), cuda(v), length, path, s * per, cuda(acc), cuda(pos), 1000 + length))
        want.append(ref.commit(k, v, length, path, acc, pos, 1000 + length, scores[:, s * per:], stats[:, s * per:]) + (acc,))
    luce.luce_tree_commit(slots, Hq, cuda(scores), cuda(stats))
    torch.cuda.synchronize()
    for sl, (k, v, acc, pos, old), path in zip(slots, want, paths):
        assert same(sl.k, k) and same(sl.v, v) and same(sl.pos, pos)
        got = sl.acc.cpu().numpy()
        end = sl.len + len(path)
        assert same(sl.acc[:, :, end:], old[:, :, end:])                # behind the last key: left as it was
        if path:
            assert np.abs(got[:, :, :end] - acc[:, :, :end]).max() <= weight_tolerance(acc, Hq // Hkv, len(path))
        else:
            assert same(sl.acc, old)


def test_commit_without_weights_moves_rows_only():
    rng = np.random.default_rng(3)
    k, v = caches(rng, 2, 3, 40)
    pos = np.zeros((2, 3, 40), dtype=np.int32)
    a = luce.CommitSlot(cuda(k), cuda(v), 10, [1, 4, 5], pos=cuda(pos), pos0=77)
    b = luce.CommitSlot(cuda(v), cuda(k), 20, [0, 1], pos0=20)
    luce.luce_tree_commit([a, b], 6)
    torch.cuda.synchronize()
    wk, wv, _, wp = ref.commit(k, v, 10, [1, 4, 5], None, pos, 77)
    assert same(a.k, wk) and same(a.v, wv) and same(a.pos, wp)
    assert same(b.k, v) and same(b.v, k)                                # a path that is where it belongs


def test_a_row_that_saw_nothing_adds_nothing():
    k = torch.zeros(1, 1, 24, 128, dtype=torch.float16, device="cuda")
    acc = torch.ones(1, 1, 24, device="cuda")
    scores = torch.full((1, 2, 2, 24), float("-inf"), device="cuda")
    stats = torch.tensor([float("-inf"), 0.0], device="cuda").repeat(1, 2, 2, 1).contiguous()
    scores[0, 1], stats[0, 1, :, 0], stats[0, 1, :, 1] = 0.0, 0.0, 10.0
    luce.luce_tree_commit([luce.CommitSlot(k, k.clone(), 8, [0, 1], 0, acc)], 2, scores, stats)
    torch.cuda.synchronize()
    # row 1: two heads of weight 1/10 for every key; two fp32 roundings of 0.1 and two sums
    want = torch.tensor([1.2] * 8 + [0.2] * 2 + [1.0] * 14, device="cuda")
    assert (acc[0, 0] - want).abs().max().item() <= 6 * 2 ** -24


def test_prepared_commit_follows_its_slots_in_streams_and_graphs():
    rng = np.random.default_rng(17)
    k, v = caches(rng, 2, 2, 64)
    scores = rng.standard_normal((2, 4, 4, 64)).astype(np.float32)
    stats = np.stack([scores.max(-1), np.full(scores.shape[:-1], 9.0, dtype=np.float32)], -1)
    acc, pos = np.zeros((2, 2, 64), dtype=np.float32), np.zeros((2, 2, 64), dtype=np.int32)
    sl = luce.CommitSlot(cuda(k), cuda(v), 10, [1, 3], 0, cuda(acc), cuda(pos), 10)
    call = luce.TreeCommit([sl], 4, cuda(scores), cuda(stats))
    want = [k, v, acc, pos]
    side = torch.cuda.Stream()
    for length, path, pos0 in ((10, [1, 3], 10), (12, [0], 40), (13, [0, 1, 2], 41)):
        sl.len, sl.path, sl.pos0 = length, path, pos0
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        torch.cuda.current_stream().wait_stream(side)
        want = list(ref.commit(want[0], want[1], length, path, want[2], want[3], pos0, scores, stats))
    sl.len, sl.path, sl.pos0 = 16, [2], 44
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):                                                   # replayed: the same commit twice
        graph.replay()
        want = list(ref.commit(want[0], want[1], 16, [2], want[2], want[3], 44, scores, stats))
    torch.cuda.synchronize()
    assert same(sl.k, want[0]) and same(sl.v, want[1]) and same(sl.pos, want[3])
    assert np.abs(sl.acc.cpu().numpy() - want[2]).max() <= 5 * weight_tolerance(want[2], 2, 3)


def test_commit_python_refusals():
    k = torch.zeros(2, 2, 24, 128, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        luce.luce_tree_commit([], 4)
    with pytest.raises(TypeError):
        luce.luce_tree_commit([luce.CommitSlot(k.float(), k, 4, [0])], 4)
    with pytest.raises(ValueError):
        luce.luce_tree_commit([luce.CommitSlot(k[:, :, ::2], k[:, :, ::2], 4, [0])], 4)
    with pytest.raises(ValueError):
        luce.luce_tree_commit([luce.CommitSlot(k, k.clone(), 4, [0], acc=torch.zeros(2, 2, 23, device="cuda"))], 4)
    with pytest.raises(TypeError):
        luce.luce_tree_commit([luce.CommitSlot(k, k.clone(), 4, [0], pos=torch.zeros(2, 2, 24, device="cuda"))], 4)
    with pytest.raises(luce.LuceError):
        luce.luce_tree_commit([luce.CommitSlot(k, k.clone(), 4, [1, 0])], 4)
    with pytest.raises(luce.LuceError):
        luce.luce_tree_commit([luce.CommitSlot(k, k, 4, [0])], 4)
    with pytest.raises(ValueError):
        luce.luce_tree_commit([luce.CommitSlot(k, k.clone(), 4, [0])], 4, torch.zeros(2, 1, 8, 24, device="cuda"),
                              torch.zeros(2, 1, 8, 2, device="cuda"))


# ------------------------------------------------------------------ eviction

def weights(rng, kind, shape):
    if kind == "ties":
        return rng.integers(0, 3, shape).astype(np.float32)
    if kind == "equal":
        return np.zeros(shape, dtype=np.float32)
    if kind == "zeros":
        return np.where(rng.random(shape) < 0.5, 0.0, -0.0).astype(np.float32)
    a = (rng.random(shape) ** 8 * 4).astype(np.float32)
    if kind == "odd":
        for x in (np.nan, np.inf, -np.inf, -1.0, 1e-40, 0.0, -0.0):
            a[rng.random(shape) < 0.08] = x
    return a


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("L,Hkv,length,budget,sinks,recent,kind", [
    (1, 1, 1, 1, 0, 0, "plain"), (1, 1, 2, 1, 0, 0, "plain"), (1, 1, 2, 1, 1, 0, "plain"), (2, 2, 5, 3, 1, 2, "plain"),
    (1, 2, 33, 32, 0, 0, "odd"), (2, 1, 100, 67, 1, 17, "odd"), (2, 2, 100, 1, 0, 1, "ties"), (1, 2, 100, 99, 0, 0, "equal"),
    (1, 1, 700, 350, 0, 0, "zeros"), (3, 2, 1023, 512, 4, 100, "ties"), (1, 2, 1024, 1023, 0, 0, "odd"),
    (1, 2, 1025, 1024, 4, 1020, "odd"), (2, 2, 2051, 2048, 4, 256, "plain"), (1, 1, 5000, 37, 5, 32, "odd"),
    (1, 2, 4100, 2049, 0, 0, "ties"), (1, 1, 9001, 8999, 4, 4000, "plain"), (1, 1, 20000, 4096, 4, 512, "odd"),
    (2, 2, 50, 50, 0, 0, "plain"), (2, 2, 50, 60, 0, 0, "plain"),
])
def test_evict(L, Hkv, length, budget, sinks, recent, kind, in_place):
    rng = np.random.default_rng(length + budget)
    cap = length + 3
    k, v = caches(rng, L, Hkv, cap)
    acc = weights(rng, kind, (L, Hkv, cap))
    pos = np.stack([rng.permutation(cap) for _ in range(L * Hkv)]).reshape(L, Hkv, cap).astype(np.int32)
    nxt = cap
    wk, wv, wa, wp = ref.evict(k, v, acc, pos, length, budget, sinks, recent, nxt)
    sl = luce.EvictSlot(cuda(k), cuda(v), cuda(acc), cuda(pos), length, budget, sinks, recent, nxt)
    keep = min(length, budget)
    if not in_place:
        sl.acc_out, sl.pos_out = torch.full_like(sl.acc, 9.0), torch.full_like(sl.pos, 9)
    luce.luce_kv_evict([sl])
    torch.cuda.synchronize()
    assert same(sl.k, wk) and same(sl.v, wv)
    if in_place:
        assert same(sl.acc, wa) and same(sl.pos, wp)
    else:
        assert same(sl.acc, acc) and same(sl.pos, pos)
        assert same(sl.acc_out[:, :, :keep], wa[:, :, :keep]) and same(sl.pos_out[:, :, :keep], wp[:, :, :keep])
        assert (sl.acc_out[:, :, keep:] == 9).all() and (sl.pos_out[:, :, keep:] == 9).all()


def test_evict_longest_cache():
    rng = np.random.default_rng(2)
    length, budget = 130816, 65001
    k, v = caches(rng, 1, 1, length)
    acc, pos = weights(rng, "plain", (1, 1, length)), np.arange(length, dtype=np.int32)[None, None]
    want = ref.evict(k, v, acc, pos, length, budget, 4, 1000, length)
    sl = luce.EvictSlot(cuda(k), cuda(v), cuda(acc), cuda(pos), length, budget, 4, 1000, length)
    luce.luce_kv_evict([sl])
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip((sl.k, sl.v, sl.acc, sl.pos), want))


def test_evict_slots_of_different_lengths():
    rng = np.random.default_rng(4)
    spec = [(2051, 2048), (10, 40), (300, 7), (9000, 1000)]
    slots, want = [], []
    for length, budget in spec:
        k, v = caches(rng, 2, 2, length + 1)
        acc, pos = weights(rng, "odd", (2, 2, length + 1)), np.tile(np.arange(length + 1, dtype=np.int32), (2, 2, 1))
        want.append(ref.evict(k, v, acc, pos, length, budget, 1, 2, length))
        slots.append(luce.EvictSlot(cuda(k), cuda(v), cuda(acc), cuda(pos), length, budget, 1, 2, length))
    luce.luce_kv_evict(slots)
    torch.cuda.synchronize()
    for sl, w in zip(slots, want):
        assert all(same(a, b) for a, b in zip((sl.k, sl.v, sl.acc, sl.pos), w))


def test_evict_protects_as_far_as_the_budget_goes():
    """Positions that repeat can protect more keys than the budget: the lowest indexes stay."""
    rng = np.random.default_rng(6)
    k, v = caches(rng, 1, 1, 40)
    acc, pos = weights(rng, "plain", (1, 1, 40)), np.zeros((1, 1, 40), dtype=np.int32)
    want = ref.evict(k, v, acc, pos, 40, 10, 5, 5, 40)
    sl = luce.EvictSlot(cuda(k), cuda(v), cuda(acc), cuda(pos), 40, 10, 5, 5, 40)
    luce.luce_kv_evict([sl])
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip((sl.k, sl.v, sl.acc, sl.pos), want))
    assert same(sl.k, k)


def test_prepared_calls_in_a_graph():
    rng = np.random.default_rng(7)
    k, v = caches(rng, 2, 2, 200)
    acc, pos = weights(rng, "plain", (2, 2, 200)), np.tile(np.arange(200, dtype=np.int32), (2, 2, 1))
    sl = luce.EvictSlot(cuda(k), cuda(v), cuda(acc), cuda(pos), 150, 100, 2, 10, 150)
    call = luce.KvEvict([sl])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    torch.cuda.synchronize()
    want = ref.evict(k, v, acc, pos, 150, 100, 2, 10, 150)
    assert all(same(a, b) for a, b in zip((sl.k, sl.v, sl.acc, sl.pos), want))


def test_evict_python_refusals():
    k = torch.zeros(2, 2, 24, 128, dtype=torch.float16, device="cuda")
    acc, pos = torch.zeros(2, 2, 24, device="cuda"), torch.zeros(2, 2, 24, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        luce.luce_kv_evict([])
    with pytest.raises(TypeError):
        luce.luce_kv_evict([luce.EvictSlot(k, k.clone(), acc.half(), pos, 4, 2)])
    with pytest.raises(TypeError):
        luce.luce_kv_evict([luce.EvictSlot(k, k.clone(), acc, pos.long(), 4, 2)])
    with pytest.raises(ValueError):
        luce.luce_kv_evict([luce.EvictSlot(k, k.clone(), acc[:, :, :20], pos, 4, 2)])
    with pytest.raises(luce.LuceError):
        luce.luce_kv_evict([luce.EvictSlot(k, k.clone(), acc, pos, 4, 0)])
    with pytest.raises(luce.LuceError):
        luce.luce_kv_evict([luce.EvictSlot(k, k, acc, pos, 4, 2)])


# ------------------------------------------------------------------ pages

def pool_of(rng, x, extra=2):
    """x [L][Hkv][cap][128] laid out in pages: (pool [n_pages][L][Hkv][128][128], table); unused rows hold NaN."""
    L, Hkv, cap, _ = x.shape
    per = -(-cap // 128)
    table = rng.permutation(per + extra)[:per].astype(np.int32)
    pool = np.full((per + extra, L, Hkv, 128, 128), np.nan, dtype=np.float16)
    for i, p in enumerate(table):
        part = x[:, :, 128 * i:128 * (i + 1)]
        pool[p, :, :, :part.shape[2]] = part
    return pool, table


@pytest.mark.parametrize("lens,paths", [([126], [[1, 2, 5]]), ([0, 300], [[0, 3], [2, 7]]), ([383, 128, 1], [[3], [0, 1, 4], []])])
def test_paged_commit(lens, paths):
    rng = np.random.default_rng(sum(lens))
    L, Hq, Hkv = 2, 6, 3
    per = 16 // len(lens)
    lds = -(-(max(lens) + 16) // 4) * 4
    scores = rng.standard_normal((L, len(lens) * per, Hq, lds)).astype(np.float32)
    stats = np.ones((L, len(lens) * per, Hq, 2), dtype=np.float32)
    slots, flat, spare = [], [], []
    for s, (n, path) in enumerate(zip(lens, paths)):
        k, v = caches(rng, L, Hkv, n + 16)
        acc, pos = rng.random((L, Hkv, n + 16)).astype(np.float32), np.zeros((L, Hkv, n + 16), dtype=np.int32)
        seed = int(rng.integers(1 << 30))
        pools = [pool_of(np.random.default_rng(seed), x) for x in (k, v)]
        flat.append(luce.CommitSlot(cuda(k), cuda(v), n, path, s * per, cuda(acc), cuda(pos), 7))
        slots.append(luce.PagedCommitSlot(cuda(pools[0][0]), cuda(pools[1][0]), pools[0][1], n, path, s * per, cuda(acc),
                                          cuda(pos), 7))
        spare.append(seed)
    luce.luce_tree_commit(flat, Hq, cuda(scores), cuda(stats))
    luce.luce_tree_commit(slots, Hq, cuda(scores), cuda(stats))
    torch.cuda.synchronize()
    for f, p, seed in zip(flat, slots, spare):
        for a, b in ((f.k, p.k_pool), (f.v, p.v_pool)):
            assert same(b, pool_of(np.random.default_rng(seed), a.cpu().numpy())[0])
        assert same(p.acc, f.acc.cpu().numpy()) and same(p.pos, f.pos.cpu().numpy())


def test_paged_evict_few_of_many():
    test_paged_evict(9000, 8990)


@pytest.mark.parametrize("length,budget", [(130, 127), (300, 290), (700, 100), (5000, 2000)])
def test_paged_evict(length, budget):
    rng = np.random.default_rng(length)
    L, Hkv = 2, 2
    k, v = caches(rng, L, Hkv, length)
    acc, pos = weights(rng, "odd", (L, Hkv, length)), np.tile(np.arange(length, dtype=np.int32), (L, Hkv, 1))
    wk, wv, wa, wp = ref.evict(k, v, acc, pos, length, budget, 2, 20, length)
    (pk, table), (pv, _) = (pool_of(np.random.default_rng(5), x) for x in (k, v))
    sl = luce.PagedEvictSlot(cuda(pk), cuda(pv), cuda(table), cuda(acc), cuda(pos), length, budget, 2, 20, length)
    luce.luce_kv_evict([sl])
    torch.cuda.synchronize()
    assert same(sl.k_pool, pool_of(np.random.default_rng(5), wk)[0]) and same(sl.v_pool, pool_of(np.random.default_rng(5), wv)[0])
    assert same(sl.acc, wa) and same(sl.pos, wp)


@pytest.mark.parametrize("length,budget", [(300, 290), (700, 300)])
def test_paged_evict_leaves_rows_of_bad_pages(length, budget):
    rng = np.random.default_rng(length + 1)
    k, v = caches(rng, 1, 2, length)
    acc, pos = weights(rng, "plain", (1, 2, length)), np.tile(np.arange(length, dtype=np.int32), (1, 2, 1))
    wk, wv, wa, wp = ref.evict(k, v, acc, pos, length, budget, 0, 0, length)
    (pk, table), (pv, _) = (pool_of(np.random.default_rng(5), x) for x in (k, v))
    bad = table.copy()
    bad[1] = 2 ** 31 - 1                                                # rows 128..255: neither read nor written
    wk[:, :, 128:256], wv[:, :, 128:256] = k[:, :, 128:256], v[:, :, 128:256]
    sl = luce.PagedEvictSlot(cuda(pk), cuda(pv), cuda(bad), cuda(acc), cuda(pos), length, budget, 0, 0, length)
    luce.luce_kv_evict([sl])
    torch.cuda.synchronize()
    assert same(sl.k_pool, pool_of(np.random.default_rng(5), wk)[0]) and same(sl.v_pool, pool_of(np.random.default_rng(5), wv)[0])
    assert same(sl.acc, wa) and same(sl.pos, wp)


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd"])
@pytest.mark.parametrize("length,leave", [(3, 2), (33, 32), (34, 33), (257, 32), (4096, 32), (4096, 1), (4097, 1), (4097, 32), (4097, 33),
                                          (8193, 2), (30011, 17)])
def test_evict_few(length, leave, kind):
    rng = np.random.default_rng(length + leave)
    k, v = caches(rng, 1, 2, length + 3)
    acc = weights(rng, kind, (1, 2, length + 3))
    pos = np.tile(rng.permutation(length + 3).astype(np.int32), (1, 2, 1))
    out = [np.full_like(acc, 5.0), np.full_like(pos, 5)]
    sinks, recent = min(2, length - leave - 1), min(7, max(length - leave - 3, 0))
    wk, wv, wa, wp = ref.evict(k, v, acc, pos, length, length - leave, sinks, recent, length)
    sl = luce.EvictSlot(cuda(k), cuda(v), cuda(acc), cuda(pos), length, length - leave, sinks, recent, length, cuda(out[0]), cuda(out[1]))
    luce.luce_kv_evict([sl])
    torch.cuda.synchronize()
    n = length - leave
    assert same(sl.k, wk) and same(sl.v, wv) and same(sl.acc, acc) and same(sl.pos, pos)
    assert same(sl.acc_out[..., :n], wa[..., :n]) and same(sl.pos_out[..., :n], wp[..., :n])
    assert bool((sl.acc_out[..., n:] == 5).all()) and bool((sl.pos_out[..., n:] == 5).all())


@pytest.mark.parametrize("length,leave,period,low", [(4000, 12, 256, 40), (4096, 32, 256, 60), (70001, 2, 512, 4), (70001, 32, 512, 60)])
def test_evict_few_when_low_weights_lie_close(length, leave, period, low):
    """The lowest keys share a few places of a period: more lie below the bound than the list holds."""
    rng = np.random.default_rng(length + low)
    k, v = caches(rng, 1, 1, length)
    acc = rng.random((1, 1, length)).astype(np.float32)
    acc = np.where(np.arange(length) % period < low, acc * np.float32(2.0 ** -20), acc + 1).astype(np.float32)
    pos = np.tile(np.arange(length, dtype=np.int32), (1, 1, 1))
    wk, wv, wa, wp = ref.evict(k, v, acc, pos, length, length - leave, 0, 3, length)
    sl = luce.EvictSlot(cuda(k), cuda(v), cuda(acc), cuda(pos), length, length - leave, 0, 3, length)
    luce.luce_kv_evict([sl])
    torch.cuda.synchronize()
    assert same(sl.k, wk) and same(sl.v, wv) and same(sl.acc, wa) and same(sl.pos, wp)


@pytest.mark.parametrize("shapes", [[(9000, 8990), (5, 5), (4097, 4096), (100, 120)], [(3000, 2990), (1, 1), (0, 4), (40, 9)],
                                    [(20000, 19968), (7000, 7000), (4100, 5000)]])
def test_evict_few_slots_of_different_lengths(shapes):
    """Slots that keep all keys next to slots that lose a few, into arrays of their own."""
    rng = np.random.default_rng(sum(n for n, _ in shapes))
    slots, want = [], []
    for n, budget in shapes:
        k, v = caches(rng, 2, 2, n + 2)
        acc, pos = weights(rng, "odd", (2, 2, n + 2)), np.tile(rng.permutation(n + 2).astype(np.int32), (2, 2, 1))
        want.append((acc, pos) + tuple(ref.evict(k, v, acc, pos, n, budget, 1, 0, n + 2)))
        out = torch.full((2, 2, n + 2), 5.0, device="cuda"), torch.full((2, 2, n + 2), 5, dtype=torch.int32, device="cuda")
        slots.append(luce.EvictSlot(cuda(k), cuda(v), cuda(acc), cuda(pos), n, budget, 1, 0, n + 2, *out))
    luce.luce_kv_evict(slots)
    torch.cuda.synchronize()
    for sl, (acc, pos, wk, wv, wa, wp) in zip(slots, want):
        keep = min(sl.len, sl.budget)
        assert same(sl.k, wk) and same(sl.v, wv) and same(sl.acc, acc) and same(sl.pos, pos)
        assert same(sl.acc_out[..., :keep], wa[..., :keep]) and same(sl.pos_out[..., :keep], wp[..., :keep])
        assert bool((sl.acc_out[..., keep:] == 5).all()) and bool((sl.pos_out[..., keep:] == 5).all())


def test_prepared_calls_follow_a_replaced_table_and_budget():
    rng = np.random.default_rng(23)
    k, v = caches(rng, 1, 2, 300)
    (pk, table), (pv, _) = (pool_of(np.random.default_rng(9), x) for x in (k, v))
    sl = luce.PagedCommitSlot(cuda(pk), cuda(pv), table, 120, [2])
    call = luce.TreeCommit([sl], 4)
    call()
    k, v = ref.commit(k, v, 120, [2])[:2]
    assert same(sl.k_pool, pool_of(np.random.default_rng(9), k)[0])
    other = np.setdiff1d(np.arange(len(pk)), table)[:1]                  # its second page moves elsewhere
    sl.k_pool[int(other[0])] = sl.k_pool[int(table[1])]
    sl.v_pool[int(other[0])] = sl.v_pool[int(table[1])]
    old = sl.k_pool[int(table[1])].clone()
    sl.table = np.array([table[0], other[0], table[2]], dtype=np.int32)
    sl.len, sl.path = 127, [0, 3]
    call()
    k, v = ref.commit(k, v, 127, [0, 3])[:2]
    got = sl.k_pool.cpu().numpy()[sl.table]                             # [3][1][2][128][128]
    assert np.array_equal(np.concatenate(list(got), axis=2)[:, :, :300].view(np.uint16), k.view(np.uint16))
    assert same(sl.k_pool[int(table[1])], old.cpu().numpy())
    sl.k_pool[int(table[1])], sl.v_pool[int(table[1])] = sl.k_pool[int(other[0])], sl.v_pool[int(other[0])]
    sl.table[1] = table[1]                                              # in place: back to the first page
    sl.len, sl.path = 129, [1, 2]
    call()
    k, v = ref.commit(k, v, 129, [1, 2])[:2]
    assert same(sl.k_pool[int(table[1])], np.ascontiguousarray(k[:, :, 128:256]))
    sl.table, sl.len, sl.path = [int(p) for p in table], 131, [4]
    call()
    k, v = ref.commit(k, v, 131, [4])[:2]
    assert same(sl.v_pool[int(table[1])], np.ascontiguousarray(v[:, :, 128:256]))

    k, v = caches(rng, 1, 2, 64)
    acc, pos = rng.random((1, 2, 64)).astype(np.float32), np.tile(np.arange(64, dtype=np.int32), (1, 2, 1))
    sl = luce.EvictSlot(cuda(k), cuda(v), cuda(acc), cuda(pos), 60, 50, 0, 0, 60)
    call = luce.KvEvict([sl])
    call()
    sl.len, sl.budget, sl.sinks, sl.recent = 50, 40, 3, 5
    call()
    for n, cut, sinks, recent in ((60, 50, 0, 0), (50, 40, 3, 5)):
        k, v, acc, pos = ref.evict(k, v, acc, pos, n, cut, sinks, recent, 60)
    torch.cuda.synchronize()
    assert same(sl.k, k) and same(sl.v, v) and same(sl.acc, acc) and same(sl.pos, pos)


# ------------------------------------------------------------------ together

def test_decode_loop_with_trees_commits_and_eviction():
    """Steps of two slots over two layers: tree attention with scores, commit of
    an accepted path, eviction once over the budget; against the plain forms."""
    rng = np.random.default_rng(11)
    L, Hq, Hkv, cap, budget, S, n = 2, 8, 2, 96, 64, 2, 8
    host = []
    for s in range(S):
        k, v = caches(rng, L, Hkv, cap)
        host.append([k, v, np.zeros((L, Hkv, cap)), np.zeros((L, Hkv, cap), dtype=np.int32), 0])
    dev = [[cuda(h[0]), cuda(h[1]), cuda(h[2].astype(np.float32)), cuda(h[3])] for h in host]
    pos0 = [0] * S
    for step in range(24):
        parents = [[-1] + [int(rng.integers(0, j)) for j in range(1, n)] for _ in range(S)]
        paths = [ref.ancestors(p, int(rng.integers(0, n))) for p in parents]
        q = rng.standard_normal((L, S * n, Hq, 128)).astype(np.float32)
        new = rng.standard_normal((2, S, L, Hkv, n, 128)).astype(np.float16)
        scores, stats = torch.zeros(L, S * n, Hq, cap, device="cuda"), torch.zeros(L, S * n, Hq, 2, device="cuda")
        for s in range(S):
            ln = host[s][4]
            for i in (0, 1):
                host[s][i][:, :, ln:ln + n] = new[i, s]
                dev[s][i][:, :, ln:ln + n] = cuda(new[i, s])
        ref_scores, ref_stats = np.zeros((L, S * n, Hq, cap)), np.zeros((L, S * n, Hq, 2))
        for layer in range(L):
            views = [luce.TreeView(dev[s][0][layer], dev[s][1][layer], host[s][4], parents[s], s * n) for s in range(S)]
            out = luce.luce_tree_attn(cuda(q[layer]), views, Hkv, SCALE, scores=scores[layer], stats=stats[layer])
            for s in range(S):
                ln = host[s][4]
                o, x, ml = ref.tree_attention(q[layer, s * n:(s + 1) * n], host[s][0][layer], host[s][1][layer], ln,
                                              parents[s], SCALE)
                tol = ref.tree_tolerance(q[layer], host[s][0][layer], host[s][1][layer], ln, n, SCALE, 1)[1]
                assert np.abs(out[s * n:(s + 1) * n].cpu().numpy() - o).max() <= tol
                ref_scores[layer, s * n:(s + 1) * n, :, :ln + n] = x
                ref_stats[layer, s * n:(s + 1) * n] = ml
        luce.luce_tree_commit([luce.CommitSlot(dev[s][0], dev[s][1], host[s][4], paths[s], s * n, dev[s][2], dev[s][3], pos0[s])
                               for s in range(S)], Hq, scores, stats)
        for s in range(S):
            h = host[s]
            h[:4] = ref.commit(*h[:2], h[4], paths[s], h[2], h[3], pos0[s], ref_scores[:, s * n:], ref_stats[:, s * n:])
            h[4] += len(paths[s])
            pos0[s] += len(paths[s])
        luce.luce_kv_evict([luce.EvictSlot(*dev[s], host[s][4], budget, 2, 8, pos0[s]) for s in range(S)])
        torch.cuda.synchronize()
        for s in range(S):
            h = host[s]
            h[:4] = ref.evict(*h[:4], h[4], budget, 2, 8, pos0[s])
            h[4] = min(h[4], budget)
            assert same(dev[s][3][:, :, :h[4]], h[3][:, :, :h[4]])       # the same keys stay
            assert same(dev[s][0][:, :, :h[4]], h[0][:, :, :h[4]]) and same(dev[s][1][:, :, :h[4]], h[1][:, :, :h[4]])
            assert np.abs(dev[s][2].cpu().numpy()[:, :, :h[4]] - h[2][:, :, :h[4]]).max() <= 1e-4
    assert max(pos0) > budget                                            # keys were evicted
