"""Caches in 8 bits: attention over sealed blocks, a tail and a draft tree, the
sealing of whole blocks, the pass that norms, rotates and appends, against plain
64-bit forms, and the bits that a row keeps whatever else is in the call."""
import numpy as np
import pytest

import q8kv_reference as ref
from cache_reference import ancestors, chain
from test_gpu_tree import tree_of

torch = pytest.importorskip("torch")
import invariant_sequence_decode_gb300 as luce  # noqa: E402

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5
D, BLOCK, PAGE = 128, 32, 128


@pytest.fixture(scope="module", autouse=True)
def lib():
    from invariant_sequence_decode_gb300 import build
    build.build()
    return luce.load_library()


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bits(t):
    return t.contiguous().view(torch.int32).cpu().numpy()


class Cache:
    """A slot's cache on the host.  What no row sees is poisoned: codes and scales of blocks that are not sealed
    (127 and NaN), the tail's rows behind the tree (NaN)."""

    def __init__(self, rng, Hq, Hkv, sealed, tail, parent, window=0, sinks=0, spread=1.0, slack=3):
        n = len(parent)
        self.sealed, self.tail, self.parent, self.window, self.sinks = sealed, tail, parent, window, sinks
        self.pages = -(-sealed // PAGE)
        k = rng.standard_normal((Hkv, sealed // BLOCK, BLOCK, D)) * (0.5 + rng.random(D))
        v = rng.standard_normal((Hkv, sealed // BLOCK, BLOCK, D)) * spread ** rng.standard_normal((Hkv, sealed // BLOCK, 1, 1))
        self.kc, self.ks = ref.quantise(k.astype(np.float16))
        self.vc, self.vs = ref.quantise(v.astype(np.float16))
        self.k = np.full((Hkv, tail + n + slack, D), np.nan, np.float16)
        self.v = self.k.copy()
        self.k[:, :tail + n] = rng.standard_normal((Hkv, tail + n, D))
        self.v[:, :tail + n] = rng.standard_normal((Hkv, tail + n, D))
        self.q = rng.standard_normal((n, Hq, D)).astype(np.float32)

    def keys(self):
        """K and V of the prefix and the nodes in float64."""
        out = []
        for c, s, t in ((self.kc, self.ks, self.k), (self.vc, self.vs, self.v)):
            Hkv = c.shape[0]
            x = (c.astype(np.float64) * s.astype(np.float64)[..., None, None]).reshape(Hkv, -1, D)
            out.append(np.concatenate([x, t[:, :self.tail + len(self.parent)].astype(np.float64)], 1))
        return out

    def pools(self, order, total):
        """The pools with the slot's page i at order[i], the rest poisoned."""
        Hkv = self.kc.shape[0]
        kp = np.full((total, Hkv, PAGE, D), 127, np.int8)
        vp = np.full((total, Hkv, D, PAGE), 127, np.int8)
        sp = np.full((total, Hkv, 2, 4), np.nan, np.float32)
        for b in range(self.sealed // BLOCK):
            p, at = order[b // 4], b % 4
            kp[p, :, at * BLOCK:(at + 1) * BLOCK] = self.kc[:, b]
            vp[p, :, :, at * BLOCK:(at + 1) * BLOCK] = self.vc[:, b].transpose(0, 2, 1)
            sp[p, :, 0, at], sp[p, :, 1, at] = self.ks[:, b], self.vs[:, b]
        return kp, vp, sp

    def flat(self, row0=0):
        pools = [cuda(x) for x in self.pools(range(self.pages), self.pages)] if self.sealed else [None] * 3
        return luce.Q8View(*pools, self.sealed, cuda(self.k), cuda(self.v), self.tail, self.parent, row0, window=self.window,
                           sinks=self.sinks)

    def paged(self, rng, row0=0, layers=1, layer=0, extra=3):
        order = rng.permutation(self.pages + extra)[:self.pages].astype(np.int32)
        pools = []
        for x in self.pools(order, self.pages + extra):
            pool = np.full((x.shape[0], layers, *x.shape[1:]), 127 if x.dtype == np.int8 else np.nan, x.dtype)
            pool[:, layer] = x
            pools.append(cuda(pool)[:, layer])
        return luce.Q8View(*pools, self.sealed, cuda(self.k), cuda(self.v), self.tail, self.parent, row0, table=cuda(order),
                           window=self.window, sinks=self.sinks)


def run(slots, views, Hkv):
    q = cuda(np.concatenate([s.q for s in slots]))
    out = torch.full_like(q, float("nan"))
    luce.luce_q8kv_attn(q, views, Hkv, SCALE, out=out)
    torch.cuda.synchronize()
    assert luce.wait_timeouts() == 0
    return out


def check(slots, out):
    r0 = 0
    for s in slots:
        n, total = len(s.parent), s.sealed + s.tail
        k, v = s.keys()
        want = ref.attention(s.q, k, v, total, s.parent, SCALE, s.window, s.sinks)
        got = out[r0:r0 + n].cpu().numpy().astype(np.float64)
        assert np.abs(got - want).max() <= ref.attention_tolerance(s.q, k, v, total, n, SCALE, 160)
        assert np.linalg.norm(got - want) <= 1e-5 * np.linalg.norm(want)
        r0 += n


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("Hq,Hkv,sealed,tail,kind,n", [
    (8, 2, 0, 0, "chain", 1), (8, 2, 0, 17, "random", 9), (8, 2, 32, 0, "star", 2), (4, 4, 64, 1, "chain", 3), (40, 8, 96, 31, "random", 16),
    (40, 8, 128, 0, "random", 5), (8, 1, 160, 5, "forest", 16), (7, 1, 256, 112, "random", 7), (6, 2, 288, 30, "chain", 4),
    (5, 1, 992, 8, "random", 13), (16, 2, 1024, 111, "star", 16), (2, 2, 4096, 1, "random", 3), (3, 1, 8192, 31, "random", 11),
    (70, 70, 320, 3, "random", 3), (200, 200, 1312, 7, "chain", 2), (8, 2, 8224, 0, "random", 16), (8, 1, 2048, 4, "random", 16),
    (4, 2, 16480, 20, "random", 6), (2, 1, 40000, 3, "random", 4), (24, 4, 2016, 31, "random", 8), (56, 8, 1984, 2, "random", 12),
])
def test_one_slot(Hq, Hkv, sealed, tail, kind, n, paged):
    rng = np.random.default_rng(sealed * 31 + n)
    s = Cache(rng, Hq, Hkv, sealed, tail, tree_of(kind, n, sealed))
    check([s], run([s], [s.paged(rng, layers=2, layer=1) if paged else s.flat()], Hkv))


@pytest.mark.parametrize("G,n", [(1, 1), (8, 2), (8, 3), (5, 6), (7, 7), (8, 8), (6, 13), (8, 11), (8, 16)])
def test_chunks_of_several_tiles(G, n):
    """Every width of the products, over chunks of more tiles than lie in flight."""
    rng = np.random.default_rng(G * n)
    s = Cache(rng, G, 1, 130784 - 4096 * (n % 3), 5, tree_of("random", n, n), window=0 if n % 2 else 100000, sinks=300)
    check([s], run([s], [s.paged(rng)], 1))


def test_longest():
    rng = np.random.default_rng(5)
    s = Cache(rng, 8, 1, 130784, 16, tree_of("random", 16, 3), slack=0)
    check([s], run([s], [s.paged(rng)], 1))


@pytest.mark.parametrize("sealed,tail,window,sinks", [
    (0, 5, 1, 0), (0, 20, 3, 2), (32, 0, 1, 0), (32, 3, 2, 1), (512, 7, 4, 0), (512, 7, 8, 0), (512, 7, 9, 40), (1024, 31, 32, 4),
    (1024, 31, 33, 4), (4096, 9, 129, 0), (4096, 9, 1000, 1), (4096, 9, 1000, 128), (4096, 9, 1000, 129), (4096, 9, 3000, 1500),
    (4096, 9, 4104, 4), (4096, 9, 4105, 4), (4096, 9, 4106, 4), (4096, 9, 2 ** 31 - 1, 0), (4096, 9, 5, 2 ** 31 - 1), (20000, 0, 4096, 4),
])
@pytest.mark.parametrize("Hq,Hkv,n", [(8, 2, 16), (5, 1, 1)])
def test_window(Hq, Hkv, n, sealed, tail, window, sinks):
    rng = np.random.default_rng(sealed + window % 1000)
    s = Cache(rng, Hq, Hkv, sealed, tail, tree_of("random", n, sealed), window, sinks)
    flat = run([s], [s.flat()], Hkv)
    check([s], flat)
    assert np.array_equal(bits(flat), bits(run([s], [s.paged(rng)], Hkv)))


def test_keys_outside_the_window_are_not_used():
    """Tail rows that no row sees may hold anything; so may the codes and scales of tiles that no row sees."""
    rng = np.random.default_rng(3)
    s = Cache(rng, 8, 2, 1024, 20, chain(3), window=6, sinks=2)
    clean = run([s], [s.flat()], 2)
    s.k[:, :10], s.v[:, :10] = np.nan, np.inf
    s.ks[:, 4:], s.vs[:, 4:] = np.nan, np.inf
    s.kc[:, 4:] = 127
    assert np.array_equal(bits(clean), bits(run([s], [s.flat()], 2)))


@pytest.mark.parametrize("sealed,tail,nodes,Hq,Hkv", [([0, 0, 512, 992], [0, 17, 1, 8], [1, 2, 3, 4], 8, 2),
                                                      ([2048, 0, 128], [3, 1, 2], [7, 8, 1], 40, 8), ([128, 8992], [0, 8], [1, 15], 12, 4),
                                                      ([2016, 2048, 1984, 2016], [31, 3, 15, 24], [4] * 4, 40, 8)])
@pytest.mark.parametrize("window", [0, 700])
def test_several_slots(sealed, tail, nodes, Hq, Hkv, window):
    rng = np.random.default_rng(sum(sealed))
    slots = [Cache(rng, Hq, Hkv, s, t, tree_of("random", n, s), window if i != 1 else 0, 4) for i, (s, t, n) in enumerate(zip(sealed, tail, nodes))]
    rows = np.cumsum([0] + nodes)
    flat = run(slots, [s.flat(int(r)) for s, r in zip(slots, rows)], Hkv)
    check(slots, flat)
    assert np.array_equal(bits(flat), bits(run(slots, [s.paged(rng, int(r)) for s, r in zip(slots, rows)], Hkv)))
    for s, r in zip(slots, rows):                              # a slot alone gives the bits it gives with others
        assert np.array_equal(bits(run([s], [s.flat()], Hkv)), bits(flat[r:r + len(s.parent)]))
    order = list(range(len(slots)))[::-1]                      # and with the views given in another order
    q = cuda(np.concatenate([s.q for s in slots]))
    assert np.array_equal(bits(luce.luce_q8kv_attn(q, [slots[i].flat(int(rows[i])) for i in order], Hkv, SCALE)), bits(flat))


@pytest.mark.parametrize("sealed,tail", [(0, 5), (192, 8), (2048, 3), (8992, 8)])
@pytest.mark.parametrize("Hq,Hkv,window", [(40, 8, 0), (3, 1, 0), (24, 4, 150), (8, 1, 7)])
def test_a_node_gives_the_bits_of_its_path_alone(sealed, tail, Hq, Hkv, window):
    rng = np.random.default_rng(sealed)
    s = Cache(rng, Hq, Hkv, sealed, tail, tree_of("random", 16, sealed), window, 3)
    out = run([s], [s.flat()], Hkv)
    for j in (0, 3, 7, 15):
        path = ancestors(s.parent, j)
        t = Cache(rng, Hq, Hkv, 0, tail, chain(len(path)), window, 3)
        for name in ("sealed", "pages", "kc", "ks", "vc", "vs"):
            setattr(t, name, getattr(s, name))
        for new, old in ((t.k, s.k), (t.v, s.v)):
            new[:, :tail] = old[:, :tail]
            new[:, tail:tail + len(path)] = old[:, [tail + a for a in path]]
        t.q[:] = s.q[path]
        assert np.array_equal(bits(run([t], [t.flat()], Hkv)[-1]), bits(out[j]))


@pytest.mark.parametrize("spread", [2.0 ** 4, 2.0 ** 12])
def test_blocks_of_unlike_size_keep_their_digits(spread):
    """V's scales of neighbouring blocks lie far apart: where the large ones' weights are small, the others' digits count."""
    rng = np.random.default_rng(9)
    s = Cache(rng, 8, 1, 640, 0, chain(2), spread=1.0)
    big = np.arange(20) % 2 == 1
    s.vs[:, big] *= np.float32(spread)
    s.ks[:, big] *= np.float32(1e-3)
    s.kc[:, ~big] = np.abs(s.kc[:, ~big])                      # scores of the small blocks far above the large ones'
    s.q[:] = np.abs(s.q) * 4
    s.v[:] = 0
    check([s], run([s], [s.flat()], 1))


def test_zero_blocks_and_zero_scale():
    rng = np.random.default_rng(2)
    s = Cache(rng, 8, 2, 256, 0, chain(1))
    for c, x in ((s.kc, s.ks), (s.vc, s.vs)):
        c[:, 1:3], x[:, 1:3] = 0, 0
    check([s], run([s], [s.flat()], 2))
    q = cuda(s.q)
    k, v = s.keys()
    got = luce.luce_q8kv_attn(q, [s.flat()], 2, 0.0).cpu().numpy()
    want = ref.attention(s.q, k, v, 256, s.parent, 0.0)
    assert np.abs(got - want).max() <= ref.attention_tolerance(s.q, k, v, 256, 1, 0.0, 160)
    got = luce.luce_q8kv_attn(q, [s.flat()], 2, -SCALE).cpu().numpy()
    want = ref.attention(s.q, k, v, 256, s.parent, -SCALE)
    assert np.abs(got - want).max() <= ref.attention_tolerance(s.q, k, v, 256, 1, SCALE, 160)


@pytest.mark.parametrize("size", [1e-30, 1e-4, 60000.0])
def test_small_and_large_q(size):
    rng = np.random.default_rng(4)
    s = Cache(rng, 8, 2, 512, 5, chain(2))
    s.q[:] = s.q / np.abs(s.q).max() * size
    k, v = s.keys()
    scale = min(SCALE / size, 1e30)
    got = luce.luce_q8kv_attn(cuda(s.q), [s.flat()], 2, scale).cpu().numpy()
    want = ref.attention(s.q, k, v, 517, s.parent, float(np.float32(scale)))
    assert np.abs(got - want).max() <= ref.attention_tolerance(s.q, k, v, 517, 2, scale, 160)


def test_pages_outside_the_pool_hold_zeros():
    rng = np.random.default_rng(6)
    s = Cache(rng, 8, 2, 512, 3, chain(2))
    view = s.paged(rng)
    view.table[1], view.table[2] = -1, view.k_codes.shape[0]
    for x in (s.kc, s.vc):
        x[:, 4:12] = 0
    check([s], run([s], [view], 2))


def test_strided_tail_and_other_stream():
    rng = np.random.default_rng(7)
    s = Cache(rng, 12, 4, 640, 9, tree_of("random", 6, 1))
    want = run([s], [s.flat()], 4)
    view = s.flat()
    cap = s.k.shape[1]
    big = torch.full((2, cap + 2, 4, 160), float("nan"), dtype=torch.float16, device="cuda")  # tokens outside, heads inside
    big[0, :cap, :, :128], big[1, :cap, :, :128] = cuda(s.k).transpose(0, 1), cuda(s.v).transpose(0, 1)
    with pytest.raises(luce.LuceError):                        # heads inside tokens: refused
        luce.luce_q8kv_attn(cuda(s.q), [luce.Q8View(view.k_codes, view.v_codes, view.scales, 640, *(b[:cap, :, :128].transpose(0, 1) for b in big), 9, s.parent)], 4, SCALE)
    wide = torch.full((2, 4, cap + 2, 160), float("nan"), dtype=torch.float16, device="cuda")
    wide[0, :, :cap, :128], wide[1, :, :cap, :128] = cuda(s.k), cuda(s.v)
    view.k, view.v = wide[0, :, :cap, :128], wide[1, :, :cap, :128]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    q = cuda(s.q)
    torch.cuda.synchronize()
    out = luce.luce_q8kv_attn(q, [view], 4, SCALE, stream=stream)
    stream.synchronize()
    assert np.array_equal(bits(out), bits(want))


def test_prepared_attention_follows_its_views():
    rng = np.random.default_rng(8)
    a, b = Cache(rng, 8, 2, 320, 9, tree_of("random", 5, 1)), Cache(rng, 8, 2, 2048, 30, chain(5), window=100, sinks=7)
    view = a.flat()
    q = cuda(a.q)
    call = luce.Q8Attention(q, [view], 2, SCALE)
    assert np.array_equal(bits(call()), bits(run([a], [a.flat()], 2)))
    view.sealed, view.len = 256, 4                             # fewer keys of the same cache
    short = a.flat()
    short.sealed, short.len = 256, 4
    assert np.array_equal(bits(call()), bits(luce.luce_q8kv_attn(q, [short], 2, SCALE)))
    other = b.flat()                                           # another cache, longer than the workspace was made for
    for name in ("k_codes", "v_codes", "scales", "sealed", "k", "v", "len", "parent", "window", "sinks"):
        setattr(view, name, getattr(other, name))
    q.copy_(cuda(b.q))
    assert np.array_equal(bits(call()), bits(run([b], [b.flat()], 2)))
    view.parent = [-1, 0]
    with pytest.raises(ValueError):
        call()
    view.parent, view.sealed = 5, 4096
    with pytest.raises(ValueError):
        call()


def test_captured_attention_is_replayed():
    rng = np.random.default_rng(11)
    slots = [Cache(rng, 40, 8, 2048, 3, chain(4)), Cache(rng, 40, 8, 960, 0, chain(2))]
    views = [slots[0].flat(0), slots[1].flat(4)]
    want = run(slots, views, 8)
    q = cuda(np.concatenate([s.q for s in slots]))
    call = luce.Q8Attention(q, views, 8, SCALE)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        call.out.fill_(float("nan"))
        g.replay()
        assert np.array_equal(bits(call.out), bits(want))


def test_repeated_calls_give_the_same_bits():
    rng = np.random.default_rng(12)
    slots = [Cache(rng, 40, 8, 2048, 3, tree_of("random", 8, 5)), Cache(rng, 40, 8, 8000, 20, tree_of("random", 8, 6), window=3000, sinks=4)]
    views = [slots[0].flat(0), slots[1].flat(8)]
    q = cuda(np.concatenate([s.q for s in slots]))
    call = luce.Q8Attention(q, views, 8, SCALE)
    want = bits(call().clone())
    for _ in range(50):
        call.out.fill_(float("nan"))
        assert np.array_equal(bits(call()), want)


# ------------------------------------------------------------ sealing

def seal_slot(rng, L, Hkv, n, sealed, cap, paged, special=False):
    k = rng.standard_normal((L, Hkv, cap, D)).astype(np.float16)
    v = (rng.standard_normal((L, Hkv, cap, D)) * 3.0 ** rng.standard_normal((L, Hkv, cap, 1))).astype(np.float16)
    if special:
        k[:, :, 0], v[:, 0, :32] = 0, 0                        # a whole block of zeros
        k[:, :, 3, 5], k[:, :, 4, 6], k[:, :, 5, 7] = np.nan, np.inf, -np.inf
        v[:, -1, 33], v[:, -1, 34, 1] = np.nan, 65504
        k[0, 0, 40, :] = 6e-8                                  # the smallest magnitude
    pages = -(-(sealed + n) // PAGE)
    total = pages + (2 if paged else 0)
    order = rng.permutation(total)[:pages].astype(np.int32) if paged else np.arange(pages, dtype=np.int32)
    pools = luce.q8_cache(max(1, total), L, Hkv)
    for p, fill in zip(pools, (11, 12, 13)):
        p.fill_(fill)
    return k, v, order, luce.Q8Slot(cuda(k), cuda(v), n, *pools, sealed, cuda(order) if paged else None)


def check_sealed(k, v, order, slot):
    n, sealed = slot.len, slot.sealed
    nb = n // BLOCK
    want = [np.full(slot.k_codes.shape, 11, np.int8), np.full(slot.v_codes.shape, 12, np.int8), np.full(slot.scales.shape, 13, np.float32)]
    for which, (x, t) in enumerate(((k, slot.k), (v, slot.v))):
        for b in range(nb):
            c, d = ref.quantise(x[:, :, b * BLOCK:(b + 1) * BLOCK])
            at = sealed // BLOCK + b
            p, span = order[at // 4], slice(at % 4 * BLOCK, (at % 4 + 1) * BLOCK)
            if which == 0:
                want[0][p, :, :, span] = c
            else:
                want[1][p, :, :, :, span] = c.transpose(0, 1, 3, 2)
            want[2][p, :, :, which, at % 4] = d
        left = x.copy()
        if nb:
            left[:, :, :n - nb * BLOCK] = x[:, :, nb * BLOCK:n]
        assert np.array_equal(t.cpu().numpy().view(np.uint16), left.view(np.uint16))
    for t, w in zip((slot.k_codes, slot.v_codes, slot.scales), want):
        assert np.array_equal(t.cpu().numpy(), w)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("L,Hkv,n,sealed", [(1, 1, 32, 0), (1, 2, 33, 0), (2, 3, 63, 96), (3, 1, 47, 32), (1, 1, 31, 64), (1, 1, 0, 0), (1, 2, 64, 0),
                                            (2, 2, 300, 64), (1, 8, 4097, 992)])
def test_seal(L, Hkv, n, sealed, paged):
    rng = np.random.default_rng(n + sealed)
    k, v, order, slot = seal_slot(rng, L, Hkv, n, sealed, n + 5, paged, special=n >= 47)
    luce.luce_q8kv_seal([slot])
    check_sealed(k, v, order, slot)


def test_seal_codes_near_a_half():
    """Quotients that lie on or next to a half: every magnitude of fp16 against scales that put it there."""
    every = np.arange(0x7C00, dtype=np.uint16).view(np.float16)
    every = np.concatenate([every, -every])
    rng = np.random.default_rng(0)
    blocks = []
    for i in range(512):
        x = rng.choice(every, (BLOCK, D))
        top = np.float16(2.0 ** rng.integers(-14, 15) * rng.choice([1, 127 / 128, 127 / 64 / 2, 1.5]))
        x = np.where(np.abs(x) > top, (np.float32(top) / 127 * (rng.integers(0, 127, x.shape) + 0.5)).astype(np.float16), x)
        x[0, 0] = top
        blocks.append(x)
    k = np.concatenate(blocks)[None, None]
    pools = luce.q8_cache(128, 1, 1)
    slot = luce.Q8Slot(cuda(k), cuda(k), 512 * BLOCK, *pools)
    luce.luce_q8kv_seal([slot])
    c, d = ref.quantise(k.reshape(512, BLOCK, D))
    assert np.array_equal(pools[0].cpu().numpy().reshape(512, BLOCK, D), c)
    assert np.array_equal(pools[1].cpu().numpy().reshape(128, D, 4, BLOCK).transpose(0, 2, 3, 1).reshape(512, BLOCK, D), c)
    assert np.array_equal(pools[2][:, 0, 0, 0].cpu().numpy().reshape(-1), d)


def test_seal_several_slots_of_one_pool():
    rng = np.random.default_rng(1)
    slots, host = [], []
    pools = luce.q8_cache(12, 2, 2)
    for p, fill in zip(pools, (11, 12, 13)):
        p.fill_(fill)
    order = rng.permutation(12).astype(np.int32)
    for i, (n, sealed) in enumerate([(32, 224), (5, 96), (130, 0), (64, 64)]):
        k, v, _, s = seal_slot(rng, 2, 2, n, sealed, 140, True)
        s.k_codes, s.v_codes, s.scales, s.table = *pools, cuda(order[3 * i:3 * i + 3])
        host.append((k, v, n, sealed, order[3 * i:3 * i + 3]))
        slots.append(s)
    luce.luce_q8kv_seal(slots)
    want_k = np.full(pools[0].shape, 11, np.int8)
    for k, v, n, sealed, table in host:
        for b in range(n // BLOCK):
            at = sealed // BLOCK + b
            want_k[table[at // 4], :, :, at % 4 * BLOCK:(at % 4 + 1) * BLOCK] = ref.quantise(k[:, :, b * BLOCK:(b + 1) * BLOCK])[0]
    assert np.array_equal(pools[0].cpu().numpy(), want_k)


def test_seal_leaves_pages_outside_the_pool():
    rng = np.random.default_rng(2)
    k, v, order, slot = seal_slot(rng, 1, 1, 300, 0, 300, True)
    slot.table[0], slot.table[1] = -1, slot.k_codes.shape[0]
    luce.luce_q8kv_seal([slot])
    torch.cuda.synchronize()
    c, _ = ref.quantise(k[:, :, 256:288])
    want = np.full(slot.k_codes.shape, 11, np.int8)
    want[order[2], :, :, :32] = c
    assert np.array_equal(slot.k_codes.cpu().numpy(), want)
    assert np.array_equal(slot.k.cpu().numpy()[:, :, :12], k[:, :, 288:300])


# ------------------------------------------------------------ norm, rotation, append

def project_tolerance(x, q, gamma, pos):
    """Per element of q: the angle is rounded to fp32 once (|r| <= pi: pi 2^-24), sine and cosine to 2 units each, two
    products, a sum; the norm's sum of 128 squares, its root, its reciprocal, two products."""
    big = np.abs(q).reshape(*q.shape[:-1], 2, D // 2)
    pair = np.repeat(np.sqrt((big ** 2).sum(-2, keepdims=True)), 2, -2).reshape(q.shape)  # |(a, b)| bounds either
    return pair * (4 * 2.0 ** -24 + 2 * 2.0 ** -22 + ref.U * (3 + (64 + 8 if gamma is not None else 0)))


@pytest.mark.parametrize("rows,Hq,Hkv,axes,norm", [
    ([1], 1, 1, 1, False), ([1], 8, 2, 1, True), ([4, 4, 4, 4], 40, 8, 1, True), ([3, 1], 5, 5, 2, True), ([7], 16, 3, 3, True),
    ([151], 8, 2, 1, False), ([152], 8, 2, 3, True), ([200, 1, 33], 40, 8, 3, True), ([160], 70, 1, 4, True), ([2], 100, 100, 1, True),
])
def test_project(rows, Hq, Hkv, axes, norm):
    rng = np.random.default_rng(sum(rows) + Hq)
    T = sum(rows)
    x = (rng.standard_normal((T, (Hq + 2 * Hkv) * D)) * 10.0 ** rng.integers(-3, 3, (T, 1))).astype(np.float32)
    x[0, :D] = 0                                               # a head of zeros
    pos = rng.integers(-5 if axes > 1 else 0, 1 << 20, (axes, T)).astype(np.int32)
    pair_axis = rng.integers(0, axes, 64).tolist()
    qg, kg = (rng.standard_normal(D).astype(np.float32) for _ in range(2)) if norm else (None, None)
    caps = [r + 9 for r in rows]
    fill = np.float16(-7)
    views, r0 = [], 0
    for r, cap in zip(rows, caps):
        k, v = (torch.full((Hkv, cap, 136), -7.0, dtype=torch.float16, device="cuda")[:, :, :128] for _ in range(2))
        views.append(luce.SeqView(k, v, 4 + r, r, r0))
        r0 += r
    q = luce.luce_qk_norm_rope(cuda(x), views, Hq, cuda(pos), 1e6, None if qg is None else cuda(qg), None if kg is None else cuda(kg), 1e-6, pair_axis)
    wq, wk, wv = ref.project(x, Hq, Hkv, qg, kg, 1e-6, pos, pair_axis, 1e6)
    tol = project_tolerance(x, wq, qg, pos)
    assert (np.abs(q.cpu().numpy() - wq) <= tol + 1e-37).all()
    r0 = 0
    for view, r in zip(views, rows):
        for got, want, t in ((view.k, wk, project_tolerance(x, wk, kg, pos)), (view.v, wv, np.zeros(wv.shape))):
            got = got.cpu().numpy()
            w = want[r0:r0 + r].transpose(1, 0, 2)
            assert (np.abs(got[:, 4:4 + r] - w) <= t[r0:r0 + r].transpose(1, 0, 2) * 1.01 + np.abs(w) * 2.0 ** -11 + 2.0 ** -25).all()
            assert (got[:, :4] == fill).all() and (got[:, 4 + r:] == fill).all()
        r0 += r


def test_project_gives_the_bits_of_rope_and_append():
    rng = np.random.default_rng(3)
    T, Hq, Hkv = 9, 10, 5
    x = rng.standard_normal((T, (Hq + 2 * Hkv) * D)).astype(np.float32)
    pos = rng.integers(0, 1 << 17, T).astype(np.int32)
    k, v, k2, v2 = (torch.zeros(Hkv, 20, D, dtype=torch.float16, device="cuda") for _ in range(4))
    q = luce.luce_qk_norm_rope(cuda(x), [luce.SeqView(k, v, 12, 9, 0)], Hq, cuda(pos), 1e6)
    h = cuda(x).view(T, -1, D)
    qk = luce.luce_rope_posvec(h[:, :Hq + Hkv].contiguous(), cuda(pos), 1e6)
    kk, vv = qk[:, Hq:].contiguous(), h[:, Hq + Hkv:].contiguous()
    for r in range(T):
        luce.luce_kv_append(kk[r:r + 1], vv[r:r + 1], [luce.SeqView(k2, v2, 4 + r, 1, 0)])
    assert np.array_equal(bits(q), bits(qk[:, :Hq]))
    assert torch.equal(k.view(torch.int16), k2.view(torch.int16)) and torch.equal(v.view(torch.int16), v2.view(torch.int16))


def test_project_rows_do_not_depend_on_company():
    """Few rows and many take different grids; a row's bits are the same."""
    rng = np.random.default_rng(4)
    T, Hq, Hkv = 400, 40, 8
    x = cuda(rng.standard_normal((T, (Hq + 2 * Hkv) * D)).astype(np.float32))
    pos = cuda(rng.integers(0, 1 << 17, (3, T)).astype(np.int32))
    g = cuda(rng.standard_normal(D).astype(np.float32))
    axes = luce.rope_sections((16, 24, 24), interleaved=True)
    k, v, k2, v2 = (torch.zeros(Hkv, T, D, dtype=torch.float16, device="cuda") for _ in range(4))
    q = luce.luce_qk_norm_rope(x, [luce.SeqView(k, v, T, T, 0)], Hq, pos, 1e4, g, g, pair_axis=axes)
    for lo, hi in ((0, 1), (1, 4), (4, 100), (100, 400)):
        part = luce.luce_qk_norm_rope(x[lo:hi], [luce.SeqView(k2, v2, hi, hi - lo, 0)], Hq, pos[:, lo:hi].contiguous(), 1e4, g, g, pair_axis=axes)
        assert np.array_equal(bits(part), bits(q[lo:hi]))
    assert torch.equal(k, k2) and torch.equal(v, v2)


def test_sections():
    assert luce.rope_sections((16, 24, 24)) == [0] * 16 + [1] * 24 + [2] * 24
    mixed = luce.rope_sections((16, 24, 24), interleaved=True)
    assert mixed[:6] == [0, 1, 2, 0, 1, 2] and mixed.count(0) == 16 and mixed[48:] == [1, 2] * 8
    with pytest.raises(ValueError):
        luce.rope_sections((16, 24))


# ------------------------------------------------------------ together

def test_decode_loop_over_a_cache_in_8_bits():
    """Prompt, sealing, then steps that verify draft trees and commit a path: each step's attention against the plain form
    over what the cache holds, and the cache's codes against those of the tokens quantised block by block."""
    rng = np.random.default_rng(21)
    Hq, Hkv, L, theta = 10, 2, 1, 1e6
    cap = 400
    k, v = (torch.zeros(L, Hkv, cap, D, dtype=torch.float16, device="cuda") for _ in range(2))
    pools = luce.q8_cache(8, L, Hkv)
    table = cuda(rng.permutation(8).astype(np.int32))
    gq, gk = (cuda((1 + 0.1 * rng.standard_normal(D)).astype(np.float32)) for _ in range(2))
    slot = luce.Q8Slot(k, v, 0, *pools, 0, table)
    tokens = [np.zeros((Hkv, 0, D), np.float16), np.zeros((Hkv, 0, D), np.float16)]  # every committed token's rows

    def project(n, depth):
        x = rng.standard_normal((n, (Hq + 2 * Hkv) * D)).astype(np.float32)
        pos = np.array([slot.sealed + slot.len + d for d in depth], np.int32)
        return luce.luce_qk_norm_rope(cuda(x), [luce.SeqView(k[0], v[0], slot.len + n, n, 0)], Hq, cuda(pos), theta, gq, gk)

    def keep(rows):
        for t, x in zip(tokens, (k, v)):
            t_new = x[0].cpu().numpy()[:, rows]
            tokens[0 if x is k else 1] = np.concatenate([t, t_new], 1)

    def seal():
        luce.luce_q8kv_seal([slot])
        slot.sealed, slot.len = slot.sealed + slot.len // BLOCK * BLOCK, slot.len % BLOCK

    project(300, range(300))
    slot.len = 300
    keep(list(range(300)))
    seal()
    assert (slot.sealed, slot.len) == (288, 12)
    for step in range(12):
        parent = tree_of("random", 6, step)
        depth = [len(ancestors(parent, j)) - 1 for j in range(6)]
        q = project(6, depth)
        view = luce.Q8View(*(p[:, 0] for p in pools), slot.sealed, k[0], v[0], slot.len, parent, 0, table=table, window=200, sinks=4)
        out = luce.luce_q8kv_attn(q, [view], Hkv, SCALE)
        # the plain form over the committed tokens, the sealed ones as codes
        host = []
        for t, x in zip(tokens, (k, v)):
            c, s = ref.quantise(t[:, :slot.sealed].reshape(Hkv, -1, BLOCK, D))
            f = (c.astype(np.float64) * s.astype(np.float64)[..., None, None]).reshape(Hkv, -1, D)
            host.append(np.concatenate([f, x[0].cpu().numpy()[:, :slot.len + 6].astype(np.float64)], 1))
        total = slot.sealed + slot.len
        want = ref.attention(q.cpu().numpy(), *host, total, parent, SCALE, 200, 4)
        got = out.cpu().numpy().astype(np.float64)
        assert np.abs(got - want).max() <= ref.attention_tolerance(q.cpu().numpy(), *host, total, 6, SCALE, 160)
        path = ancestors(parent, 5)
        luce.luce_tree_commit([luce.CommitSlot(k, v, slot.len, path)], Hq)
        keep([slot.len + i for i in range(len(path))])
        slot.len += len(path)
        seal()
    c, s = ref.quantise(tokens[0][:, :slot.sealed].reshape(Hkv, -1, BLOCK, D))
    pages = pools[0][table.long()[:-(-slot.sealed // PAGE)], 0].cpu().numpy().transpose(1, 0, 2, 3).reshape(Hkv, -1, D)
    assert slot.sealed > 288 and np.array_equal(pages[:, :slot.sealed], c.reshape(Hkv, -1, D))
