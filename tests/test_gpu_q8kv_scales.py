"""Scales of caches in 8 bits at the ends of what attention takes: blocks that no row sees inside
tiles that some row does, V's scales up to the least and the most."""
import numpy as np
import pytest

import q8kv_reference as ref
from cache_reference import chain
from test_gpu_q8kv import D, SCALE, Cache, bits, lib, run  # noqa: F401
from test_gpu_tree import tree_of

pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
BAD = [np.nan, np.inf, -np.inf, -1.0, 0.0, 3e38, 1e-45]


@pytest.mark.parametrize("Hq,Hkv,n", [(8, 2, 3), (5, 1, 1), (8, 1, 3), (8, 1, 10), (7, 1, 16)])
@pytest.mark.parametrize("window,sinks,unseen", [
    (6, 2, range(1, 32)),              # the first tile's first block alone is seen
    (230, 33, range(2, 25)),           # blocks between the sinks and the window, in both of their tiles
    (230, 0, range(0, 25)),            # ahead of the window's first block, inside its tile
])
def test_unseen_blocks_of_a_seen_tile_are_not_used(Hq, Hkv, n, window, sinks, unseen):
    """1,024 sealed keys and a tail of 20: with a window of 230 the first key that a node without ancestors sees
    is 1044 - 229 = 815, in block 25 of tile 6 (blocks 24 to 27)."""
    rng = np.random.default_rng(n)
    s = Cache(rng, Hq, Hkv, 1024, 20, tree_of("random", n, 4), window=window, sinks=sinks)
    clean = bits(run([s], [s.flat()], Hkv))
    assert np.isfinite(clean.view(np.float32)).all()
    unseen = list(unseen)
    for ks, vs, code in [(1.0, v, 127) for v in BAD] + [(k, 1.0, -128) for k in BAD] + [(np.inf, np.inf, -128), (np.nan, np.inf, 0)]:
        s.ks[:, unseen], s.vs[:, unseen] = ks, vs
        s.kc[:, unseen] = s.vc[:, unseen] = code
        assert np.array_equal(clean, bits(run([s], [s.flat()], Hkv))), (ks, vs, code)


def near(s, got):
    """A relative bound on the whole result.  A weight's relative error: its score is a sum of 16 steps of the tensor cores and
    a product, each within 2^-23 of the score's partial sums (a few units: 16 x 4 x 2^-23 at the very most, 8e-6, were all to
    err alike; as they do not, a quarter), the three numbers that its exponent is formed from round at 2^-19 at most (each is
    below 128); weights are two f16 parts.  out is a mean of values under these weights: 1e-5."""
    k, v = s.keys()
    want = ref.attention(s.q, k, v, s.sealed + s.tail, s.parent, SCALE, s.window, s.sinks)
    got = got.cpu().numpy().astype(np.float64)
    assert np.linalg.norm(got - want) <= 1e-5 * np.linalg.norm(want)


LEAST, MOST = 2.0 ** -50, 2.0 ** 35  # V's scales but 0
EDGES = [LEAST, float(np.nextafter(np.float32(LEAST), np.float32(1))), 1e-15, 1e-12, 2.0 ** -32, 2.0 ** -31, 2.0 ** -24 / 127, 1.0, MOST]


@pytest.mark.parametrize("Hq,Hkv,n", [(8, 2, 1), (8, 1, 4), (8, 1, 6), (8, 1, 8), (8, 1, 10), (8, 1, 12), (8, 1, 16)])
@pytest.mark.parametrize("scale", EDGES)
def test_small_scales_of_v_count_as_they_are(scale, Hq, Hkv, n):
    """All of V's blocks of one scale: the result is as small (or large) as they are.  Every width of the products."""
    rng = np.random.default_rng(3)
    s = Cache(rng, Hq, Hkv, 2016, 5, tree_of("random", n, 2))
    s.vs[:] = scale
    s.v[:] = 0
    near(s, run([s], [s.flat()], Hkv))


@pytest.mark.parametrize("window", [0, 300])
@pytest.mark.parametrize("small", [LEAST, 1e-15, 1e-12])
@pytest.mark.parametrize("Hq,Hkv,n", [(8, 2, 1), (5, 1, 5), (8, 1, 16)])
def test_small_scales_beside_others(Hq, Hkv, n, small, window):
    """Their weights stay in the sum, their values are as small as the scale says.  The others' values are small too,
    so that a code times 2^-31 would be seen."""
    rng = np.random.default_rng(4)
    s = Cache(rng, Hq, Hkv, 640, 3, chain(n), window, 4)
    s.vs[:, 1::2] = small
    s.vs[:, ::2] *= np.float32(1e-9) / s.vs[:, ::2]
    s.v[:] = 0
    near(s, run([s], [s.flat()], Hkv))


@pytest.mark.parametrize("small", [0.0, 1e-45, 1e-30, LEAST / 2])
@pytest.mark.parametrize("Hq,Hkv,n", [(8, 2, 1), (8, 1, 5), (8, 1, 16)])
def test_a_scale_below_the_least_counts_as_it(Hq, Hkv, n, small):
    rng = np.random.default_rng(6)
    s = Cache(rng, Hq, Hkv, 640, 3, chain(n))
    s.v[:] = 0
    s.vs[:, 1::2] = LEAST
    want = bits(run([s], [s.flat()], Hkv))
    s.vs[:, 1::2] = small
    assert np.array_equal(want, bits(run([s], [s.flat()], Hkv)))


@pytest.mark.parametrize("large", [1.0, 2.0 ** 10, MOST])
@pytest.mark.parametrize("Hq,Hkv,n", [(8, 2, 1), (8, 1, 5)])
def test_zero_blocks_beside_large_scales_keep_their_weight(Hq, Hkv, n, large):
    """What a block of zeros adds to the sum of weights is still there next to one of a large scale."""
    rng = np.random.default_rng(5)
    s = Cache(rng, Hq, Hkv, 512, 0, chain(n))
    s.vc[:, ::2], s.vs[:, ::2] = 0, 0
    s.vs[:, 1::2] = large
    s.v[:] = 0
    near(s, run([s], [s.flat()], Hkv))


@pytest.fixture(scope="module")
def longest():
    return Cache(np.random.default_rng(7), 5, 1, 130784, 0, chain(1))


@pytest.mark.parametrize("large", [1.0, 2.0 ** 10, MOST])
@pytest.mark.parametrize("below", [3, 13, 27])
def test_chunks_of_zeros_beside_a_large_scale_keep_their_weight(longest, below, large):
    """One key of a large value, 2^below times as heavy as each of 130,783 keys of zeros in other chunks: at 2^27 these are
    1e-3 of the sum of weights."""
    s = longest
    s.kc[:], s.ks[:], s.vc[:], s.vs[:] = 0, 1, 0, 0
    s.k[:], s.v[:] = 0, 0
    s.kc[:, 5, 3, 0] = below
    s.vc[:, 5, 3], s.vs[:, 5] = np.arange(D) - 70, large
    s.q[:] = 0
    s.q[:, :, 0] = np.log(2) / SCALE
    got = run([s], [s.flat()], 1).cpu().numpy().astype(np.float64)
    w = 2.0 ** (below * float(np.float32(np.log(2) / SCALE)) * float(np.float32(SCALE)) / np.log(2))
    want = np.repeat(s.vc[:, 5, 3].astype(np.float64) * large * w / (w + 130784), 5, 0)[None]
    # (the score is one product of a scale's, exact parts: 2^-24 of `below`, and three numbers' roundings as above)
    assert np.linalg.norm(got - want) <= 1e-5 * np.linalg.norm(want)
