"""Scales of caches in 8 bits at the ends of what attention takes: blocks that no row sees inside
tiles that some row does."""
import numpy as np
import pytest

from test_gpu_q8kv import SCALE, Cache, bits, lib, run  # noqa: F401
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
