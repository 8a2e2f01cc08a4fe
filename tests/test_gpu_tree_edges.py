"""Tree attention at its edges: views of unlike kinds in one call."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import invariant_sequence_decode_gb300 as luce  # noqa: E402
from test_gpu_tree import Slot, bits, check, run, tree_of  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from invariant_sequence_decode_gb300 import build
    build.build()
    return luce.load_library()


@pytest.mark.parametrize("lens", [[0, 300], [300, 64], [5, 65, 64], [65, 0, 1000, 3], [1, 2, 3, 129]])
def test_short_and_cut_prefixes_in_one_call(lens):
    rng = np.random.default_rng(sum(lens))
    slots = [Slot(rng, 8, 2, L, tree_of("random", 3, L)) for L in lens]
    for views in ([s.flat(3 * i) for i, s in enumerate(slots)], [s.paged(3 * i, rng) for i, s in enumerate(slots)]):
        out, sc, st = run(slots, views, 2, scores=True)
        check(slots, out, sc, st, 2)
    for i, s in enumerate(slots):
        alone, _, _ = run([s], [s.flat(0)], 2)
        assert np.array_equal(bits(alone), bits(out[3 * i:3 * i + 3]))
