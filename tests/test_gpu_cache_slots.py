"""Slots of commits and evictions: the fields that may be left out."""
import numpy as np
import pytest

import cache_reference as ref

torch = pytest.importorskip("torch")
import invariant_sequence_decode_gb300 as luce  # noqa: E402
from test_gpu_cache import cuda, same  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from invariant_sequence_decode_gb300 import build
    build.build()
    return luce.load_library()


@pytest.mark.parametrize("length,budget", [(40, 35), (300, 100), (5000, 4990)])
@pytest.mark.parametrize("first", [0, 7000])
def test_eviction_without_positions_of_its_own_goes_by_weight(length, budget, first):
    """Also where earlier evictions left positions past the cache's length."""
    rng = np.random.default_rng(length)
    L, Hkv, cap = 2, 2, length + 3
    k, v = (rng.standard_normal((L, Hkv, cap, 128)).astype(np.float16) for _ in range(2))
    acc = rng.random((L, Hkv, cap)).astype(np.float32)
    pos = (first + rng.permuted(np.tile(np.arange(cap), (L, Hkv, 1)), axis=-1)).astype(np.int32)
    want = ref.evict(k, v, acc, pos, length, budget, 0, 0, 2 ** 31 - 1)
    slot = luce.EvictSlot(cuda(k), cuda(v), cuda(acc), cuda(pos), length, budget)
    luce.luce_kv_evict([slot])
    torch.cuda.synchronize()
    for t, w in zip((slot.k, slot.v, slot.acc, slot.pos), want):
        assert same(t[:, :, :budget], w[:, :, :budget])
