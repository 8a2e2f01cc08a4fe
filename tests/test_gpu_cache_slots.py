"""Slots of commits and evictions: the fields that may be left out."""
import numpy as np
import pytest

import cache_reference as ref

torch = pytest.importorskip("torch")
import invariant_sequence_decode_gb300 as luce  # noqa: E402
from test_gpu_cache import cuda, same, weight_tolerance  # noqa: E402

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


@pytest.mark.parametrize("paged", [False, True])
def test_a_commit_without_pos0_continues_the_cache(paged):
    rng = np.random.default_rng(3)
    L, Hkv, length, path = 2, 2, 200, [0, 3, 4]
    pos = cuda(np.tile(np.arange(256, dtype=np.int32), (L, Hkv, 1)))
    pos[:, :, length:] = -1
    if paged:
        pool = [cuda(rng.standard_normal((3, L, Hkv, 128, 128)).astype(np.float16)) for _ in range(2)]
        slot = luce.PagedCommitSlot(*pool, np.array([2, 0], dtype=np.int32), length, path, pos=pos)
    else:
        slot = luce.CommitSlot(*(cuda(rng.standard_normal((L, Hkv, 256, 128)).astype(np.float16)) for _ in range(2)), length, path, pos=pos)
    luce.luce_tree_commit([slot], 4)
    torch.cuda.synchronize()
    assert (pos[:, :, :length + 3].cpu() == torch.arange(length + 3)).all() and (pos[:, :, length + 3:] == -1).all()


@pytest.mark.parametrize("length,budget", [(300, 290), (700, 300)])
def test_a_prepared_eviction_follows_a_replaced_table(length, budget):
    """The same keys in other pages, by the same prepared call."""
    rng = np.random.default_rng(length)
    L, Hkv, per = 2, 2, -(-length // 128)
    k, v = (rng.standard_normal((L, Hkv, per * 128, 128)).astype(np.float16) for _ in range(2))
    acc = rng.random((L, Hkv, length)).astype(np.float32)
    pos = np.tile(np.arange(length, dtype=np.int32), (L, Hkv, 1))
    pools = [torch.zeros(2 * per, L, Hkv, 128, 128, dtype=torch.float16, device="cuda") for _ in range(2)]
    want = ref.evict(k, v, acc, pos, length, budget, 0, 0, length)
    slot = luce.PagedEvictSlot(*pools, cuda(np.arange(per, dtype=np.int32)), cuda(acc), cuda(pos), length, budget, next_pos=length,
                               acc_out=torch.zeros_like(cuda(acc)), pos_out=torch.zeros_like(cuda(pos)))
    call = luce.KvEvict([slot])
    for pages in (range(per), range(2 * per - 1, per - 1, -1)):
        table = np.array(list(pages), dtype=np.int32)
        slot.table = cuda(table)
        for pool, x in zip(pools, (k, v)):
            pool[torch.from_numpy(table).long()] = cuda(x.reshape(L, Hkv, per, 128, 128).transpose(2, 0, 1, 3, 4))
        call()
        torch.cuda.synchronize()
        for pool, w in zip(pools, want[:2]):
            got = pool[torch.from_numpy(table).long()].cpu().numpy().transpose(1, 2, 0, 3, 4).reshape(L, Hkv, per * 128, 128)
            assert np.array_equal(got.view(np.uint16), w.view(np.uint16))


@pytest.mark.parametrize("m", [float("-inf"), 0.0, -50.0, 3.0])
@pytest.mark.parametrize("length", [1, 70, 1300])
def test_a_row_without_weights_adds_nothing_whatever_its_scores(m, length):
    rng = np.random.default_rng(length)
    L, Hq, Hkv, n, path = 2, 4, 2, 3, [0, 2]
    cap = length + n
    k, v = (cuda(rng.standard_normal((L, Hkv, cap, 128)).astype(np.float16)) for _ in range(2))
    acc = rng.random((L, Hkv, cap)).astype(np.float32)
    scores = rng.standard_normal((L, n, Hq, -(-cap // 4) * 4)).astype(np.float32)
    stats = np.stack([scores.max(-1), np.exp(scores - scores.max(-1, keepdims=True)).sum(-1)], -1).astype(np.float32)
    scores[:, 2] = 100 * np.abs(scores[:, 2]) + 100             # e^s is past fp32
    scores[:, 2, :, ::3] = -np.inf
    stats[:, 2] = m, 0
    _, _, want, _ = ref.commit(k.cpu().numpy(), v.cpu().numpy(), length, path, acc, scores=scores, stats=stats)
    slot = luce.CommitSlot(k, v, length, path, acc=cuda(acc))
    luce.luce_tree_commit([slot], Hq, cuda(scores), cuda(stats))
    got = slot.acc.cpu().numpy()[:, :, :length + 2]
    assert np.abs(got - want[:, :, :length + 2]).max() <= weight_tolerance(want, Hq // Hkv, len(path))
