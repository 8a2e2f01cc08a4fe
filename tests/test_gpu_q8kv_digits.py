"""Attention over caches in 8 bits held to a relative error of the whole result, where a bound by the worst
element would let a real mistake pass: extreme units of q, scales of 0 and below, a decode loop's every step."""
import numpy as np
import pytest

import q8kv_reference as ref
from cache_reference import ancestors
from test_gpu_q8kv import BLOCK, D, SCALE, Cache, cuda, lib  # noqa: F401
from test_gpu_tree import tree_of

torch = pytest.importorskip("torch")
import invariant_sequence_decode_gb300 as luce  # noqa: E402

pytestmark = pytest.mark.gpu


def near(got, want):
    """1e-5 of the result's norm.  A weight is off by what its score is, a sum of 16 steps of the tensor cores within 2^-23 of
    partial sums of a few units (8e-6 at the very most, were all to err alike), and by 2^-19 at most from its exponent; out is
    a mean of values under these weights.  One sink less, a low part of q lost or a scale 1 % off are far outside."""
    torch.cuda.synchronize()
    assert luce.wait_timeouts() == 0
    got = got.cpu().numpy().astype(np.float64)
    assert np.linalg.norm(got - want) <= 1e-5 * np.linalg.norm(want)


@pytest.mark.parametrize("Hq,Hkv,n", [(8, 2, 2), (8, 1, 3), (8, 1, 11)])
@pytest.mark.parametrize("size", [1e-38, 1e-36, 1e-30, 1e-4, 60000.0, 65500.0])
def test_small_and_large_q(size, Hq, Hkv, n):
    rng = np.random.default_rng(4)
    s = Cache(rng, Hq, Hkv, 512, 5, tree_of("random", n, 3))
    s.q[:] = s.q / np.abs(s.q).max() * size
    scale = float(np.float32(SCALE / size))
    near(luce.luce_q8kv_attn(cuda(s.q), [s.flat()], Hkv, scale),
         ref.attention(s.q, *s.keys(), 517, s.parent, scale))


def test_rows_of_unlike_size():
    """Each row of q has a unit of its own."""
    rng = np.random.default_rng(5)
    s = Cache(rng, 8, 2, 1024, 7, tree_of("random", 9, 1))
    s.q *= (10.0 ** rng.integers(-3, 1, s.q.shape[:2]))[..., None].astype(np.float32)
    near(luce.luce_q8kv_attn(cuda(s.q), [s.flat()], 2, SCALE), ref.attention(s.q, *s.keys(), 1031, s.parent, SCALE))


@pytest.mark.parametrize("scale", [0.0, -SCALE, -2 * SCALE, 1e-30])
@pytest.mark.parametrize("Hq,Hkv,n,window", [(8, 2, 1, 0), (5, 1, 5, 0), (8, 1, 16, 100)])
def test_zero_and_negative_scale(Hq, Hkv, n, window, scale):
    rng = np.random.default_rng(6)
    s = Cache(rng, Hq, Hkv, 256, 9, tree_of("random", n, 2), window, 3)
    for c, x in ((s.kc, s.ks), (s.vc, s.vs)):
        c[:, 1:3], x[:, 1:3] = 0, 0
    near(luce.luce_q8kv_attn(cuda(s.q), [s.flat()], Hkv, scale),
         ref.attention(s.q, *s.keys(), 265, s.parent, scale, window, 3))


@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 4), (33, 40), (5, 0)])
def test_every_step_of_a_decode_loop(window, sinks):
    """Steps that append a tree's rows, attend, commit a path and seal, against the plain form over the tokens committed."""
    rng = np.random.default_rng(7)
    Hq, Hkv, n = 10, 2, 7
    k, v = (torch.zeros(1, Hkv, 400, D, dtype=torch.float16, device="cuda") for _ in range(2))
    pools = luce.q8_cache(8, 1, Hkv)
    table = cuda(rng.permutation(8).astype(np.int32))
    slot = luce.Q8Slot(k, v, 0, *pools, 0, table)
    ones = torch.ones(D, device="cuda")
    tokens = [np.zeros((Hkv, 0, D), np.float16) for _ in range(2)]

    def append(rows, depth):
        x = cuda(rng.standard_normal((rows, (Hq + 2 * Hkv) * D)).astype(np.float32))
        pos = cuda(np.array([slot.sealed + slot.len + d for d in depth], np.int32))
        return luce.luce_qk_norm_rope(x, [luce.SeqView(k[0], v[0], slot.len + rows, rows, 0)], Hq, pos, 1e6, ones, ones)

    def commit(rows):
        for i, x in enumerate((k, v)):
            tokens[i] = np.concatenate([tokens[i], x[0].cpu().numpy()[:, rows]], 1)

    append(271, range(271))
    slot.len = 271
    commit(list(range(271)))
    for step in range(14):
        luce.luce_q8kv_seal([slot])
        slot.sealed, slot.len = slot.sealed + slot.len // BLOCK * BLOCK, slot.len % BLOCK
        parent = tree_of("random", n, step)
        q = append(n, [len(ancestors(parent, j)) - 1 for j in range(n)])
        view = luce.Q8View(*(p[:, 0] for p in pools), slot.sealed, k[0], v[0], slot.len, parent, table=table, window=window, sinks=sinks)
        out = luce.luce_q8kv_attn(q, [view], Hkv, SCALE)
        keys = []
        for t, x in zip(tokens, (k, v)):
            c, d = ref.quantise(t[:, :slot.sealed].reshape(Hkv, -1, BLOCK, D))
            f = (c.astype(np.float64) * d.astype(np.float64)[..., None, None]).reshape(Hkv, -1, D)
            keys.append(np.concatenate([f, x[0].cpu().numpy()[:, :slot.len + n].astype(np.float64)], 1))
        near(out, ref.attention(q.cpu().numpy(), *keys, slot.sealed + slot.len, parent, SCALE, window, sinks))
        path = ancestors(parent, n - 1 - step % 3)
        commit([slot.len + a for a in path])
        luce.luce_tree_commit([luce.CommitSlot(k, v, slot.len, path)], Hq)
        slot.len += len(path)
