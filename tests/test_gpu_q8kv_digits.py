"""Attention over caches in 8 bits held to a relative error of the whole result, where a bound by the worst
element would let a real mistake pass: extreme units of q."""
import numpy as np
import pytest

import q8kv_reference as ref
from test_gpu_q8kv import SCALE, Cache, cuda, lib  # noqa: F401
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
