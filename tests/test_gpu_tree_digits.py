"""Digits of tree attention's weights and of q, held relative to the output.

The inputs make the scores exact: q has one non-zero element and K's column is
what it picks, so a tolerance has no term for the products."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import invariant_sequence_decode_gb300 as luce  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -23   # a unit of an fp32 sum, a truncating add's


@pytest.fixture(scope="module", autouse=True)
def lib():
    from invariant_sequence_decode_gb300 import build
    build.build()
    return luce.load_library()


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def sums(length):
    """Units that positive sums and the exponentials cost relative to the result: 128 keys of a tile, the tiles, the
    merge's chunks (at most 160) and path; e^x of |x| <= 64 through one product with log2 e (64 / 2 units each for the
    product, the constant and the reference), 4 of exp2; once in the weighted sum, once in the sum of weights."""
    return U * 2 * (128 + -(-length // 128) + 160 + 16 + 3 * 32 + 4)


@pytest.mark.parametrize("gap", [0, 8, 12, 16, 17, 18, 20])
@pytest.mark.parametrize("Hkv,length,at", [(152, 2000, 5), (8, 20000, 3), (1, 100, 99), (2, 70, 0)])
@pytest.mark.parametrize("spread", [0, 1])
def test_small_weights_keep_their_digits_beside_a_dominant_key(Hkv, length, at, gap, spread):
    """An attention sink: one key far above the others, its V zero, so the output is the sum of the small weights.

    A weight of e^-x of the largest is held as two f16 parts of 2^15 e^-x: within 2^-22 of it, and within 2^-25 in all.
    """
    rng = np.random.default_rng(length + gap)
    n, cap = 2, length + 2
    q = np.zeros((n, Hkv, 128), dtype=np.float32)
    q[:, :, 7] = 1
    score = (spread * rng.random((Hkv, cap)) - spread).astype(np.float16)   # in [-1, 0], exact
    score[:, at] = gap
    k = np.zeros((Hkv, cap, 128), dtype=np.float16)
    k[:, :, 7] = score
    v = (0.5 + rng.random((Hkv, cap, 128))).astype(np.float16)
    v[:, at] = 0
    out = luce.luce_tree_attn(cuda(q), [luce.TreeView(cuda(k), cuda(v), length, [-1, -1])], Hkv, 1.0)
    got = out.cpu().numpy().astype(np.float64)
    tol = sums(length) + 2.0 ** -22 + 2.0 ** -40 * np.exp(gap + spread)
    for j in range(n):
        keys = [*range(length), length + j]
        p = np.exp(score[:, keys].astype(np.float64) - gap)
        want = np.einsum("gk,gkd->gd", p, v[:, keys].astype(np.float64)) / p.sum(1, keepdims=True)
        assert (np.abs(got[j] - want) / want).max() <= tol


@pytest.mark.parametrize("size", [1e-30, 1e-10, 1e-6, 1e-5, 1e-3, 1.0, 6e4])
@pytest.mark.parametrize("Hq,Hkv,length", [(40, 8, 300), (3, 1, 1000), (8, 8, 70)])
def test_q_keeps_its_digits_whatever_its_size(Hq, Hkv, length, size):
    """Scores of about 1 from small q and large K, or the other way round.

    A score is two times 128 products in fp32 sums (a unit each) and one with scale; an element of q is held within
    2^-22 of itself or 2^-39 of its row's largest.  K's own error is none: the reference takes the binary16 values.
    """
    rng = np.random.default_rng(length)
    n, cap = 3, length + 3
    kscale = 1.0 if size >= 1 else 4000.0
    q = (size * (rng.random((n, Hq, 128)) - 0.5)).astype(np.float32)
    q[1, :, 5] = size                                         # small elements beside a large one
    q[1, :, 6:] *= np.float32(2.0 ** -12)
    k = (kscale * (rng.random((Hkv, cap, 128)) - 0.5)).astype(np.float16)
    v = rng.standard_normal((Hkv, cap, 128)).astype(np.float16)
    scale = 1.0 / (size * kscale)
    lds = -(-cap // 4) * 4
    sc, st = torch.zeros(n, Hq, lds, device="cuda"), torch.zeros(n, Hq, 2, device="cuda")
    out = luce.luce_tree_attn(cuda(q), [luce.TreeView(cuda(k), cuda(v), length, n)], Hkv, scale, scores=sc, stats=st)
    out, sc = out.cpu().numpy().astype(np.float64), sc.cpu().numpy().astype(np.float64)
    scale = float(np.float32(scale))
    for j in range(n):
        for h in range(Hq):
            K, V, Q = (x.astype(np.float64) for x in (k[h // (Hq // Hkv), :length + j + 1], v[h // (Hq // Hkv), :length + j + 1], q[j, h]))
            size_of = scale * (np.abs(K) @ np.abs(Q))
            tol = size_of * (260 * U + 2.0 ** -22) + 2.0 ** -39 * scale * np.abs(Q).max() * np.abs(K).sum(1)
            s = scale * (K @ Q)
            assert (np.abs(sc[j, h, :length + j + 1] - s) <= tol).all()
            p = np.exp(s - s.max())
            want = p @ V / p.sum()
            rel = 2 * tol.max() + sums(length) + 2.0 ** -22
            assert (np.abs(out[j, h] - want) <= rel * (p @ np.abs(V)) / p.sum() * 2).all()
