"""Plain 64-bit forms (numpy) of the operators over a slot's cache in 8 bits, and
the tolerances that their 32-bit forms are held to."""
import numpy as np

from cache_reference import ancestors

D, BLOCK, PAGE = 128, 32, 128
U = 2.0 ** -23   # one unit of an fp32 sum, a truncating add's


def quantise(x):
    """x [.., BLOCK, D] fp16 -> (codes int8, scales fp32 [..]) of its blocks, by the definition: fp32 divisions,
    halves away from zero, infinities and NaN outside the maximum."""
    x = x.astype(np.float32)
    top = np.where(np.isfinite(x), np.abs(x), 0).max((-2, -1)).astype(np.float32)
    d = (top / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = (x / d[..., None, None]).astype(np.float32)
    q = np.where(np.isnan(q) | (d[..., None, None] == 0), 0, q).astype(np.float64)
    return np.clip(np.copysign(np.floor(np.abs(q) + 0.5), q), -127, 127).astype(np.int8), d


def attention(q, k, v, total, parent, scale, window=0, sinks=0):
    """q [n][Hq][D]; k, v [Hkv][total + n][D] in float64 (the prefix, then the nodes) -> out [n][Hq][D]."""
    q, n, Hq, G = q.astype(np.float64), len(parent), q.shape[1], q.shape[1] // k.shape[0]
    out = np.zeros(q.shape)
    for j in range(n):
        path = ancestors(parent, j)
        pos = total + len(path) - 1
        keys = [(i, i) for i in range(total)] + [(total + e, total + a) for e, a in enumerate(path)]
        keys = [row for i, row in keys if window == 0 or i < sinks or pos - i < window]
        for h in range(Hq):
            s = scale * (k[h // G, keys] @ q[j, h])
            p = np.exp(s - s.max())
            out[j, h] = p @ v[h // G, keys] / p.sum()
    return out


def attention_tolerance(q, k, v, total, n, scale, chunks):
    """An absolute error bound of the 32-bit form.  A score is a sum of 2 x 128 products (q in two parts, within 2^-22
    of q together), a product with the scale and one with the block's; e^x off by d is off by a factor of 1 + d, once
    in the weight and once in their sum; the argument of a weight is formed from three numbers (score, maximum,
    logarithm of V's scale), each below 128 in all weights that count: 3 x 128 / 2 units, exp2 and log2 of 4 each; a tile's
    sums run over 128 keys, the chunks' over their tiles, the merge's over the chunks, the tail and the path."""
    a = np.abs(q.astype(np.float64)).max(axis=(0, 1))
    b = np.abs(k).max(axis=(0, 1))
    ds = U * (256 + 6) * abs(scale) * float((a * b).sum())
    rel = 2 * ds + 2 * U * (192 + 8 + min(total, 128) + -(-total // 128) + 2 * chunks + 128 + 8)
    return rel * float(np.abs(v).max())


def project(x, Hq, Hkv, q_gamma, k_gamma, eps, pos, pair_axis, theta):
    """x [T][(Hq + 2 Hkv) D], pos [axes][T] -> (q, k, v) [T][heads][D] in float64."""
    T = x.shape[0]
    x = x.astype(np.float64).reshape(T, -1, D)
    i = np.arange(D // 2)
    angle = pos.astype(np.float64)[np.asarray(pair_axis)].T * theta ** (-2.0 * i / D)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]

    def turned(h, gamma):
        if gamma is not None:
            h = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * gamma.astype(np.float64)
        a, b = h[..., :D // 2], h[..., D // 2:]
        return np.concatenate([a * c - b * s, a * s + b * c], -1)

    return turned(x[:, :Hq], q_gamma), turned(x[:, Hq:Hq + Hkv], k_gamma), x[:, Hq + Hkv:]
