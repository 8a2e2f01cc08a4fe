"""Plain 64-bit forms (numpy) of the operators over a slot's cache, and the
tolerances that their 32-bit forms are held to."""
import numpy as np

D = 128


def ancestors(parent, j):
    path = []
    while j >= 0:
        path.insert(0, j)
        j = parent[j]
    return path


def chain(n):
    return list(range(-1, n - 1))


def tree_attention(q, k, v, length, parent, scale):
    """q [n][Hq][D]; k, v [Hkv][cap][D] -> (out [n][Hq][D], scores [n][Hq][length + n], stats [n][Hq][2]) in float64."""
    q, n, Hq, Hkv = q.astype(np.float64), len(parent), q.shape[1], k.shape[0]
    G = Hq // Hkv
    out, scores = np.zeros(q.shape), np.full((n, Hq, length + n), -np.inf)
    stats = np.zeros((n, Hq, 2))
    for j in range(n):
        keys = np.array(list(range(length)) + [length + a for a in ancestors(parent, j)])
        for h in range(Hq):
            K, V = k[h // G, keys].astype(np.float64), v[h // G, keys].astype(np.float64)
            s = scale * (K @ q[j, h])
            m = s.max()
            p = np.exp(s - m)
            out[j, h] = p @ V / p.sum()
            scores[j, h, keys] = s
            stats[j, h] = m, p.sum()
    return out, scores, stats


def tree_tolerance(q, k, v, length, n, scale, chunks):
    """(score, out, l) absolute error bounds of the 32-bit form.  One unit of an
    fp32 sum is taken as 2^-23, a truncating add's.  A score is a sum of 2 x 128
    products (q in two f16 parts, together within 2^-22 of q) and one product
    with scale; e^x of a score off by d is off by a factor of 1 + d, once in the
    weight and once in their sum, plus 4 units of exp and its argument's (times
    |x| <= 88: weights below e^-88 are nothing); a chunk's sums run over 128
    keys of a tile and at most 1,024 tiles, the merge's over the chunks and the
    path."""
    u = 2.0 ** -23
    a = np.abs(q.astype(np.float64)).max(axis=(0, 1))
    b = np.abs(np.nan_to_num(k[:, :length + n].astype(np.float64))).max(axis=(0, 1))
    ds = u * (256 + 4) * abs(scale) * float((a * b).sum())
    rel = 2 * ds + u * (4 + 88 + min(length, 128) + -(-length // 128) + 2 * chunks + 2 * n + 8)
    vmax = float(np.abs(np.nan_to_num(v[:, :length + n].astype(np.float64))).max())
    return ds, 2 * rel * vmax, rel * (length + n)


def commit(k, v, length, path, acc=None, pos=None, pos0=0, scores=None, stats=None):
    """k, v [L][Hkv][cap][D] -> new (k, v, acc float64, pos); scores, stats: the slot's own rows [L][n][Hq][..]."""
    k, v = k.copy(), v.copy()
    old_k, old_v = k.copy(), v.copy()
    for i, a in enumerate(path):
        k[:, :, length + i], v[:, :, length + i] = old_k[:, :, length + a], old_v[:, :, length + a]
    if acc is not None:
        acc = acc.astype(np.float64)
        L, Hkv = acc.shape[:2]
        cols = max([length] + [length + a + 1 for a in path])
        w = np.zeros((L, Hkv, cols))
        for a in path:
            s, st = scores[:, a, :, :cols].astype(np.float64), stats[:, a].astype(np.float64)
            with np.errstate(divide="ignore", invalid="ignore"):
                p = np.exp(s - st[..., :1]) / st[..., 1:]
            p = np.where(st[..., 1:] == 0, 0.0, p)
            w += p.reshape(L, Hkv, -1, cols).sum(2)
        acc[:, :, :length] += w[:, :, :length]
        for i, a in enumerate(path):
            acc[:, :, length + i] = w[:, :, length + a]
    if pos is not None:
        pos = pos.copy()
        for i in range(len(path)):
            pos[:, :, length + i] = pos0 + i
    return k, v, acc, pos


def evict(k, v, acc, pos, length, budget, sinks, recent, next_pos):
    """-> new (k, v, acc, pos); rows at or past the budget are the old ones."""
    k, v, acc, pos = k.copy(), v.copy(), acc.copy(), pos.copy()
    n = length - budget
    if n <= 0:
        return k, v, acc, pos
    for layer in range(k.shape[0]):
        for g in range(k.shape[1]):
            a, p = acc[layer, g, :length], pos[layer, g, :length]
            held = (p < sinks) | (p >= next_pos - recent)
            key = [(bool(held[j]), 0 if held[j] else (-np.inf if np.isnan(a[j]) else float(a[j])), 0 if held[j] or not np.isnan(a[j]) else -1, -j)
                   for j in range(length)]
            # a NaN is below every weight, -inf too
            key = [(h, (0, 0.0) if nan == -1 else (1, x), j) for h, x, nan, j in key]
            leave = set(sorted(range(length), key=lambda j: key[j])[:n])
            holes = [j for j in range(budget) if j in leave]
            come = [j for j in range(budget, length) if j not in leave]
            assert len(holes) == len(come)
            for to, frm in zip(holes, come):
                for x in (k, v, acc, pos):
                    x[layer, g, to] = x[layer, g, frm]
    return k, v, acc, pos
