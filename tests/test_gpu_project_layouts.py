"""The pass that norms, rotates and appends, into caches that lie between one another: the values and bits that
caches of their own get, and nothing else written."""
import numpy as np
import pytest

from test_gpu_q8kv import D, cuda, lib  # noqa: F401

torch = pytest.importorskip("torch")
import invariant_sequence_decode_gb300 as luce  # noqa: E402

pytestmark = pytest.mark.gpu
Hq, Hkv, CAP, ROWS = 8, 2, 20, [3, 1, 5, 200]


def caches(layout, cap):
    """(K, V) of each slot in one tensor, and that tensor."""
    if layout == "pool":                                  # slices along the tokens
        t = torch.full((2, Hkv, len(ROWS) * cap, D), -7.0, dtype=torch.float16, device="cuda")
        return [(t[0, :, s * cap:(s + 1) * cap], t[1, :, s * cap:(s + 1) * cap]) for s in range(len(ROWS))], t
    if layout == "token":                                 # K and V of a token side by side
        t = torch.full((len(ROWS), Hkv, cap, 2, D), -7.0, dtype=torch.float16, device="cuda")
        return [(x[:, :, 0], x[:, :, 1]) for x in t], t
    t = torch.full((len(ROWS), Hkv, 2, cap, D), -7.0, dtype=torch.float16, device="cuda")  # of a head
    return [(x[:, 0], x[:, 1]) for x in t], t


@pytest.mark.parametrize("layout", ["pool", "token", "head"])
def test_caches_between_one_another(layout):
    rng = np.random.default_rng(1)
    cap, T = max(ROWS) + 4, sum(ROWS)
    x = cuda(rng.standard_normal((T, (Hq + 2 * Hkv) * D)).astype(np.float32))
    pos = cuda(rng.integers(0, 1 << 15, T).astype(np.int32))
    g = cuda(rng.standard_normal(D).astype(np.float32))
    pairs, whole = caches(layout, cap)
    own = [tuple(torch.full((Hkv, cap, D), -7.0, dtype=torch.float16, device="cuda") for _ in range(2)) for _ in ROWS]
    row0 = np.cumsum([0] + ROWS)
    q = [luce.luce_qk_norm_rope(x, [luce.SeqView(*p, 2 + r, r, int(r0)) for p, r, r0 in zip(to, ROWS, row0)], Hq, pos, 1e6, g, g)
         for to in (pairs, own)]
    assert torch.equal(q[0], q[1])
    for a, b in zip(pairs, own):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    # (each cache equals one of its own, which is -7 outside of the rows; together they are all of the tensor)
    assert sum(t.numel() for p in pairs for t in p) == whole.numel()


def test_one_cache_in_two_views():
    rng = np.random.default_rng(2)
    x = cuda(rng.standard_normal((9, (Hq + 2 * Hkv) * D)).astype(np.float32))
    pos = cuda(np.arange(9, dtype=np.int32))
    a, b = ([torch.zeros(Hkv, CAP, D, dtype=torch.float16, device="cuda") for _ in range(2)] for _ in range(2))
    q = luce.luce_qk_norm_rope(x, [luce.SeqView(*a, 9, 5, 4), luce.SeqView(*a, 4, 4, 0)], Hq, pos, 1e6)
    want = luce.luce_qk_norm_rope(x, [luce.SeqView(*b, 9, 9, 0)], Hq, pos, 1e6)
    assert torch.equal(q, want) and all(torch.equal(s, t) for s, t in zip(a, b))
