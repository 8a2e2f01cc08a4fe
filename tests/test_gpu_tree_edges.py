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


@pytest.mark.parametrize("paged", [False, True])
def test_a_prepared_call_follows_the_trees_of_a_loop(paged):
    rng = np.random.default_rng(21)
    views = []
    for L in (300, 40, 9000):                               # each cache holds six rows behind its prefix
        s = Slot(rng, 8, 2, L, tree_of("random", 6, L), slack=0)
        views.append(s.paged(0, rng) if paged else s.flat(0))
    *views, longer = views
    views[1].parent, views[1].row0 = 2, 6
    q = torch.randn(8, 8, 128, device="cuda")
    call, fn = luce.TreeAttention(q, views, 2, 0.09), luce.luce_tree_attn_paged if paged else luce.luce_tree_attn
    for step, sizes in enumerate(([6, 2], [4, 4], [4, 4], [2, 6], [5, 3], [5, 3])):
        if step == 4:                                       # the first slot goes on with a longer cache
            for name in vars(longer):
                setattr(views[0], name, getattr(longer, name))
        for i, (v, n) in enumerate(zip(views, sizes)):
            v.parent, v.row0 = tree_of("random", n, 10 * step + i), sum(sizes[:i])
        got = call().clone()
        assert np.array_equal(bits(got), bits(fn(q, views, 2, 0.09)))


def test_an_expired_wait_is_counted_and_leaves_the_context_usable():
    lib = luce.load_library()
    stream = torch.cuda.current_stream().cuda_stream
    luce.wait_timeouts(reset=True)
    assert lib.luce_test_tree_wait_expiry(5_000_000, stream) == 0
    torch.cuda.synchronize()
    assert luce.wait_timeouts() == 1                        # (read, not reset)
    assert lib.luce_test_tree_wait_expiry(1_000_000, stream) == lib.luce_test_wait_expiry(1_000_000, stream) == 0
    torch.cuda.synchronize()
    assert luce.wait_timeouts(reset=True) == 3              # the rings' and the trees' together
    assert luce.wait_timeouts() == 0
    s = Slot(np.random.default_rng(2), 8, 2, 700, tree_of("random", 5, 2))
    check([s], *run([s], [s.flat(0)], 2, scores=True), 2)


@pytest.mark.parametrize("Hkv,lens", [(2, [300, 40]), (1, [129, 1000]), (8, [700])])
def test_a_layer_of_a_pool_of_several(Hkv, lens):
    """The pools that the step, the commit and eviction take: the same bits as a pool of the layer alone."""
    rng = np.random.default_rng(sum(lens))
    slots = [Slot(rng, 4 * Hkv, Hkv, L, tree_of("random", 3, L)) for L in lens]
    views = [s.paged(3 * i, rng) for i, s in enumerate(slots)]
    want = run(slots, views, Hkv, scores=True)
    for layers, layer in ((3, 0), (3, 2), (2, 1)):
        wide = []
        for v in views:
            pools = []
            for x in (v.k_pool, v.v_pool):
                pool = torch.full((x.shape[0], layers, *x.shape[1:]), float("nan"), dtype=torch.float16, device="cuda")
                pool[:, layer] = x
                pools.append(pool[:, layer])
            wide.append(luce.PagedTreeView(*pools, v.table, v.len, v.parent, v.row0))
        got = run(slots, wide, Hkv, scores=True)
        assert all(np.array_equal(bits(a), bits(b)) for a, b in zip(got, want))
    v = views[0]
    with pytest.raises(ValueError):                             # pages whose heads lie apart
        k = torch.zeros(4, 2 * Hkv, 128, 128, dtype=torch.float16, device="cuda")[:, ::2]
        k = k if Hkv > 1 else torch.zeros(4, 1, 256, 128, dtype=torch.float16, device="cuda")[:, :, ::2]
        luce.luce_tree_attn_paged(torch.zeros(3, 4 * Hkv, 128, device="cuda"), [luce.PagedTreeView(k, k, v.table, 100, 3)], Hkv, 0.1)
