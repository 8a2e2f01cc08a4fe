"""Caches in 8 bits, called as a server would: several heads one after the other in a CTA, two streams
at once, captured and replayed, slots that share their prefix."""
import numpy as np
import pytest

import q8kv_reference as ref
from cache_reference import chain
from test_gpu_q8kv import SCALE, Cache, bits, check, check_sealed, cuda, lib, run, seal_slot  # noqa: F401
from test_gpu_tree import tree_of

torch = pytest.importorskip("torch")
import invariant_sequence_decode_gb300 as luce  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G,n", [(1, 1), (4, 4), (5, 4), (5, 8), (8, 8), (5, 16), (6, 16), (8, 16)])
def test_a_cta_takes_several_heads(G, n):
    """More KV heads than CTAs run at once, at every width of the products."""
    rng = np.random.default_rng(100 * G + n)
    Hkv = 640
    s = Cache(rng, G * Hkv, Hkv, 160, 3, tree_of("random", n, G), window=170 if n == 4 else 0, sinks=5)
    check([s], run([s], [s.flat()], Hkv))


def calls(rng, shapes):
    """Prepared attention of several slots each, with the wanted bits."""
    out = []
    for Hq, Hkv, sealed, n in shapes:
        s = Cache(rng, Hq, Hkv, sealed, 7, tree_of("random", n, n))
        out.append((luce.Q8Attention(cuda(s.q), [s.flat()], Hkv, SCALE), bits(run([s], [s.flat()], Hkv))))
    return out


def test_two_streams_at_once():
    pairs = calls(np.random.default_rng(21), [(40, 8, 8192, 4), (40, 8, 4096, 16), (8, 2, 2048, 1)])
    streams = [torch.cuda.Stream() for _ in pairs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (call, _), stream in zip(pairs, streams):
            with torch.cuda.stream(stream):
                call.out.fill_(float("nan"))
                call()
    torch.cuda.synchronize()
    assert luce.wait_timeouts() == 0
    for call, want in pairs:
        assert np.array_equal(bits(call.out), want)


def test_two_captured_graphs_at_once():
    """Each prepared call has a workspace of its own, so their graphs may overlap."""
    pairs = calls(np.random.default_rng(22), [(40, 8, 8192, 16), (40, 8, 8192, 4)])
    graphs = []
    for call, _ in pairs:
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call.out.zero_()
            call()
        graphs.append((g, torch.cuda.Stream()))
    for _ in range(20):
        for g, stream in graphs:
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    assert luce.wait_timeouts() == 0
    for call, want in pairs:
        assert np.array_equal(bits(call.out), want)


def test_captured_seal_and_projection_are_replayed():
    rng = np.random.default_rng(23)
    k, v, order, slot = seal_slot(rng, 2, 4, 75, 96, 80, True)
    x, pos = cuda(rng.standard_normal((3, 12 * 128)).astype(np.float32)), cuda(np.array([5, 6, 9], np.int32))
    cache = [torch.zeros(2, 16, 128, dtype=torch.float16, device="cuda") for _ in range(2)]
    project = luce.QkNormRope(x, [luce.SeqView(*cache, 8, 3, 0)], 8, pos, 1e4, cuda(np.ones(128, np.float32)), None)
    seal = luce.Q8Seal([slot])
    want = project().clone(), [c.clone() for c in cache]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        project()
        seal()
    k0, v0 = cuda(k), cuda(v)
    for _ in range(3):
        slot.k.copy_(k0)
        slot.v.copy_(v0)
        for p, fill in zip((slot.k_codes, slot.v_codes, slot.scales), (11, 12, 13)):
            p.fill_(fill)
        project.out.zero_()
        for c in cache:
            c.zero_()
        g.replay()
        torch.cuda.synchronize()
        check_sealed(k, v, order, slot)
        assert torch.equal(project.out, want[0]) and all(torch.equal(c, w) for c, w in zip(cache, want[1]))


def test_slots_share_the_pages_of_their_prefix():
    rng = np.random.default_rng(24)
    s = Cache(rng, 40, 8, 2048, 9, chain(4))
    one = s.paged(rng)
    views = [luce.Q8View(one.k_codes, one.v_codes, one.scales, 2048, one.k, one.v, 9, s.parent, r, table=one.table) for r in (0, 4, 8, 12)]
    out = run([s] * 4, views, 8)
    want = bits(run([s], [one], 8))
    for r in (0, 4, 8, 12):
        assert np.array_equal(bits(out[r:r + 4]), want)


def test_sealing_then_attending_needs_no_wait_between():
    """The two on one stream, many times: codes and scales that the sealing kernel writes are read by the next."""
    rng = np.random.default_rng(25)
    Hkv, n = 8, 64
    k, v, order, slot = seal_slot(rng, 1, Hkv, n, 0, n + 1, False)
    q = cuda(rng.standard_normal((1, 40, 128)).astype(np.float32))
    slot.k[:, :, n:] = 1
    seal = luce.Q8Seal([slot])
    row = torch.ones(Hkv, 1, 128, dtype=torch.float16, device="cuda")
    attend = luce.Q8Attention(q, [luce.Q8View(slot.k_codes[:, 0], slot.v_codes[:, 0], slot.scales[:, 0], n, row, row, 0, 1)], Hkv, SCALE)
    k0, v0 = cuda(k), cuda(v)
    seal()
    first = bits(attend())
    torch.cuda.synchronize()
    outs = []
    for i in range(30):
        slot.k.copy_(k0 * (1 + i % 3))
        slot.v.copy_(v0 * (1 + i % 3))
        seal()
        outs.append(attend().clone())
    torch.cuda.synchronize()
    for i in (0, 3, 27):
        assert np.array_equal(bits(outs[i]), first)
    for i in range(3, 30):
        assert np.array_equal(bits(outs[i]), bits(outs[i % 3]))
    assert not np.array_equal(bits(outs[1]), first)


def test_an_expired_wait_is_counted_and_the_context_stays_usable(lib):  # noqa: F811
    rng = np.random.default_rng(26)
    s = Cache(rng, 40, 8, 1024, 5, chain(3))
    want = bits(run([s], [s.flat()], 8))                       # (no wait expired)
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.luce_test_q8kv_wait_expiry(1_000_000, stream) == lib.luce_test_tree_wait_expiry(1_000_000, stream) == 0
    assert luce.wait_timeouts(reset=True) == 2
    assert np.array_equal(bits(run([s], [s.flat()], 8)), want)
