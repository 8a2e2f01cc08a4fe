"""Paged slots whose tables change between the steps of a decode loop."""
import numpy as np
import pytest

from invariant_sequence_decode_gb300 import workloads as wl

torch = pytest.importorskip("torch")
import invariant_sequence_decode_gb300 as luce  # noqa: E402
from test_gpu_tree_step import LAYERS, VOCAB, bits, cuda, lib, model, step  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def plain(model, slots, x):
    logits, am = torch.empty(1, VOCAB, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    luce.luce_decode_step_paged(model, slots, [1], x, model.workspace(1, 600), logits, am)
    torch.cuda.synchronize()
    return x, logits, am


@pytest.mark.parametrize("kind", ["tree", "plain"])
def test_a_step_follows_a_grown_and_a_remapped_table(model, kind):  # noqa: F811
    d = wl.TINY_LAYER
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn(9, LAYERS, d.n_kv_heads, 128, 128, generator=g, device="cuda").half() for _ in range(2))
    make = luce.PagedTreeSlot if kind == "tree" else luce.PagedSlot
    run = step if kind == "tree" else plain
    slot = make(k.clone(), v.clone(), np.array([2]), 100)

    def agrees():
        """The step's bits are those of a slot made anew."""
        x = cuda(wl.acts(3, 1, d.hidden, sub=8))
        fresh = make(slot.k_pool.clone(), slot.v_pool.clone(), np.array(slot.table), slot.len)
        got, want = run(model, [slot], x.clone()), run(model, [fresh], x.clone())
        assert all(np.array_equal(bits(a), bits(b)) for a, b in zip(got, want))
        assert torch.equal(slot.k_pool.view(torch.int16), fresh.k_pool.view(torch.int16))

    agrees()
    slot.table, slot.len = np.array([2, 7, 0, 5]), 300       # the cache grew by pages
    agrees()
    slot.table[1] = 4                                        # a page moved
    agrees()
    slot.table, slot.len = [8, 3], 130                       # the slot serves another sequence
    agrees()


def test_a_captured_step_keeps_its_table(model):  # noqa: F811
    d = wl.TINY_LAYER
    k, v = (torch.randn(6, LAYERS, d.n_kv_heads, 128, 128, device="cuda").half() for _ in range(2))
    slot = luce.PagedTreeSlot(k, v, np.array([1, 4]), 200)
    xh = cuda(wl.acts(3, 1, d.hidden, sub=9))
    x, ws = xh.clone(), model.tree_workspace(1, 300)
    luce.luce_decode_step_tree(model, [slot], x, ws)
    torch.cuda.synchronize()
    want, graph = bits(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        luce.luce_decode_step_tree(model, [slot], x, ws)
    slot.table = np.array([5, 0, 2])
    luce.luce_decode_step_tree(model, [slot], xh.clone(), ws)          # a new device copy; the graph's one stays
    junk = [torch.full((2,), -1, dtype=torch.int32, device="cuda") for _ in range(64)]
    x.copy_(xh)
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(bits(x), want) and junk
    slot.table = np.array([0, 1])
    with pytest.raises(RuntimeError, match="before the capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            luce.luce_decode_step_tree(model, [slot], x, ws)
    torch.cuda.synchronize()
    luce.luce_decode_step_tree(model, [slot], x, ws)
    torch.cuda.synchronize()


def test_a_capture_on_a_stream_that_is_not_the_current_one(model):  # noqa: F811
    d = wl.TINY_LAYER
    k, v = (torch.randn(6, LAYERS, d.n_kv_heads, 128, 128, device="cuda").half() for _ in range(2))
    slot = luce.PagedTreeSlot(k, v, np.array([1, 4]), 200)
    xh = cuda(wl.acts(3, 1, d.hidden, sub=9))
    x, ws, side, graph = xh.clone(), model.tree_workspace(1, 300), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    luce.luce_decode_step_tree(model, [slot], x, ws)
    torch.cuda.synchronize()
    want, first = bits(x), slot.table_dev
    with torch.cuda.stream(side):
        graph.capture_begin()
    try:
        luce.luce_decode_step_tree(model, [slot], x, ws, stream=side)
        slot.table = np.array([5, 0, 2])
        with pytest.raises(RuntimeError, match="before the capture"):
            luce.luce_decode_step_tree(model, [slot], x, ws, stream=side)
    finally:
        with torch.cuda.stream(side):
            graph.capture_end()
    luce.luce_decode_step_tree(model, [slot], xh.clone(), ws)
    assert slot.table_dev is not first and any(t is first for t in slot._captured)
    x.copy_(xh)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(bits(x), want)
