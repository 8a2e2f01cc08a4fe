"""Calls over a slot's cache whose arrays overlap are refused before anything is
enqueued; arrays that only touch are not."""
import ctypes

import pytest

import invariant_sequence_decode_gb300 as luce
from invariant_sequence_decode_gb300 import build
from test_cache_refusals import BIG, E, P, attn, model, ptslot, view

S = luce.LUCE_ENOSPACE
Q, OUT, SC, ST, WS = (P + i * BIG for i in range(2, 7))
ROW = 8 * 128 * 4            # a row of q and out


@pytest.fixture(scope="module")
def lib():
    build.build()
    return luce.load_library()


def flat(lib, **kw):
    a = dict(q=Q, out=OUT, scores=SC, lds=12, stats=ST, ws=WS)
    a.update(kw)
    return attn(lib, [view()], **a)


def paged(lib, **kw):
    a = dict(q=Q, out=OUT, scores=SC, lds=12, stats=ST, ws=WS, ws_bytes=1 << 20)
    a.update(kw)
    arr = (luce.PagedTreeViewC * 1)(luce.PagedTreeViewC(P, P + BIG, P + 9 * BIG, 4, 10, 2, 0, None))
    return lib.luce_tree_attn_paged(a["q"], arr, 1, 8, 2, 128, 0.1, a["out"], a["scores"], a["lds"], a["stats"], a["ws"],
                                    a["ws_bytes"], None)


@pytest.mark.parametrize("call", [flat, paged])
@pytest.mark.parametrize("kw", [
    dict(out=P), dict(out=P + BIG + 64), dict(out=Q + 4), dict(out=Q + 2 * ROW - 4), dict(out=Q - 2 * ROW + 4), dict(out=WS + 128),
    dict(scores=Q), dict(scores=OUT + 16), dict(scores=P + 1024), dict(stats=SC + 8), dict(stats=Q + 8), dict(stats=P + BIG),
    dict(ws=Q), dict(ws=OUT), dict(ws=SC), dict(ws=ST), dict(ws=P + 256), dict(ws=P + BIG),
])
def test_tree_attention_refuses_overlaps(lib, call, kw):
    before = luce.launch_count()
    assert call(lib, **kw) == E and b"overlaps" in lib.luce_last_error()
    assert luce.launch_count() == before


def test_tree_attention_refuses_an_output_over_its_table(lib):
    assert paged(lib, out=P + 9 * BIG) == E and b"table" in lib.luce_last_error()


@pytest.mark.parametrize("kw", [
    dict(scores=P), dict(scores=P + BIG + 4096), dict(stats=P + 64), dict(stats=P + BIG), dict(stats=SC + 16),
    dict(scores=P + 2 * 2 * 128 * 128 * 2 * 4 - 16),     # the pool's last bytes
])
def test_paged_tree_step_refuses_scores_and_stats_over_its_pools(lib, kw):
    a = dict(scores=SC, stats=ST)
    a.update(kw)
    arr = (luce.PagedTreeSlotC * 1)(ptslot())
    assert lib.luce_decode_step_tree_paged(ctypes.byref(model()), arr, 1, Q, None, None, None if a["scores"] is None else a["scores"],
                                           12, a["stats"], WS, 1 << 30, None) == E
    assert b"overlaps" in lib.luce_last_error()


def test_arrays_that_touch_are_not_refused(lib):
    """The last check before the launch is the overlap's: these get as far as the next call's status."""
    arr = (luce.PagedTreeSlotC * 1)(ptslot())
    end = P + 2 * 2 * 128 * 128 * 2 * 4
    assert lib.luce_decode_step_tree_paged(ctypes.byref(model()), arr, 1, Q, None, None, end, 12, ST, WS, 1024, None) == S


def test_the_trees_expiry_hook_takes_a_limit(lib):
    for bad in (0, 999, 1_000_000_001, -5):
        assert lib.luce_test_tree_wait_expiry(bad, None) == E and b"limit_ns" in lib.luce_last_error()


@pytest.mark.parametrize("stride", [2 * 128 * 128 - 8, 2 * 128 * 128 + 4, -(1 << 20), 1 << 38, 8])
def test_paged_tree_attention_refuses_pages_that_are_not_apart(lib, stride):
    arr = (luce.PagedTreeViewC * 1)(luce.PagedTreeViewC(P, P + BIG, P + 9 * BIG, 4, 10, 2, 0, None, stride))
    assert lib.luce_tree_attn_paged(Q, arr, 1, 8, 2, 128, 0.1, OUT, None, 0, None, WS, 1 << 20, None) == E
    assert b"page_stride" in lib.luce_last_error()


def test_a_layer_reaches_to_its_own_end_of_the_pool(lib):
    """Layer 1 of 2: what lies behind the last page's layer 1 is not the view's."""
    page = 2 * 128 * 128
    end = P + 2 * (7 * page + page)                      # 4 pages x 2 layers
    arr = (luce.PagedTreeViewC * 1)(luce.PagedTreeViewC(P + 2 * page, P + BIG, P + 9 * BIG, 4, 10, 2, 0, None, 2 * page))
    call = lambda out: lib.luce_tree_attn_paged(Q, arr, 1, 8, 2, 128, 0.1, out, SC, 12, SC, WS, 1 << 20, None)  # noqa: E731
    assert call(end - 16) == E and b"overlaps the K" in lib.luce_last_error()
    assert call(end) == E and b"stats overlaps the scores" in lib.luce_last_error()
