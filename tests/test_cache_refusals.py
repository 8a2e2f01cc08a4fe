"""The entry points over a slot's cache refuse invalid calls with a status
before anything is enqueued (no device needed: validation precedes launches)."""
import ctypes

import pytest

import invariant_sequence_decode_gb300 as luce
from invariant_sequence_decode_gb300 import build

P = 0x10000
BIG = 0x100000000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return luce.load_library()


def ints(values):
    return (ctypes.c_int32 * max(1, len(values)))(*values)


def view(length=10, nodes=2, row0=0, cap=4096, head=4096 * 128, tok=128, parent=None, k=P, v=P + BIG):
    return luce.TreeViewC(k, v, length, nodes, row0, cap, head, tok, None if parent is None else ints(parent))


def attn(lib, views, q=P, Hq=8, Hkv=2, D=128, scale=0.1, out=P, scores=None, lds=0, stats=None, ws=P, ws_bytes=1 << 40, n=None):
    arr = (luce.TreeViewC * max(1, len(views)))(*views)
    return lib.luce_tree_attn(q, arr, len(views) if n is None else n, Hq, Hkv, D, scale, out, scores, lds, stats, ws,
                              ws_bytes, None)


E, U, S = luce.LUCE_EINVAL, luce.LUCE_EUNSUPPORTED, luce.LUCE_ENOSPACE


@pytest.mark.parametrize("want,kw", [
    (E, dict(q=0)), (E, dict(q=P + 8)), (E, dict(out=0)), (E, dict(ws=0)), (E, dict(ws=P + 16)),
    (E, dict(Hq=9)), (E, dict(Hkv=0)), (E, dict(Hq=0)), (U, dict(Hq=18)), (U, dict(D=64)),
    (E, dict(scale=float("nan"))), (E, dict(scale=float("inf"))),
    (E, dict(scores=P, lds=0)), (E, dict(scores=P, lds=14)), (E, dict(scores=P + 4, lds=16)), (E, dict(scores=P, lds=8)),
    (E, dict(stats=P + 4)), (S, dict(ws_bytes=16)),
])
def test_tree_attention_refuses_arguments(lib, want, kw):
    assert attn(lib, [view()], **kw) == want and lib.luce_last_error()


@pytest.mark.parametrize("want,views", [
    (E, []), (E, [view(row0=2 * i) for i in range(5)]),
    (E, [view(nodes=0)]), (E, [view(nodes=17)]), (E, [view(nodes=-1)]),
    (E, [view(length=-1)]), (E, [view(length=4095)]), (U, [view(length=130815, cap=1 << 20, head=1 << 27)]),
    (E, [view(row0=1)]), (E, [view(row0=-1)]), (E, [view(nodes=4, row0=13)]),
    (E, [view(), view()]), (E, [view(nodes=8), view(nodes=9, row0=8)]),
    (E, [view(parent=[0, 0])]), (E, [view(parent=[-1, 1])]), (E, [view(parent=[-2, 0])]), (E, [view(parent=[-1, 5])]),
    (E, [view(k=0)]), (E, [view(v=0)]), (E, [view(k=P + 8)]),
    (E, [view(tok=120)]), (E, [view(tok=132)]), (E, [view(head=4096 * 128 - 8)]), (E, [view(head=4096 * 128 + 4)]),
    (E, [view(tok=1 << 33, head=1 << 37)]), (E, [view(tok=1 << 31, cap=1 << 10, head=1 << 41)]),
])
def test_tree_attention_refuses_views(lib, want, views):
    assert attn(lib, views) == want and lib.luce_last_error()


def test_tree_attention_refuses_a_span_beyond_the_maps(lib):
    assert attn(lib, [view(tok=1 << 30, cap=1 << 9)], Hkv=1) == E and b"2^38" in lib.luce_last_error()


def test_tree_attention_null_views(lib):
    assert lib.luce_tree_attn(P, None, 1, 8, 2, 128, 0.1, P, None, 0, None, P, 1 << 30, None) == E


@pytest.mark.parametrize("want,kw", [
    (E, dict(k=0)), (E, dict(v=P + 2)), (E, dict(table=0)), (E, dict(table=P + 2)), (E, dict(pages=0)), (E, dict(length=-1)),
    (U, dict(length=130815)), (E, dict(nodes=0)), (E, dict(nodes=17)), (E, dict(row0=1)), (E, dict(parent=[1, 0])),
])
def test_paged_tree_attention_refusals(lib, want, kw):
    a = dict(k=P, v=P, table=P, pages=4, length=10, nodes=2, row0=0, parent=None)
    a.update(kw)
    v = luce.PagedTreeViewC(a["k"], a["v"], a["table"], a["pages"], a["length"], a["nodes"], a["row0"],
                            None if a["parent"] is None else ints(a["parent"]))
    arr = (luce.PagedTreeViewC * 1)(v)
    assert lib.luce_tree_attn_paged(P, arr, 1, 8, 2, 128, 0.1, P, None, 0, None, P, 1 << 40, None) == want


def test_tree_workspace_sizes(lib):
    size = lib.luce_tree_attn_workspace_size
    assert size(0, 8, 2, 128, 10) == size(17, 8, 2, 128, 10) == size(1, 8, 2, 64, 10) == size(1, 8, 2, 128, 200000) == 0
    assert size(1, 0, 1, 128, 10) == size(1, 8, 0, 128, 10) == size(1, 8, 3, 128, 10) == size(1, 18, 2, 128, 10) == 0
    assert size(1, 8, 2, 128, -1) == 0 and size(1, 8, 2, 128, 0) >= 256
    for hkv in (1, 2, 3, 8, 40, 200, 700):
        last = 0
        for n in (1, 128, 129, 1000, 8192, 8193, 32768, 32769, 100000, 130816):
            assert size(4, 4 * hkv, hkv, 128, n) >= last  # a workspace for longer prefixes serves shorter ones
            last = size(4, 4 * hkv, hkv, 128, n)


def slot(k=P, v=P + BIG, length=10, cap=64, path=(0, 2), row0=0, acc=None, pos=None, pos0=10, n=None):
    return luce.CommitSlotC(k, v, length, cap, len(path) if n is None else n, row0, ints(path), acc, pos, pos0)


def commit(lib, slots, L=2, Hq=8, Hkv=2, D=128, scores=None, rows=0, lds=0, stats=None, n=None):
    arr = (luce.CommitSlotC * max(1, len(slots)))(*slots)
    return lib.luce_tree_commit(arr, len(slots) if n is None else n, L, Hq, Hkv, D, scores, rows, lds, stats, None)


ACC, POS, SC, ST = P + 2 * BIG, P + 3 * BIG, P + 4 * BIG, P + 5 * BIG


@pytest.mark.parametrize("want,slots,kw", [
    (E, [], {}), (E, [slot()] * 5, {}), (E, [slot()], dict(L=0)), (E, [slot()], dict(Hkv=0)), (U, [slot()], dict(D=64)),
    (E, [slot()], dict(Hq=9)), (U, [slot()], dict(Hq=32)), (E, [slot()], dict(L=1 << 20)),
    (E, [slot(k=0)], {}), (E, [slot(v=P + BIG + 8)], {}), (E, [slot(length=-1)], {}), (E, [slot(length=65)], {}),
    (E, [slot(n=17)], {}), (E, [slot(n=-1)], {}), (E, [slot(path=(2, 0))], {}), (E, [slot(path=(1, 1))], {}),
    (E, [slot(path=(0, 16))], {}), (E, [slot(path=(-1,))], {}), (E, [slot(length=60, path=(0, 4))], {}),
    (E, [slot(pos0=-1)], {}), (E, [slot(v=P)], {}), (E, [slot(), slot()], {}),
    (E, [slot(acc=ACC)], {}), (E, [slot(acc=ACC)], dict(scores=SC, rows=4, lds=16)),
    (E, [slot(acc=ACC)], dict(scores=SC, rows=2, lds=16, stats=ST)),     # row 2 outside two rows
    (E, [slot(acc=ACC)], dict(scores=SC, rows=17, lds=16, stats=ST)),
    (E, [slot(acc=ACC)], dict(scores=SC, rows=4, lds=12, stats=ST)),     # column 12 outside
    (E, [slot(acc=ACC)], dict(scores=SC, rows=4, lds=15, stats=ST)),
    (E, [slot(acc=ACC)], dict(scores=SC + 4, rows=4, lds=16, stats=ST)),
    (E, [slot(acc=ACC, row0=-1)], dict(scores=SC, rows=4, lds=16, stats=ST)),
    (E, [slot(acc=ACC, pos=ACC)], dict(scores=SC, rows=4, lds=16, stats=ST)),
    (E, [slot(acc=SC)], dict(scores=SC, rows=4, lds=16, stats=ST)),
    (E, [slot(acc=ACC + 2)], dict(scores=SC, rows=4, lds=16, stats=ST)), (E, [slot(acc=ACC)], dict(scores=SC, rows=4, lds=16, stats=ST + 4)),
    (U, [slot(length=130815, cap=130900)], {}), (U, [slot(length=2 ** 30, cap=2 ** 31 - 1)], {}),
])
def test_commit_refusals(lib, want, slots, kw):
    assert commit(lib, slots, **kw) == want and lib.luce_last_error()


def test_commit_of_nothing_enqueues_nothing(lib):
    before = luce.launch_count()
    assert commit(lib, [slot(path=()), slot(k=P + 6 * BIG, v=P + 7 * BIG, path=())]) == luce.LUCE_OK
    assert luce.launch_count() == before


def eslot(k=P, v=P + BIG, acc=ACC, pos=POS, acc_out=ACC, pos_out=POS, length=20, cap=64, budget=10, sinks=1, recent=4, nxt=20):
    return luce.EvictSlotC(k, v, acc, pos, acc_out, pos_out, length, cap, budget, sinks, recent, nxt)


def evict(lib, slots, L=2, Hkv=2, D=128):
    arr = (luce.EvictSlotC * max(1, len(slots)))(*slots)
    return lib.luce_kv_evict(arr, len(slots), L, Hkv, D, None)


@pytest.mark.parametrize("want,slots,kw", [
    (E, [], {}), (E, [eslot()] * 5, {}), (E, [eslot()], dict(L=0)), (U, [eslot()], dict(D=64)),
    (E, [eslot(k=0)], {}), (E, [eslot(k=P + 8)], {}), (E, [eslot(acc=0)], {}), (E, [eslot(pos_out=0)], {}),
    (E, [eslot(acc=ACC + 1)], {}), (E, [eslot(length=65)], {}), (E, [eslot(length=-1)], {}),
    (U, [eslot(length=130817, cap=130900)], {}), (E, [eslot(budget=0)], {}), (E, [eslot(sinks=-1)], {}),
    (E, [eslot(recent=-1)], {}), (E, [eslot(sinks=6, recent=5)], {}), (E, [eslot(sinks=2**31 - 1, recent=2**31 - 1)], {}),
    (E, [eslot(nxt=-1)], {}), (E, [eslot(), eslot()], {}), (E, [eslot(v=P)], {}),
    (E, [eslot(acc_out=ACC + 4)], {}), (E, [eslot(acc_out=POS)], {}), (E, [eslot(pos_out=POS + 64)], {}),
])
def test_evict_refusals(lib, want, slots, kw):
    assert evict(lib, slots, **kw) == want and lib.luce_last_error()


def test_evict_within_budget_in_place_enqueues_nothing(lib):
    before = luce.launch_count()
    assert evict(lib, [eslot(budget=20), eslot(P + 6 * BIG, P + 7 * BIG, P + 8 * BIG, P + 9 * BIG, P + 8 * BIG, P + 9 * BIG,
                                               length=0)]) == luce.LUCE_OK
    assert luce.launch_count() == before


def model(n_layers=2, vocab=0, hq=4, hkv=2):
    layers = (luce.LayerC * n_layers)(*[luce.LayerC(*([P] * 10)) for _ in range(n_layers)])
    m = luce.ModelC(n_layers, 256, hq, hkv, 128, 512, vocab, 1e-6, 1e6, layers, P, P, P)
    return m


def tslot(k=P, v=P + BIG, length=10, cap=64, pos0=10, nodes=2, parent=None):
    return luce.TreeSlotC(k, v, length, cap, pos0, nodes, None if parent is None else ints(parent))


def step(lib, slots, m=None, x=P, logits=None, argmax=None, scores=None, lds=0, stats=None, ws=0x100000, ws_bytes=1 << 40, n=None):
    arr = (luce.TreeSlotC * max(1, len(slots)))(*slots)
    return lib.luce_decode_step_tree(ctypes.byref(m or model()), arr, len(slots) if n is None else n, x, logits, argmax,
                                     scores, lds, stats, ws, ws_bytes, None)


@pytest.mark.parametrize("want,slots,kw", [
    (E, [], {}), (E, [tslot()] * 5, {}), (E, [tslot(k=0)], {}), (E, [tslot(v=P + BIG + 8)], {}), (E, [tslot(nodes=0)], {}),
    (E, [tslot(nodes=17)], {}), (E, [tslot(nodes=9), tslot(P + 2 * BIG, P + 3 * BIG, nodes=8)], {}), (E, [tslot(length=63)], {}),
    (E, [tslot(length=-1)], {}), (U, [tslot(length=130815, cap=1 << 20)], {}), (E, [tslot(pos0=-1)], {}),
    (E, [tslot(pos0=2 ** 31 - 1)], {}), (E, [tslot(parent=[0, 0])], {}), (E, [tslot(parent=[-1, 1])], {}),
    (E, [tslot(), tslot()], {}), (E, [tslot(v=P)], {}), (E, [tslot()], dict(scores=SC, lds=10)),
    (E, [tslot()], dict(scores=SC, lds=8)), (E, [tslot()], dict(scores=SC + 8, lds=12)), (E, [tslot()], dict(stats=ST + 4)),
    (E, [tslot()], dict(scores=P, lds=12)), (E, [tslot()], dict(x=0)), (E, [tslot()], dict(ws=0)), (E, [tslot()], dict(logits=P)),
    (S, [tslot()], dict(ws_bytes=1024)),
])
def test_tree_step_refusals(lib, want, slots, kw):
    assert step(lib, slots, **kw) == want and lib.luce_last_error()


def test_tree_step_layout(lib):
    m, a, b = model(), luce.StepLayoutC(), luce.StepLayoutC()
    assert lib.luce_decode_step_tree_layout(ctypes.byref(m), 0, 10, ctypes.byref(a)) == E
    assert lib.luce_decode_step_tree_layout(ctypes.byref(m), 17, 10, ctypes.byref(a)) == E
    assert lib.luce_decode_step_tree_layout(ctypes.byref(m), 4, -1, ctypes.byref(a)) == E
    assert lib.luce_decode_step_tree_layout(ctypes.byref(m), 4, 130817, ctypes.byref(a)) == E
    assert lib.luce_decode_step_tree_layout(ctypes.byref(m), 4, 10, None) == E
    assert lib.luce_decode_step_tree_layout(ctypes.byref(m), 4, 1000, ctypes.byref(a)) == luce.LUCE_OK
    assert lib.luce_decode_step_layout(ctypes.byref(m), 4, 1000, ctypes.byref(b)) == luce.LUCE_OK
    assert all(getattr(a, f) == getattr(b, f) for f in luce._LAYOUT_FIELDS if f != "total")


def pslot(k=P, v=P + BIG, table=(0, 1, 2), n_pages=4, length=130, cap=400, path=(0, 2), row0=0, acc=None, pos=None, pos0=10):
    return luce.PagedCommitSlotC(k, v, ints(table) if table is not None else None, len(table or ()), n_pages, length, cap,
                                 len(path), row0, ints(path), acc, pos, pos0)


def pcommit(lib, slots, L=2, Hq=8, Hkv=2, D=128, scores=None, rows=0, lds=0, stats=None):
    arr = (luce.PagedCommitSlotC * max(1, len(slots)))(*slots)
    return lib.luce_tree_commit_paged(arr, len(slots), L, Hq, Hkv, D, scores, rows, lds, stats, None)


@pytest.mark.parametrize("want,slots,kw", [
    (E, [], {}), (U, [pslot()], dict(D=64)), (E, [pslot(k=0)], {}), (E, [pslot(v=P)], {}), (E, [pslot(k=P + 8)], {}),
    (E, [pslot(table=None)], {}), (E, [pslot(n_pages=0)], {}), (E, [pslot(table=(0, 4))], {}), (E, [pslot(table=(0, -1))], {}),
    (E, [pslot(table=(0,))], {}), (E, [pslot(length=126, path=(0, 2), table=(0, 9))], {}), (E, [pslot(path=(2, 1))], {}),
    (E, [pslot(length=399, path=(0, 1))], {}), (E, [pslot(), pslot()], {}), (E, [pslot(acc=ACC)], {}),
    (E, [pslot(path=(1, 3)), pslot(table=(3, 1), length=133, path=(0,))], {}),   # writes key 133's row, which the other reads
    (E, [pslot(acc=ACC, pos=ACC)], dict(scores=SC, rows=4, lds=136, stats=ST)),
    (E, [pslot(pos=P + 256)], {}), (E, [pslot(acc=P + BIG)], dict(scores=SC, rows=4, lds=136, stats=ST)),       # within a pool
    (E, [pslot(), pslot(k=P + 2 * 2 * 128 * 256, table=(3, 3, 3))], {}), (E, [pslot(), pslot(P + BIG, P, (3, 3, 3))], {}),
    (U, [pslot(length=130815, cap=1 << 20, table=(0,) * 1023)], {}),
])
def test_paged_commit_refusals(lib, want, slots, kw):
    assert pcommit(lib, slots, **kw) == want and lib.luce_last_error()


def peslot(k=P, v=P + BIG, table=P, acc=ACC, pos=POS, acc_out=ACC, pos_out=POS, n_pages=4, length=20, cap=64, budget=10, sinks=1,
           recent=4, nxt=20):
    return luce.PagedEvictSlotC(k, v, table, acc, pos, acc_out, pos_out, n_pages, length, cap, budget, sinks, recent, nxt)


@pytest.mark.parametrize("want,slot,kw", [
    (U, peslot(), dict(D=64)), (E, peslot(k=0), {}), (E, peslot(v=P), {}), (E, peslot(table=0), {}), (E, peslot(table=P + 2), {}),
    (E, peslot(n_pages=0), {}), (E, peslot(acc=0), {}), (E, peslot(length=65), {}), (E, peslot(budget=0), {}),
    (E, peslot(sinks=6, recent=5), {}), (E, peslot(acc_out=POS), {}), (U, peslot(length=130817, cap=130900), {}),
    (E, peslot(acc_out=P + 256), {}), (E, peslot(pos=P + BIG, pos_out=P + BIG), {}), (U, peslot(n_pages=1 << 22), {}),
])
def test_paged_evict_refusals(lib, want, slot, kw):
    arr = (luce.PagedEvictSlotC * 1)(slot)
    assert lib.luce_kv_evict_paged(arr, 1, 2, 2, kw.get("D", 128), None) == want and lib.luce_last_error()


def ptslot(k=P, v=P + BIG, table=P, host=(0, 1), n_pages=4, length=10, pos0=10, nodes=2, parent=None):
    return luce.PagedTreeSlotC(k, v, table, ints(host), len(host), n_pages, length, pos0, nodes,
                               None if parent is None else ints(parent))


@pytest.mark.parametrize("want,slots", [
    (E, []), (E, [ptslot(k=0)]), (E, [ptslot(v=P)]), (E, [ptslot(table=0)]), (E, [ptslot(host=(4, 0))]), (E, [ptslot(host=())]),
    (E, [ptslot(length=255)]), (E, [ptslot(nodes=0)]), (E, [ptslot(nodes=17)]), (E, [ptslot(parent=[0, 0])]), (E, [ptslot(pos0=-1)]),
    (E, [ptslot(), ptslot()]), (U, [ptslot(length=130815)]),
])
def test_paged_tree_step_refusals(lib, want, slots):
    arr = (luce.PagedTreeSlotC * max(1, len(slots)))(*slots)
    assert lib.luce_decode_step_tree_paged(ctypes.byref(model()), arr, len(slots), P, None, None, None, 0, None, 0x100000,
                                           1 << 40, None) == want
    assert lib.luce_last_error()
