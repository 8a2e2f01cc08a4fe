"""Layouts and numbers that the prepared calls over caches in 8 bits refuse or hand on, seen by a stand-in for
the library: no device needed, the tensors lie on the host."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
import invariant_sequence_decode_gb300 as luce  # noqa: E402
from test_prepared_calls import library, prepared, record  # noqa: E402,F401
from test_q8kv_prepared import q8_slot  # noqa: E402

i32 = ctypes.c_int32


@pytest.fixture
def host(prepared, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    prepared.luce_q8kv_attn_workspace_size = lambda *a: 1000
    return prepared


def attention(host, fields=("page_stride", "n_pages")):
    """(make a prepared call of one view, what the library saw)."""
    seen = []

    def call(q, views, n, Hq, Hkv, D, scale, out, ws, ws_bytes, stream):
        seen.append(tuple(getattr(views[0], f) for f in fields))
        return 0

    call.argtypes = [ctypes.c_void_p, None, i32, i32, i32, i32, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    host.luce_q8kv_attn = call
    return lambda view: luce.Q8Attention(torch.zeros(1, 4, 128), [view], 2, 0.1), seen


def pools(n_pages, layers=1):
    return [torch.zeros(n_pages, layers, 2, 128, 128, dtype=torch.int8) for _ in range(2)] + [torch.zeros(n_pages, layers, 2, 2, 4)]


def view_of(k_codes, v_codes, scales, **kw):
    tail = torch.zeros(2, 8, 128, dtype=torch.float16)
    return luce.Q8View(k_codes, v_codes, scales, 32, tail, tail.clone(), **kw)


def test_pages_that_lie_on_one_another_are_refused(host):
    """One page expanded to several has a stride of 0 from page to page, which the library takes as pages in a row."""
    make, seen = attention(host)
    one = [p[:, 0] for p in pools(1)]
    with pytest.raises(ValueError, match="apart"):
        make(view_of(*(p.expand(3, *p.shape[1:]) for p in one)))
    with pytest.raises(ValueError, match="apart"):
        make(view_of(*(p.expand(3, *p.shape[1:]) for p in one), table=torch.zeros(2, dtype=torch.int32)))
    many = [p[:, 0] for p in pools(3)]
    with pytest.raises(ValueError, match="apart"):
        make(view_of(many[0], many[1], one[2].expand(3, -1, -1, -1)))
    run = make(view_of(*many))
    run()
    run = make(view_of(*(p[:, 1] for p in pools(3, layers=4))))
    run()
    run = make(view_of(*one))
    run()
    assert seen == [(2 * 128 * 128, 3), (4 * 2 * 128 * 128, 3), (0, 1)]


def test_a_view_put_right_after_a_refusal_is_taken_again(host):
    """What a refused call has handed to the library's structs of a view does not stay there."""
    make, seen = attention(host, ("sealed", "len", "n_nodes", "row0"))
    view = view_of(*(p[:, 0] for p in pools(3)), len=2)
    run = make(view)
    run()
    view.parent, view.sealed = 4, 4096                   # more keys than the pages hold, and another tree
    with pytest.raises(ValueError, match="pages hold"):
        run()
    view.parent, view.sealed = 1, 32
    run()
    view.parent = [-1, 0]                                # a row too many
    with pytest.raises(ValueError, match="rows"):
        run()
    view.parent = 1
    run()
    assert seen == [(32, 2, 1, 0)] * 3


def test_a_projection_put_right_after_a_refusal_is_taken_again(host):
    seen = []

    def call(qkv, ld, views, n, *rest):
        seen.append(tuple((v.len, v.n_q, v.row0) for v in views))
        return 0

    vp = ctypes.c_void_p
    call.argtypes = [vp, ctypes.c_int64, None, i32, i32, i32, i32, vp, vp, ctypes.c_float, vp, i32, vp, ctypes.c_double, vp, vp]
    host.luce_qk_norm_rope = call
    cache = lambda: torch.zeros(2, 16, 128, dtype=torch.float16)  # noqa: E731
    views = [luce.SeqView(cache(), cache(), 9, 4, 0), luce.SeqView(cache(), cache(), 5, 5, 4)]
    run = luce.QkNormRope(torch.zeros(9, 8 * 128), views, 4, torch.zeros(9, dtype=torch.int32), 1e4)
    run()
    views[1].n_q = views[1].len = 4                      # a row too few
    with pytest.raises(ValueError, match="rows"):
        run()
    views[1].n_q = views[1].len = 5
    run()
    views[0].n_q, views[1].row0, views[1].n_q = 5, 5, 4  # another split of the same rows
    run()
    assert seen == [((9, 4, 0), (5, 5, 4))] * 2 + [((9, 5, 0), (5, 4, 5))]


BIG = 2 ** 32


@pytest.mark.parametrize("field,value", [("sinks", BIG), ("window", BIG + 4096), ("len", BIG + 2), ("row0", -BIG), ("sealed", -BIG + 32),
                                         ("parent", BIG + 1), ("window", 2 ** 31)])
def test_numbers_of_a_view_that_32_bits_do_not_hold_are_refused(host, field, value):
    """(sinks of 2^32, meant as all keys, would be none)"""
    make, seen = attention(host, ("sealed", "len", "n_nodes", "row0", "window", "sinks"))
    view = view_of(*(p[:, 0] for p in pools(3)), len=2, window=100, sinks=3)
    run = make(view)
    run()
    was = getattr(view, field)
    setattr(view, field, value)
    for _ in range(2):
        with pytest.raises(ValueError, match="32 bits"):
            run()
    setattr(view, field, was)
    run()
    assert seen == [(32, 2, 1, 0, 100, 3)] * 2
    setattr(view, field, value)
    with pytest.raises(ValueError, match="32 bits"):
        make(view)


def test_numbers_of_a_slot_that_32_bits_do_not_hold_are_refused(host):
    seen = record(host, "luce_q8kv_seal", ("len", "sealed"), [None, i32, i32, i32, i32, None])
    slot = q8_slot(40, 64)
    seal = luce.Q8Seal([slot])
    for field, value in (("len", -BIG + 40), ("sealed", -BIG), ("sealed", -BIG + 64)):
        was = getattr(slot, field)
        setattr(slot, field, value)
        for _ in range(2):
            with pytest.raises(ValueError, match="32 bits"):
                seal()
        setattr(slot, field, was)
    seal()
    assert seen == [(40, 64)]


def test_numbers_of_a_projection_that_32_bits_do_not_hold_are_refused(host):
    seen = []

    def call(qkv, ld, views, n, *rest):
        seen.append((views[0].len, views[0].n_q, views[0].row0))
        return 0

    vp = ctypes.c_void_p
    call.argtypes = [vp, ctypes.c_int64, None, i32, i32, i32, i32, vp, vp, ctypes.c_float, vp, i32, vp, ctypes.c_double, vp, vp]
    host.luce_qk_norm_rope = call
    view = luce.SeqView(*(torch.zeros(2, 16, 128, dtype=torch.float16) for _ in range(2)), 9, 4, 0)
    run = luce.QkNormRope(torch.zeros(4, 8 * 128), [view], 4, torch.zeros(4, dtype=torch.int32), 1e4)
    view.len = BIG + 9
    with pytest.raises(ValueError, match="32 bits"):
        run()
    view.len = 9
    view.n_q, view.row0 = 4 - BIG, BIG                   # 4 rows, by their sum
    with pytest.raises(ValueError, match="32 bits"):
        run()
    view.n_q, view.row0 = 4, 0
    run()
    assert seen == [(9, 4, 0)]
