"""The entry points of caches in 8 bits refuse invalid calls with a status before
anything is enqueued (no device needed: validation precedes launches)."""
import ctypes

import pytest

import invariant_sequence_decode_gb300 as luce
from invariant_sequence_decode_gb300 import build

P = 0x10000
M = 1 << 36          # arrays that lie apart
E, U, S = luce.LUCE_EINVAL, luce.LUCE_EUNSUPPORTED, luce.LUCE_ENOSPACE


@pytest.fixture(scope="module")
def lib():
    build.build()
    return luce.load_library()


def ints(values):
    return (ctypes.c_int32 * max(1, len(values)))(*values)


def view(kc=P + M, vc=P + 2 * M, sc=P + 3 * M, table=None, k=P + 4 * M, v=P + 5 * M, page=0, head=128 * 128, tok=128, pages=20, sealed=2048,
         length=10, cap=128, nodes=2, row0=0, window=0, sinks=0, parent=None):
    return luce.Q8ViewC(kc, vc, sc, table, k, v, page, head, tok, pages, sealed, length, cap, nodes, row0, window, sinks,
                        None if parent is None else ints(parent))


def attn(lib, views, q=P, Hq=8, Hkv=2, D=128, scale=0.1, out=P + 6 * M, ws=P + 7 * M, ws_bytes=1 << 35, n=None):
    arr = (luce.Q8ViewC * max(1, len(views)))(*views)
    return lib.luce_q8kv_attn(q, arr, len(views) if n is None else n, Hq, Hkv, D, scale, out, ws, ws_bytes, None)


@pytest.mark.parametrize("want,kw", [
    (E, dict(q=0)), (E, dict(q=P + 8)), (E, dict(out=0)), (E, dict(out=P + 6 * M + 2)), (E, dict(ws=0)), (E, dict(ws=P + 7 * M + 16)),
    (E, dict(Hq=9)), (E, dict(Hkv=0)), (E, dict(Hq=0)), (U, dict(Hq=18)), (U, dict(D=64)), (U, dict(Hq=8194, Hkv=4097)),
    (E, dict(scale=float("nan"))), (E, dict(scale=float("inf"))), (S, dict(ws_bytes=16)), (E, dict(n=0)), (E, dict(n=5)),
    (E, dict(out=P + M)), (E, dict(out=P + 4 * M)), (E, dict(ws=P + 3 * M)), (E, dict(ws=P + 6 * M)), (E, dict(out=P + 4)),
])
def test_attention_refuses_arguments(lib, want, kw):
    assert attn(lib, [view()], **kw) == want and lib.luce_last_error()


@pytest.mark.parametrize("want,views", [
    (E, [view(nodes=0)]), (E, [view(nodes=17)]), (E, [view(sealed=-32)]), (E, [view(sealed=2040)]), (E, [view(length=-1)]),
    (U, [view(length=113, cap=300, head=300 * 128)]), (U, [view(sealed=130816, pages=1022, length=0)]),
    (E, [view(cap=11)]), (E, [view(window=-1)]), (E, [view(sinks=-1)]), (E, [view(tok=120)]), (E, [view(tok=132)]),
    (E, [view(head=128 * 128 - 8)]), (E, [view(head=128 * 128 + 4)]), (E, [view(tok=1 << 33, head=1 << 37)]),
    (E, [view(row0=1)]), (E, [view(row0=-1)]), (E, [view(nodes=4, row0=13)]), (E, [view(), view()]),
    (E, [view(parent=[0, 0])]), (E, [view(parent=[-1, 1])]), (E, [view(parent=[-2, 0])]),
    (E, [view(kc=0)]), (E, [view(vc=0)]), (E, [view(sc=0)]), (E, [view(kc=P + M + 8)]), (E, [view(sc=P + 3 * M + 4)]),
    (E, [view(table=P + 2)]), (E, [view(pages=15)]), (E, [view(pages=0, table=P + 8 * M)]), (E, [view(k=0)]), (E, [view(v=P + 5 * M + 8)]),
    (E, [view(page=16384)]), (E, [view(page=32768 + 128)]), (E, [view(page=1 << 38)]),
])
def test_attention_refuses_views(lib, want, views):
    assert attn(lib, views) == want and lib.luce_last_error()


def test_attention_workspace(lib):
    size = lib.luce_q8kv_attn_workspace_size
    assert size(1, 8, 2, 128, 0) == 256
    assert size(16, 40, 8, 128, 130816) > size(4, 40, 8, 128, 2048) > 0
    for bad in ((0, 8, 2, 128, 0), (17, 8, 2, 128, 0), (1, 9, 2, 128, 0), (1, 18, 2, 128, 0), (1, 8, 2, 64, 0), (1, 8, 2, 128, -1),
                (1, 8, 2, 128, 130817), (1, 8, 0, 128, 0)):
        assert size(*bad) == 0
    # a size by the longest cache is enough for every shorter one, whatever its window
    for top in (2048, 40960, 130784):
        room = size(2, 8, 2, 128, top)
        for sealed in (32, 128, 160, 1024, 2048, 16384, 40960, 130784):
            for window, sinks in ((0, 0), (1, 0), (500, 4), (5000, 1000), (30000, 4)):
                if sealed <= top:
                    v = view(sealed=sealed, pages=1022, window=window, sinks=sinks)
                    # (passes the workspace's check: what it then meets is the overlap of out and q's view)
                    assert attn(lib, [v], out=P + M, ws_bytes=room) == E and b"overlaps" in lib.luce_last_error()


def slot(k=P + M, v=P + 2 * M, length=40, cap=64, kc=P + 3 * M, vc=P + 4 * M, sc=P + 5 * M, table=None, pages=4, sealed=64):
    return luce.Q8SlotC(k, v, length, cap, kc, vc, sc, table, pages, sealed)


def seal(lib, slots, L=1, Hkv=2, D=128, n=None):
    arr = (luce.Q8SlotC * max(1, len(slots)))(*slots)
    return lib.luce_q8kv_seal(arr, len(slots) if n is None else n, L, Hkv, D, None)


@pytest.mark.parametrize("want,slots,kw", [
    (E, [slot()], dict(n=0)), (E, [slot()] * 5, {}), (U, [slot()], dict(D=64)), (E, [slot()], dict(L=0)), (E, [slot()], dict(Hkv=0)),
    (E, [slot(k=0)], {}), (E, [slot(v=P + 2)], {}), (E, [slot(length=65)], {}), (E, [slot(length=-1)], {}), (E, [slot(cap=0, length=0)], {}),
    (E, [slot(sealed=-32)], {}), (E, [slot(sealed=40)], {}), (U, [slot(sealed=130784)], {}), (E, [slot(pages=-1)], {}),
    (E, [slot(pages=0)], {}), (E, [slot(sealed=512)], {}), (E, [slot(kc=0)], {}), (E, [slot(vc=P + 8)], {}), (E, [slot(sc=0)], {}),
    (E, [slot(sc=P + 5 * M + 4)], {}), (E, [slot(table=P + 1)], {}),
    (E, [slot(), slot()], {}),                               # two slots of one tail
    (E, [slot(kc=P + M)], {}), (E, [slot(vc=P + 3 * M)], {}), (E, [slot(sc=P + 4 * M + 16)], {}), (E, [slot(table=P + 5 * M)], {}),
    (E, [slot(v=P + M + 256)], {}),
])
def test_seal_refusals(lib, want, slots, kw):
    assert seal(lib, slots, **kw) == want and lib.luce_last_error()


def test_nothing_to_seal_enqueues_nothing(lib):
    before = lib.luce_launch_count()
    assert seal(lib, [slot(length=31, kc=0, vc=0, sc=0, pages=0), slot(k=P + 8 * M, v=P + 9 * M, length=0)]) == luce.LUCE_OK
    assert lib.luce_launch_count() == before


def seq(k=P + M, v=P + 2 * M, length=10, n=4, row0=0, cap=64, head=64 * 128, tok=128):
    return luce.SeqViewC(k, v, length, n, row0, cap, head, tok)


def project(lib, views=None, qkv=P, ld=12 * 128, Hq=8, Hkv=2, D=128, qg=None, kg=None, eps=1e-6, pos=P + 3 * M, axes=1, pair=None, theta=1e6,
            q=P + 4 * M, n=None):
    views = [seq()] if views is None else views
    arr = (luce.SeqViewC * max(1, len(views)))(*views)
    pair = None if pair is None else ctypes.addressof(pair)
    return lib.luce_qk_norm_rope(qkv, ld, arr, len(views) if n is None else n, Hq, Hkv, D, qg, kg, eps, pos, axes, pair, theta, q, None)


THREE = (ctypes.c_uint8 * 64)(*[i % 3 for i in range(64)])


@pytest.mark.parametrize("want,kw", [
    (E, dict(qkv=0)), (E, dict(qkv=P + 4)), (E, dict(pos=0)), (E, dict(pos=P + 3 * M + 2)), (E, dict(q=0)), (E, dict(q=P + 4 * M + 8)),
    (E, dict(ld=12 * 128 - 4)), (E, dict(ld=12 * 128 + 2)), (E, dict(Hq=0)), (E, dict(Hkv=0)), (U, dict(D=64)), (E, dict(qg=P + 5 * M + 4)),
    (E, dict(kg=P + 5 * M + 4)), (E, dict(eps=-1.0)), (E, dict(eps=float("nan"))), (E, dict(theta=0.0)), (E, dict(theta=float("inf"))),
    (E, dict(axes=0)), (E, dict(axes=5)), (E, dict(axes=3)), (E, dict(axes=2, pair=THREE)), (E, dict(n=0)), (E, dict(n=5)),
    (E, dict(views=[seq(k=0)])), (E, dict(views=[seq(v=P + 8)])), (E, dict(views=[seq(n=0)])), (E, dict(views=[seq(n=11)])),
    (E, dict(views=[seq(length=65)])), (E, dict(views=[seq(tok=120)])), (E, dict(views=[seq(tok=130)])), (E, dict(views=[seq(head=64 * 128 - 8)])),
    (E, dict(views=[seq(row0=1)])), (E, dict(views=[seq(row0=-1)])), (E, dict(views=[seq(), seq(k=P + 6 * M, v=P + 7 * M, row0=3)])),
    (E, dict(views=[seq(row0=2 ** 31 - 2)])), (E, dict(views=[seq(), seq(row0=4)])),      # (the same cache twice, at the same rows)
    (E, dict(q=P)), (E, dict(q=P + M + 10 * 256 - 512)), (E, dict(qg=P + 4 * M)), (E, dict(views=[seq(k=P + 4 * M)])),
])
def test_project_refusals(lib, want, kw):
    assert project(lib, **kw) == want and lib.luce_last_error()


def test_seal_reads_32_bytes_at_a_time(lib):
    for kw in (dict(k=P + M + 16), dict(v=P + 2 * M + 16)):
        assert seal(lib, [slot(**kw)]) == E and b"32-byte" in lib.luce_last_error()


def test_sizes_that_pass_64_bits(lib):
    assert project(lib, ld=1 << 62) == E and b"2^28" in lib.luce_last_error()
    assert seal(lib, [slot(pages=2 ** 31 - 1)], L=1 << 19) == E and b"out of range" in lib.luce_last_error()
    assert attn(lib, [view(pages=2 ** 31 - 1, page=1 << 37)]) == E and b"out of range" in lib.luce_last_error()


def test_wait_expiry_refuses_limits(lib):
    for bad in (0, 999, 1_000_000_001, -1):
        assert lib.luce_test_q8kv_wait_expiry(bad, None) == E and b"limit_ns" in lib.luce_last_error()
