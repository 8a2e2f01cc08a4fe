"""What the prepared calls over caches in 8 bits hand to the library, seen by a stand-in for it: no
device needed, the tensors lie on the host."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
import invariant_sequence_decode_gb300 as luce  # noqa: E402
from test_prepared_calls import ints, library, prepared, record  # noqa: E402,F401


def q8_slot(length=40, sealed=0):
    kv = lambda: torch.zeros(1, 2, 64, 128, dtype=torch.float16)  # noqa: E731
    pools = [torch.zeros(3, 1, 2, 128, 128, dtype=torch.int8) for _ in range(2)] + [torch.zeros(3, 1, 2, 2, 4)]
    return luce.Q8Slot(kv(), kv(), length, *pools, sealed)


def test_a_prepared_seal_follows_its_slot(prepared, monkeypatch):
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    i32 = ctypes.c_int32
    seen = record(prepared, "luce_q8kv_seal", ("k", "len", "cap", "k_codes", "n_pages", "sealed", "table"), [None, i32, i32, i32, i32, None])
    slot = q8_slot()
    call = luce.Q8Seal([slot])
    call()
    slot.sealed, slot.len = 32, 33                       # the caller continues behind the sealed block
    call()
    slot.k_codes = torch.zeros(5, 1, 2, 128, 128, dtype=torch.int8)
    with pytest.raises(ValueError):                      # the pools disagree
        call()
    slot.v_codes, slot.scales = slot.k_codes.clone(), torch.zeros(5, 1, 2, 2, 4)
    slot.table = torch.tensor([4, 1], dtype=torch.int32)
    call()
    slot.sealed, slot.len = 224, 40                      # two pages hold 256 keys: 224 + 32
    call()
    slot.len = 64
    with pytest.raises(ValueError, match="pages hold 256"):
        call()
    first = (slot.k.data_ptr(), 40, 64)
    assert [s[:3] for s in seen] == [first, (first[0], 33, 64), (first[0], 33, 64), first]
    assert [s[4:6] for s in seen] == [(3, 0), (3, 32), (5, 32), (5, 224)]
    assert seen[0][6] is None and seen[2][6] == slot.table.data_ptr() and seen[2][3] == slot.k_codes.data_ptr()


def test_prepared_attention_over_8_bits_follows_its_views(prepared, monkeypatch):
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    i32, vp, size = ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t
    asked = []
    prepared.luce_q8kv_attn_workspace_size = lambda *a: asked.append(a) or 1000 + a[-1]
    seen = []

    def call(q, views, n, Hq, Hkv, D, scale, out, ws, ws_bytes, stream):
        v = views[0]
        seen.append((v.sealed, v.len, v.n_nodes, v.window, v.sinks, v.n_pages, ints(v.parent, v.n_nodes) if v.parent else None, ws_bytes.value))
        return 0

    call.argtypes = [vp, None, i32, i32, i32, i32, ctypes.c_float, vp, vp, size, vp]
    prepared.luce_q8kv_attn = call
    slot = q8_slot(40, 256)
    view = luce.Q8View(slot.k_codes[:, 0], slot.v_codes[:, 0], slot.scales[:, 0], 256, slot.k[0], slot.v[0], 8, [-1, 0, 0])
    run = luce.Q8Attention(torch.zeros(3, 4, 128), [view], 2, 0.1)
    run()
    view.sealed, view.len, view.window, view.sinks = 288, 9, 100, 4
    view.parent[2] = 1                                   # the same list, another tree
    run()
    big = [torch.zeros(9, 2, 128, 128, dtype=torch.int8) for _ in range(2)] + [torch.zeros(9, 2, 2, 4)]
    view.k_codes, view.v_codes, view.scales = big        # more pages: more room
    view.sealed = 1152
    run()
    assert [s[:7] for s in seen] == [(256, 8, 3, 0, 0, 3, [-1, 0, 0]), (288, 9, 3, 100, 4, 3, [-1, 0, 1]),
                                     (1152, 9, 3, 100, 4, 9, [-1, 0, 1])]
    assert seen[0][7] == seen[1][7] == 1000 + 384 and seen[2][7] == 1000 + 1152
    view.parent = [-1, 0]
    with pytest.raises(ValueError):
        run()
