"""Prepared calls whose views lose their tensors: refused at every call, not the first alone.  No device needed."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
import invariant_sequence_decode_gb300 as luce  # noqa: E402
from test_prepared_calls import library, prepared  # noqa: E402,F401

vp, i32, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float
KV_PAIR = luce._kv_pair


@pytest.fixture
def host(prepared, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    monkeypatch.setattr(luce, "_kv_pair", KV_PAIR)       # (the real check)
    for name in ("luce_tree_attn_workspace_size", "luce_q8kv_attn_workspace_size"):
        setattr(prepared, name, lambda *a: 1000)
    prepared.calls = []
    for name, types in (("luce_tree_attn", [vp, None, i32, i32, i32, i32, f32, vp, vp, ctypes.c_int64, vp, vp, ctypes.c_size_t, vp]),
                        ("luce_q8kv_attn", [vp, None, i32, i32, i32, i32, f32, vp, vp, ctypes.c_size_t, vp]),
                        ("luce_qk_norm_rope", [vp, ctypes.c_int64, None, i32, i32, i32, i32, vp, vp, f32, vp, i32, vp, ctypes.c_double, vp, vp])):
        def call(*a):
            prepared.calls.append(1)
            return 0
        call.argtypes = types
        setattr(prepared, name, call)
    return prepared


def cache():
    return torch.zeros(2, 16, 128, dtype=torch.float16)


@pytest.mark.parametrize("make", [
    lambda: (lambda v: (v, luce.TreeAttention(torch.zeros(1, 4, 128), [v], 2, 0.1)))(luce.TreeView(cache(), cache(), 5, 1)),
    lambda: (lambda v: (v, luce.Q8Attention(torch.zeros(1, 4, 128), [v], 2, 0.1)))(luce.Q8View(None, None, None, 0, cache(), cache(), 5)),
    lambda: (lambda v: (v, luce.QkNormRope(torch.zeros(4, 8 * 128), [v], 4, torch.zeros(4, dtype=torch.int32), 1e4)))(luce.SeqView(cache(), cache(), 9, 4, 0)),
])
def test_an_emptied_view_is_refused_at_every_call(host, make):
    view, run = make()
    run()
    k, v = view.k, view.v
    view.k = view.v = None
    for _ in range(3):
        with pytest.raises(TypeError):
            run()
    view.k, view.v = k, v
    run()
    assert len(host.calls) == 2
