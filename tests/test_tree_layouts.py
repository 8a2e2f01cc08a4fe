"""Layouts of paged pools that the prepared tree attention refuses, seen by a stand-in for the library: no device
needed, the tensors lie on the host."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
import invariant_sequence_decode_gb300 as luce  # noqa: E402
from test_prepared_calls import library, prepared  # noqa: E402,F401

vp, i32 = ctypes.c_void_p, ctypes.c_int32


def test_pages_that_lie_on_one_another_are_refused(prepared):  # noqa: F811
    """One page expanded to several has a stride of 0 from page to page, which the library takes as pages in a row."""
    seen = []

    def call(q, views, *rest):
        seen.append((views[0].page_stride, views[0].n_pages))
        return 0

    call.argtypes = [vp, None, i32, i32, i32, i32, ctypes.c_float, vp, vp, ctypes.c_int64, vp, vp, ctypes.c_size_t, vp]
    prepared.luce_tree_attn_paged = call
    prepared.luce_tree_attn_workspace_size = lambda *a: 1000
    pools = lambda n, layers: [torch.zeros(n, layers, 2, 128, 128, dtype=torch.float16)[:, 0] for _ in range(2)]  # noqa: E731
    table = torch.zeros(3, dtype=torch.int32)

    def run(k, v):
        luce.TreeAttention(torch.zeros(1, 4, 128), [luce.PagedTreeView(k, v, table, 200, 1)], 2, 0.1)()

    with pytest.raises(ValueError, match="on one another"):
        run(*(p.expand(3, -1, -1, -1) for p in pools(1, 1)))
    run(*pools(3, 1))
    run(*pools(3, 4))
    run(*pools(1, 4))
    assert seen == [(2 * 128 * 128, 3), (4 * 2 * 128 * 128, 3), (0, 1)]
