"""What the Python calls hand to the library, seen by a stand-in for it: no
device needed, the tensors lie on the host."""
import contextlib
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import invariant_sequence_decode_gb300 as luce  # noqa: E402


def ints(p, n):
    return np.ctypeslib.as_array(ctypes.cast(p, ctypes.POINTER(ctypes.c_int32)), (n,)).tolist()


@pytest.fixture
def library(monkeypatch):
    """Stands in for the library: names' functions are set by the tests."""
    class Library:
        luce_last_error = staticmethod(lambda: b"refused")

        def __getitem__(self, name):
            return getattr(self, name)

    lib = Library()
    monkeypatch.setattr(luce, "load_library", lambda *a: lib)
    monkeypatch.setattr(luce, "_need", lambda *a: None)
    monkeypatch.setattr(luce, "_kv_pair", lambda *a: None)
    monkeypatch.setattr(luce, "_stream", lambda stream=None: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    return lib


class TinyModel:
    layers, n_kv_heads, n_q_heads, vocab, hidden = [None], 2, 4, 0, 256
    c = luce.ModelC()


def paged_steps(library):
    """(make a slot, step over it): what a step sees as its host and its device table."""
    seen = []

    def step(model, slots, *rest):
        s = slots[0]
        seen.append((ints(s.table_host, s.n_table), ints(s.table, s.n_table)))
        return 0

    library.luce_decode_step_paged = library.luce_decode_step_tree_paged = step
    pool = lambda: torch.zeros(8, 1, 2, 128, 128, dtype=torch.float16)  # noqa: E731
    x, ws = torch.zeros(1, 256), torch.zeros(1024, dtype=torch.uint8)
    return seen, {
        "tree": (lambda t: luce.PagedTreeSlot(pool(), pool(), t, 130, 1),
                 lambda s: luce.luce_decode_step_tree(TinyModel, [s], x, ws)),
        "plain": (lambda t: luce.PagedSlot(pool(), pool(), t, 130),
                  lambda s: luce.luce_decode_step_paged(TinyModel, [s], [1], x, ws)),
    }


@pytest.mark.parametrize("kind", ["tree", "plain"])
def test_a_paged_step_reads_the_table_it_was_given_last(library, kind):
    seen, steps = paged_steps(library)
    make, step = steps[kind]
    slot = make([3, 1])
    step(slot)
    first = slot.table_dev
    step(slot)
    assert slot.table_dev is first                       # nothing changed, nothing copied
    slot.table[1] = 5                                    # a page was remapped
    step(slot)
    slot.table = np.array([3, 5, 7, 0])                  # the cache grew
    step(slot)
    slot.table = [2, 6]
    step(slot)
    want = [[3, 1], [3, 1], [3, 5], [3, 5, 7, 0], [2, 6]]
    assert seen == [(t, t) for t in want]


def state(dtype, cap=40):
    return torch.zeros(1, 2, cap, dtype=dtype)


def evict_slot(**kw):
    kv = lambda: torch.zeros(1, 2, 40, 128, dtype=torch.float16)  # noqa: E731
    return luce.EvictSlot(kv(), kv(), state(torch.float32), state(torch.int32), 30, 20, **kw)


def record(library, name, fields, argtypes):
    """The named function as one that notes its first slot's fields."""
    seen = []

    def call(slots, n, *rest):
        seen.append(tuple(getattr(slots[0], f) for f in fields))
        return 0

    call.argtypes = argtypes
    setattr(library, name, call)
    return seen


@pytest.fixture
def prepared(library, monkeypatch):
    """The library for prepared calls, whose device and stream are the host's."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: None, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    return library


@pytest.fixture
def evictions(prepared):
    library, i32 = prepared, ctypes.c_int32
    for name in ("luce_kv_evict", "luce_kv_evict_paged"):
        seen = record(library, name, ("len", "budget", "sinks", "recent", "next_pos"), [None, i32, i32, i32, i32, None])
        setattr(library, name + "_seen", seen)
    return library.luce_kv_evict_seen


def test_eviction_without_a_next_position_protects_none_as_recent(evictions):
    luce.luce_kv_evict([evict_slot()])
    luce.luce_kv_evict([evict_slot(sinks=2)])
    assert evictions == [(30, 20, 0, 0, 2 ** 31 - 1), (30, 20, 2, 0, 2 ** 31 - 1)]
    with pytest.raises(ValueError, match="next_pos"):
        luce.luce_kv_evict([evict_slot(recent=4)])
    luce.luce_kv_evict([evict_slot(recent=4, next_pos=31)])
    assert evictions[2:] == [(30, 20, 0, 4, 31)]


def test_a_commit_takes_len_as_its_first_position_unless_told(prepared):
    i32, vp = ctypes.c_int32, ctypes.c_void_p
    seen = record(prepared, "luce_tree_commit", ("len", "pos0", "n_path"), [None, i32, i32, i32, i32, i32, vp, i32, ctypes.c_int64, vp, vp])
    kv = lambda: torch.zeros(1, 2, 40, 128, dtype=torch.float16)  # noqa: E731
    slot = luce.CommitSlot(kv(), kv(), 30, [0, 2], pos=state(torch.int32))
    call = luce.TreeCommit([slot], 4)
    call()
    slot.len = 32
    call()
    slot.pos0 = 0
    call()
    slot.pos0 = 70
    call()
    assert seen == [(30, 30, 2), (32, 32, 2), (32, 0, 2), (32, 70, 2)]


def test_prepared_evictions_and_commits_follow_replaced_tensors(prepared, monkeypatch):
    monkeypatch.setattr(luce, "_state", lambda *a: None)
    monkeypatch.setattr(luce, "_pools", lambda *a: None)
    i32, vp, i64 = ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64
    evict_fields = ("k_pool", "v_pool", "table", "acc", "pos", "acc_out", "pos_out", "n_pages", "cap")
    seen = record(prepared, "luce_kv_evict_paged", evict_fields, [None, i32, i32, i32, i32, vp])
    pool = lambda n=3: torch.zeros(n, 1, 2, 128, 128, dtype=torch.float16)  # noqa: E731
    table = lambda n=2: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    s = luce.PagedEvictSlot(pool(), pool(), table(), state(torch.float32, 256), state(torch.int32, 256), 200, 100)
    call = luce.KvEvict([s])

    def want():
        outs = (s.acc if s.acc_out is None else s.acc_out, s.pos if s.pos_out is None else s.pos_out)
        return tuple(t.data_ptr() for t in (s.k_pool, s.v_pool, s.table, s.acc, s.pos, *outs)) + (len(s.k_pool), s.acc.shape[-1])

    for change in ({}, {"table": table()}, {"k_pool": pool(5), "v_pool": pool(5)}, {"acc_out": state(torch.float32, 256)},
                   {"acc": state(torch.float32, 256)}, {"pos": state(torch.int32, 256)}, {"table": table(4)}):
        for name, t in change.items():
            setattr(s, name, t)
        call()
        assert seen[-1] == want()
    s.len = 513
    with pytest.raises(ValueError, match="does not hold"):
        call()
    s.len, s.table = 300, table(2)
    with pytest.raises(ValueError):
        call()
    commit_fields = ("k", "v", "acc", "pos", "cap")
    seen = record(prepared, "luce_tree_commit", commit_fields, [None, i32, i32, i32, i32, i32, vp, i32, i64, vp, vp])
    kv = lambda n=40: torch.zeros(1, 2, n, 128, dtype=torch.float16)  # noqa: E731
    c = luce.CommitSlot(kv(), kv(), 30, [0, 2], acc=state(torch.float32), pos=state(torch.int32))
    call = luce.TreeCommit([c], 4)
    for change in ({}, {"k": kv(), "v": kv()}, {"acc": state(torch.float32)}, {"pos": None}, {"k": kv(50), "v": kv(50), "acc": None}):
        for name, t in change.items():
            setattr(c, name, t)
        call()
        assert seen[-1] == tuple(None if t is None else t.data_ptr() for t in (c.k, c.v, c.acc, c.pos)) + (c.k.shape[2],)


@pytest.fixture
def attention(prepared):
    """Notes each call's views as (k, parents or None, len, row0, nodes), and the workspace's bytes."""
    i32, i64, f32, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
    seen = []

    def call(q, views, n, Hq, Hkv, D, scale, out, scores, lds, stats, ws, ws_bytes, stream):
        seen.append([(v.k, ints(v.parent, v.n_nodes) if v.parent else None, v.len, v.row0, v.n_nodes) for v in views])
        prepared.ws_bytes = ws_bytes.value
        return 0

    call.argtypes = [vp, None, i32, i32, i32, i32, f32, vp, vp, i64, vp, vp, sz, vp]
    prepared.luce_tree_attn = call
    prepared.luce_tree_attn_workspace_size = lambda T, Hq, Hkv, D, max_len: max_len * 10
    return seen


def test_a_prepared_tree_attention_follows_trees_rows_and_caches(attention, prepared):
    kv = lambda cap=64: torch.zeros(2, cap, 128, dtype=torch.float16)  # noqa: E731
    a, b = luce.TreeView(kv(), kv(), 10, [-1, 0, 0], 0), luce.TreeView(kv(), kv(), 20, 2, 3)
    call = luce.TreeAttention(torch.zeros(5, 4, 128), [a, b], 2, 0.1)

    def check():
        call()
        for v, got in zip((a, b), attention[-1]):
            tree = None if isinstance(v.parent, int) else list(v.parent)
            assert got == (v.k.data_ptr(), tree, v.len, v.row0, v.parent if tree is None else len(tree))

    check()
    a.parent = [-1, -1, 1]                       # the next step's tree
    check()
    a.parent[2] = 0                              # edited where it lies
    check()
    a.parent, b.parent, b.row0 = (-1, 0), [-1, 0, 1], 2
    check()
    a.parent = np.array([-1, -1])
    check()
    a.parent[1] = 0
    check()
    b.row0, a.row0 = 0, 3
    check()
    a.k, a.v, a.len = kv(), kv(), 30
    check()
    first = prepared.ws_bytes
    b.k, b.v, b.len = kv(500), kv(500), 400      # a longer cache asks for more workspace
    check()
    assert prepared.ws_bytes > first and prepared.ws_bytes >= 10 * 400
    calls = len(attention)
    for bad in ({"parent": [-1] * 3}, {"parent": [-1]}, {"parent": 2, "row0": 4}):
        keep = {name: getattr(a, name) for name in bad}
        for name, x in bad.items():
            setattr(a, name, x)
        for _ in range(2):                       # refused until it is put right
            with pytest.raises(ValueError, match="rows"):
                call()
        for name, x in keep.items():
            setattr(a, name, x)
    b.len = 498
    with pytest.raises(ValueError, match="exceed"):
        call()
    assert len(attention) == calls
    b.len = 497
    check()


def test_two_threads_on_two_streams_keep_to_their_own(prepared, monkeypatch):
    """A second call comes between a call's look at its stream and its launch, as another thread's may."""
    i32, vp, streams, launched, between = ctypes.c_int32, ctypes.c_void_p, [11], [], [True]

    def evict(slots, n, L, Hkv, D, stream):
        launched.append(stream.value)
        return 0

    evict.argtypes = [None, i32, i32, i32, i32, vp]
    prepared.luce_kv_evict = evict
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: streams[-1], raising=False)

    def device():
        if between.pop() if between else False:
            streams.append(22)
            call()
            streams.pop()

    monkeypatch.setattr(torch._C, "_cuda_getDevice", device, raising=False)
    call = luce.KvEvict([evict_slot()])
    call()
    assert launched == [22, 11]
    call()
    assert launched == [22, 11, 11]


@pytest.mark.parametrize("bad", [dict(x=torch.zeros(1, 255)), dict(x=torch.zeros(1, 2, 128)), dict(x=torch.zeros(2, 256)),
                                 dict(logits=torch.zeros(1, 9)), dict(argmax=torch.zeros(0, dtype=torch.int32))])
def test_a_tree_step_refuses_buffers_that_are_too_small(library, bad):
    """They would be read or written past their ends."""
    class Model(TinyModel):
        vocab = 10

    calls = []
    library.luce_decode_step_tree = lambda *a: calls.append(a) or 0
    library.luce_decode_step_tree.argtypes = None
    kv = lambda: torch.zeros(1, 2, 40, 128, dtype=torch.float16)  # noqa: E731
    a = dict(x=torch.zeros(1, 256), logits=torch.zeros(1, 10), argmax=torch.zeros(1, dtype=torch.int32))
    run = lambda **kw: luce.luce_decode_step_tree(Model, [luce.TreeSlot(kv(), kv(), 10, 1)], ws=torch.zeros(64, dtype=torch.uint8), **kw)  # noqa: E731
    run(**a)
    a.update(bad)
    with pytest.raises(ValueError):
        run(**a)
    assert len(calls) == 1
