"""Batch-invariant concurrent decode step for GB300 (sm_103a).

Thin Python binding over ``libluce.so`` (the C ABI declared in
``include/luce.h``).  Functions take torch CUDA tensors, check dtypes and
layouts, and pass raw pointers and the current CUDA stream to the library:
argument marshalling only, every step of the path runs in the library's CUDA
kernels.  There is no fallback: a missing library raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import List, Optional, Sequence

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libluce.so")

QK = 32
MAX_SEQ = 4
MAX_ROWS_PER_SEQ = 4
MAX_ROWS = 16
HEAD_DIM = 128
MAX_KEYS = 130816
MAX_TREE = 16
LAST_POS = 2 ** 31 - 1  # no key is this far

LUCE_OK, LUCE_EINVAL, LUCE_EUNSUPPORTED, LUCE_ECUDA, LUCE_ENOSPACE = 0, -1, -2, -3, -4


class LuceError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"luce status {status}: {msg}")
        self.status = status


# ------------------------------------------------------------ ctypes mirror of luce.h

class SeqViewC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("len", ctypes.c_int32),
                ("n_q", ctypes.c_int32), ("row0", ctypes.c_int32), ("cap", ctypes.c_int32),
                ("head_stride", ctypes.c_int64), ("tok_stride", ctypes.c_int64)]


class LayerC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "attn_norm", "wqkv_q", "wqkv_d", "wo_q", "wo_d", "ffn_norm", "wgu_q", "wgu_d", "wdown_q", "wdown_d")]


class ModelC(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("hidden", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("ffn", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_double),
                ("layers", ctypes.POINTER(LayerC)), ("final_norm", ctypes.c_void_p),
                ("head_q", ctypes.c_void_p), ("head_d", ctypes.c_void_p)]


class SlotC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("len", ctypes.c_int32), ("cap", ctypes.c_int32)]


class PagedViewC(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("len", ctypes.c_int32), ("n_q", ctypes.c_int32), ("row0", ctypes.c_int32)]


class PagedSlotC(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("table_host", ctypes.POINTER(ctypes.c_int32)), ("n_table", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("len", ctypes.c_int32)]


class TreeViewC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("len", ctypes.c_int32), ("n_nodes", ctypes.c_int32),
                ("row0", ctypes.c_int32), ("cap", ctypes.c_int32), ("head_stride", ctypes.c_int64),
                ("tok_stride", ctypes.c_int64), ("parent", ctypes.POINTER(ctypes.c_int32))]


class PagedTreeViewC(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("n_pages", ctypes.c_int32), ("len", ctypes.c_int32), ("n_nodes", ctypes.c_int32),
                ("row0", ctypes.c_int32), ("parent", ctypes.POINTER(ctypes.c_int32)), ("page_stride", ctypes.c_int64)]


class TreeSlotC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("len", ctypes.c_int32), ("cap", ctypes.c_int32),
                ("pos0", ctypes.c_int32), ("n_nodes", ctypes.c_int32), ("parent", ctypes.POINTER(ctypes.c_int32))]


class PagedTreeSlotC(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("table_host", ctypes.POINTER(ctypes.c_int32)), ("n_table", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("len", ctypes.c_int32), ("pos0", ctypes.c_int32),
                ("n_nodes", ctypes.c_int32), ("parent", ctypes.POINTER(ctypes.c_int32))]


class CommitSlotC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("len", ctypes.c_int32), ("cap", ctypes.c_int32),
                ("n_path", ctypes.c_int32), ("row0", ctypes.c_int32), ("path", ctypes.POINTER(ctypes.c_int32)),
                ("acc", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("pos0", ctypes.c_int32)]


class PagedCommitSlotC(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("table_host", ctypes.POINTER(ctypes.c_int32)), ("n_table", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("len", ctypes.c_int32), ("cap", ctypes.c_int32),
                ("n_path", ctypes.c_int32), ("row0", ctypes.c_int32), ("path", ctypes.POINTER(ctypes.c_int32)),
                ("acc", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("pos0", ctypes.c_int32)]


class EvictSlotC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("acc", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("acc_out", ctypes.c_void_p), ("pos_out", ctypes.c_void_p), ("len", ctypes.c_int32),
                ("cap", ctypes.c_int32), ("budget", ctypes.c_int32), ("sinks", ctypes.c_int32),
                ("recent", ctypes.c_int32), ("next_pos", ctypes.c_int32)]


class PagedEvictSlotC(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("acc", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("acc_out", ctypes.c_void_p),
                ("pos_out", ctypes.c_void_p), ("n_pages", ctypes.c_int32), ("len", ctypes.c_int32),
                ("cap", ctypes.c_int32), ("budget", ctypes.c_int32), ("sinks", ctypes.c_int32),
                ("recent", ctypes.c_int32), ("next_pos", ctypes.c_int32)]


_LAYOUT_FIELDS = ("xn", "xn_q", "xn_d", "qkv", "q_rot", "part", "attn", "attn_q", "attn_d", "x1",
                  "xn2", "xn2_q", "xn2_d", "gu", "h", "h_q", "h_d", "xf", "xf_q", "xf_d", "total")


class StepLayoutC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in _LAYOUT_FIELDS]


EXPORTS = ("luce_last_error", "luce_version", "luce_launch_count", "luce_q8_quantize_act", "luce_q8_matvec_batch",
           "luce_q8_block_dots", "luce_rope_posvec", "luce_kv_append", "luce_decode_attn_multiseq",
           "luce_decode_attn_workspace_size", "luce_decode_step_layout", "luce_decode_step",
           "luce_decode_attn_multiseq_noalloc", "luce_decode_attn_noalloc_max_bytes", "luce_decode_attn_paged",
           "luce_decode_step_paged", "luce_wait_timeouts", "luce_decode_step_host",
           "luce_test_wait_expiry", "luce_test_tree_wait_expiry", "luce_q8_matvec_batch_path", "luce_q8_quantize_act_f16", "luce_rmsnorm_q8",
           "luce_swiglu_q8", "luce_step_graph_create", "luce_step_graph_run", "luce_step_graph_stats",
           "luce_step_graph_destroy", "luce_tree_attn", "luce_tree_attn_paged", "luce_tree_attn_workspace_size",
           "luce_tree_commit", "luce_kv_evict", "luce_decode_step_tree", "luce_decode_step_tree_layout",
           "luce_decode_step_tree_paged", "luce_tree_commit_paged", "luce_kv_evict_paged")

_lib = None


def load_library(path: str = LIB_PATH):
    """Load libluce.so (built by ``invariant_sequence_decode_gb300.build``).  Raises if missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run `python -m invariant_sequence_decode_gb300.build`")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz, f32, f64 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t,
                                  ctypes.c_float, ctypes.c_double)
    lib.luce_last_error.restype = ctypes.c_char_p
    lib.luce_last_error.argtypes = []
    lib.luce_version.restype = i32
    lib.luce_launch_count.restype = ctypes.c_uint64
    lib.luce_launch_count.argtypes = []
    lib.luce_q8_quantize_act.argtypes = [vp, i32, i32, i64, vp, vp, vp]
    lib.luce_q8_quantize_act_f16.argtypes = [vp, i32, i32, i64, vp, vp, vp]
    lib.luce_rmsnorm_q8.argtypes = [vp, i32, i32, vp, f32, vp, vp, vp, i32, vp]
    lib.luce_swiglu_q8.argtypes = [vp, i32, i32, vp, vp, vp, i32, vp]
    lib.luce_q8_matvec_batch.argtypes = [vp, vp, i32, i32, vp, vp, i32, vp, i64, vp]
    lib.luce_q8_matvec_batch_path.argtypes = [vp, vp, i32, i32, vp, vp, i32, vp, i64, i32, vp]
    lib.luce_q8_block_dots.argtypes = [vp, i32, i32, vp, i32, vp, vp]
    lib.luce_rope_posvec.argtypes = [vp, i32, i32, i32, i64, vp, f64, vp]
    lib.luce_kv_append.argtypes = [vp, vp, i64, i32, i32, ctypes.POINTER(SeqViewC), i32, vp]
    lib.luce_decode_attn_multiseq.argtypes = [vp, ctypes.POINTER(SeqViewC), i32, i32, i32, i32, f32, vp, vp, sz, vp]
    lib.luce_decode_attn_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.luce_decode_attn_workspace_size.restype = sz
    lib.luce_decode_step_layout.argtypes = [ctypes.POINTER(ModelC), i32, i32, ctypes.POINTER(StepLayoutC)]
    lib.luce_decode_step.argtypes = [ctypes.POINTER(ModelC), ctypes.POINTER(SlotC), ctypes.POINTER(ctypes.c_int32),
                                     i32, vp, vp, vp, vp, sz, vp]
    lib.luce_decode_attn_multiseq_noalloc.argtypes = [vp, ctypes.POINTER(SeqViewC), i32, i32, i32, i32, f32, vp, vp]
    lib.luce_decode_attn_noalloc_max_bytes.argtypes = []
    lib.luce_decode_attn_paged.argtypes = [vp, ctypes.POINTER(PagedViewC), i32, i32, i32, i32, f32, vp, vp, sz, vp]
    lib.luce_decode_step_paged.argtypes = [ctypes.POINTER(ModelC), ctypes.POINTER(PagedSlotC),
                                           ctypes.POINTER(ctypes.c_int32), i32, vp, vp, vp, vp, sz, vp]
    lib.luce_decode_attn_noalloc_max_bytes.restype = sz
    lib.luce_wait_timeouts.argtypes = [ctypes.POINTER(ctypes.c_uint32), i32]
    lib.luce_test_wait_expiry.argtypes = [i64, vp]
    lib.luce_test_tree_wait_expiry.argtypes = [i64, vp]
    lib.luce_decode_step_host.argtypes = [ctypes.POINTER(ModelC), ctypes.POINTER(SlotC), ctypes.POINTER(ctypes.c_int32),
                                          i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.luce_step_graph_create.argtypes = [ctypes.POINTER(ModelC), ctypes.POINTER(SlotC),
                                           ctypes.POINTER(ctypes.c_int32), i32, vp, vp, vp, vp, vp, vp, vp, sz,
                                           ctypes.POINTER(vp)]
    lib.luce_step_graph_run.argtypes = [vp, ctypes.POINTER(ctypes.c_int32), vp]
    lib.luce_step_graph_stats.argtypes = [vp, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64),
                                          ctypes.POINTER(ctypes.c_int32)]
    lib.luce_step_graph_destroy.argtypes = [vp]
    lib.luce_tree_attn.argtypes = [vp, ctypes.POINTER(TreeViewC), i32, i32, i32, i32, f32, vp, vp, i64, vp, vp, sz, vp]
    lib.luce_tree_attn_paged.argtypes = [vp, ctypes.POINTER(PagedTreeViewC), i32, i32, i32, i32, f32, vp, vp, i64, vp,
                                         vp, sz, vp]
    lib.luce_tree_attn_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    lib.luce_tree_attn_workspace_size.restype = sz
    lib.luce_decode_step_tree.argtypes = [ctypes.POINTER(ModelC), ctypes.POINTER(TreeSlotC), i32, vp, vp, vp, vp, i64, vp,
                                          vp, sz, vp]
    lib.luce_decode_step_tree_paged.argtypes = [ctypes.POINTER(ModelC), ctypes.POINTER(PagedTreeSlotC), i32, vp, vp, vp,
                                                vp, i64, vp, vp, sz, vp]
    lib.luce_tree_commit_paged.argtypes = [ctypes.POINTER(PagedCommitSlotC), i32, i32, i32, i32, i32, vp, i32, i64, vp, vp]
    lib.luce_kv_evict_paged.argtypes = [ctypes.POINTER(PagedEvictSlotC), i32, i32, i32, i32, vp]
    lib.luce_decode_step_tree_layout.argtypes = [ctypes.POINTER(ModelC), i32, i32, ctypes.POINTER(StepLayoutC)]
    lib.luce_tree_commit.argtypes = [ctypes.POINTER(CommitSlotC), i32, i32, i32, i32, i32, vp, i32, i64, vp, vp]
    lib.luce_kv_evict.argtypes = [ctypes.POINTER(EvictSlotC), i32, i32, i32, i32, vp]
    for name in EXPORTS:
        if name not in ("luce_last_error", "luce_version", "luce_launch_count", "luce_decode_attn_workspace_size",
                        "luce_decode_attn_noalloc_max_bytes", "luce_tree_attn_workspace_size"):
            getattr(lib, name).restype = i32
    _lib = lib
    return lib


def launch_count() -> int:
    """Kernel launches the library has enqueued so far (all threads)."""
    return int(load_library().luce_launch_count())


def wait_timeouts(reset: bool = False) -> int:
    """Bounded device waits that expired on the current device (0 on a healthy run)."""
    n = ctypes.c_uint32(0)
    _check(load_library().luce_wait_timeouts(ctypes.byref(n), 1 if reset else 0))
    return int(n.value)


def _check(rc: int):
    if rc != LUCE_OK:
        raise LuceError(rc, load_library().luce_last_error().decode())


def _stream(stream=None) -> int:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t, dtype, name):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA {dtype} tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


# ------------------------------------------------------------ kernels

def luce_q8_quantize_act(x, q=None, d=None, stream=None):
    """fp32 [T][K] -> (int8 [T][K], fp32 [T][K/32]) q8_0 activation blocks."""
    import torch
    _need(x, torch.float32, "x")
    T, K = x.shape
    q = torch.empty((T, K), dtype=torch.int8, device=x.device) if q is None else q
    d = torch.empty((T, K // QK), dtype=torch.float32, device=x.device) if d is None else d
    _check(load_library().luce_q8_quantize_act(x.data_ptr(), T, K, K, q.data_ptr(), d.data_ptr(), _stream(stream)))
    return q, d


def luce_q8_quantize_act_f16(x, q=None, d=None, stream=None):
    """fp32 [T][K] -> (int8 [T][K], binary16 scales as float16 [T][K/32]): the half-scale form."""
    import torch
    _need(x, torch.float32, "x")
    T, K = x.shape
    q = torch.empty((T, K), dtype=torch.int8, device=x.device) if q is None else q
    d = torch.empty((T, K // QK), dtype=torch.float16, device=x.device) if d is None else d
    _check(load_library().luce_q8_quantize_act_f16(x.data_ptr(), T, K, K, q.data_ptr(), d.data_ptr(),
                                                   _stream(stream)))
    return q, d


def luce_rmsnorm_q8(x, gamma, eps: float, half_scale: bool = False, stream=None):
    """RMSNorm of fp32 rows [T][H] and its q8_0 blocks: (xn fp32, q int8, d fp32 or float16)."""
    import torch
    _need(x, torch.float32, "x")
    _need(gamma, torch.float32, "gamma")
    T, H = x.shape
    xn = torch.empty_like(x)
    q = torch.empty((T, H), dtype=torch.int8, device=x.device)
    d = torch.empty((T, H // QK), dtype=torch.float16 if half_scale else torch.float32, device=x.device)
    _check(load_library().luce_rmsnorm_q8(x.data_ptr(), T, H, gamma.data_ptr(), float(eps), xn.data_ptr(),
                                          q.data_ptr(), d.data_ptr(), 1 if half_scale else 0, _stream(stream)))
    return xn, q, d


def luce_swiglu_q8(gu, half_scale: bool = False, stream=None):
    """SwiGLU of gate||up rows [T][2F] and its q8_0 blocks: (h fp32, q int8, d fp32 or float16)."""
    import torch
    _need(gu, torch.float32, "gu")
    T, F2 = gu.shape
    F = F2 // 2
    h = torch.empty((T, F), dtype=torch.float32, device=gu.device)
    q = torch.empty((T, F), dtype=torch.int8, device=gu.device)
    d = torch.empty((T, F // QK), dtype=torch.float16 if half_scale else torch.float32, device=gu.device)
    _check(load_library().luce_swiglu_q8(gu.data_ptr(), T, F, h.data_ptr(), q.data_ptr(), d.data_ptr(),
                                         1 if half_scale else 0, _stream(stream)))
    return h, q, d


def luce_q8_matvec_batch(wq, wd, aq, ad, y=None, stream=None):
    """q8_0 weights (int8 [N][K], fp16 [N][K/32]) x q8_0 activations -> fp32 [T][N]."""
    import torch
    _need(wq, torch.int8, "wq")
    _need(aq, torch.int8, "aq")
    _need(ad, torch.float32, "ad")
    if wd.dtype not in (torch.float16, torch.int16, torch.uint16):
        raise TypeError("wd: expected fp16 scales")
    N, K = wq.shape
    T = aq.shape[0]
    y = torch.empty((T, N), dtype=torch.float32, device=wq.device) if y is None else y
    _check(load_library().luce_q8_matvec_batch(wq.data_ptr(), wd.data_ptr(), N, K, aq.data_ptr(), ad.data_ptr(),
                                               T, y.data_ptr(), y.stride(0), _stream(stream)))
    return y


MATVEC_AUTO, MATVEC_REGISTER, MATVEC_RING, MATVEC_TENSOR = 0, 1, 2, 3


def luce_q8_matvec_batch_path(wq, wd, aq, ad, path: int, y=None, stream=None):
    """luce_q8_matvec_batch through one named kernel (MATVEC_*); raises LuceError
    (LUCE_EUNSUPPORTED) when that kernel does not serve the shape."""
    import torch
    _need(wq, torch.int8, "wq")
    _need(aq, torch.int8, "aq")
    _need(ad, torch.float32, "ad")
    N, K = wq.shape
    T = aq.shape[0]
    y = torch.empty((T, N), dtype=torch.float32, device=wq.device) if y is None else y
    _check(load_library().luce_q8_matvec_batch_path(wq.data_ptr(), wd.data_ptr(), N, K, aq.data_ptr(), ad.data_ptr(),
                                                    T, y.data_ptr(), y.stride(0), int(path), _stream(stream)))
    return y


def luce_q8_block_dots(wq, aq, stream=None):
    import torch
    N, K = wq.shape
    T = aq.shape[0]
    out = torch.empty((T, N, K // QK), dtype=torch.int32, device=wq.device)
    _check(load_library().luce_q8_block_dots(wq.data_ptr(), N, K, aq.data_ptr(), T, out.data_ptr(), _stream(stream)))
    return out


def luce_rope_posvec(x, pos, theta: float, stream=None):
    """In-place RoPE of fp32 x [T][n_heads][128] at per-row positions pos (int32 [T])."""
    import torch
    _need(x, torch.float32, "x")
    _need(pos, torch.int32, "pos")
    T, nh, D = x.shape
    _check(load_library().luce_rope_posvec(x.data_ptr(), T, nh, D, nh * D, pos.data_ptr(), float(theta),
                                           _stream(stream)))
    return x


@dataclass
class SeqView:
    """A sequence's cache for one layer (fp16 [Hkv][cap][128] K and V) with ``len``
    keys including this step's ``n_q`` rows, which are rows row0.. of q/out."""
    k: object
    v: object
    len: int
    n_q: int = 1
    row0: int = 0

    def c(self) -> SeqViewC:
        Hkv, cap, D = self.k.shape
        return SeqViewC(self.k.data_ptr(), self.v.data_ptr(), self.len, self.n_q, self.row0, cap,
                        self.k.stride(0), self.k.stride(1))


def _views(views: Sequence[SeqView]):
    arr = (SeqViewC * max(1, len(views)))()
    for i, v in enumerate(views):
        arr[i] = v.c()
    return arr


def luce_kv_append(k, v, views: Sequence[SeqView], stream=None):
    """Append fp32 rows k, v ([T][Hkv][128]) as fp16 at each view's positions."""
    import torch
    _need(k, torch.float32, "k")
    _need(v, torch.float32, "v")
    T, Hkv, D = k.shape
    _check(load_library().luce_kv_append(k.data_ptr(), v.data_ptr(), Hkv * D, Hkv, D, _views(views), len(views),
                                         _stream(stream)))


def luce_decode_attn_workspace_size(n_rows: int, Hq: int, D: int, max_len: int) -> int:
    return int(load_library().luce_decode_attn_workspace_size(n_rows, Hq, D, max_len))


def luce_decode_attn_multiseq(q, views: Sequence[SeqView], n_kv_heads: int, scale: float, out=None, ws=None,
                              stream=None):
    """Decode attention of fp32 q [T][Hq][128] against each row's own fp16 cache."""
    import torch
    _need(q, torch.float32, "q")
    T, Hq, D = q.shape
    out = torch.empty_like(q) if out is None else out
    if ws is None:
        max_len = max(v.len for v in views)
        ws = torch.empty(luce_decode_attn_workspace_size(T, Hq, D, max_len), dtype=torch.uint8, device=q.device)
    _check(load_library().luce_decode_attn_multiseq(q.data_ptr(), _views(views), len(views), Hq, n_kv_heads, D,
                                                    float(scale), out.data_ptr(), ws.data_ptr(), ws.numel(),
                                                    _stream(stream)))
    return out


PAGE_KEYS = 128


@dataclass
class PagedView:
    """A sequence's K/V for one layer in pages: pools fp16 [n_pages][Hkv][128][128],
    ``table`` (device int32) the pool page of each 128-key span; ``len`` keys
    including this step's ``n_q`` rows, which are rows row0.. of q/out."""
    k_pool: object
    v_pool: object
    table: object
    len: int
    n_q: int = 1
    row0: int = 0


def luce_decode_attn_paged(q, views: Sequence[PagedView], n_kv_heads: int, scale: float, out=None, ws=None,
                           stream=None):
    """luce_decode_attn_multiseq over paged caches (the same bits as a flat cache)."""
    import torch
    _need(q, torch.float32, "q")
    T, Hq, D = q.shape
    out = torch.empty_like(q) if out is None else out
    if ws is None:
        max_len = max(v.len for v in views)
        ws = torch.empty(luce_decode_attn_workspace_size(T, Hq, D, max_len), dtype=torch.uint8, device=q.device)
    vc = (PagedViewC * len(views))(*[PagedViewC(v.k_pool.data_ptr(), v.v_pool.data_ptr(), v.table.data_ptr(), v.len,
                                                v.n_q, v.row0) for v in views])
    _check(load_library().luce_decode_attn_paged(q.data_ptr(), vc, len(views), Hq, n_kv_heads, D, float(scale),
                                                 out.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)))
    return out


def luce_decode_attn_multiseq_noalloc(q, views: Sequence[SeqView], n_kv_heads: int, scale: float, out=None,
                                      stream=None):
    """luce_decode_attn_multiseq using the library's fixed scratch array instead
    of a workspace, for callers that cannot allocate device memory.  Calls that
    can overlap on the GPU share that array and must be ordered."""
    import torch
    _need(q, torch.float32, "q")
    T, Hq, D = q.shape
    out = torch.empty_like(q) if out is None else out
    _check(load_library().luce_decode_attn_multiseq_noalloc(q.data_ptr(), _views(views), len(views), Hq, n_kv_heads,
                                                            D, float(scale), out.data_ptr(), _stream(stream)))
    return out


# ------------------------------------------------------------ decode step

@dataclass
class LayerTensors:
    attn_norm: object
    wqkv_q: object
    wqkv_d: object
    wo_q: object
    wo_d: object
    ffn_norm: object
    wgu_q: object
    wgu_d: object
    wdown_q: object
    wdown_d: object


class Model:
    """Device weights of a decoder stack plus the C struct that points at them."""

    def __init__(self, layers: List[LayerTensors], hidden: int, n_q_heads: int, n_kv_heads: int, ffn: int,
                 head_dim: int = HEAD_DIM, rms_eps: float = 1e-6, rope_theta: float = 1e6,
                 final_norm=None, head_q=None, head_d=None):
        self.layers = layers
        self.hidden, self.n_q_heads, self.n_kv_heads, self.ffn, self.head_dim = hidden, n_q_heads, n_kv_heads, ffn, head_dim
        self.rms_eps, self.rope_theta = rms_eps, rope_theta
        self.final_norm, self.head_q, self.head_d = final_norm, head_q, head_d
        self.vocab = 0 if head_q is None else head_q.shape[0]
        self._layers_c = (LayerC * max(1, len(layers)))()
        for i, L in enumerate(layers):
            self._layers_c[i] = LayerC(*[getattr(L, n).data_ptr() for n, _ in LayerC._fields_])
        self.c = ModelC(len(layers), hidden, n_q_heads, n_kv_heads, head_dim, ffn, self.vocab, rms_eps, rope_theta,
                        self._layers_c, _ptr(final_norm), _ptr(head_q), _ptr(head_d))

    def layout(self, n_rows: int, max_ctx: int) -> dict:
        out = StepLayoutC()
        _check(load_library().luce_decode_step_layout(ctypes.byref(self.c), n_rows, max_ctx, ctypes.byref(out)))
        return {n: getattr(out, n) for n in _LAYOUT_FIELDS}

    def workspace(self, n_rows: int, max_ctx: int, device="cuda"):
        import torch
        return torch.empty(self.layout(n_rows, max_ctx)["total"], dtype=torch.uint8, device=device)

    def tree_layout(self, n_rows: int, max_ctx: int) -> dict:
        """The workspace layout of luce_decode_step_tree for prefixes of at most max_ctx keys."""
        out = StepLayoutC()
        _check(load_library().luce_decode_step_tree_layout(ctypes.byref(self.c), n_rows, max_ctx, ctypes.byref(out)))
        return {n: getattr(out, n) for n in _LAYOUT_FIELDS}

    def tree_workspace(self, n_rows: int, max_ctx: int, device="cuda"):
        import torch
        return torch.empty(self.tree_layout(n_rows, max_ctx)["total"], dtype=torch.uint8, device=device)


@dataclass
class Slot:
    """A sequence's K/V cache for every layer: fp16 [n_layers][Hkv][cap][128] each,
    with ``len`` tokens already cached."""
    k: object
    v: object
    len: int

    @property
    def cap(self) -> int:
        return self.k.shape[2]


class _TableMirror:
    """A slot whose host int32 ``table`` may be replaced or edited between calls;
    ``table_dev`` is its copy on the device."""

    def __post_init__(self):
        self._array = self._mirrored = None
        self._captured = []
        self.mirror_table()
        self.table = self._array

    def mirror_table(self, stream=None):
        """Bring table_dev up to date for a call on ``stream`` and return the host
        table.  A changed table gets a new device copy (calls under way and
        captured ones keep theirs), which cannot be made during a capture."""
        return _mirror_tables([self], stream)[0]

    def _mirror(self, stream, now, capturing):
        import numpy as np
        import torch
        table = self.table
        if table is not self._array:  # (an int32 array stays itself, anything else is copied at every call)
            table = self._array = np.ascontiguousarray(table, dtype=np.int32)
            self._host = table.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))  # (1.5 us)
        contents = table.tobytes()
        if contents != self._mirrored:
            if capturing:
                raise RuntimeError("the slot's table changed: call mirror_table() before the capture")
            self.table_dev, self._mirrored, self._home = torch.from_numpy(table.copy()).to(self.k_pool.device), contents, now
        if capturing:
            self._captured.append(self.table_dev)
        elif stream != self._home:
            self.table_dev.record_stream(torch.cuda.ExternalStream(stream, device=self.k_pool.device))
        return table


def _mirror_tables(slots, stream):
    """The slots' host tables, their device copies brought up to date for a call on ``stream``."""
    import torch
    device = slots[0].k_pool.device if slots else None
    if device is None or device.type != "cuda":
        return [s._mirror(None, None, False) for s in slots]
    now = torch._C._cuda_getCurrentRawStream(device.index)
    at = now if stream is None else stream.cuda_stream
    if at == now:
        capturing = torch.cuda.is_current_stream_capturing()
    else:
        with torch.cuda.stream(stream):
            capturing = torch.cuda.is_current_stream_capturing()
    return [s._mirror(at, now, capturing) for s in slots]


@dataclass
class PagedSlot(_TableMirror):
    """A slot in pages of 128 tokens: pools fp16 [n_pages][n_layers][Hkv][128][128];
    ``table`` lists the pool page of each 128-token span (a host int32 array,
    mirrored on the device; each call takes what it holds by then)."""
    k_pool: object
    v_pool: object
    table: object  # numpy int32
    len: int


def luce_decode_step_paged(model: "Model", slots: Sequence[PagedSlot], rows_per_slot: Sequence[int], x, ws,
                           logits=None, argmax=None, stream=None):
    """luce_decode_step over paged slots (the same bits as flat caches)."""
    import torch
    _need(x, torch.float32, "x")
    n = len(slots)
    sc = (PagedSlotC * max(1, n))()
    for i, (s, t) in enumerate(zip(slots, _mirror_tables(slots, stream))):
        sc[i] = PagedSlotC(s.k_pool.data_ptr(), s.v_pool.data_ptr(), s.table_dev.data_ptr(),
                           s._host, t.size, s.k_pool.shape[0], s.len)
    rows = (ctypes.c_int32 * max(1, n))(*rows_per_slot)
    _check(load_library().luce_decode_step_paged(ctypes.byref(model.c), sc, rows, n, x.data_ptr(), _ptr(logits),
                                                 _ptr(argmax), ws.data_ptr(), ws.numel(), _stream(stream)))
    return x


def luce_decode_step(model: Model, slots: Sequence[Slot], rows_per_slot: Sequence[int], x, ws,
                     logits=None, argmax=None, stream=None):
    """One batched decode step (all layers, optional head) over the given slots.
    x: fp32 [T][hidden] in/out.  The slots' caches get this step's K/V rows."""
    import torch
    _need(x, torch.float32, "x")
    n = len(slots)
    sc = (SlotC * max(1, n))()
    for i, s in enumerate(slots):
        sc[i] = SlotC(s.k.data_ptr(), s.v.data_ptr(), s.len, s.cap)
    rows = (ctypes.c_int32 * max(1, n))(*rows_per_slot)
    _check(load_library().luce_decode_step(ctypes.byref(model.c), sc, rows, n, x.data_ptr(), _ptr(logits),
                                           _ptr(argmax), ws.data_ptr(), ws.numel(), _stream(stream)))
    return x


def luce_decode_step_host(model: Model, slots: Sequence[Slot], rows_per_slot: Sequence[int], x_in, x, ws,
                          x_out=None, logits=None, argmax=None, argmax_out=None, stream=None):
    """luce_decode_step with host rows: x_in (CPU fp32 [T][hidden], ideally
    pinned) is copied to x (device) on the stream, the step runs, and x (and
    argmax) are copied back to x_out (and argmax_out) when given.  Nothing
    waits: synchronise the stream before reading x_out."""
    import torch
    _need(x, torch.float32, "x")
    if x_in.device.type != "cpu" or x_in.dtype != torch.float32 or not x_in.is_contiguous():
        raise TypeError("x_in: expected a contiguous CPU float32 tensor")
    if x_in.shape != x.shape or (x_out is not None and x_out.shape != x.shape):
        raise ValueError("x_in, x and x_out must have the same shape")
    n = len(slots)
    sc = (SlotC * max(1, n))()
    for i, s in enumerate(slots):
        sc[i] = SlotC(s.k.data_ptr(), s.v.data_ptr(), s.len, s.cap)
    rows = (ctypes.c_int32 * max(1, n))(*rows_per_slot)
    _check(load_library().luce_decode_step_host(ctypes.byref(model.c), sc, rows, n, x_in.data_ptr(), x.data_ptr(),
                                                _ptr(x_out), _ptr(logits), _ptr(argmax), _ptr(argmax_out),
                                                ws.data_ptr(), ws.numel(), _stream(stream)))
    return x_out


class DeviceStep:
    """luce_decode_step with its arguments marshalled once, for repeated steps
    over the same slots and buffers (x on the device): each call copies the
    slots' current ``len`` into the prepared slot array and makes the C call
    (nothing else is re-checked).  The stream is the one given, or the current
    stream at construction."""

    def __init__(self, model: Model, slots: Sequence[Slot], rows_per_slot: Sequence[int], x, ws, logits=None,
                 argmax=None, stream=None):
        import torch
        _need(x, torch.float32, "x")
        self.slots = list(slots)
        n = len(self.slots)
        self._sc = (SlotC * max(1, n))()
        for i, s in enumerate(self.slots):
            self._sc[i] = SlotC(s.k.data_ptr(), s.v.data_ptr(), s.len, s.cap)
        self._rows = (ctypes.c_int32 * max(1, n))(*rows_per_slot)
        self._keep = (model, x, ws, logits, argmax)
        self._fn = load_library().luce_decode_step
        self._args = (ctypes.byref(model.c), self._sc, self._rows, n, x.data_ptr(), _ptr(logits), _ptr(argmax),
                      ws.data_ptr(), ws.numel(), _stream(stream))

    def __call__(self):
        sc = self._sc
        for i, s in enumerate(self.slots):
            sc[i].len = s.len
        _check(self._fn(*self._args))


class HostStep:
    """luce_decode_step_host with its arguments marshalled once, for repeated
    steps over the same slots and buffers: each call copies the slots' current
    ``len`` into the prepared slot array and makes the C call (nothing else is
    re-checked).  The stream is the one given, or the current stream at
    construction.  Synchronise the stream before reading x_out."""

    def __init__(self, model: Model, slots: Sequence[Slot], rows_per_slot: Sequence[int], x_in, x, ws,
                 x_out=None, logits=None, argmax=None, argmax_out=None, stream=None):
        import torch
        _need(x, torch.float32, "x")
        if x_in.device.type != "cpu" or x_in.dtype != torch.float32 or not x_in.is_contiguous():
            raise TypeError("x_in: expected a contiguous CPU float32 tensor")
        if x_in.shape != x.shape or (x_out is not None and x_out.shape != x.shape):
            raise ValueError("x_in, x and x_out must have the same shape")
        self.slots = list(slots)
        n = len(self.slots)
        self._sc = (SlotC * max(1, n))()
        for i, s in enumerate(self.slots):
            self._sc[i] = SlotC(s.k.data_ptr(), s.v.data_ptr(), s.len, s.cap)
        self._rows = (ctypes.c_int32 * max(1, n))(*rows_per_slot)
        self._keep = (model, x_in, x, ws, x_out, logits, argmax, argmax_out)
        self._fn = load_library().luce_decode_step_host
        self._args = (ctypes.byref(model.c), self._sc, self._rows, n, x_in.data_ptr(), x.data_ptr(), _ptr(x_out),
                      _ptr(logits), _ptr(argmax), _ptr(argmax_out), ws.data_ptr(), ws.numel(), _stream(stream))

    def __call__(self):
        sc = self._sc
        for i, s in enumerate(self.slots):
            sc[i].len = s.len
        _check(self._fn(*self._args))


class StepGraph:
    """luce_step_graph: the step of HostStep (same arguments) kept as one CUDA
    graph.  Each call passes the slots' current ``len`` to luce_step_graph_run,
    which refreshes the graph's changed nodes (or captures it anew) and
    launches it on the stream given at construction (else the current stream).
    Synchronise the stream before reading x_out.  close() (or garbage
    collection) releases the graph once the stream has finished its runs."""

    def __init__(self, model: Model, slots: Sequence[Slot], rows_per_slot: Sequence[int], x_in, x, ws,
                 x_out=None, logits=None, argmax=None, argmax_out=None, stream=None):
        import torch
        _need(x, torch.float32, "x")
        if x_in.device.type != "cpu" or x_in.dtype != torch.float32 or not x_in.is_contiguous():
            raise TypeError("x_in: expected a contiguous CPU float32 tensor")
        if x_in.shape != x.shape or (x_out is not None and x_out.shape != x.shape):
            raise ValueError("x_in, x and x_out must have the same shape")
        self.slots = list(slots)
        n = len(self.slots)
        sc = (SlotC * max(1, n))()
        for i, s in enumerate(self.slots):
            sc[i] = SlotC(s.k.data_ptr(), s.v.data_ptr(), s.len, s.cap)
        rows = (ctypes.c_int32 * max(1, n))(*rows_per_slot)
        self._lens = (ctypes.c_int32 * max(1, n))()
        self._keep = (model, x_in, x, ws, x_out, logits, argmax, argmax_out)
        self._lib = load_library()
        self._stream = _stream(stream)
        h = ctypes.c_void_p()
        _check(self._lib.luce_step_graph_create(ctypes.byref(model.c), sc, rows, n, x_in.data_ptr(), x.data_ptr(),
                                                _ptr(x_out), _ptr(logits), _ptr(argmax), _ptr(argmax_out),
                                                ws.data_ptr(), ws.numel(), ctypes.byref(h)))
        self._h = h

    def __call__(self):
        lens = self._lens
        for i, s in enumerate(self.slots):
            lens[i] = s.len
        _check(self._lib.luce_step_graph_run(self._h, lens, self._stream))

    def stats(self) -> dict:
        """Captures and node refreshes so far, and the graph's kernel nodes."""
        c, u, k = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int32()
        _check(self._lib.luce_step_graph_stats(self._h, ctypes.byref(c), ctypes.byref(u), ctypes.byref(k)))
        return {"captures": c.value, "node_updates": u.value, "kernels": k.value}

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            self._lib.luce_step_graph_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------------------ draft trees and eviction

@dataclass
class TreeView:
    """A slot's tree of drafted tokens over its cache for one layer (fp16
    [Hkv][cap][128] K and V): ``len`` prefix keys, node j's rows at cache
    position len + j and at row row0 + j of q/out, ``parent[j]`` in [-1, j)
    (-1: follows the prefix).  An int n instead of a list is the chain of n."""
    k: object
    v: object
    len: int
    parent: object = 1
    row0: int = 0


@dataclass
class PagedTreeView:
    """The same over pools fp16 [n_pages][Hkv][128][128] (or a layer pool[:, l] of
    pools [n_pages][n_layers][Hkv][128][128]) and a device int32 ``table`` of
    the pool page of each 128-key span."""
    k_pool: object
    v_pool: object
    table: object
    len: int
    parent: object = 1
    row0: int = 0


@dataclass
class TreeSlot:
    """A slot of luce_decode_step_tree: its K/V cache for every layer (fp16
    [n_layers][Hkv][cap][128]), ``len`` keys cached, ``pos0`` the position of a
    node that follows them (default len), ``parent`` as in TreeView."""
    k: object
    v: object
    len: int
    parent: object = 1
    pos0: Optional[int] = None


@dataclass
class PagedTreeSlot(_TableMirror):
    """The same in pages of 128 tokens: pools fp16 [n_pages][n_layers][Hkv][128][128]
    and ``table``, the pool page of each 128-token span (a host int32 array,
    mirrored on the device as table_dev; each call takes what it holds by then)."""
    k_pool: object
    v_pool: object
    table: object  # numpy int32
    len: int
    parent: object = 1
    pos0: Optional[int] = None


@dataclass
class CommitSlot:
    """A slot's cache of every layer (fp16 [n_layers][Hkv][cap][128]) whose tree's
    nodes ``path`` (ascending) were accepted; ``row0`` is the score row of node
    0, ``acc`` (fp32) and ``pos`` (int32), [n_layers][Hkv][cap], its keys'
    accumulated weights and positions, ``pos0`` the first accepted node's
    (default len, as in TreeSlot)."""
    k: object
    v: object
    len: int
    path: object
    row0: int = 0
    acc: object = None
    pos: object = None
    pos0: Optional[int] = None


@dataclass
class PagedCommitSlot:
    """The same over pools fp16 [n_pages][n_layers][Hkv][128][128] and a host
    int32 ``table``; acc and pos are [n_layers][Hkv][keys]."""
    k_pool: object
    v_pool: object
    table: object  # numpy int32
    len: int
    path: object
    row0: int = 0
    acc: object = None
    pos: object = None
    pos0: Optional[int] = None


@dataclass
class EvictSlot:
    """A slot's cache with its keys' accumulated weights and positions (as in
    CommitSlot), to be cut to ``budget`` keys; keys at positions < sinks and
    >= next_pos - recent stay (``recent`` needs ``next_pos``, the position of
    the slot's next token); acc_out and pos_out default to acc and pos
    themselves."""
    k: object
    v: object
    acc: object
    pos: object
    len: int
    budget: int
    sinks: int = 0
    recent: int = 0
    next_pos: Optional[int] = None
    acc_out: object = None
    pos_out: object = None


@dataclass
class PagedEvictSlot:
    """The same over pools fp16 [n_pages][n_layers][Hkv][128][128] and a device
    int32 ``table``; the pages of indexes >= budget are free afterwards."""
    k_pool: object
    v_pool: object
    table: object
    acc: object
    pos: object
    len: int
    budget: int
    sinks: int = 0
    recent: int = 0
    next_pos: Optional[int] = None
    acc_out: object = None
    pos_out: object = None


def _tree(parent):
    """(n_nodes, host int32 array or None) of a parent list or a chain's length."""
    if isinstance(parent, int):
        return parent, None
    p = [int(v) for v in parent]
    return len(p), (ctypes.c_int32 * max(1, len(p)))(*p)


def _same_device(first, *tensors):
    for t in tensors:
        if t is not None and t.device != first.device:
            raise ValueError(f"tensors on {first.device} and {t.device}: one call works on one device")


def _kv_pair(k, v, rank, name):
    import torch
    for t, w in ((k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float16 or not t.is_cuda:
            raise TypeError(f"{name}.{w}: expected a CUDA float16 tensor")
        if t.dim() != rank or t.shape[-1] != HEAD_DIM or t.stride(-1) != 1:
            raise ValueError(f"{name}.{w}: expected {rank} dims, the last of {HEAD_DIM} contiguous values")
    if k.shape != v.shape or k.stride() != v.stride():
        raise ValueError(f"{name}: k and v must have the same shape and strides")


class _Prepared:
    """A C call with its arguments marshalled once.  The call goes to the stream
    given at construction, else to the device's current stream at each call;
    memory that the object allocated itself belongs to the stream of its
    construction and is kept from reuse until a call on another one is done."""

    _owned = ()
    _home = None
    _lent = frozenset()

    def _bind(self, name, args, device, stream, keep):
        """The C function and its arguments but the stream, as C values: converting
        them at every call takes ctypes 0.7 us."""
        import torch
        lib = load_library()
        self._fn = lib[name]  # (a function object of its own, without argument types)
        self._args = tuple(v if isinstance(v, ctypes.Array) else t(v) for t, v in zip(getattr(lib, name).argtypes, args))
        self._index, self._keep = device.index, (stream, keep)
        self._stream = None if stream is None else stream.cuda_stream
        self._at = (None, None)  # the last call's stream, also as a C value
        self._device_now, self._stream_now = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream

    def _allocate(self, shape, dtype, device, stream):
        import torch
        if stream is None:
            t = torch.empty(shape, dtype=dtype, device=device)
            home = torch._C._cuda_getCurrentRawStream(device.index)
        else:
            with torch.cuda.stream(stream):
                t = torch.empty(shape, dtype=dtype, device=device)
            home = stream.cuda_stream
        self._home = home if self._home in (None, home) else -1  # (of several streams: every call lends)
        self._owned, self._lent, self._at = self._owned + (t,), frozenset(), (None, None)
        return t

    def _lend(self, stream):
        """The object's own memory is used on another stream than its own."""
        import torch
        for t in self._owned:
            t.record_stream(torch.cuda.ExternalStream(stream, device=t.device))
        self._lent = self._lent | {stream}

    def _call(self):
        s = self._stream if self._stream is not None else self._stream_now(self._index)
        at = self._at  # (read once: another thread's call may put its own there)
        if s != at[0]:
            if s != self._home and self._owned and s not in self._lent:
                self._lend(s)
            at = self._at = (s, ctypes.c_void_p(s))
        if self._device_now() == self._index:
            rc = self._fn(*self._args, at[1])
        else:
            import torch
            with torch.cuda.device(self._index):
                rc = self._fn(*self._args, at[1])
        if rc != LUCE_OK:
            _check(rc)


_NOTHING = (None,) * 8  # what no view holds


class TreeAttention(_Prepared):
    """luce_tree_attn (or luce_tree_attn_paged, for PagedTreeViews) with its
    arguments marshalled once, for repeated calls over the same buffers: q fp32
    [T][Hq][128], ``out`` as q, ``scores`` fp32 [T][Hq][lds] and ``stats`` fp32
    [T][Hq][2] when given.  Each call takes what the views hold by then (another
    tree, other rows of the T, a longer cache) and checks tensors that were
    replaced.  The object owns its workspace (sized for the views' capacity)
    unless one is given, so calls of one object must not overlap on the GPU, and
    a graph that captured a call needs the object and the call's caches alive."""

    def __init__(self, q, views, n_kv_heads: int, scale: float, out=None, scores=None, stats=None, ws=None, stream=None):
        import torch
        _need(q, torch.float32, "q")
        if q.dim() != 3:
            raise ValueError("q: expected [T][Hq][128]")
        T, Hq, D = q.shape
        self.views = list(views)
        if not self.views:
            raise ValueError("views: expected at least one")
        paged = isinstance(self.views[0], PagedTreeView)
        if not all(isinstance(v, PagedTreeView if paged else TreeView) for v in self.views):
            raise TypeError("views: expected TreeViews or PagedTreeViews, of one kind")
        self.out = self._allocate(q.shape, torch.float32, q.device, stream) if out is None else out
        _need(self.out, torch.float32, "out")
        if self.out.shape != q.shape:
            raise ValueError("out: expected q's shape")
        lds = 0
        if scores is not None:
            _need(scores, torch.float32, "scores")
            if scores.dim() != 3 or scores.shape[:2] != q.shape[:2]:
                raise ValueError("scores: expected [T][Hq][lds]")
            lds = scores.shape[2]
        if stats is not None:
            _need(stats, torch.float32, "stats")
            if stats.shape != (T, Hq, 2):
                raise ValueError("stats: expected [T][Hq][2]")
        n = len(self.views)
        self._paged, self._q, self._shape = paged, q, (T, Hq, int(n_kv_heads), D)
        self._vc = ((PagedTreeViewC if paged else TreeViewC) * n)()
        self._items, self._caps, self._seen = [self._vc[i] for i in range(n)], [0] * n, [None] * n
        for i, v in enumerate(self.views):
            self._take(i, v)
        self._check_rows()
        _same_device(q, self.out, scores, stats, ws)
        self._own_ws = ws is None
        if ws is None:
            ws = self._allocate((self._ws_bytes(),), torch.uint8, q.device, stream)
        _need(ws, torch.uint8, "ws")
        args = (q.data_ptr(), self._vc, n, Hq, int(n_kv_heads), D, float(scale), self.out.data_ptr(), _ptr(scores), lds,
                _ptr(stats), ws.data_ptr(), ws.numel())
        self._ws_args = len(args) - 2
        self._bind("luce_tree_attn_paged" if paged else "luce_tree_attn", args, q.device, stream, (q, scores, stats, ws))

    def _take(self, i, v):
        """View i's tensors, then its tree."""
        import torch
        c, Hkv = self._items[i], self._shape[2]
        self._seen[i] = (i, v, *_NOTHING)  # (until all is checked)
        if self._paged:
            _kv_pair(v.k_pool, v.v_pool, 4, f"views[{i}]")
            _need(v.table, torch.int32, f"views[{i}].table")
            page, stride = (Hkv, PAGE_KEYS, HEAD_DIM), v.k_pool.stride()
            if v.k_pool.shape[1:] != page or stride[2] != HEAD_DIM or (Hkv > 1 and stride[1] != PAGE_KEYS * HEAD_DIM):
                raise ValueError(f"views[{i}]: expected pools [n_pages][{Hkv}][128][128], each page contiguous")
            c.page_stride = stride[0] if v.k_pool.shape[0] > 1 else 0
            _same_device(self._q, v.k_pool, v.v_pool, v.table)
            self._caps[i] = min(v.table.numel() * PAGE_KEYS, MAX_KEYS)
            c.k_pool, c.v_pool, c.table, c.n_pages = v.k_pool.data_ptr(), v.v_pool.data_ptr(), v.table.data_ptr(), v.k_pool.shape[0]
            self._take_tree(i, v, (v.k_pool, v.v_pool, v.table))
        else:
            _kv_pair(v.k, v.v, 3, f"views[{i}]")
            if v.k.shape[0] != Hkv:
                raise ValueError(f"views[{i}]: {v.k.shape[0]} heads, expected {Hkv}")
            _same_device(self._q, v.k, v.v)
            self._caps[i] = min(v.k.shape[1], MAX_KEYS)
            c.k, c.v, c.cap = v.k.data_ptr(), v.v.data_ptr(), v.k.shape[1]
            c.head_stride, c.tok_stride = v.k.stride(0), v.k.stride(1)
            self._take_tree(i, v, (v.k, v.v, None))

    def _take_tree(self, i, v, tensors):
        """View i's tree, rows and length."""
        c, seen = self._items[i], self._seen[i]
        # the tree as given, to tell whether it changed (one that has no == of its own is taken at every call)
        kind = v.parent.__class__ if v.parent.__class__ in (int, list, tuple) else None
        same = kind is not None and kind is seen[7] and v.parent == seen[8]
        nn, par, parent = (c.n_nodes, seen[9], seen[8]) if same else (*_tree(v.parent), list(v.parent) if kind is list else v.parent)
        if v.len + nn > self._caps[i]:
            raise ValueError(f"len {v.len} and the tree exceed the cache")
        if not same or v.row0 != seen[5]:
            self._rows = None
        c.len, c.n_nodes, c.row0, c.parent = v.len, nn, v.row0, par
        self._seen[i] = (i, v, *tensors, v.row0, v.len, kind, parent, par)

    def _check_rows(self):
        rows, T = max(c.row0 + c.n_nodes for c in self._items), self._shape[0]
        if rows != T:
            raise ValueError(f"q has {T} rows, the views name {rows}")
        self._rows = rows

    def _ws_bytes(self):
        return max(256, luce_tree_attn_workspace_size(*self._shape, max(0, *(cap - c.n_nodes for cap, c in zip(self._caps, self._items)))))

    def _retake(self, i, v):
        """View i changed: more room is asked for where its cache grew."""
        import torch
        seen, at = self._seen[i], self._ws_args
        if (v.k_pool is seen[2] and v.v_pool is seen[3] and v.table is seen[4]) if self._paged else (v.k is seen[2] and v.v is seen[3]):
            self._take_tree(i, v, seen[2:5])
            return
        self._take(i, v)
        if self._own_ws and self._ws_bytes() > self._args[at + 1].value:
            ws = self._allocate((self._ws_bytes(),), torch.uint8, self._q.device, self._keep[0])
            self._args = (*self._args[:at], ctypes.c_void_p(ws.data_ptr()), ctypes.c_size_t(ws.numel()))

    def __call__(self):
        if self._paged:
            for i, v, k, vv, table, row0, length, kind, parent, _ in self._seen:
                if v.k_pool is not k or v.v_pool is not vv or v.table is not table or v.row0 != row0 or v.len != length or \
                        v.parent.__class__ is not kind or v.parent != parent:
                    self._retake(i, v)
        else:
            for i, v, k, vv, _, row0, length, kind, parent, _ in self._seen:
                if v.k is not k or v.v is not vv or v.row0 != row0 or v.len != length or \
                        v.parent.__class__ is not kind or v.parent != parent:
                    self._retake(i, v)
        if self._rows is None:
            self._check_rows()
        self._call()
        return self.out


def luce_tree_attn_workspace_size(n_rows: int, Hq: int, Hkv: int, D: int, max_len: int) -> int:
    return int(load_library().luce_tree_attn_workspace_size(n_rows, Hq, Hkv, D, max_len))


def luce_tree_attn(q, views: Sequence[TreeView], n_kv_heads: int, scale: float, out=None, scores=None, stats=None,
                   ws=None, stream=None):
    """Attention of the views' draft trees: fp32 q [T][Hq][128] against each
    node's prefix, ancestors and itself.  Optional ``scores`` [T][Hq][lds] and
    ``stats`` [T][Hq][2] receive the scaled scores and (max, sum)."""
    return TreeAttention(q, views, n_kv_heads, scale, out, scores, stats, ws, stream)()


def luce_tree_attn_paged(q, views: Sequence[PagedTreeView], n_kv_heads: int, scale: float, out=None, scores=None,
                         stats=None, ws=None, stream=None):
    """luce_tree_attn over paged caches (the same bits as a flat cache)."""
    return TreeAttention(q, views, n_kv_heads, scale, out, scores, stats, ws, stream)()


def luce_decode_step_tree(model: "Model", slots: Sequence[TreeSlot], x, ws, logits=None, argmax=None, scores=None,
                          stats=None, stream=None):
    """One batched decode step over the slots' draft trees (luce_decode_step for
    rows that are nodes of trees, or whose caches had keys evicted).  x: fp32
    [T][hidden] in/out, a slot's nodes in consecutive rows; scores
    [n_layers][T][Hq][lds] and stats [n_layers][T][Hq][2] are what
    luce_tree_commit takes."""
    import torch
    _need(x, torch.float32, "x")
    n, T, L, Hkv = len(slots), x.shape[0], len(model.layers), model.n_kv_heads
    paged = n > 0 and isinstance(slots[0], PagedTreeSlot)
    if not all(isinstance(s, PagedTreeSlot if paged else TreeSlot) for s in slots):
        raise TypeError("slots: expected TreeSlots or PagedTreeSlots, of one kind")
    trees = [_tree(s.parent) for s in slots]
    if sum(t[0] for t in trees) != T:
        raise ValueError(f"x has {T} rows, the trees {sum(t[0] for t in trees)}")
    if x.shape != (T, model.hidden):
        raise ValueError(f"x: expected [T][{model.hidden}]")
    if logits is not None:
        _need(logits, torch.float32, "logits")
        if logits.numel() < T * model.vocab:
            raise ValueError(f"logits: expected [{T}][{model.vocab}]")
    if argmax is not None:
        _need(argmax, torch.int32, "argmax")
        if argmax.numel() < T:
            raise ValueError(f"argmax: expected [{T}]")
    _need(ws, torch.uint8, "ws")
    sc = ((PagedTreeSlotC if paged else TreeSlotC) * max(1, n))()
    tables = _mirror_tables(slots, stream) if paged else [None] * n
    for i, (s, (nn, par), t) in enumerate(zip(slots, trees, tables)):
        pos0 = s.len if s.pos0 is None else s.pos0
        if paged:
            _pools(s.k_pool, s.v_pool, L, Hkv, f"slots[{i}]")
            _same_device(x, s.k_pool, s.v_pool, s.table_dev)
            sc[i] = PagedTreeSlotC(s.k_pool.data_ptr(), s.v_pool.data_ptr(), s.table_dev.data_ptr(),
                                   s._host, t.size, s.k_pool.shape[0], s.len, pos0, nn, par)
        else:
            _caches(s.k, s.v, L, Hkv, f"slots[{i}]")
            _same_device(x, s.k, s.v)
            sc[i] = TreeSlotC(s.k.data_ptr(), s.v.data_ptr(), s.len, s.k.shape[2], pos0, nn, par)
    lds = 0
    if scores is not None:
        _need(scores, torch.float32, "scores")
        lds = scores.shape[-1]
        if scores.numel() != len(model.layers) * T * model.n_q_heads * lds:
            raise ValueError("scores: expected [n_layers][T][Hq][lds]")
    if stats is not None:
        _need(stats, torch.float32, "stats")
        if stats.numel() != len(model.layers) * T * model.n_q_heads * 2:
            raise ValueError("stats: expected [n_layers][T][Hq][2]")
    _same_device(x, ws, logits, argmax, scores, stats)
    lib = load_library()
    fn = lib.luce_decode_step_tree_paged if paged else lib.luce_decode_step_tree
    with torch.cuda.device(x.device):
        _check(fn(ctypes.byref(model.c), sc, n, x.data_ptr(), _ptr(logits), _ptr(argmax), _ptr(scores), lds, _ptr(stats),
                  ws.data_ptr(), ws.numel(), _stream(stream)))
    return x


def _caches(k, v, L, Hkv, name):
    import torch
    _kv_pair(k, v, 4, name)
    _need(k, torch.float16, name + ".k")
    _need(v, torch.float16, name + ".v")
    if k.shape[:2] != (L, Hkv):
        raise ValueError(f"{name}: expected caches [{L} layers][{Hkv} KV heads][cap][128]")


def _pools(k, v, L, Hkv, name):
    import torch
    _kv_pair(k, v, 5, name)
    _need(k, torch.float16, name + ".k_pool")
    _need(v, torch.float16, name + ".v_pool")
    if k.shape[1:4] != (L, Hkv, PAGE_KEYS):
        raise ValueError(f"{name}: expected pools [n_pages][{L} layers][{Hkv} KV heads][128][128]")


def _state(t, dtype, L, Hkv, cap, name):
    _need(t, dtype, name)
    if t.dim() != 3 or t.shape[:2] != (L, Hkv) or (cap is not None and t.shape[2] != cap):
        raise ValueError(f"{name}: expected [{L} layers][{Hkv} KV heads][cap]")


def _kind(slots, flat, paged):
    """Whether the slots are paged ones; they are all of one kind."""
    if not slots:
        raise ValueError("slots: expected at least one")
    is_paged = isinstance(slots[0], paged)
    if not all(isinstance(s, paged if is_paged else flat) for s in slots):
        raise TypeError(f"slots: expected {flat.__name__}s or {paged.__name__}s, of one kind")
    return is_paged


class TreeCommit(_Prepared):
    """luce_tree_commit (or luce_tree_commit_paged, for PagedCommitSlots) with its
    arguments marshalled once: each call takes what the slots hold by then, and
    checks tensors that were replaced.  ``scores`` [n_layers][n_rows][Hq][lds] and
    ``stats`` [n_layers][n_rows][Hq][2] (the n_layers dimension may be left out
    for one layer) are what luce_tree_attn gave."""

    def __init__(self, slots: Sequence[CommitSlot], n_q_heads: int, scores=None, stats=None, stream=None):
        import torch
        self.slots = list(slots)
        self._paged = paged = _kind(self.slots, CommitSlot, PagedCommitSlot)
        first = self.slots[0].k_pool if paged else self.slots[0].k
        L, Hkv = first.shape[1:3] if paged else first.shape[:2]
        n_rows = lds = 0
        if scores is not None:
            _need(scores, torch.float32, "scores")
            _need(stats, torch.float32, "stats")
            n_rows, hq, lds = scores.shape[-3:]
            if hq != n_q_heads or scores.numel() != L * n_rows * hq * lds or stats.numel() != L * n_rows * hq * 2:
                raise ValueError("scores, stats: expected [n_layers][n_rows][Hq][lds] and [n_layers][n_rows][Hq][2]")
        n = len(self.slots)
        self._first, self._heads = first, (L, Hkv)
        _same_device(first, scores, stats)
        self._sc = ((PagedCommitSlotC if paged else CommitSlotC) * n)()
        self._items, self._seen = [self._sc[i] for i in range(n)], [None] * n
        self._now, self._arrays, self._tables = [None] * n, [None] * n, [None] * n
        for i, s in enumerate(self.slots):
            self._take(i, s)
        args = (self._sc, n, L, int(n_q_heads), Hkv, HEAD_DIM, _ptr(scores), n_rows, lds, _ptr(stats))
        self._bind("luce_tree_commit_paged" if paged else "luce_tree_commit", args, first.device, stream, (scores, stats))

    def _take(self, i, s):
        """Slot i's tensors."""
        import torch
        (L, Hkv), c = self._heads, self._items[i]
        if self._paged:
            _pools(s.k_pool, s.v_pool, L, Hkv, f"slots[{i}]")
            k, v, cap = s.k_pool, s.v_pool, next((t.shape[-1] for t in (s.acc, s.pos) if t is not None), MAX_KEYS)
        else:
            _caches(s.k, s.v, L, Hkv, f"slots[{i}]")
            k, v, cap = s.k, s.v, s.k.shape[2]
        if s.acc is not None:
            _state(s.acc, torch.float32, L, Hkv, cap, f"slots[{i}].acc")
        if s.pos is not None:
            _state(s.pos, torch.int32, L, Hkv, cap, f"slots[{i}].pos")
        _same_device(self._first, k, v, s.acc, s.pos)
        if self._paged:
            c.k_pool, c.v_pool, c.n_pages = k.data_ptr(), v.data_ptr(), k.shape[0]
        else:
            c.k, c.v = k.data_ptr(), v.data_ptr()
        c.cap, c.acc, c.pos = cap, _ptr(s.acc), _ptr(s.pos)
        self._seen[i] = (i, s, k, v, s.acc, s.pos)

    def _take_path(self, i, s):
        path, c = list(s.path), self._items[i]
        self._arrays[i] = (ctypes.c_int32 * max(1, len(path)))(*path)
        c.len, c.row0, c.path, c.n_path = s.len, s.row0, self._arrays[i], len(path)
        c.pos0 = s.len if s.pos0 is None else s.pos0
        self._now[i] = (s.len, s.row0, s.pos0, *path)

    def _take_table(self, i, s):
        import numpy as np
        t = np.ascontiguousarray(s.table, dtype=np.int32)
        self._tables[i] = t  # (an int32 array is read where it lies, anything else copied at every call)
        self._items[i].table_host = t.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
        self._items[i].n_table = t.size

    def __call__(self):
        if self._paged:
            for i, s, k, v, acc, pos in self._seen:
                if s.k_pool is not k or s.v_pool is not v or s.acc is not acc or s.pos is not pos:
                    self._take(i, s)
                if s.table is not self._tables[i]:
                    self._take_table(i, s)
                if (s.len, s.row0, s.pos0, *s.path) != self._now[i]:
                    self._take_path(i, s)
        else:
            for i, s, k, v, acc, pos in self._seen:
                if s.k is not k or s.v is not v or s.acc is not acc or s.pos is not pos:
                    self._take(i, s)
                if (s.len, s.row0, s.pos0, *s.path) != self._now[i]:
                    self._take_path(i, s)
        self._call()


def luce_tree_commit(slots: Sequence[CommitSlot], n_q_heads: int, scores=None, stats=None, stream=None):
    """Make the accepted paths of verified trees the slots' next keys: their K/V
    rows move to len, len + 1, ..; acc and pos follow where given.  The caller
    adds the path's length to ``len``."""
    TreeCommit(slots, n_q_heads, scores, stats, stream)()


class KvEvict(_Prepared):
    """luce_kv_evict (or luce_kv_evict_paged, for PagedEvictSlots) with its
    arguments marshalled once: each call takes what the slots hold by then, and
    checks tensors that were replaced."""

    def __init__(self, slots: Sequence[EvictSlot], stream=None):
        self.slots = list(slots)
        self._paged = paged = _kind(self.slots, EvictSlot, PagedEvictSlot)
        first = self.slots[0].k_pool if paged else self.slots[0].k
        L, Hkv = first.shape[1:3] if paged else first.shape[:2]
        n = len(self.slots)
        self._first, self._heads = first, (L, Hkv)
        self._sc = ((PagedEvictSlotC if paged else EvictSlotC) * n)()
        self._items, self._seen, self._pages = [self._sc[i] for i in range(n)], [None] * n, [0] * n
        for i, s in enumerate(self.slots):
            self._take(i, s)
        args = (self._sc, n, L, Hkv, HEAD_DIM)
        self._bind("luce_kv_evict_paged" if paged else "luce_kv_evict", args, first.device, stream, None)

    def _take(self, i, s):
        """Slot i's tensors."""
        import torch
        (L, Hkv), c, table = self._heads, self._items[i], None
        if self._paged:
            _pools(s.k_pool, s.v_pool, L, Hkv, f"slots[{i}]")
            _need(s.table, torch.int32, f"slots[{i}].table")
            k, v, cap, table = s.k_pool, s.v_pool, s.acc.shape[-1], s.table
            if table.numel() * PAGE_KEYS < min(s.len, cap):
                raise ValueError(f"slots[{i}].table: {table.numel()} pages do not hold {s.len} keys")
        else:
            _caches(s.k, s.v, L, Hkv, f"slots[{i}]")
            k, v, cap = s.k, s.v, s.k.shape[2]
        acc_out = s.acc if s.acc_out is None else s.acc_out
        pos_out = s.pos if s.pos_out is None else s.pos_out
        for t, dt, w in ((s.acc, torch.float32, "acc"), (acc_out, torch.float32, "acc_out"),
                         (s.pos, torch.int32, "pos"), (pos_out, torch.int32, "pos_out")):
            _state(t, dt, L, Hkv, cap, f"slots[{i}].{w}")
        _same_device(self._first, k, v, s.acc, s.pos, acc_out, pos_out, table)
        if self._paged:
            c.k_pool, c.v_pool, c.n_pages, c.table = k.data_ptr(), v.data_ptr(), k.shape[0], table.data_ptr()
            self._pages[i] = table.numel() * PAGE_KEYS
        else:
            c.k, c.v = k.data_ptr(), v.data_ptr()
        c.acc, c.pos, c.acc_out, c.pos_out = s.acc.data_ptr(), s.pos.data_ptr(), acc_out.data_ptr(), pos_out.data_ptr()
        c.cap = cap
        self._seen[i] = (i, s, k, v, table, s.acc, s.pos, s.acc_out, s.pos_out, None)

    def _take_sizes(self, i, s):
        if self._paged and s.len > self._pages[i]:
            raise ValueError(f"slots[{i}].table does not hold {s.len} keys")
        if s.next_pos is None and s.recent:
            raise ValueError(f"slots[{i}]: recent={s.recent} needs next_pos, the position of the next token")
        c = self._items[i]
        c.len, c.budget, c.sinks, c.recent = s.len, s.budget, s.sinks, s.recent
        c.next_pos = LAST_POS if s.next_pos is None else s.next_pos
        self._seen[i] = (*self._seen[i][:-1], (s.len, s.next_pos, s.budget, s.sinks, s.recent))

    def __call__(self):
        paged = self._paged
        for i, s, k, v, table, acc, pos, acc_out, pos_out, now in self._seen:
            if (s.k_pool is not k or s.v_pool is not v or s.table is not table if paged else s.k is not k or s.v is not v) or \
                    s.acc is not acc or s.pos is not pos or s.acc_out is not acc_out or s.pos_out is not pos_out:
                now = self._take(i, s)
            if (s.len, s.next_pos, s.budget, s.sinks, s.recent) != now:
                self._take_sizes(i, s)
        self._call()


def luce_kv_evict(slots: Sequence[EvictSlot], stream=None):
    """Cut the slots' caches to their budgets by accumulated attention weight,
    per layer and KV head.  The caller continues with min(len, budget) keys."""
    KvEvict(slots, stream)()
