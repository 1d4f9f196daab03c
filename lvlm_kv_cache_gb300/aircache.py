"""Thin ctypes binding of the AirCache C ABI (include/aircache.h).

Argument marshalling only: every step of the compression runs in the CUDA
library ``libaircache.so`` built from ``csrc/``.  If that library is missing the
binding raises; there is no fallback path.

Tensors are torch CUDA tensors; the functions take the same arguments as the C
entry points (device buffers are tensors, the stream is a torch stream or None
for the current one) and raise ``AirCacheError`` on a non-zero status.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# AIRCACHE_TIMELINE=1 selects the measurement build whose kernels record their
# entry and exit times (build.build(timeline=True)); the default is the product build
LIB_PATH = os.path.join(HERE, "libaircache_timeline.so" if os.environ.get("AIRCACHE_TIMELINE") == "1"
                        else "libaircache.so")

OK = 0
DECODE_EARLY_CACHE = 1
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED = -2
ERR_WORKSPACE = -3
ERR_CUDA = -4
ERR_DEVICE_TIMEOUT = -5
ERR_DEVICE_BOUNDS = -6
ERR_ELITE_OVERFLOW = -7
ERR_CAPACITY = -8

F32, BF16, INT8 = 0, 1, 2
MAX_LAYERS = 256
# test hook of the variant word: the first kernel's bounded wait runs out (see aircache.h)
VARIANT_WAIT_TEST = 1 << 24


class AirCacheError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({status_string(status)})")


class ProblemStruct(ctypes.Structure):
    _fields_ = [
        ("num_layers", ctypes.c_int32),
        ("num_requests", ctypes.c_int32),
        ("h_q", ctypes.c_int32),
        ("h_kv", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("max_visual", ctypes.c_int32),
        ("max_text", ctypes.c_int32),
        ("max_elite", ctypes.c_int32),
        ("variant", ctypes.c_int32),
        ("total_tokens", ctypes.c_int64),
        ("total_visual", ctypes.c_int64),
        ("cu_seqlens", ctypes.c_void_p),
        ("cu_visual", ctypes.c_void_p),
        ("q_text", ctypes.POINTER(ctypes.c_void_p)),
        ("k", ctypes.POINTER(ctypes.c_void_p)),
        ("v", ctypes.POINTER(ctypes.c_void_p)),
        ("q_stride_tok", ctypes.c_int64),
        ("q_stride_head", ctypes.c_int64),
        ("kv_stride_tok", ctypes.c_int64),
        ("kv_stride_head", ctypes.c_int64),
        ("alpha", ctypes.c_double),
        ("r", ctypes.c_double),
        ("n_prefix", ctypes.c_void_p),
        ("q_visual", ctypes.POINTER(ctypes.c_void_p)),
    ]


_lib = None


class DecodeProblemStruct(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32), ("h_q", ctypes.c_int32), ("h_kv", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
        ("kv_rows", ctypes.c_int64), ("max_rows", ctypes.c_int64),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("row_begin", ctypes.c_void_p), ("row_end", ctypes.c_void_p),
        ("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p),
        ("q_stride_seq", ctypes.c_int64), ("q_stride_head", ctypes.c_int64),
        ("kv_stride_row", ctypes.c_int64), ("kv_stride_head", ctypes.c_int64),
        ("new_stride_seq", ctypes.c_int64), ("new_stride_head", ctypes.c_int64),
        ("out", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("flags", ctypes.c_int32), ("reserved1", ctypes.c_int32),
        ("row_index", ctypes.c_void_p), ("index_len", ctypes.c_int64),
    ]


class QuantProblemStruct(ctypes.Structure):
    _fields_ = [
        ("num_units", ctypes.c_int32), ("h_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("reserved0", ctypes.c_int32), ("reserved1", ctypes.c_int32),
        ("rows", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("kv_stride_row", ctypes.c_int64), ("kv_stride_head", ctypes.c_int64),
        ("offsets", ctypes.c_void_p), ("k8", ctypes.c_void_p), ("v8", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
    ]


class PagesStruct(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32), ("h_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32), ("page_rows", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("num_pages", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("stride_page", ctypes.c_int64), ("stride_row", ctypes.c_int64), ("stride_head", ctypes.c_int64),
        ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("lens", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("mass", ctypes.c_void_p), ("order", ctypes.c_void_p),
    ]


class RotateProblemStruct(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64), ("num_seqs", ctypes.c_int32), ("h_q", ctypes.c_int32),
        ("h_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("axes", ctypes.c_int32),
        ("section0", ctypes.c_int32), ("section1", ctypes.c_int32), ("eps", ctypes.c_float),
        ("reserved0", ctypes.c_int32),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("q_stride_tok", ctypes.c_int64), ("q_stride_head", ctypes.c_int64),
        ("k_stride_tok", ctypes.c_int64), ("k_stride_head", ctypes.c_int64),
        ("v_stride_tok", ctypes.c_int64), ("v_stride_head", ctypes.c_int64),
        ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p),
        ("qo_stride_tok", ctypes.c_int64), ("qo_stride_head", ctypes.c_int64),
        ("ko_stride_tok", ctypes.c_int64), ("ko_stride_head", ctypes.c_int64),
        ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("turns", ctypes.c_void_p),
        ("positions", ctypes.c_void_p), ("cu_tokens", ctypes.c_void_p), ("seen", ctypes.c_void_p),
        ("pages", ctypes.POINTER(PagesStruct)),
    ]


class PagedDecodeProblemStruct(ctypes.Structure):
    _fields_ = [
        ("pages", ctypes.POINTER(PagesStruct)), ("h_q", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("scale", ctypes.c_float), ("reserved0", ctypes.c_int32), ("total_rows", ctypes.c_int64),
        ("q", ctypes.c_void_p), ("q_stride_seq", ctypes.c_int64), ("q_stride_head", ctypes.c_int64),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("mass_out", ctypes.c_void_p),
    ]


class EvictProblemStruct(ctypes.Structure):
    _fields_ = [
        ("pages", ctypes.POINTER(PagesStruct)), ("keep", ctypes.c_void_p), ("seen", ctypes.c_void_p),
        ("lens_out", ctypes.c_void_p), ("mass_out", ctypes.c_void_p), ("order_out", ctypes.c_void_p),
        ("sink", ctypes.c_int32), ("recent", ctypes.c_int32), ("max_rows", ctypes.c_int64),
    ]


class PagedAttendProblemStruct(ctypes.Structure):
    _fields_ = [
        ("pages", ctypes.POINTER(PagesStruct)), ("num_tokens", ctypes.c_int64), ("h_q", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("causal", ctypes.c_int32), ("reserved0", ctypes.c_int32),
        ("scale", ctypes.c_float), ("reserved1", ctypes.c_float),
        ("cu_tokens", ctypes.c_void_p), ("row_begin", ctypes.c_void_p), ("row_end", ctypes.c_void_p),
        ("q", ctypes.c_void_p), ("q_stride_tok", ctypes.c_int64), ("q_stride_head", ctypes.c_int64),
        ("out", ctypes.c_void_p), ("out_stride_tok", ctypes.c_int64), ("out_stride_head", ctypes.c_int64),
        ("lse", ctypes.c_void_p),
    ]


class SharedDecodeProblemStruct(ctypes.Structure):
    _fields_ = [
        ("own", PagedDecodeProblemStruct), ("prefix", ctypes.POINTER(PagesStruct)), ("cu_seqs", ctypes.c_void_p),
    ]


def lib():
    """The loaded CUDA library (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing; build it with `python -m lvlm_kv_cache_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(ProblemStruct)
        vp, sz, i64, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_int
        L.aircache_workspace_size.argtypes = [P]
        L.aircache_workspace_size.restype = sz
        L.aircache_compress_bound.argtypes = [P]
        L.aircache_compress_bound.restype = i64
        L.aircache_score.argtypes = [P, vp, sz, vp, vp, vp, vp]
        L.aircache_score.restype = i32
        L.aircache_budget.argtypes = [P, vp, vp, sz, vp, vp, vp]
        L.aircache_budget.restype = i32
        L.aircache_budget_noalloc.argtypes = [P, vp, vp, vp, vp, vp]
        L.aircache_budget_noalloc.restype = i32
        L.aircache_select.argtypes = [P, vp, vp, vp, sz, vp, vp]
        L.aircache_select.restype = i32
        L.aircache_compact.argtypes = [P, vp, vp, vp, sz, vp, vp, vp, i64, vp]
        L.aircache_compact.restype = i32
        L.aircache_compress.argtypes = [P, vp, sz, vp, vp, vp, i64, vp, vp, vp, vp]
        L.aircache_compress.restype = i32
        L.aircache_get_error.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_int32)]
        L.aircache_get_error.restype = i32
        L.aircache_status_string.argtypes = [i32]
        L.aircache_status_string.restype = ctypes.c_char_p
        L.aircache_compress_launches.argtypes = [P]
        L.aircache_compress_launches.restype = i32
        L.aircache_compress_profile.argtypes = [P, vp, sz, vp, vp, vp, i64, vp, vp, vp,
                                                ctypes.POINTER(ctypes.c_void_p), i32, vp]
        L.aircache_compress_profile.restype = i32
        pv = ctypes.POINTER(ctypes.c_void_p)
        L.aircache_prefill.argtypes = [P, pv, i64, i64, pv, i64, i64, vp, sz, vp]
        L.aircache_prefill.restype = i32
        L.aircache_prefill_compress.argtypes = [P, pv, i64, i64, pv, i64, i64, vp, sz, vp, vp, vp, i64, vp, vp,
                                                vp, vp]
        L.aircache_prefill_compress.restype = i32
        L.aircache_kernel_name.argtypes = [P, i32]
        L.aircache_kernel_name.restype = ctypes.c_char_p
        L.aircache_row_index.argtypes = [P, vp, vp, vp, vp, sz, vp, i64, vp]
        L.aircache_row_index.restype = i32
        L.aircache_quantize_int8.argtypes = [ctypes.POINTER(QuantProblemStruct), vp, vp]
        L.aircache_quantize_int8.restype = i32
        DP = ctypes.POINTER(DecodeProblemStruct)
        L.aircache_decode_workspace_size.argtypes = [DP]
        L.aircache_decode_workspace_size.restype = sz
        L.aircache_decode_splits.argtypes = [DP]
        L.aircache_decode_splits.restype = i32
        L.aircache_decode.argtypes = [DP, vp, sz, vp]
        L.aircache_decode.restype = i32
        L.aircache_rotate.argtypes = [ctypes.POINTER(RotateProblemStruct), vp, vp]
        L.aircache_rotate.restype = i32
        PD = ctypes.POINTER(PagedDecodeProblemStruct)
        L.aircache_paged_decode_workspace_size.argtypes = [PD]
        L.aircache_paged_decode_workspace_size.restype = sz
        L.aircache_paged_decode.argtypes = [PD, vp, sz, vp]
        L.aircache_paged_decode.restype = i32
        EV = ctypes.POINTER(EvictProblemStruct)
        L.aircache_evict_workspace_size.argtypes = [EV]
        L.aircache_evict_workspace_size.restype = sz
        L.aircache_evict.argtypes = [EV, vp, sz, vp]
        L.aircache_evict.restype = i32
        PA = ctypes.POINTER(PagedAttendProblemStruct)
        L.aircache_paged_attend_workspace_size.argtypes = [PA]
        L.aircache_paged_attend_workspace_size.restype = sz
        L.aircache_paged_attend.argtypes = [PA, vp, sz, vp]
        L.aircache_paged_attend.restype = i32
        SD = ctypes.POINTER(SharedDecodeProblemStruct)
        L.aircache_shared_decode_workspace_size.argtypes = [SD]
        L.aircache_shared_decode_workspace_size.restype = sz
        L.aircache_shared_decode.argtypes = [SD, vp, sz, vp]
        L.aircache_shared_decode.restype = i32
        _lib = L
    return _lib


def status_string(status: int) -> str:
    try:
        return lib().aircache_status_string(int(status)).decode()
    except ImportError:
        return "library not loaded"


def _check(status: int, where: str):
    if status != OK:
        raise AirCacheError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


class Problem:
    """A compression problem over torch tensors (kept alive by this object).

    q, k, v: either stacked tensors [L, T, H, D] or lists of per-layer [T, H, D]
    tensors (same strides for every layer); q holds the text rows only.
    cu_seqlens, cu_visual: int32 device tensors [B+1].
    max_visual, max_text: host maxima over the requests.
    """

    def __init__(self, q, k, v, cu_seqlens, cu_visual, max_visual, max_text, alpha=0.9, r=0.1,
                 max_elite=0, total_tokens=None, total_visual=None, window_mode=0, budget_mode=0,
                 n_prefix=None, head_sets=False, q_visual=None, wait_test=False):
        qs = list(q.unbind(0)) if torch.is_tensor(q) else list(q)
        ks = list(k.unbind(0)) if torch.is_tensor(k) else list(k)
        vs = list(v.unbind(0)) if torch.is_tensor(v) else list(v)
        L = len(qs)
        if not (len(ks) == len(vs) == L) or L < 1 or L > MAX_LAYERS:
            raise ValueError("q, k, v must have the same number of layers (1..256)")
        dt = qs[0].dtype
        if dt not in (torch.float32, torch.bfloat16) or any(t.dtype != dt for t in qs + ks + vs):
            raise TypeError("q, k, v must all be float32 or all bfloat16")
        self.dtype = dt
        self.layers = (qs, ks, vs)  # keep alive
        B = cu_seqlens.numel() - 1
        T = int(total_tokens) if total_tokens is not None else int(ks[0].shape[0])
        TV = int(total_visual) if total_visual is not None else None
        if TV is None:
            TV = int(cu_visual[-1].item())
        self.B, self.L = B, L
        self.head_sets = bool(head_sets)
        self.h_q, self.h_kv, self.d = int(qs[0].shape[1]), int(ks[0].shape[1]), int(ks[0].shape[2])
        self.total_tokens, self.total_visual = T, TV
        self.cu_seqlens, self.cu_visual = cu_seqlens, cu_visual
        arr = ctypes.c_void_p * L
        self._q = arr(*[t.data_ptr() for t in qs])
        self._k = arr(*[t.data_ptr() for t in ks])
        self._v = arr(*[t.data_ptr() for t in vs])
        self.c = ProblemStruct(
            num_layers=L, num_requests=B, h_q=self.h_q, h_kv=self.h_kv, head_dim=self.d,
            dtype=BF16 if dt == torch.bfloat16 else F32,
            max_visual=int(max_visual), max_text=int(max_text), max_elite=int(max_elite),
            variant=int(window_mode) | (int(budget_mode) << 8) | ((1 << 16) if head_sets else 0)
            | (VARIANT_WAIT_TEST if wait_test else 0),
            total_tokens=T, total_visual=TV,
            cu_seqlens=cu_seqlens.data_ptr(), cu_visual=cu_visual.data_ptr(),
            q_text=ctypes.cast(self._q, ctypes.POINTER(ctypes.c_void_p)),
            k=ctypes.cast(self._k, ctypes.POINTER(ctypes.c_void_p)),
            v=ctypes.cast(self._v, ctypes.POINTER(ctypes.c_void_p)),
            q_stride_tok=qs[0].stride(0), q_stride_head=qs[0].stride(1),
            kv_stride_tok=ks[0].stride(0), kv_stride_head=ks[0].stride(1),
            alpha=float(alpha), r=float(r),
            n_prefix=n_prefix.data_ptr() if n_prefix is not None else None,
        )
        if q_visual is not None:  # window 4: the visual tokens' queries, per layer [total_visual, H_q, D]
            qvs = list(q_visual.unbind(0)) if torch.is_tensor(q_visual) else list(q_visual)
            if len(qvs) != L or any(t.stride() != qs[0].stride() for t in qvs):
                raise ValueError("q_visual: one tensor per layer with q's strides")
            self._qv = arr(*[t.data_ptr() for t in qvs])
            self.c.q_visual = ctypes.cast(self._qv, ctypes.POINTER(ctypes.c_void_p))
            self.q_visual = qvs  # keep alive
        self.n_prefix = n_prefix  # keep alive
        for t in ks + vs + qs:
            if t.stride(2) != 1:
                raise ValueError("head_dim must be contiguous")
        if any(t.stride() != ks[0].stride() for t in ks + vs) or any(t.stride() != qs[0].stride() for t in qs):
            raise ValueError("every layer must share the same strides")

    @property
    def ref(self):
        return ctypes.byref(self.c)

    def workspace_size(self) -> int:
        n = lib().aircache_workspace_size(self.ref)
        if n == 0:
            raise AirCacheError(ERR_INVALID_ARG, "aircache_workspace_size")
        return int(n)

    def compress_bound(self) -> int:
        n = lib().aircache_compress_bound(self.ref)
        if n < 0:
            raise AirCacheError(ERR_INVALID_ARG, "aircache_compress_bound")
        return int(n)

    def launches(self) -> int:
        return int(lib().aircache_compress_launches(self.ref))

    @property
    def max_text(self):
        return self.c.max_text

    def new_workspace(self, device=None) -> torch.Tensor:
        """A 256-byte-aligned device workspace (torch allocations are 512-B aligned)."""
        dev = device or self.layers[1][0].device
        return torch.empty(self.workspace_size(), dtype=torch.uint8, device=dev)


# ------------------------------------------------------------------ entry points

def aircache_score(prob: Problem, ws, iv, elite, n_tk, stream=None):
    _check(lib().aircache_score(prob.ref, _ptr(ws), ws.numel(), _ptr(iv), _ptr(elite), _ptr(n_tk),
                                _stream(stream)), "aircache_score")


def aircache_budget(prob: Problem, iv, ws, stats, keep, stream=None):
    _check(lib().aircache_budget(prob.ref, _ptr(iv), _ptr(ws), ws.numel(), _ptr(stats), _ptr(keep),
                                 _stream(stream)), "aircache_budget")


def aircache_budget_noalloc(prob: Problem, iv, stats, keep, device_status=None, stream=None):
    """aircache_budget with the library's fixed device scratch instead of a
    workspace (for callers that cannot allocate; at most
    AIRCACHE_NOALLOC_MAX_UNITS layer-request pairs; calls must not overlap)."""
    _check(lib().aircache_budget_noalloc(prob.ref, _ptr(iv), _ptr(stats), _ptr(keep), _ptr(device_status),
                                         _stream(stream)), "aircache_budget_noalloc")


def aircache_select(prob: Problem, iv, keep, ws, idx, stream=None):
    _check(lib().aircache_select(prob.ref, _ptr(iv), _ptr(keep), _ptr(ws), ws.numel(), _ptr(idx),
                                 _stream(stream)), "aircache_select")


def aircache_compact(prob: Problem, idx, keep, ws, out_k, out_v, out_offsets, stream=None):
    cap = out_k.shape[0]
    _check(lib().aircache_compact(prob.ref, _ptr(idx), _ptr(keep), _ptr(ws), ws.numel(), _ptr(out_k),
                                  _ptr(out_v), _ptr(out_offsets), cap, _stream(stream)),
           "aircache_compact")


def aircache_compress(prob: Problem, ws, out_k, out_v, out_offsets, keep, idx=None, iv=None, stream=None):
    cap = out_k.shape[0]
    _check(lib().aircache_compress(prob.ref, _ptr(ws), ws.numel(), _ptr(out_k), _ptr(out_v),
                                   _ptr(out_offsets), cap, _ptr(keep), _ptr(idx), _ptr(iv),
                                   _stream(stream)), "aircache_compress")


def _layer_array(ts):
    arr = (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])
    return arr, ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p))


def aircache_prefill(prob: Problem, q_all, attn_out, ws, stream=None):
    """Causal prefill attention of every layer: q_all [L][T][H_q][D] (every
    prompt row), attn_out [L][T][H_q][D] bf16 (written)."""
    qs = list(q_all.unbind(0)) if torch.is_tensor(q_all) else list(q_all)
    os_ = list(attn_out.unbind(0)) if torch.is_tensor(attn_out) else list(attn_out)
    qa, qp = _layer_array(qs)
    oa, op = _layer_array(os_)
    _check(lib().aircache_prefill(prob.ref, qp, qs[0].stride(0), qs[0].stride(1), op, os_[0].stride(0),
                                  os_[0].stride(1), _ptr(ws), ws.numel(), _stream(stream)), "aircache_prefill")


def aircache_prefill_compress(prob: Problem, q_all, attn_out, ws, out_k, out_v, out_offsets, keep, idx=None,
                              iv=None, stream=None):
    """The prefill attention and, from its own logits, the whole compression."""
    qs = list(q_all.unbind(0)) if torch.is_tensor(q_all) else list(q_all)
    os_ = list(attn_out.unbind(0)) if torch.is_tensor(attn_out) else list(attn_out)
    qa, qp = _layer_array(qs)
    oa, op = _layer_array(os_)
    cap = out_k.shape[0]
    _check(lib().aircache_prefill_compress(prob.ref, qp, qs[0].stride(0), qs[0].stride(1), op, os_[0].stride(0),
                                           os_[0].stride(1), _ptr(ws), ws.numel(), _ptr(out_k), _ptr(out_v),
                                           _ptr(out_offsets), cap, _ptr(keep), _ptr(idx), _ptr(iv),
                                           _stream(stream)), "aircache_prefill_compress")


def prefill_compress(prob: Problem, q_all, attn_out=None, ws=None, out=None, stream=None, check=True):
    """aircache_prefill_compress with allocated outputs; returns (attn_out, out dict)."""
    ws = prob.new_workspace() if ws is None else ws
    out = alloc_outputs(prob) if out is None else out
    if attn_out is None:
        attn_out = torch.empty(q_all.shape, dtype=torch.bfloat16, device=q_all.device)
    aircache_prefill_compress(prob, q_all, attn_out, ws, out["out_k"], out["out_v"], out["out_offsets"],
                              out["keep"], out["idx"], out["iv"], stream)
    if check:
        st = aircache_get_error(ws, stream)
        if st != OK:
            raise AirCacheError(st, "aircache_prefill_compress (device)")
    return attn_out, out


def aircache_compress_profile(prob: Problem, ws, out_k, out_v, out_offsets, keep, events, idx=None,
                              iv=None, stream=None):
    """aircache_compress recording torch.cuda.Event objects around each kernel
    (len(events) == prob.launches() + 1)."""
    cap = out_k.shape[0]
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check(lib().aircache_compress_profile(prob.ref, _ptr(ws), ws.numel(), _ptr(out_k), _ptr(out_v),
                                           _ptr(out_offsets), cap, _ptr(keep), _ptr(idx), _ptr(iv),
                                           arr, len(events), _stream(stream)),
           "aircache_compress_profile")


def kernel_names(prob: "Problem"):
    """Names of the kernels one aircache_compress call on `prob` launches, in order."""
    n = prob.launches()
    return [lib().aircache_kernel_name(prob.ref, i).decode() for i in range(n)]


def aircache_get_error(ws, stream=None) -> int:
    st = ctypes.c_int32(0)
    _check(lib().aircache_get_error(_ptr(ws), _stream(stream), ctypes.byref(st)), "aircache_get_error")
    return int(st.value)


# ------------------------------------------------------------------ conveniences

def alloc_outputs(prob: Problem, device=None):
    """Device buffers for aircache_compress: out_k, out_v ([bound, H_kv, D]),
    out_offsets [L*B+1], keep [L*B], idx and iv [L, total_visual]."""
    dev = device or prob.layers[1][0].device
    rows = prob.compress_bound()
    L, B = prob.L, prob.B
    return {
        "out_k": torch.empty((rows, prob.h_kv, prob.d), dtype=prob.dtype, device=dev),
        "out_v": torch.empty((rows, prob.h_kv, prob.d), dtype=prob.dtype, device=dev),
        "out_offsets": torch.empty(L * B + 1, dtype=torch.int64, device=dev),
        "keep": torch.empty(L * B, dtype=torch.int32, device=dev),
        "idx": torch.empty((L, prob.h_kv, prob.total_visual) if prob.head_sets else (L, prob.total_visual),
                           dtype=torch.int32, device=dev),
        "iv": torch.empty((L, prob.total_visual), dtype=torch.float32, device=dev),
    }


def compress(prob: Problem, ws=None, out=None, stream=None, check=True):
    """One fused compression; returns the output dict (see alloc_outputs).
    With check=True the device error word is read (this synchronises)."""
    ws = prob.new_workspace() if ws is None else ws
    out = alloc_outputs(prob) if out is None else out
    aircache_compress(prob, ws, out["out_k"], out["out_v"], out["out_offsets"], out["keep"],
                      out["idx"], out["iv"], stream)
    if check:
        st = aircache_get_error(ws, stream)
        if st != OK:
            raise AirCacheError(st, "aircache_compress (device)")
    return out


def compress_host(q, k, v, cu_seqlens, cu_visual, max_visual, max_text, alpha=0.9, r=0.1,
                  device="cuda", stream=None):
    """End-to-end from HOST tensors: copies q, k and the offsets to the device,
    compresses, and copies the compacted cache and its offsets back.  Values in
    page-locked memory (v.is_pinned()) stay on the host: only the compaction
    reads them, and only the rows it keeps; other values are copied first.
    Returns (out_k, out_v, out_offsets) as host tensors trimmed to the rows used."""
    dq = q.to(device, non_blocking=True)
    dk = k.to(device, non_blocking=True)
    dv = v if v.is_pinned() else v.to(device, non_blocking=True)
    dcs = cu_seqlens.to(device, non_blocking=True)
    dcv = cu_visual.to(device, non_blocking=True)
    prob = Problem(dq, dk, dv, dcs, dcv, max_visual, max_text, alpha, r,
                   total_tokens=k.shape[1], total_visual=int(cu_visual[-1]))
    out = compress(prob, stream=stream)
    offs = out["out_offsets"].cpu()
    rows = int(offs[-1])
    return out["out_k"][:rows].cpu(), out["out_v"][:rows].cpu(), offs


def math_bound(L, B, total_text, total_visual, r):
    """The compress_bound formula, for host-side sizing without the library."""
    return L * total_text + math.ceil(r * L * total_visual) + B * (2 * L + 1)


# ------------------------------------------------------------------ decode

class DecodeProblem:
    """One decode step over cached rows (see aircache_decode in the header).

    q: [S, H_q, D] bf16 (one query row per sequence); k, v: arenas
    [rows, H_kv, D] bf16, or int8 codes with k_scale, v_scale [S, H_kv] fp32;
    row_begin, row_end: int64 device tensors [S] (or one offsets tensor [S+1]
    via ``offsets=``); k_new, v_new: optional [S, H_kv, D] bf16; out: fp32
    [S, H_q, D] (allocated when None).  max_rows: the expected longest range
    (sizes the split; not a limit).  early_cache: AIRCACHE_DECODE_EARLY_CACHE
    (programmatic dependent launch; the kernel launched just before on the
    stream must not write the ranges or the cached rows)."""

    def __init__(self, q, k, v, row_begin=None, row_end=None, max_rows=0, k_new=None, v_new=None,
                 out=None, offsets=None, k_scale=None, v_scale=None, early_cache=False, row_index=None):
        if offsets is not None:
            row_begin, row_end = offsets[:-1], offsets[1:]
        S, h_q, d = (int(x) for x in q.shape)
        h_kv = int(k.shape[1])
        if out is None:
            out = torch.empty((S, h_q, d), dtype=torch.float32, device=q.device)
        for t in (q, k, v) + ((k_new, v_new) if k_new is not None else ()):
            if t.stride(-1) != 1:
                raise ValueError("head_dim must be contiguous")
        if k.stride() != v.stride() or (k_new is not None and k_new.stride() != v_new.stride()):
            raise ValueError("k and v (and k_new and v_new) must share strides")
        if row_begin.dtype != torch.int64 or row_end.dtype != torch.int64:
            raise TypeError("row ranges are int64")
        if not out.is_contiguous() or tuple(out.shape) != (S, h_q, d) or out.dtype != torch.float32:
            raise ValueError("out must be a dense fp32 [S, H_q, D] tensor")
        q8 = k.dtype == torch.int8
        if q8 and (k_scale is None or v_scale is None or not k_scale.is_contiguous() or not v_scale.is_contiguous()):
            raise ValueError("int8 caches need contiguous k_scale and v_scale [S, H_kv]")
        if row_index is not None and (row_index.dtype != torch.int32 or not row_index.is_contiguous()):
            raise TypeError("row_index is a contiguous int32 tensor")
        self.keep = (q, k, v, row_begin, row_end, k_new, v_new, out, k_scale, v_scale, row_index)
        self.out = out
        self.c = DecodeProblemStruct(
            num_seqs=S, h_q=h_q, h_kv=h_kv, head_dim=d,
            dtype=BF16 if q.dtype == torch.bfloat16 else F32, kv_dtype=INT8 if q8 else BF16,
            kv_rows=int(k.shape[0]), max_rows=int(max_rows),
            q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(),
            row_begin=row_begin.data_ptr(), row_end=row_end.data_ptr(),
            k_new=k_new.data_ptr() if k_new is not None else None,
            v_new=v_new.data_ptr() if v_new is not None else None,
            q_stride_seq=q.stride(0), q_stride_head=q.stride(1),
            kv_stride_row=k.stride(0), kv_stride_head=k.stride(1),
            new_stride_seq=k_new.stride(0) if k_new is not None else 0,
            new_stride_head=k_new.stride(1) if k_new is not None else 0,
            out=out.data_ptr(),
            k_scale=k_scale.data_ptr() if q8 else None, v_scale=v_scale.data_ptr() if q8 else None,
            flags=DECODE_EARLY_CACHE if early_cache else 0, reserved1=0,
            row_index=row_index.data_ptr() if row_index is not None else None,
            index_len=row_index.numel() if row_index is not None else 0,
        )

    @property
    def ref(self):
        return ctypes.byref(self.c)

    def workspace_size(self) -> int:
        n = lib().aircache_decode_workspace_size(self.ref)
        if n == 0:
            raise AirCacheError(ERR_INVALID_ARG, "aircache_decode_workspace_size")
        return int(n)

    def splits(self) -> int:
        return int(lib().aircache_decode_splits(self.ref))

    def new_workspace(self, device=None) -> torch.Tensor:
        """A zeroed decode workspace (zeroed once; every call leaves it zeroed
        again, apart from a recorded device error)."""
        return torch.zeros(self.workspace_size(), dtype=torch.uint8, device=device or self.out.device)


def aircache_decode(prob: DecodeProblem, ws, stream=None):
    _check(lib().aircache_decode(prob.ref, _ptr(ws), ws.numel(), _stream(stream)), "aircache_decode")


def decode(prob: DecodeProblem, ws=None, stream=None, check=True):
    """One decode step; returns prob.out.  check=True reads the device error word (synchronises)."""
    ws = prob.new_workspace() if ws is None else ws
    aircache_decode(prob, ws, stream)
    if check:
        st = aircache_get_error(ws, stream)
        if st != OK:
            raise AirCacheError(st, "aircache_decode (device)")
    return prob.out


# ------------------------------------------------------------------ int8 storage

def aircache_quantize_int8(k, v, offsets, k8, v8, k_scale, v_scale, status=None, stream=None):
    """int8 codes and per-(unit, KV head) scales of the bf16 arenas k, v
    ([rows, H_kv, D]); units are offsets[u] .. offsets[u+1]-1 (int64 device)."""
    c = QuantProblemStruct(
        num_units=offsets.numel() - 1, h_kv=int(k.shape[1]), head_dim=int(k.shape[2]),
        dtype=BF16 if k.dtype == torch.bfloat16 else F32, reserved0=0, reserved1=0,
        rows=int(k.shape[0]), k=k.data_ptr(), v=v.data_ptr(),
        kv_stride_row=k.stride(0), kv_stride_head=k.stride(1), offsets=offsets.data_ptr(),
        k8=k8.data_ptr(), v8=v8.data_ptr(), k_scale=k_scale.data_ptr(), v_scale=v_scale.data_ptr())
    if k.stride() != v.stride() or k.stride(2) != 1:
        raise ValueError("k and v must share strides, head_dim contiguous")
    _check(lib().aircache_quantize_int8(ctypes.byref(c), _ptr(status), _stream(stream)), "aircache_quantize_int8")


def quantize_int8(k, v, offsets, stream=None, check=True):
    """Allocates and returns (k8, v8, k_scale, v_scale) for the arenas k, v."""
    U = offsets.numel() - 1
    k8 = torch.empty(k.shape, dtype=torch.int8, device=k.device)
    v8 = torch.empty(v.shape, dtype=torch.int8, device=v.device)
    ks = torch.empty((U, k.shape[1]), dtype=torch.float32, device=k.device)
    vs = torch.empty((U, k.shape[1]), dtype=torch.float32, device=k.device)
    st = torch.zeros(1, dtype=torch.int32, device=k.device) if check else None
    aircache_quantize_int8(k, v, offsets, k8, v8, ks, vs, st, stream)
    if check and int(st.item()) != OK:
        raise AirCacheError(int(st.item()), "aircache_quantize_int8 (device)")
    return k8, v8, ks, vs


def aircache_row_index(prob: Problem, keep, idx, out_offsets, ws, row_index, stream=None):
    _check(lib().aircache_row_index(prob.ref, _ptr(keep), _ptr(idx), _ptr(out_offsets), _ptr(ws), ws.numel(),
                                    _ptr(row_index), row_index.numel(), _stream(stream)), "aircache_row_index")


def row_index(prob: Problem, out, ws=None, stream=None, check=True):
    """The compacted rows' prompt positions (int32 [rows]) for a gather-fused
    decode from the full cache; `out` is aircache_compress's output dict."""
    ws = prob.new_workspace() if ws is None else ws
    rows = int(out["out_offsets"][-1])
    ri = torch.empty(max(rows, 1), dtype=torch.int32, device=out["keep"].device)
    aircache_row_index(prob, out["keep"], out["idx"], out["out_offsets"], ws, ri, stream)
    if check:
        st = aircache_get_error(ws, stream)
        if st != OK:
            raise AirCacheError(st, "aircache_row_index (device)")
    return ri


# ------------------------------------------------------------------ paged cache

MAX_EVICT_ROWS = 393216


def _same_device(*ts):
    """Every given tensor lies on one CUDA device, which is returned."""
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("the tensors must be on a CUDA device")
        if dev is not None and t.device != dev:
            raise ValueError("the tensors must be on one device")
        dev = t.device
    return dev


def _dense(t, dtype, shape, name):
    if t is None:
        return
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a dense {dtype} tensor of shape {tuple(shape)}")


def _paged_stream(prob, ws, stream):
    """The stream handle of a call on `prob` (by default the current stream of the problem's device)."""
    if ws is not None and ws.device != prob.device:
        raise ValueError("the workspace must be on the problem's device")
    return torch._C._cuda_getCurrentRawStream(prob.device.index) if stream is None else stream.cuda_stream


def _on_stream(prob, stream, make):
    """make() with its allocations and kernels on the stream that a call on `prob` will use."""
    with torch.cuda.device(prob.device), torch.cuda.stream(stream):  # (None: the current stream)
        return make()


def _check_device(prob, word, stream, where):
    """Waits for the call's stream and raises what the device recorded in `word`."""
    if prob.empty:
        return
    with torch.cuda.device(prob.device):
        st = aircache_get_error(word, stream)
    if st != OK:
        raise AirCacheError(st, where + " (device)")


def _run_paged(fn, where, prob, *args):
    """fn(problem, *args) on the problem's device, whichever the current one is."""
    if torch._C._cuda_getDevice() == prob.device.index:
        st = fn(prob.ref, *args)
    else:
        with torch.cuda.device(prob.device):
            st = fn(prob.ref, *args)
    if st != OK:
        raise AirCacheError(st, where)


class PagedCache:
    """One layer's cache in pages (aircache_pages in the header).

    k, v: [P, page_rows, H_kv, D] bf16 with equal strides, or int8 codes with
    k_scale, v_scale [P, H_kv, page_rows] fp32; table: int32 [S, max_pages]
    (rows may be strided); lens: int32 [S], the rows of each sequence; mass
    fp32 and order int32 [P, H_kv, page_rows] are optional.  The tensors are
    the caller's and are updated in place by the calls that write them."""

    def __init__(self, k, v, table, lens, k_scale=None, v_scale=None, mass=None, order=None):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("k and v are [P, page_rows, H_kv, D] of one type and one layout, head_dim contiguous")
        if k.dtype not in (torch.bfloat16, torch.int8):
            raise TypeError("cached rows are bfloat16 or int8 codes")
        P, page_rows, h_kv, d = (int(x) for x in k.shape)
        if table.dtype != torch.int32 or table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
            raise ValueError("table is an int32 [S, max_pages] tensor with contiguous rows")
        S, max_pages = (int(x) for x in table.shape)
        if S > 1 and table.stride(0) < max_pages:
            raise ValueError("the table's rows must not overlap")
        _dense(lens, torch.int32, (S,), "lens")
        q8 = k.dtype == torch.int8
        if q8 != (k_scale is not None) or q8 != (v_scale is not None):
            raise ValueError("int8 codes come with k_scale and v_scale, bf16 rows without")
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale"), (mass, "mass")):
            _dense(t, torch.float32, (P, h_kv, page_rows), name)
        _dense(order, torch.int32, (P, h_kv, page_rows), "order")
        self.device = _same_device(k, v, table, lens, k_scale, v_scale, mass, order)
        self.k, self.v, self.table, self.lens = k, v, table, lens
        self.k_scale, self.v_scale, self.mass, self.order = k_scale, v_scale, mass, order
        self.num_seqs, self.max_pages, self.num_pages, self.page_rows = S, max_pages, P, page_rows
        self.h_kv, self.d = h_kv, d
        adr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self.c = PagesStruct(
            num_seqs=S, h_kv=h_kv, head_dim=d, kv_dtype=INT8 if q8 else BF16, page_rows=page_rows,
            max_pages=max_pages, num_pages=P, k=adr(k), v=adr(v), stride_page=k.stride(0), stride_row=k.stride(1),
            stride_head=k.stride(2), table=adr(table), table_stride=max(table.stride(0), max_pages), lens=adr(lens),
            k_scale=adr(k_scale), v_scale=adr(v_scale), mass=adr(mass), order=adr(order))


def rotation_table(inv_freq):
    """The rotation's frequencies as aircache_rotate takes them: fp32
    [n, 2], inv_freq / (2 pi) as a sum of two floats.  inv_freq: fp64 tensor or
    sequence of n angular frequencies (radians per position)."""
    f = torch.as_tensor(inv_freq, dtype=torch.float64)
    turns = f / (2 * math.pi)
    hi = turns.to(torch.float32)
    return torch.stack((hi, (turns - hi.to(torch.float64)).to(torch.float32)), dim=-1).contiguous()


class RotateProblem:
    """Per-head norms, rotation and append of one layer's projections (see
    aircache_rotate in the header).

    q: [T, H_q, D], k and v: [T, H_kv, D] bf16 (any strides that are multiples
    of 8 with D contiguous, such as views of one fused projection); q_out,
    k_out: bf16 outputs (q_out is allocated when None; k_out when None and
    there is no cache; in place: pass q, k).  cache: a PagedCache that the rows
    are appended to.  cu_tokens, seen: int32 [S + 1], [S]; positions: int32 [T], or [3, T] with
    sections (n0, n1, n2) frequencies to each axis.  turns: rotation_table's
    output on the device (None: no rotation)."""

    def __init__(self, q=None, k=None, v=None, q_out=None, k_out=None, cache=None, cu_tokens=None, seen=None,
                 positions=None, sections=None, turns=None, q_weight=None, k_weight=None, eps=1e-6,
                 interleaved=False):
        if q is None and k is None:
            raise ValueError("q or k must be given")
        some = q if q is not None else k
        T, d = int(some.shape[0]), int(some.shape[2])
        if q is not None and q_out is None:
            q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        if k is not None and k_out is None and cache is None:
            k_out = torch.empty(k.shape, dtype=torch.bfloat16, device=k.device)
        for t, like in ((q, None), (k, None), (v, k), (q_out, q), (k_out, k)):
            if t is None:
                continue
            if t.dtype != torch.bfloat16 or t.dim() != 3 or t.shape[0] != T or t.shape[2] != d or t.stride(2) != 1:
                raise ValueError("q, k, v and their outputs are bf16 [T, heads, D] with head_dim contiguous")
            if like is not None and t.shape != like.shape:
                raise ValueError("v, q_out and k_out have the shapes of k, q and k")
        if (q_out is not None and q is None) or (k_out is not None and k is None):
            raise ValueError("an output needs its input")
        for w in (q_weight, k_weight):
            _dense(w, torch.bfloat16, (d,), "a norm's weight")
        rot = 0
        if turns is not None:
            rot = 2 * int(turns.shape[0])
            _dense(turns, torch.float32, (rot // 2, 2), "turns")
        axes, n0, n1 = 1, 0, 0
        if positions is not None:
            if positions.dim() == 2:
                axes = 3
                if sections is None or len(sections) != 3 or sum(sections) != rot // 2 or min(sections) < 0:
                    raise ValueError("positions of three axes need sections that add up to rotary_dim / 2")
                n0, n1 = int(sections[0]), int(sections[1])
            _dense(positions, torch.int32, (3, T) if axes == 3 else (T,), "positions")
        S = cu_tokens.numel() - 1 if cu_tokens is not None else 0
        _dense(cu_tokens, torch.int32, (S + 1,), "cu_tokens")
        _dense(seen, torch.int32, (S,), "seen")
        if cache is not None and (cu_tokens is None or cache.num_seqs != S or k is None or v is None
                                  or cache.h_kv != k.shape[1] or cache.d != d):
            raise ValueError("a cache needs k, v and cu_tokens of its sequences, KV heads and head_dim")
        self.device = _same_device(q, k, v, q_out, k_out, cu_tokens, seen, positions, turns, q_weight, k_weight,
                                   cache.k if cache is not None else None)
        self.keep = (q, k, v, cu_tokens, seen, positions, turns, q_weight, k_weight, cache)
        self.empty = T == 0 or (cu_tokens is not None and S == 0)
        self.q_out, self.k_out = q_out, k_out
        adr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        st = lambda t, i: 0 if t is None else t.stride(i)  # noqa: E731
        self.c = RotateProblemStruct(
            num_tokens=T, num_seqs=S, h_q=0 if q is None else int(q.shape[1]), h_kv=0 if k is None else int(k.shape[1]),
            head_dim=d, dtype=BF16, rotary_dim=rot, interleaved=1 if interleaved else 0, axes=axes, section0=n0,
            section1=n1, eps=float(eps), reserved0=0, q=adr(q), k=adr(k), v=adr(v),
            q_stride_tok=st(q, 0), q_stride_head=st(q, 1), k_stride_tok=st(k, 0), k_stride_head=st(k, 1),
            v_stride_tok=st(v, 0), v_stride_head=st(v, 1), q_out=adr(q_out), k_out=adr(k_out),
            qo_stride_tok=st(q_out, 0), qo_stride_head=st(q_out, 1), ko_stride_tok=st(k_out, 0),
            ko_stride_head=st(k_out, 1), q_weight=adr(q_weight), k_weight=adr(k_weight), turns=adr(turns),
            positions=adr(positions), cu_tokens=adr(cu_tokens), seen=adr(seen),
            pages=ctypes.pointer(cache.c) if cache is not None else None)
        self.ref = ctypes.byref(self.c)


def aircache_rotate(prob: RotateProblem, status=None, stream=None):
    if status is not None and (status.dtype != torch.int32 or status.numel() < 1):
        raise ValueError("status is an int32 tensor")
    if prob.empty:  # (tensors without storage)
        return
    s = _paged_stream(prob, status, stream)
    _run_paged(lib().aircache_rotate, "aircache_rotate", prob, None if status is None else status.data_ptr(), s)


def rotate(prob: RotateProblem, stream=None, check=True):
    """One call; returns (q_out, k_out).  check=True reads the device status (synchronises)."""
    st = _on_stream(prob, stream, lambda: torch.zeros(1, dtype=torch.int32, device=prob.device)) if check else None
    aircache_rotate(prob, st, stream)
    if check:
        _check_device(prob, st, stream, "aircache_rotate")
    return prob.q_out, prob.k_out


class PagedDecodeProblem:
    """One decode step over a PagedCache (see aircache_paged_decode in the header).

    q: [S, H_q, D] bf16; out: bf16 [S, H_q, D] (allocated when None); lse:
    True (allocated) or an fp32 [S, H_q] tensor; scale: the logits' factor
    (None: 1 / sqrt(D)); accumulate: add the weights to cache.mass in place, or
    pass mass_out for another array; total_rows: a bound of the sum of
    cache.lens (0: what the pages and the table can hold; give it when
    sequences share pages)."""

    def __init__(self, q, cache, out=None, lse=None, scale=None, accumulate=False, mass_out=None, total_rows=0):
        if q.dim() != 3 or q.dtype != torch.bfloat16 or q.stride(2) != 1:
            raise ValueError("q is bf16 [S, H_q, D], head_dim contiguous")
        S, h_q, d = (int(x) for x in q.shape)
        if S != cache.num_seqs or d != cache.d:
            raise ValueError("q must have the cache's sequences and head_dim")
        if out is None:
            out = torch.empty((S, h_q, d), dtype=torch.bfloat16, device=q.device)
        if isinstance(lse, bool):
            lse = torch.empty((S, h_q), dtype=torch.float32, device=q.device) if lse else None
        _dense(out, torch.bfloat16, (S, h_q, d), "out")
        _dense(lse, torch.float32, (S, h_q), "lse")
        if accumulate and mass_out is None:
            mass_out = cache.mass
        if (accumulate or mass_out is not None) and cache.mass is None:
            raise ValueError("the cache has no mass to accumulate")
        _dense(mass_out, torch.float32, (cache.num_pages, cache.h_kv, cache.page_rows), "mass_out")
        if not total_rows:
            total_rows = min(S * cache.max_pages, cache.num_pages) * cache.page_rows
        self.device = _same_device(q, out, lse, mass_out, cache.k)
        self.keep = (q, cache)
        self.empty = S == 0
        self.out, self.lse, self.mass_out = out, lse, mass_out
        adr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self.c = PagedDecodeProblemStruct(
            pages=ctypes.pointer(cache.c), h_q=h_q, dtype=BF16, scale=float(d ** -0.5 if scale is None else scale),
            reserved0=0, total_rows=int(total_rows), q=adr(q), q_stride_seq=q.stride(0),
            q_stride_head=q.stride(1), out=adr(out), lse=adr(lse), mass_out=adr(mass_out))
        self.ref = ctypes.byref(self.c)

    def workspace_size(self) -> int:
        if self.empty:
            return 256
        with torch.cuda.device(self.device):
            n = lib().aircache_paged_decode_workspace_size(self.ref)
            if n == 0:  # (the call itself names the reason, before it looks at a workspace)
                raise AirCacheError(lib().aircache_paged_decode(self.ref, None, 0, None), "aircache_paged_decode_workspace_size")
        return int(n)

    def new_workspace(self) -> torch.Tensor:
        """A zeroed workspace (zeroed once; every call leaves it ready for the next)."""
        return torch.zeros(self.workspace_size(), dtype=torch.uint8, device=self.device)


def aircache_paged_decode(prob: PagedDecodeProblem, ws, stream=None):
    if prob.empty:
        return
    s = _paged_stream(prob, ws, stream)
    _run_paged(lib().aircache_paged_decode, "aircache_paged_decode", prob, ws.data_ptr(), ws.numel(), s)


def paged_decode(prob: PagedDecodeProblem, ws=None, stream=None, check=True):
    """One decode step; returns prob.out.  check=True reads the device error word (synchronises)."""
    ws = _on_stream(prob, stream, prob.new_workspace) if ws is None else ws
    aircache_paged_decode(prob, ws, stream)
    if check:
        _check_device(prob, ws, stream, "aircache_paged_decode")
    return prob.out


class EvictProblem:
    """Eviction from a PagedCache by its mass (see aircache_evict in the header).

    keep: int32 [S], rows each sequence keeps; lens_out: int32 [S], not
    cache.lens itself; seen: int32 [S], tokens appended so far (needed with
    recent); sink, recent: the first and the newest tokens, always kept;
    mass_out, order_out: other arrays than the cache's (None: in place);
    max_rows: a bound of cache.lens (0: the table's capacity, or the longest that
    an eviction takes, MAX_EVICT_ROWS, if it is less)."""

    def __init__(self, cache, keep, lens_out, seen=None, sink=0, recent=0, mass_out=None, order_out=None, max_rows=0):
        S = cache.num_seqs
        for t, name in ((keep, "keep"), (lens_out, "lens_out"), (seen, "seen")):
            _dense(t, torch.int32, (S,), name)
        if cache.mass is None:
            raise ValueError("the cache has no mass to evict by")
        mass_out = cache.mass if mass_out is None else mass_out
        order_out = cache.order if order_out is None else order_out
        shape = (cache.num_pages, cache.h_kv, cache.page_rows)
        _dense(mass_out, torch.float32, shape, "mass_out")
        _dense(order_out, torch.int32, shape, "order_out")
        self.device = _same_device(cache.k, keep, lens_out, seen, mass_out, order_out)
        self.keep_alive = (cache, keep, seen)
        self.empty = S == 0
        self.lens_out, self.mass_out, self.order_out = lens_out, mass_out, order_out
        adr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self.c = EvictProblemStruct(
            pages=ctypes.pointer(cache.c), keep=adr(keep), seen=adr(seen), lens_out=adr(lens_out),
            mass_out=adr(mass_out), order_out=adr(order_out), sink=int(sink), recent=int(recent),
            max_rows=int(max_rows) or min(cache.max_pages * cache.page_rows, MAX_EVICT_ROWS))
        self.ref = ctypes.byref(self.c)

    def workspace_size(self) -> int:
        if self.empty:
            return 256
        with torch.cuda.device(self.device):
            n = lib().aircache_evict_workspace_size(self.ref)
            if n == 0:  # (the call itself names the reason, before it looks at a workspace)
                raise AirCacheError(lib().aircache_evict(self.ref, None, 0, None), "aircache_evict_workspace_size")
        return int(n)

    def new_workspace(self) -> torch.Tensor:
        """A zeroed workspace (zeroed once; every call leaves it ready for the next)."""
        return torch.zeros(self.workspace_size(), dtype=torch.uint8, device=self.device)


def aircache_evict(prob: EvictProblem, ws, stream=None):
    if prob.empty:
        return
    s = _paged_stream(prob, ws, stream)
    _run_paged(lib().aircache_evict, "aircache_evict", prob, ws.data_ptr(), ws.numel(), s)


def evict(prob: EvictProblem, ws=None, stream=None, check=True):
    """One eviction; returns prob.lens_out.  check=True reads the device error word (synchronises)."""
    ws = _on_stream(prob, stream, prob.new_workspace) if ws is None else ws
    aircache_evict(prob, ws, stream)
    if check:
        _check_device(prob, ws, stream, "aircache_evict")
    return prob.lens_out


class PagedAttendProblem:
    """Attention of several tokens of each sequence over a PagedCache (see
    aircache_paged_attend in the header).

    q: [T, H_q, D] bf16; cu_tokens: int32 [S + 1], the tokens of each sequence;
    out: bf16 [T, H_q, D] (allocated when None); lse: True (allocated) or an fp32
    [T, H_q] tensor; scale: the logits' factor (None: 1 / sqrt(D)).  A token sees
    all rows of its sequence; causal: the tokens' own rows are the cache's last
    and each sees those up to its own; row_begin, row_end: int32 [T], only rows
    of [row_begin, row_end) (either may be None)."""

    def __init__(self, q, cache, cu_tokens, out=None, lse=None, scale=None, causal=False, row_begin=None, row_end=None):
        if q.dim() != 3 or q.dtype != torch.bfloat16 or q.stride(2) != 1:
            raise ValueError("q is bf16 [T, H_q, D], head_dim contiguous")
        T, h_q, d = (int(x) for x in q.shape)
        if d != cache.d:
            raise ValueError("q must have the cache's head_dim")
        _dense(cu_tokens, torch.int32, (cache.num_seqs + 1,), "cu_tokens")
        if out is None:
            out = torch.empty((T, h_q, d), dtype=torch.bfloat16, device=q.device)
        if out.dtype != torch.bfloat16 or out.shape != q.shape or out.stride(2) != 1:
            raise ValueError("out is bf16 of q's shape, head_dim contiguous")
        if isinstance(lse, bool):
            lse = torch.empty((T, h_q), dtype=torch.float32, device=q.device) if lse else None
        _dense(lse, torch.float32, (T, h_q), "lse")
        for t, name in ((row_begin, "row_begin"), (row_end, "row_end")):
            _dense(t, torch.int32, (T,), name)
        self.device = _same_device(q, cu_tokens, out, lse, row_begin, row_end, cache.k)
        self.keep = (q, cache, cu_tokens, row_begin, row_end)
        self.empty = T == 0 or cache.num_seqs == 0
        self.out, self.lse = out, lse
        adr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self.c = PagedAttendProblemStruct(
            pages=ctypes.pointer(cache.c), num_tokens=T, h_q=h_q, dtype=BF16, causal=1 if causal else 0, reserved0=0,
            scale=float(d ** -0.5 if scale is None else scale), reserved1=0.0, cu_tokens=adr(cu_tokens),
            row_begin=adr(row_begin), row_end=adr(row_end), q=adr(q), q_stride_tok=q.stride(0),
            q_stride_head=q.stride(1), out=adr(out), out_stride_tok=out.stride(0), out_stride_head=out.stride(1),
            lse=adr(lse))
        self.ref = ctypes.byref(self.c)

    def workspace_size(self) -> int:
        if self.empty:
            return 256
        with torch.cuda.device(self.device):
            n = lib().aircache_paged_attend_workspace_size(self.ref)
            if n == 0:  # (the call itself names the reason, before it looks at a workspace)
                raise AirCacheError(lib().aircache_paged_attend(self.ref, None, 0, None), "aircache_paged_attend_workspace_size")
        return int(n)

    def new_workspace(self) -> torch.Tensor:
        """A zeroed workspace (zeroed once; every call leaves it ready for the next)."""
        return torch.zeros(self.workspace_size(), dtype=torch.uint8, device=self.device)


def aircache_paged_attend(prob: PagedAttendProblem, ws, stream=None):
    if prob.empty:
        return
    s = _paged_stream(prob, ws, stream)
    _run_paged(lib().aircache_paged_attend, "aircache_paged_attend", prob, ws.data_ptr(), ws.numel(), s)


def paged_attend(prob: PagedAttendProblem, ws=None, stream=None, check=True):
    """One call; returns prob.out.  check=True reads the device error word (synchronises)."""
    ws = _on_stream(prob, stream, prob.new_workspace) if ws is None else ws
    aircache_paged_attend(prob, ws, stream)
    if check:
        _check_device(prob, ws, stream, "aircache_paged_attend")
    return prob.out


class SharedDecodeProblem(PagedDecodeProblem):
    """One decode step of sequences that share prefixes (see aircache_shared_decode
    in the header): a PagedDecodeProblem over the sequences' own rows, q and cache,
    with prefix, a PagedCache of the prefixes, and cu_seqs: int32 [prefixes + 1],
    sequences cu_seqs[i] .. cu_seqs[i + 1] - 1 continue prefix i.  total_rows
    bounds the own rows."""

    def __init__(self, q, cache, prefix, cu_seqs, out=None, lse=None, scale=None, accumulate=False, mass_out=None,
                 total_rows=0):
        super().__init__(q, cache, out=out, lse=lse, scale=scale, accumulate=accumulate, mass_out=mass_out,
                         total_rows=total_rows)
        if prefix.d != cache.d or prefix.h_kv != cache.h_kv:
            raise ValueError("prefix must have the cache's KV heads and head_dim")
        _dense(cu_seqs, torch.int32, (prefix.num_seqs + 1,), "cu_seqs")
        self.device = _same_device(q, cache.k, prefix.k, cu_seqs)
        self.keep += (prefix, cu_seqs)
        self.c = SharedDecodeProblemStruct(own=self.c, prefix=ctypes.pointer(prefix.c), cu_seqs=cu_seqs.data_ptr())
        self.ref = ctypes.byref(self.c)

    def workspace_size(self) -> int:
        if self.empty:
            return 256
        with torch.cuda.device(self.device):
            n = lib().aircache_shared_decode_workspace_size(self.ref)
            if n == 0:  # (the call itself names the reason, before it looks at a workspace)
                raise AirCacheError(lib().aircache_shared_decode(self.ref, None, 0, None), "aircache_shared_decode_workspace_size")
        return int(n)


def aircache_shared_decode(prob: SharedDecodeProblem, ws, stream=None):
    if prob.empty:
        return
    s = _paged_stream(prob, ws, stream)
    _run_paged(lib().aircache_shared_decode, "aircache_shared_decode", prob, ws.data_ptr(), ws.numel(), s)


def shared_decode(prob: SharedDecodeProblem, ws=None, stream=None, check=True):
    """One decode step; returns prob.out.  check=True reads the device error word (synchronises)."""
    ws = _on_stream(prob, stream, prob.new_workspace) if ws is None else ws
    aircache_shared_decode(prob, ws, stream)
    if check:
        _check_device(prob, ws, stream, "aircache_shared_decode")
    return prob.out
