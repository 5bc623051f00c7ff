"""Batched decode attention over a paged KV cache, for one GB300 (sm_103a).

Thin Python binding of ``libfadecode.so`` (C ABI in ``include/fa_decode.h``):
argument marshalling only.  Every step of the decode path runs in the
library's CUDA kernels; PyTorch supplies device memory and streams.  If the
library has not been built, the first call into it raises RuntimeError -
there is no fallback implementation.

The calls follow the plan/run split of the page "FlashDecoding + FlashInfer -
the decode-time attention story" (section "The API you actually use"):
``plan`` once per batch shape, ``run`` on the hot path, plus ``merge_states``
for the merge rule of section "FlashDecoding - the split-KV trick".
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

__all__ = [
    "FA_OK", "FaError", "DecodePlan", "plan", "plan_multi_token", "plan_ragged_q", "run",
    "merge_states",
    "CascadePlan", "cascade_plan",
    "RotaryTable", "AppendPlan", "plan_append", "append_workspace_size",
    "PrefillPlan", "plan_prefill", "plan_prefill_host",
    "WeightsPlan", "plan_weights", "EvictPlan", "plan_evict",
    "workspace_size", "plan_work_host", "plan_work_host_buckets",
    "BatchDecodeWithPagedKVCacheWrapper",
    "LIB_PATH", "EXPORTED_SYMBOLS", "library", "library_stats",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfadecode.so")

# Entry points declared in include/fa_decode.h.
EXPORTED_SYMBOLS = (
    "fa_status_string", "fa_decode_workspace_size", "fa_decode_plan",
    "fa_decode_run", "fa_merge_states", "fa_decode_plan_destroy",
    "fa_decode_plan_get_info", "fa_decode_plan_get_work", "fa_plan_work_host",
    "fa_decode_check", "fa_decode_set_timing_events", "fa_decode_static",
    "fa_decode_run_token_scales", "fa_decode_plan_multi_token",
    "fa_cascade_workspace_size", "fa_cascade_plan", "fa_cascade_run", "fa_cascade_plan_destroy",
    "fa_cascade_check", "fa_decode_run_unified_max", "fa_decode_unified_max_fallbacks",
    "fa_cascade_set_timing_events", "fa_decode_static_check", "fa_library_get_stats",
    "fa_decode_plan_ragged_q", "fa_decode_workspace_size_ragged_q", "fa_cascade_run_scaled",
    "fa_plan_work_host_buckets",
    "fa_decode_run_head_scales", "fa_plan_work_host_heads",
    "fa_decode_run_block_scales",
    "fa_append_workspace_size", "fa_append_plan", "fa_append_run", "fa_append_run_head_scales",
    "fa_append_run_token_scales", "fa_append_run_block_scales", "fa_append_check",
    "fa_append_plan_destroy", "fa_cascade_run_block_scales", "fa_append_plan_axes",
    "fa_prefill_workspace_size", "fa_prefill_plan", "fa_prefill_run", "fa_prefill_run_head_scales",
    "fa_prefill_run_token_scales", "fa_prefill_run_block_scales", "fa_prefill_check",
    "fa_prefill_plan_destroy", "fa_plan_prefill_host",
    "fa_weights_workspace_size", "fa_weights_plan", "fa_weights_run", "fa_weights_run_head_scales",
    "fa_weights_run_token_scales", "fa_weights_run_block_scales", "fa_weights_check",
    "fa_weights_plan_destroy", "fa_evict_workspace_size", "fa_evict_plan", "fa_evict_run",
    "fa_evict_check", "fa_evict_plan_destroy",
)

FA_OK = 0
SEGMENT_INTS = 8
MERGE_INTS = 4
DTYPE_CODES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2,
               torch.float8_e4m3fn: 3}

class FaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_L().fa_status_string(status).decode()} ({status})")


class PlanInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "batch", "num_qo_heads", "num_kv_heads", "head_dim", "page_size",
        "num_ctas", "ctas_per_sm", "num_sms", "num_segments", "num_merge_units",
        "num_partial_slots", "threads_per_cta", "smem_bytes_per_cta", "stages")] + [
        ("total_pages", ctypes.c_int64), ("total_tokens", ctypes.c_int64),
        ("workspace_bytes_used", ctypes.c_size_t), ("plan_upload_bytes", ctypes.c_size_t),
        ("tensor_cores", ctypes.c_int), ("fused_merge", ctypes.c_int), ("q_len", ctypes.c_int),
        ("unified_max", ctypes.c_int), ("num_pool_segments", ctypes.c_int),
        ("pool_pages", ctypes.c_int64), ("ragged_q", ctypes.c_int),
        ("total_q_rows", ctypes.c_int64), ("num_buckets", ctypes.c_int),
        ("bucket_first_cta", ctypes.c_int * 4), ("bucket_q_len", ctypes.c_int * 4)]

    def as_dict(self) -> dict:
        out = {}
        for n, _ in self._fields_:
            v = getattr(self, n)
            out[n] = list(v) if isinstance(v, ctypes.Array) else v
        return out


# fa_rows of k, v and q in a row: {address, token stride, head stride} each
_Rows3 = ctypes.c_int64 * 9
_Rows = ctypes.c_int64 * 3
_ROWS_BYTES = 24


class LibraryStats(ctypes.Structure):
    _fields_ = [("pinned_host_allocations", ctypes.c_int64), ("pinned_host_bytes", ctypes.c_int64),
                ("staged_uploads", ctypes.c_int64)]


def library_stats() -> dict:
    """The library's own host-side resource counters (fa_library_get_stats)."""
    s = LibraryStats()
    _check(_L().fa_library_get_stats(ctypes.byref(s)), "fa_library_get_stats")
    return {n: int(getattr(s, n)) for n, _ in s._fields_}


def _load() -> ctypes.CDLL:
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                            ctypes.c_float, ctypes.c_size_t)
    lib.fa_status_string.argtypes = [i32]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_decode_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.fa_decode_workspace_size.restype = sz
    lib.fa_decode_plan.argtypes = [P, P, P, i32, i32, i32, i32, i32, i32, i32,
                                   P, sz, P, ctypes.POINTER(P)]
    lib.fa_decode_plan.restype = i32
    lib.fa_decode_plan_multi_token.argtypes = [P, P, P, i32, i32, i32, i32, i32, i32, i32, i32,
                                               P, sz, P, ctypes.POINTER(P)]
    lib.fa_decode_plan_multi_token.restype = i32
    lib.fa_decode_plan_ragged_q.argtypes = [P, P, P, P, i32, i32, i32, i32, i32, i32, i32,
                                            P, sz, P, ctypes.POINTER(P)]
    lib.fa_decode_plan_ragged_q.restype = i32
    lib.fa_decode_workspace_size_ragged_q.argtypes = [i32, i32, i32, i32]
    lib.fa_decode_workspace_size_ragged_q.restype = sz
    lib.fa_decode_run.argtypes = [P, P, P, i64, f32, f32, f32, P, P, P]
    lib.fa_decode_run.restype = i32
    lib.fa_decode_run_token_scales.argtypes = [P, P, P, i64, f32, P, P, P, P, P]
    lib.fa_decode_run_token_scales.restype = i32
    lib.fa_decode_run_head_scales.argtypes = [P, P, P, i64, f32, P, P, P, P, P]
    lib.fa_decode_run_head_scales.restype = i32
    lib.fa_decode_run_block_scales.argtypes = [P, P, P, i64, f32, P, P, P, P, P]
    lib.fa_decode_run_block_scales.restype = i32
    lib.fa_cascade_run_block_scales.argtypes = [P, P, P, i64, f32, P, P, P, P, P]
    lib.fa_cascade_run_block_scales.restype = i32
    lib.fa_append_workspace_size.argtypes = [i32, i64]
    lib.fa_append_workspace_size.restype = sz
    lib.fa_append_plan.argtypes = [P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32, P, i32, i32,
                                   P, sz, P, ctypes.POINTER(P)]
    lib.fa_append_plan.restype = i32
    lib.fa_append_plan_axes.argtypes = [P, P, P, P, P, i32, P, i32, i32, i32, i32, i32, i32, i32,
                                        P, i32, i32, P, sz, P, ctypes.POINTER(P)]
    lib.fa_append_plan_axes.restype = i32
    lib.fa_weights_workspace_size.argtypes = [i32, i64]
    lib.fa_weights_workspace_size.restype = sz
    lib.fa_weights_plan.argtypes = [P, P, P, P, i32, i32, i32, i32, i32, i32, i32, P, sz, P,
                                    ctypes.POINTER(P)]
    lib.fa_weights_plan.restype = i32
    lib.fa_weights_run.argtypes = [P, P, P, i64, f32, f32, P, P, P]
    lib.fa_weights_run.restype = i32
    for name in ("fa_weights_run_head_scales", "fa_weights_run_token_scales",
                 "fa_weights_run_block_scales"):
        f = getattr(lib, name)
        f.argtypes = [P, P, P, i64, f32, P, P, P, P]
        f.restype = i32
    lib.fa_evict_workspace_size.argtypes = [i32, i64, i32]
    lib.fa_evict_workspace_size.restype = sz
    lib.fa_evict_plan.argtypes = [P, P, P, P, P, i32, i32, i32, i32, i32, P, sz, P,
                                  ctypes.POINTER(P)]
    lib.fa_evict_plan.restype = i32
    lib.fa_evict_run.argtypes = [P, P, i64, P, P, P, P]
    lib.fa_evict_run.restype = i32
    for kind in ("weights", "evict"):
        f = getattr(lib, f"fa_{kind}_check")
        f.argtypes = [P, P, ctypes.POINTER(i32)]
        f.restype = i32
        f = getattr(lib, f"fa_{kind}_plan_destroy")
        f.argtypes = [P]
        f.restype = i32
    lib.fa_prefill_workspace_size.argtypes = [P, P, P, i32, i32, i32, i32, i32, i32]
    lib.fa_prefill_workspace_size.restype = sz
    lib.fa_prefill_plan.argtypes = [P, P, P, P, i32, i32, i32, i32, i32, i32, i32, P, sz, P,
                                    ctypes.POINTER(P)]
    lib.fa_prefill_plan.restype = i32
    lib.fa_prefill_run.argtypes = [P, P, P, i64, f32, f32, f32, P, P, P]
    lib.fa_prefill_run.restype = i32
    for name in ("fa_prefill_run_head_scales", "fa_prefill_run_token_scales",
                 "fa_prefill_run_block_scales"):
        f = getattr(lib, name)
        f.argtypes = [P, P, P, i64, f32, P, P, P, P, P]
        f.restype = i32
    lib.fa_prefill_check.argtypes = [P, P, ctypes.POINTER(i32)]
    lib.fa_prefill_check.restype = i32
    lib.fa_prefill_plan_destroy.argtypes = [P]
    lib.fa_prefill_plan_destroy.restype = i32
    ip = ctypes.POINTER(i32)
    lib.fa_plan_prefill_host.argtypes = [P, P, P, i32, i32, i32, i32, P, P, i32, P, i32, ip, ip,
                                         ip, ip]
    lib.fa_plan_prefill_host.restype = i32
    lib.fa_append_run.argtypes = [P, P, P, P, P, P, i64, f32, f32, P]
    lib.fa_append_run.restype = i32
    for name in ("fa_append_run_head_scales", "fa_append_run_token_scales",
                 "fa_append_run_block_scales"):
        f = getattr(lib, name)
        f.argtypes = [P, P, P, P, P, P, i64, P, P, P]
        f.restype = i32
    lib.fa_append_check.argtypes = [P, P, ctypes.POINTER(i32)]
    lib.fa_append_check.restype = i32
    lib.fa_append_plan_destroy.argtypes = [P]
    lib.fa_append_plan_destroy.restype = i32
    lib.fa_decode_run_unified_max.argtypes = [P, P, P, i64, f32, f32, f32, f32, P, P, P]
    lib.fa_decode_run_unified_max.restype = i32
    lib.fa_decode_unified_max_fallbacks.argtypes = [P, P, ctypes.POINTER(i32)]
    lib.fa_decode_unified_max_fallbacks.restype = i32
    lib.fa_cascade_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.fa_cascade_workspace_size.restype = sz
    lib.fa_cascade_plan.argtypes = [P, i32, P, P, P, i32, i32, i32, i32, i32, i32, i32, P, sz, P,
                                    ctypes.POINTER(P)]
    lib.fa_cascade_plan.restype = i32
    lib.fa_cascade_run.argtypes = [P, P, P, i64, f32, P, P, P]
    lib.fa_cascade_run.restype = i32
    lib.fa_cascade_run_scaled.argtypes = [P, P, P, i64, f32, f32, f32, P, P, P]
    lib.fa_cascade_run_scaled.restype = i32
    lib.fa_cascade_plan_destroy.argtypes = [P]
    lib.fa_cascade_plan_destroy.restype = i32
    lib.fa_cascade_check.argtypes = [P, P, ctypes.POINTER(i32)]
    lib.fa_cascade_check.restype = i32
    lib.fa_merge_states.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, P]
    lib.fa_merge_states.restype = i32
    lib.fa_decode_plan_destroy.argtypes = [P]
    lib.fa_decode_plan_destroy.restype = i32
    lib.fa_decode_plan_get_info.argtypes = [P, ctypes.POINTER(PlanInfo)]
    lib.fa_decode_plan_get_info.restype = i32
    pp = ctypes.POINTER(ctypes.POINTER(ctypes.c_int32))
    lib.fa_decode_plan_get_work.argtypes = [P, pp, pp, pp]
    lib.fa_decode_plan_get_work.restype = i32
    lib.fa_plan_work_host.argtypes = [P, P, i32, i32, i32, i32, i32, ctypes.c_double, P, P, P,
                                      ctypes.POINTER(i32), ctypes.POINTER(i32),
                                      ctypes.POINTER(i32), ctypes.POINTER(i32)]
    lib.fa_plan_work_host.restype = i32
    lib.fa_plan_work_host_heads.argtypes = [P, P, i32, i32, i32, i32, i32, P, P, P, P, P, P, P]
    lib.fa_plan_work_host_heads.restype = i32
    lib.fa_plan_work_host_buckets.argtypes = [P, P, P, i32, i32, i32, i32, i32, P, i32,
                                              ctypes.c_int64, P, P, P, P, P, P, P, P, P, P]
    lib.fa_plan_work_host_buckets.restype = i32
    lib.fa_decode_check.argtypes = [P, P, ctypes.POINTER(i32)]
    lib.fa_decode_check.restype = i32
    lib.fa_decode_set_timing_events.argtypes = [P, P, P]
    lib.fa_decode_set_timing_events.restype = i32
    lib.fa_cascade_set_timing_events.argtypes = [P, P, P]
    lib.fa_cascade_set_timing_events.restype = i32
    lib.fa_decode_static.argtypes = [P, P, P, i32, i32, i32, i32, i32, i32, i32, P, P, i64,
                                     f32, f32, f32, P, P, P]
    lib.fa_decode_static.restype = i32
    lib.fa_decode_static_check.argtypes = [P, ctypes.POINTER(i32)]
    lib.fa_decode_static_check.restype = i32
    lib.fa_library_get_stats.argtypes = [ctypes.POINTER(LibraryStats)]
    lib.fa_library_get_stats.restype = i32
    return lib


_lib_handle: ctypes.CDLL | None = None


def _L() -> ctypes.CDLL:
    """The loaded library.  Raises if it was never built: there is no fallback."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it first with "
                "`python -c 'import __graft_entry__ as g; g.build()'` (nvcc, sm_103a)")
        _lib_handle = _load()
    return _lib_handle


def library() -> ctypes.CDLL:
    """Load (once) and return the ctypes handle of libfadecode.so."""
    return _L()


def _check(status: int, what: str) -> None:
    if status != FA_OK:
        raise FaError(status, what)


# torch's current stream of a device as a raw handle, without building a
# Stream object (a few microseconds a call on the plan and run paths)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream) -> int | None:
    if stream is None:
        if _current_raw_stream is not None:
            return _current_raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _as_stream(stream) -> torch.cuda.Stream:
    """A torch stream, or one of a raw handle."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    # (an ExternalStream of the null handle would be a new stream)
    return torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()


def _empty(shape, dtype, device, stream, **kw) -> torch.Tensor:
    """A tensor that a call running on `stream` (None: the current one) writes.
    It comes from that stream's memory: what the current stream has freed may
    still be in use there.  And it is given back once the current stream, whose
    caller gets it, is done with it too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device, **kw)
    stream = _as_stream(stream)
    current = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device, **kw)
    if t.is_cuda:
        t.record_stream(current)
    return t


def _host_i32(t) -> np.ndarray:
    if isinstance(t, torch.Tensor):
        if t.device.type == "cpu" and t.dtype == torch.int32 and t.is_contiguous():
            return t.detach().numpy()  # no copy
        t = t.detach().to("cpu").numpy()
    if isinstance(t, np.ndarray) and t.dtype == np.int32 and t.flags.c_contiguous:
        return t
    t = np.asarray(t)
    try:
        with np.errstate(invalid="ignore"):
            a = np.ascontiguousarray(t, dtype=np.int32)
        fits = t.dtype == np.int32 or np.array_equal(a, t.reshape(a.shape))
    except OverflowError:
        fits = False
    if not fits:
        raise ValueError("host arrays must hold whole numbers of 32 bits")
    return a


def _host_i32_ptr(t):
    """(owner, address, length) of a host int32 array: a contiguous CPU int32
    tensor is passed as it is, anything else goes through _host_i32."""
    if (isinstance(t, torch.Tensor) and t.device.type == "cpu" and t.dtype == torch.int32
            and t.dim() == 1 and t.is_contiguous()):
        return t, t.data_ptr(), t.shape[0]
    a = _host_i32(t)
    return a, a.ctypes.data, a.shape[0]


def _reachable(t: torch.Tensor) -> bool:
    """Device memory, or page-locked host memory that the kernels read and
    write directly over the CPU-GPU link (on a GB300 node, NVLink-C2C)."""
    return t.is_cuda or t.is_pinned()


def _i32_at(address: int, i: int) -> int:
    """Element i of a host int32 array (indexing a tensor takes 3 us of a plan)."""
    return ctypes.c_int32.from_address(address + 4 * i).value


def _check_indices(indices: torch.Tensor, indptr: int, batch: int) -> None:
    """The page table of a batch: the kernels read indptr[batch] entries of it."""
    if indices.dtype != torch.int32 or not _reachable(indices) or not indices.is_contiguous():
        raise ValueError("indices must be a contiguous int32 CUDA or page-locked tensor")
    if batch > 0 and indices.numel() < _i32_at(indptr, batch):
        raise ValueError(f"indices holds {indices.numel()} pages, indptr asks for "
                         f"{_i32_at(indptr, batch)}")


def _cuda_device(t: torch.Tensor) -> torch.device:
    """The device a tensor lives on, or the current CUDA device for host memory."""
    return t.device if t.is_cuda else torch.device("cuda", torch.cuda.current_device())


def _dtype_code(dt) -> int:
    if dt not in DTYPE_CODES:
        raise ValueError(f"unsupported dtype {dt}")
    return DTYPE_CODES[dt]


def workspace_size(batch: int, num_qo_heads: int, num_kv_heads: int, head_dim: int) -> int:
    """Bytes of device workspace a plan of this batch may need (current device)."""
    n = _L().fa_decode_workspace_size(batch, num_qo_heads, num_kv_heads, head_dim)
    if n == 0:
        raise ValueError("invalid shape or no CUDA device")
    return int(n)


class DecodePlan:
    """A planned decode batch.  Holds the library's plan handle and keeps the
    tensors it refers to (indices, workspace) alive."""

    def __init__(self, handle, indices, workspace, q_dtype, kv_dtype, shape, q_len=1,
                 total_q_rows=None):
        self._h = handle
        self._indices = indices
        self._workspace = workspace
        self.q_dtype = q_dtype
        self.kv_dtype = kv_dtype
        self.q_len = q_len
        self.total_q_rows = total_q_rows  # ragged plans: rows of q / o
        self.batch, self.num_qo_heads, self.num_kv_heads, self.head_dim, self.page_size = shape
        B, Hq, D = self.batch, self.num_qo_heads, self.head_dim
        if total_q_rows is not None:
            self._q_shape = (total_q_rows, Hq, D)
        else:
            self._q_shape = (B, Hq, D) if q_len == 1 else (B, q_len, Hq, D)
        self._page_shape = (2, self.page_size, self.num_kv_heads, D)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            _L().fa_decode_plan_destroy(h)
            self._h = None

    @property
    def info(self) -> dict:
        i = PlanInfo()
        _check(_L().fa_decode_plan_get_info(self._h, ctypes.byref(i)), "fa_decode_plan_get_info")
        return i.as_dict()

    def work(self):
        """(cta_offsets [num_ctas+1], segments [n, 8], merge [m, 4]) as numpy int32."""
        info = self.info
        co = ctypes.POINTER(ctypes.c_int32)()
        sg = ctypes.POINTER(ctypes.c_int32)()
        mg = ctypes.POINTER(ctypes.c_int32)()
        _check(_L().fa_decode_plan_get_work(self._h, ctypes.byref(co), ctypes.byref(sg),
                                            ctypes.byref(mg)), "fa_decode_plan_get_work")
        n_c, n_s, n_m = info["num_ctas"], info["num_segments"], info["num_merge_units"]
        cta = np.ctypeslib.as_array(co, shape=(n_c + 1,)).copy()
        seg = (np.ctypeslib.as_array(sg, shape=(n_s * SEGMENT_INTS,)).reshape(n_s, SEGMENT_INTS).copy()
               if n_s else np.zeros((0, SEGMENT_INTS), np.int32))
        mer = (np.ctypeslib.as_array(mg, shape=(n_m * MERGE_INTS,)).reshape(n_m, MERGE_INTS).copy()
               if n_m else np.zeros((0, MERGE_INTS), np.int32))
        return cta, seg, mer

    def run(self, q: torch.Tensor, paged_kv: torch.Tensor, *, sm_scale: float | None = None,
            k_scale: float = 1.0, v_scale: float = 1.0, out: torch.Tensor | None = None,
            lse: torch.Tensor | None = None, return_lse: bool = True, stream=None):
        """Decode attention; returns (o, lse) (lse None if return_lse is False)."""
        out, lse = self._outputs(q, paged_kv, out, lse, return_lse, stream)
        _check(_L().fa_decode_run(
            self._h, q.data_ptr(), paged_kv.data_ptr(), paged_kv.shape[0],
            0.0 if sm_scale is None else float(sm_scale), float(k_scale), float(v_scale),
            out.data_ptr(), lse.data_ptr() if lse is not None else None,
            _stream_handle(stream)), "fa_decode_run")
        return out, lse

    def run_unified_max(self, q: torch.Tensor, paged_kv: torch.Tensor, max_bound: float, *,
                        sm_scale: float | None = None, k_scale: float = 1.0,
                        v_scale: float = 1.0, out: torch.Tensor | None = None,
                        lse: torch.Tensor | None = None, return_lse: bool = True, stream=None):
        """Decode attention with the softmax referenced to a static bound
        `max_bound` on the logits sm_scale * k_scale * (q . k) instead of a
        running maximum (bf16 plans, groups 2/4/8); returns (o, lse)."""
        out, lse = self._outputs(q, paged_kv, out, lse, return_lse, stream)
        _check(_L().fa_decode_run_unified_max(
            self._h, q.data_ptr(), paged_kv.data_ptr(), paged_kv.shape[0],
            0.0 if sm_scale is None else float(sm_scale), float(k_scale), float(v_scale),
            float(max_bound), out.data_ptr(), lse.data_ptr() if lse is not None else None,
            _stream_handle(stream)), "fa_decode_run_unified_max")
        return out, lse

    def run_head_scales(self, q: torch.Tensor, paged_kv: torch.Tensor, k_scales: torch.Tensor,
                        v_scales: torch.Tensor, *, sm_scale: float | None = None,
                        out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                        return_lse: bool = True, stream=None):
        """Decode over an E4M3 cache with one scale per kv head: k_scales /
        v_scales [num_kv_heads] float32 CUDA tensors; returns (o, lse)."""
        for s in (k_scales, v_scales):
            if (s.dtype != torch.float32 or tuple(s.shape) != (self.num_kv_heads,)
                    or not s.is_contiguous() or not s.is_cuda):
                raise ValueError(f"scales must be contiguous float32 CUDA tensors "
                                 f"[{self.num_kv_heads}]")
        out, lse = self._outputs(q, paged_kv, out, lse, return_lse, stream)
        _check(_L().fa_decode_run_head_scales(
            self._h, q.data_ptr(), paged_kv.data_ptr(), paged_kv.shape[0],
            0.0 if sm_scale is None else float(sm_scale), k_scales.data_ptr(),
            v_scales.data_ptr(), out.data_ptr(), lse.data_ptr() if lse is not None else None,
            _stream_handle(stream)), "fa_decode_run_head_scales")
        return out, lse

    def run_block_scales(self, q: torch.Tensor, paged_kv: torch.Tensor, k_scales: torch.Tensor,
                         v_scales: torch.Tensor, *, sm_scale: float | None = None,
                         out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                         return_lse: bool = True, stream=None):
        """Decode over an E4M3 cache with one scale per block of tokens (a page)
        and kv head: k_scales / v_scales [num_pages, num_kv_heads] float32 CUDA
        tensors, as AppendPlan.run_block_scales writes them; returns (o, lse)."""
        out, lse = self._outputs(q, paged_kv, out, lse, return_lse, stream)
        device = self._workspace.get_device()
        if paged_kv.get_device() != device:
            raise ValueError("paged_kv must be on the plan's device")
        if ((q.get_device() != device and q.is_cuda) or (out.get_device() != device and out.is_cuda)
                or (lse is not None and lse.get_device() != device and lse.is_cuda)):
            raise ValueError("q / out / lse must be on the plan's device, or page-locked")
        _check_scales((k_scales, v_scales), (paged_kv.shape[0], self.num_kv_heads), paged_kv)
        _check(_L().fa_decode_run_block_scales(
            self._h, q.data_ptr(), paged_kv.data_ptr(), paged_kv.shape[0],
            0.0 if sm_scale is None else float(sm_scale), k_scales.data_ptr(),
            v_scales.data_ptr(), out.data_ptr(), lse.data_ptr() if lse is not None else None,
            _stream_handle(stream)), "fa_decode_run_block_scales")
        return out, lse

    def unified_max_fallbacks(self, stream=None) -> int:
        """Synchronise; return and clear the count of unified-max re-centrings."""
        n = ctypes.c_int(0)
        _check(_L().fa_decode_unified_max_fallbacks(self._h, _stream_handle(stream),
                                                    ctypes.byref(n)),
               "fa_decode_unified_max_fallbacks")
        return int(n.value)

    def _outputs(self, q, paged_kv, out, lse, return_lse, stream):
        """Check q / paged_kv against the plan; allocate missing outputs."""
        if q.dtype is not self.q_dtype or paged_kv.dtype is not self.kv_dtype:
            raise TypeError("q / paged_kv dtype differs from the plan")
        if q.shape != self._q_shape or not q.is_contiguous() or not _reachable(q):
            raise ValueError(f"q must be a contiguous CUDA or page-locked tensor "
                             f"{list(self._q_shape)}")
        if (paged_kv.dim() != 5 or paged_kv.shape[1:] != self._page_shape
                or not paged_kv.is_contiguous() or not paged_kv.is_cuda):
            raise ValueError("paged_kv must be a contiguous CUDA tensor "
                             "[num_pages, 2, page_size, num_kv_heads, head_dim]")
        pinned = {} if q.is_cuda else {"pin_memory": True}  # outputs follow q: device, or
        if out is not None:                                 # page-locked host memory
            _room(out, q.nbytes)
        elif stream is None:
            out = torch.empty_like(q, **pinned)
        else:
            out = _empty(q.shape, q.dtype, q.device, stream, **pinned)
        if lse is not None:
            _room(lse, q.numel() // self.head_dim * 4)
        elif return_lse:
            lse = _empty(q.shape[:-1], torch.float32, q.device, stream, **pinned)
        for t in (out, lse):
            if t is not None and (not _reachable(t) or not t.is_contiguous()):
                raise ValueError("out / lse must be contiguous CUDA or page-locked tensors")
        return out, lse

    def run_token_scales(self, q: torch.Tensor, paged_kv: torch.Tensor, k_scales: torch.Tensor,
                         v_scales: torch.Tensor, *, sm_scale: float | None = None,
                         out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                         return_lse: bool = True, stream=None):
        """Decode over an E4M3 cache with per-token, per-kv-head scales
        k_scales / v_scales [num_pages, num_kv_heads, page_size] float32."""
        B, Hq, D = self.batch, self.num_qo_heads, self.head_dim
        if q.dtype != self.q_dtype or paged_kv.dtype != self.kv_dtype:
            raise TypeError("q / paged_kv dtype differs from the plan")
        want = (paged_kv.shape[0], self.num_kv_heads, self.page_size)
        for t in (k_scales, v_scales):
            if (t.dtype != torch.float32 or tuple(t.shape) != want or not t.is_contiguous()
                    or not t.is_cuda):
                raise ValueError(f"scales must be contiguous float32 CUDA tensors {want}")
        if tuple(q.shape) != (B, Hq, D) or not q.is_contiguous():
            raise ValueError(f"q must be a contiguous CUDA tensor [{B}, {Hq}, {D}]")
        if out is None:
            out = _empty((B, Hq, D), q.dtype, q.device, stream)
        if return_lse and lse is None:
            lse = _empty((B, Hq), torch.float32, q.device, stream)
        _room(out, q.nbytes)
        if lse is not None:
            _room(lse, B * Hq * 4)
        _check(_L().fa_decode_run_token_scales(
            self._h, q.data_ptr(), paged_kv.data_ptr(), paged_kv.shape[0],
            0.0 if sm_scale is None else float(sm_scale), k_scales.data_ptr(),
            v_scales.data_ptr(), out.data_ptr(), lse.data_ptr() if lse is not None else None,
            _stream_handle(stream)), "fa_decode_run_token_scales")
        return out, lse

    def check(self, stream=None) -> int:
        """Synchronise and return the device-check flags (0 = clean)."""
        flags = ctypes.c_int(0)
        st = _L().fa_decode_check(self._h, _stream_handle(stream), ctypes.byref(flags))
        if st not in (FA_OK, -5):
            _check(st, "fa_decode_check")
        return int(flags.value)

    def set_timing_events(self, before, after) -> None:
        """Record torch.cuda.Events around the launches of later runs: the decode
        kernel, and the merge kernel or a ragged plan's other buckets where the
        plan has them (None = off).

        torch creates an event lazily at its first record, so record each
        event once from torch before handing it over."""
        _check(_L().fa_decode_set_timing_events(self._h, *_event_handles(before, after)),
               "fa_decode_set_timing_events")


def _room(t, nbytes) -> torch.Tensor:
    """An output of the caller's, if it holds what a run writes."""
    if t.nbytes < nbytes:
        raise ValueError(f"out / lse too small: {t.nbytes} bytes, a run writes {nbytes}")
    return t


def _check_scales(scales, shape, paged_kv) -> None:
    device = paged_kv.get_device()
    for s in scales:
        if (s.dtype is not torch.float32 or s.shape != shape or not s.is_contiguous()
                or s.get_device() != device):
            raise ValueError(f"scales must be contiguous float32 tensors {list(shape)} on the "
                             "device of paged_kv")


def _event_handles(before, after):
    """CUDA event handles of two recorded torch.cuda.Events (None = off).
    torch creates an event lazily at its first record, so record each event
    once from torch before handing it over."""
    for ev in (before, after):
        if ev is not None and not ev.cuda_event:
            raise ValueError("record the torch.cuda.Event once before passing it")
    return (ctypes.c_void_p(before.cuda_event) if before is not None else None,
            ctypes.c_void_p(after.cuda_event) if after is not None else None)


def plan(indptr, indices: torch.Tensor, last_page_len, num_qo_heads: int, num_kv_heads: int,
         head_dim: int, page_size: int, *, q_data_type=torch.bfloat16,
         kv_data_type=None, workspace: torch.Tensor | None = None, stream=None) -> DecodePlan:
    """Plan a decode batch.  indptr/last_page_len may live on the host or the
    device (they are read on the host); indices must be an int32 CUDA tensor."""
    kv_data_type = q_data_type if kv_data_type is None else kv_data_type
    indptr_h, indptr_p, n_indptr = _host_i32_ptr(indptr)
    last_h, last_p, n_last = _host_i32_ptr(last_page_len)
    B = n_indptr - 1
    if n_last < B:
        raise ValueError("last_page_len shorter than the batch")
    _check_indices(indices, indptr_p, B)
    if workspace is None:
        workspace = _empty(workspace_size(B, num_qo_heads, num_kv_heads, head_dim), torch.uint8,
                           _cuda_device(indices), stream)
    handle = ctypes.c_void_p()
    _check(_L().fa_decode_plan(
        indptr_p, indices.data_ptr() if indices.numel() else None,
        last_p if B else None, B, num_qo_heads, num_kv_heads, head_dim, page_size,
        _dtype_code(q_data_type), _dtype_code(kv_data_type), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_handle(stream),
        ctypes.byref(handle)), "fa_decode_plan")
    return DecodePlan(handle.value, indices, workspace, q_data_type, kv_data_type,
                      (B, num_qo_heads, num_kv_heads, head_dim, page_size))


def plan_multi_token(indptr, indices: torch.Tensor, last_page_len, q_len: int, num_qo_heads: int,
                     num_kv_heads: int, head_dim: int, page_size: int, *,
                     q_data_type=torch.bfloat16, kv_data_type=None,
                     workspace: torch.Tensor | None = None, stream=None) -> DecodePlan:
    """Plan multi-token decode: q_len query tokens per request (the last q_len
    cache positions), query token i attending to positions <= len - q_len + i.
    run() then takes q [B, q_len, Hq, D] and returns o of that shape and lse
    [B, q_len, Hq]."""
    kv_data_type = q_data_type if kv_data_type is None else kv_data_type
    indptr_h, indptr_p, n_indptr = _host_i32_ptr(indptr)
    last_h, last_p, n_last = _host_i32_ptr(last_page_len)
    B = n_indptr - 1
    if n_last < B:
        raise ValueError("last_page_len shorter than the batch")
    _check_indices(indices, indptr_p, B)
    if workspace is None:
        if (num_qo_heads // max(1, num_kv_heads)) * q_len > 8:   # the ragged-q kernels
            n = _L().fa_decode_workspace_size_ragged_q(B, num_qo_heads, num_kv_heads, head_dim)
        else:
            n = workspace_size(B, num_qo_heads * q_len, num_kv_heads, head_dim)
        if n == 0:
            raise ValueError("invalid shape or no CUDA device")
        workspace = _empty(int(n), torch.uint8, _cuda_device(indices), stream)
    handle = ctypes.c_void_p()
    _check(_L().fa_decode_plan_multi_token(
        indptr_p, indices.data_ptr() if indices.numel() else None,
        last_p if B else None, B, q_len, num_qo_heads, num_kv_heads, head_dim,
        page_size, _dtype_code(q_data_type), _dtype_code(kv_data_type), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_handle(stream),
        ctypes.byref(handle)), "fa_decode_plan_multi_token")
    return DecodePlan(handle.value, indices, workspace, q_data_type, kv_data_type,
                      (B, num_qo_heads, num_kv_heads, head_dim, page_size), q_len=q_len)


def plan_ragged_q(indptr, indices: torch.Tensor, last_page_len, qo_indptr, num_qo_heads: int,
                  num_kv_heads: int, head_dim: int, page_size: int, *,
                  q_data_type=torch.bfloat16, kv_data_type=None,
                  workspace: torch.Tensor | None = None, stream=None) -> DecodePlan:
    """Plan decode with qo_indptr[i+1] - qo_indptr[i] query tokens for request
    i (the last positions of its cache, causal among themselves).  run() then
    takes q [qo_indptr[-1], Hq, D] and returns o of that shape and lse
    [qo_indptr[-1], Hq]."""
    kv_data_type = q_data_type if kv_data_type is None else kv_data_type
    indptr_h, indptr_p, n_indptr = _host_i32_ptr(indptr)
    last_h, last_p, n_last = _host_i32_ptr(last_page_len)
    qo_h, qo_p, n_qo = _host_i32_ptr(qo_indptr)
    B = n_indptr - 1
    if n_last < B or n_qo != B + 1:
        raise ValueError("last_page_len shorter than the batch, or qo_indptr not batch + 1 long")
    _check_indices(indices, indptr_p, B)
    if workspace is None:
        n = _L().fa_decode_workspace_size_ragged_q(B, num_qo_heads, num_kv_heads, head_dim)
        if n == 0:
            raise ValueError("invalid shape or no CUDA device")
        workspace = _empty(int(n), torch.uint8, _cuda_device(indices), stream)
    handle = ctypes.c_void_p()
    _check(_L().fa_decode_plan_ragged_q(
        indptr_p, indices.data_ptr() if indices.numel() else None,
        last_p if B else None, qo_p, B, num_qo_heads, num_kv_heads, head_dim,
        page_size, _dtype_code(q_data_type), _dtype_code(kv_data_type), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_handle(stream),
        ctypes.byref(handle)), "fa_decode_plan_ragged_q")
    total_q = int(np.asarray(qo_h)[B]) if B >= 0 else 0
    return DecodePlan(handle.value, indices, workspace, q_data_type, kv_data_type,
                      (B, num_qo_heads, num_kv_heads, head_dim, page_size),
                      total_q_rows=total_q)


def run(p: DecodePlan, q, paged_kv, **kw):
    return p.run(q, paged_kv, **kw)


def merge_states(o_a: torch.Tensor, lse_a: torch.Tensor, o_b: torch.Tensor, lse_b: torch.Tensor,
                 *, out: torch.Tensor | None = None, lse_out: torch.Tensor | None = None,
                 stream=None):
    """Merge two sets of states o [n, H, D] (f32/bf16/f16) with lse [n, H] fp32."""
    if o_a.shape != o_b.shape or lse_a.shape != lse_b.shape or o_a.dtype != o_b.dtype:
        raise ValueError("state shapes / dtypes differ")
    if o_a.dim() != 3 or tuple(lse_a.shape) != tuple(o_a.shape[:2]):
        raise ValueError("o must be [n, H, D] and lse [n, H]")
    for t in (o_a, o_b, lse_a, lse_b):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("inputs must be contiguous CUDA tensors")
    if lse_a.dtype != torch.float32 or lse_b.dtype != torch.float32:
        raise TypeError("lse must be float32")
    n, H, D = o_a.shape
    out = _empty(o_a.shape, o_a.dtype, o_a.device, stream) if out is None else out
    if lse_out is None:
        lse_out = _empty(lse_a.shape, lse_a.dtype, lse_a.device, stream)
    _check(_L().fa_merge_states(o_a.data_ptr(), lse_a.data_ptr(), o_b.data_ptr(),
                                lse_b.data_ptr(), out.data_ptr(), lse_out.data_ptr(), n, H, D,
                                _dtype_code(o_a.dtype), _stream_handle(stream)),
           "fa_merge_states")
    return out, lse_out


def plan_work_host(indptr, last_page_len, num_kv_heads: int, page_size: int, max_ctas: int,
                   min_pages_per_cta: int = 8, pool_fraction: float = 0.0, heads: bool = False):
    """Host-only work-list builder (no GPU).  Returns (cta_offsets, segments [n,8],
    merge [m,4], n_slots); segments cta_offsets[-1]: are the run-time pool.
    heads=True: the head-grouped plan fa_decode_plan makes by default
    (fa_plan_work_host_heads; no pool)."""
    indptr_h, indptr_p, n_indptr = _host_i32_ptr(indptr)
    last_h, last_p, n_last = _host_i32_ptr(last_page_len)
    B = n_indptr - 1
    if n_last < B:
        raise ValueError("last_page_len shorter than the batch")
    cuts = max_ctas * 7 + 1
    cta = np.zeros(max_ctas + 1, np.int32)
    seg = np.zeros(((B * num_kv_heads + cuts) * SEGMENT_INTS,), np.int32)
    mer = np.zeros((cuts * MERGE_INTS,), np.int32)
    n_c, n_s, n_m, n_sl = (ctypes.c_int() for _ in range(4))
    if heads:
        _check(_L().fa_plan_work_host_heads(
            indptr_p, last_p if B else None, B, num_kv_heads, page_size, max_ctas,
            min_pages_per_cta, cta.ctypes.data, seg.ctypes.data, mer.ctypes.data,
            ctypes.byref(n_c), ctypes.byref(n_s), ctypes.byref(n_m), ctypes.byref(n_sl)),
            "fa_plan_work_host_heads")
    else:
        _check(_L().fa_plan_work_host(indptr_p, last_p if B else None, B,
                                      num_kv_heads, page_size, max_ctas, min_pages_per_cta,
                                      float(pool_fraction), cta.ctypes.data, seg.ctypes.data,
                                      mer.ctypes.data, ctypes.byref(n_c), ctypes.byref(n_s),
                                      ctypes.byref(n_m), ctypes.byref(n_sl)), "fa_plan_work_host")
    return (cta[: n_c.value + 1].copy(), seg[: n_s.value * SEGMENT_INTS].reshape(-1, SEGMENT_INTS).copy(),
            mer[: n_m.value * MERGE_INTS].reshape(-1, MERGE_INTS).copy(), n_sl.value)


def plan_work_host_buckets(indptr, last_page_len, qo_indptr, group: int, num_kv_heads: int,
                           page_size: int, widest_tiles: int, max_ctas_by_tiles,
                           one_tile_own: bool = False, min_own_units: int = 0,
                           all_buckets: bool = False):
    """Host-only buckets of a ragged plan (fa_plan_work_host_buckets, no GPU).
    Returns None when the batch stays one launch of the widest kernel, else
    (cta_offsets, segments [n,8], merge [m,4], bucket_tiles, bucket_first_cta,
    slot_columns) for the buckets' concatenated work list."""
    indptr_h, indptr_p, n_indptr = _host_i32_ptr(indptr)
    last_h, last_p, n_last = _host_i32_ptr(last_page_len)
    qo_h, qo_p, n_qo = _host_i32_ptr(qo_indptr)
    B = n_indptr - 1
    if n_last < B or n_qo < B + 1:
        raise ValueError("last_page_len / qo_indptr shorter than the batch")
    mc = np.zeros(4, np.int32)
    mc[:len(max_ctas_by_tiles)] = max_ctas_by_tiles
    total = int(mc.sum())
    cuts = sum(int(m) * 7 + 1 for m in mc)
    cta = np.zeros(total + 1, np.int32)
    seg = np.zeros(((B * num_kv_heads + cuts) * SEGMENT_INTS,), np.int32)
    mer = np.zeros((cuts * MERGE_INTS,), np.int32)
    tiles = np.zeros(4, np.int32)
    first = np.zeros(4, np.int32)
    n_c, n_s, n_m, n_b = (ctypes.c_int() for _ in range(4))
    cols = ctypes.c_int64()
    flags = (1 if one_tile_own else 0) | (2 if all_buckets else 0)
    _check(_L().fa_plan_work_host_buckets(
        indptr_p, last_p if B else None, qo_p, B, group, num_kv_heads, page_size, widest_tiles,
        mc.ctypes.data, flags, int(min_own_units), cta.ctypes.data, seg.ctypes.data,
        mer.ctypes.data, ctypes.byref(n_c), ctypes.byref(n_s), ctypes.byref(n_m),
        ctypes.byref(n_b), tiles.ctypes.data, first.ctypes.data, ctypes.byref(cols)),
        "fa_plan_work_host_buckets")
    if n_b.value == 0:
        return None
    nb = n_b.value
    return (cta[: n_c.value + 1].copy(),
            seg[: n_s.value * SEGMENT_INTS].reshape(-1, SEGMENT_INTS).copy(),
            mer[: n_m.value * MERGE_INTS].reshape(-1, MERGE_INTS).copy(),
            tiles[:nb].copy(), first[:nb].copy(), cols.value)


class CascadePlan:
    """A planned cascade batch: one shared prefix of whole pages, then each
    request's own pages.  Keeps the index tensors and the workspace alive."""

    def __init__(self, handle, keep, q_dtype, shape, kv_dtype=None):
        self._h = handle
        self._keep = keep
        self.q_dtype = q_dtype
        self.kv_dtype = q_dtype if kv_dtype is None else kv_dtype
        self.batch, self.num_qo_heads, self.num_kv_heads, self.head_dim = shape

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            _L().fa_cascade_plan_destroy(h)
            self._h = None

    def run(self, q: torch.Tensor, paged_kv: torch.Tensor, *, sm_scale: float | None = None,
            k_scale: float = 1.0, v_scale: float = 1.0, out: torch.Tensor | None = None,
            lse: torch.Tensor | None = None, return_lse: bool = True, stream=None):
        """Cascade decode; k_scale / v_scale are an E4M3 cache's per-tensor
        scales (1 for a 16-bit cache)."""
        out, lse = self._outputs(q, paged_kv, out, lse, return_lse, stream)
        _check(_L().fa_cascade_run_scaled(
            self._h, q.data_ptr(), paged_kv.data_ptr(), paged_kv.shape[0],
            0.0 if sm_scale is None else float(sm_scale), float(k_scale), float(v_scale),
            out.data_ptr(), lse.data_ptr() if lse is not None else None,
            _stream_handle(stream)), "fa_cascade_run_scaled")
        return out, lse

    def run_block_scales(self, q: torch.Tensor, paged_kv: torch.Tensor, k_scales: torch.Tensor,
                         v_scales: torch.Tensor, *, sm_scale: float | None = None,
                         out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                         return_lse: bool = True, stream=None):
        """Cascade decode over an E4M3 cache with one scale per page and kv head:
        k_scales / v_scales [num_pages, num_kv_heads] float32."""
        for t in (q, out, lse):
            if t is not None and (t.device != paged_kv.device or not t.is_contiguous()):
                raise ValueError("q / out / lse must be contiguous, on the device of paged_kv")
        want = (2, 16, self.num_kv_heads, self.head_dim)
        if paged_kv.shape[1:] != want or paged_kv.get_device() != self._keep[-1].get_device():
            raise ValueError(f"paged_kv must be [num_pages, {', '.join(map(str, want))}] on the "
                             "plan's device")
        out, lse = self._outputs(q, paged_kv, out, lse, return_lse, stream)
        _check_scales((k_scales, v_scales), (paged_kv.shape[0], self.num_kv_heads), paged_kv)
        _check(_L().fa_cascade_run_block_scales(
            self._h, q.data_ptr(), paged_kv.data_ptr(), paged_kv.shape[0],
            0.0 if sm_scale is None else float(sm_scale), k_scales.data_ptr(),
            v_scales.data_ptr(), out.data_ptr(), lse.data_ptr() if lse is not None else None,
            _stream_handle(stream)), "fa_cascade_run_block_scales")
        return out, lse

    def _outputs(self, q, paged_kv, out, lse, return_lse, stream):
        """Check q / paged_kv against the plan; allocate missing outputs."""
        B, Hq, D = self.batch, self.num_qo_heads, self.head_dim
        if q.dtype != self.q_dtype or paged_kv.dtype != self.kv_dtype:
            raise TypeError("q / paged_kv dtype differs from the plan")
        if tuple(q.shape) != (B, Hq, D) or not q.is_contiguous() or not paged_kv.is_contiguous():
            raise ValueError(f"q must be a contiguous CUDA tensor [{B}, {Hq}, {D}]")
        if out is None:
            out = _empty((B, Hq, D), q.dtype, q.device, stream)
        if return_lse and lse is None:
            lse = _empty((B, Hq), torch.float32, q.device, stream)
        _room(out, q.nbytes)
        if lse is not None:
            _room(lse, B * Hq * 4)
        return out, lse

    def set_timing_events(self, before, after) -> None:
        """Record torch.cuda.Events around the prefix kernel of later runs (None = off)."""
        _check(_L().fa_cascade_set_timing_events(self._h, *_event_handles(before, after)),
               "fa_cascade_set_timing_events")

    def check(self, stream=None) -> int:
        flags = ctypes.c_int(0)
        st = _L().fa_cascade_check(self._h, _stream_handle(stream), ctypes.byref(flags))
        if st not in (FA_OK, -5):
            _check(st, "fa_cascade_check")
        return int(flags.value)


def cascade_plan(prefix_indices: torch.Tensor, indptr, indices: torch.Tensor, last_page_len,
                 num_qo_heads: int, num_kv_heads: int, head_dim: int, page_size: int, *,
                 q_data_type=torch.bfloat16, kv_data_type=None,
                 workspace: torch.Tensor | None = None, stream=None) -> CascadePlan:
    """Plan cascade decode: prefix_indices are the shared (full) pages every
    request starts with; indptr/indices/last_page_len describe each request's
    own pages after them."""
    indptr_h, indptr_p, n_indptr = _host_i32_ptr(indptr)
    last_h, last_p, n_last = _host_i32_ptr(last_page_len)
    B = n_indptr - 1
    if n_last < B:
        raise ValueError("last_page_len shorter than the batch")
    for t in (prefix_indices, indices):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("index arrays must be contiguous int32 CUDA tensors")
    _check_indices(indices, indptr_p, B)
    if workspace is None:
        n = _L().fa_cascade_workspace_size(B, num_qo_heads, num_kv_heads, head_dim)
        if n == 0:
            raise ValueError("invalid shape or no CUDA device")
        workspace = _empty(int(n), torch.uint8, prefix_indices.device, stream)
    handle = ctypes.c_void_p()
    kv_data_type = q_data_type if kv_data_type is None else kv_data_type
    _check(_L().fa_cascade_plan(
        prefix_indices.data_ptr(), prefix_indices.numel(), indptr_p,
        indices.data_ptr() if indices.numel() else None, last_p if B else None, B, num_qo_heads,
        num_kv_heads, head_dim, page_size, _dtype_code(q_data_type), _dtype_code(kv_data_type),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _stream_handle(stream), ctypes.byref(handle)), "fa_cascade_plan")
    return CascadePlan(handle.value, (prefix_indices, indices, workspace), q_data_type,
                       (B, num_qo_heads, num_kv_heads, head_dim), kv_dtype=kv_data_type)


class RotaryTable:
    """The rotation of a model's positions: rotary_dim dims turn, pair j by
    position * inv_freq[j] radians.  inv_freq defaults to
    theta ** (-2 j / rotary_dim); pass it (rotary_dim / 2 values, kept in 64
    bits) for scaled variants.  interleaved: pairs (2j, 2j + 1) instead of
    (j, j + rotary_dim / 2).  axes: for tokens with a position on several axes
    (time, height, width), the axis that each pair turns by (rotary_dim / 2
    numbers from 0), e.g. np.repeat([0, 1, 2], [16, 24, 24])."""

    def __init__(self, rotary_dim: int, theta: float = 10000.0, *, inv_freq=None,
                 interleaved: bool = False, axes=None):
        if rotary_dim <= 0 or rotary_dim % 16:
            raise ValueError("rotary_dim must be a positive multiple of 16")
        if inv_freq is None:
            inv_freq = float(theta) ** (-2.0 * np.arange(rotary_dim // 2) / rotary_dim)
        elif isinstance(inv_freq, torch.Tensor):
            inv_freq = inv_freq.detach().to("cpu", torch.float64).numpy()
        self.inv_freq = np.array(inv_freq, dtype=np.float64)
        if (self.inv_freq.shape != (rotary_dim // 2,)
                or not (np.abs(self.inv_freq) <= 2.0 ** 32).all()):
            raise ValueError(f"inv_freq must be {rotary_dim // 2} values of at most 2^32")
        self.rotary_dim = int(rotary_dim)
        self.interleaved = bool(interleaved)
        self.axes = None
        if axes is not None:
            given = _host_i32(axes)
            if given.shape != (rotary_dim // 2,) or (given < 0).any():
                raise ValueError(f"axes must be {rotary_dim // 2} axis numbers from 0")
            self.axes = given.copy()
            self.num_axes = int(given.max()) + 1


def append_workspace_size(batch: int, num_tokens: int) -> int:
    """Bytes of device workspace a plan_append of this batch may need."""
    n = _L().fa_append_workspace_size(batch, num_tokens)
    if n == 0:
        raise ValueError("invalid batch or token count")
    return int(n)


class AppendPlan:
    """A planned append: where a batch's new tokens go in the paged cache.
    Keeps the index tensor, the positions and the workspace alive."""

    def __init__(self, handle, indices, workspace, q_dtype, kv_dtype, shape, num_tokens):
        self._h = handle
        self._indices = indices
        self._workspace = workspace
        self.q_dtype = q_dtype
        self.kv_dtype = kv_dtype
        self.batch, self.num_qo_heads, self.num_kv_heads, self.head_dim, self.page_size = shape
        self.num_tokens = num_tokens
        self._device = workspace.get_device()
        self._itemsize = q_dtype.itemsize
        self._page_shape = (2, self.page_size, self.num_kv_heads, self.head_dim)
        self._kv_shape = (num_tokens, self.num_kv_heads, self.head_dim)
        self._q_shape = (num_tokens, self.num_qo_heads, self.head_dim)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            _L().fa_append_plan_destroy(h)
            self._h = None

    def run(self, k: torch.Tensor, v: torch.Tensor, paged_kv: torch.Tensor, *,
            q: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
            k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
        """Append k and v [num_tokens, Hkv, D] (innermost dim contiguous, other
        strides free) to the cache; with q [num_tokens, Hq, D], also rotate it
        and return it (in q_out, contiguous; q itself to rotate in place).
        k_scale / v_scale are an E4M3 cache's per-tensor scales."""
        rows, q_out, out = self._rows(k, v, paged_kv, q, q_out, stream)
        at = ctypes.addressof(rows)
        _check(_L().fa_append_run(
            self._h, at, at + _ROWS_BYTES, at + 2 * _ROWS_BYTES if q is not None else None, out,
            paged_kv.data_ptr(), paged_kv.shape[0], float(k_scale), float(v_scale),
            _stream_handle(stream)), "fa_append_run")
        return q_out

    def run_head_scales(self, k: torch.Tensor, v: torch.Tensor, paged_kv: torch.Tensor,
                        k_scales: torch.Tensor, v_scales: torch.Tensor, *,
                        q: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                        stream=None):
        """As run, into an E4M3 cache with one given scale per kv head:
        k_scales / v_scales [num_kv_heads] float32."""
        return self._run_scales("fa_append_run_head_scales", (self.num_kv_heads,), k, v,
                                paged_kv, k_scales, v_scales, q, q_out, stream)

    def run_token_scales(self, k: torch.Tensor, v: torch.Tensor, paged_kv: torch.Tensor,
                         k_scales: torch.Tensor, v_scales: torch.Tensor, *,
                         q: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                         stream=None):
        """As run, into an E4M3 cache with one scale per token and kv head, which
        it writes to k_scales / v_scales [num_pages, num_kv_heads, page_size]
        float32."""
        shape = (paged_kv.shape[0], self.num_kv_heads, self.page_size)
        return self._run_scales("fa_append_run_token_scales", shape, k, v, paged_kv, k_scales,
                                v_scales, q, q_out, stream)

    def run_block_scales(self, k: torch.Tensor, v: torch.Tensor, paged_kv: torch.Tensor,
                         k_scales: torch.Tensor, v_scales: torch.Tensor, *,
                         q: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                         stream=None):
        """As run, into an E4M3 cache with one power-of-two scale per page and
        kv head, k_scales / v_scales [num_pages, num_kv_heads] float32, which
        it writes - and raises, re-rounding the page, where a page goes on."""
        return self._run_scales("fa_append_run_block_scales",
                                (paged_kv.shape[0], self.num_kv_heads), k, v, paged_kv, k_scales,
                                v_scales, q, q_out, stream)

    def check(self, stream=None) -> int:
        """Synchronise and return the device-check flags (0 = clean)."""
        flags = ctypes.c_int(0)
        st = _L().fa_append_check(self._h, _stream_handle(stream), ctypes.byref(flags))
        if st not in (FA_OK, -5):
            _check(st, "fa_append_check")
        return int(flags.value)

    def _run_scales(self, name, shape, k, v, paged_kv, k_scales, v_scales, q, q_out, stream):
        rows, q_out, out = self._rows(k, v, paged_kv, q, q_out, stream)
        _check_scales((k_scales, v_scales), shape, paged_kv)
        at = ctypes.addressof(rows)
        _check(getattr(_L(), name)(
            self._h, at, at + _ROWS_BYTES, at + 2 * _ROWS_BYTES if q is not None else None, out,
            paged_kv.data_ptr(), paged_kv.shape[0], k_scales.data_ptr(), v_scales.data_ptr(),
            _stream_handle(stream)), name)
        return q_out

    def _rows(self, k, v, paged_kv, q, q_out, stream):
        """Check the tensors against the plan; fa_rows of k, v and q, q_out, its
        address (None without q)."""
        if paged_kv.dtype is not self.kv_dtype:
            raise TypeError("paged_kv dtype differs from the plan")
        if (paged_kv.shape[1:] != self._page_shape or not paged_kv.is_contiguous()
                or paged_kv.get_device() != self._device):
            raise ValueError("paged_kv must be a contiguous CUDA tensor "
                             "[num_pages, 2, page_size, num_kv_heads, head_dim] on the plan's "
                             "device")
        if q is None:
            if q_out is not None:
                raise ValueError("q_out without q")
            return _Rows3(*self._row(k, self._kv_shape), *self._row(v, self._kv_shape)), None, None
        rows = self._plain_rows(k, v, q)
        if rows is None:  # refused there, or with strides that are never taken
            rows = _Rows3(*self._row(k, self._kv_shape), *self._row(v, self._kv_shape),
                          *self._row(q, self._q_shape))
        if q_out is None:
            q_out = _empty(self._q_shape, q.dtype, q.device, stream)
        elif (q_out.dtype is not q.dtype or q_out.shape != self._q_shape
              or not q_out.is_contiguous() or q_out.get_device() != self._device):
            raise ValueError(f"q_out must be a contiguous tensor {list(self._q_shape)} of q's "
                             "dtype on its device")
        return rows, q_out, q_out.data_ptr()

    def _plain_rows(self, k, v, q):
        """fa_rows of k, v and q where each passes the checks of _row at once (a
        small append is bound by the time of this call), else None."""
        dtype, device, kv_shape = self.q_dtype, self._device, self._kv_shape
        if (k.dtype is not dtype or v.dtype is not dtype or q.dtype is not dtype
                or k.shape != kv_shape or v.shape != kv_shape or q.shape != self._q_shape
                or k.get_device() != device or v.get_device() != device
                or q.get_device() != device or not self.num_tokens):
            return None
        (kt, kh, ki), (vt, vh, vi), (qt, qh, qi) = k.stride(), v.stride(), q.stride()
        kp, vp, qp = k.data_ptr(), v.data_ptr(), q.data_ptr()
        if (ki != 1 or vi != 1 or qi != 1
                or (kp | vp | qp | (kt | kh | vt | vh | qt | qh) * self._itemsize) & 15):
            return None
        return _Rows3(kp, kt, kh, vp, vt, vh, qp, qt, qh)

    def _row(self, t, shape):
        """(address, token stride, head stride) of a k, v or q."""
        if t.dtype is not self.q_dtype:
            raise TypeError("k / v / q dtype differs from the plan")
        if t.shape != shape or t.get_device() != self._device:
            raise ValueError(f"k / v / q must be CUDA tensors on the plan's device, here "
                             f"{list(shape)}")
        if not shape[0]:
            return 0, 0, 0
        address, (token, head, inner) = t.data_ptr(), t.stride()
        # a stride that is never taken may be anything
        if shape[0] == 1:
            token = 0
        if shape[1] == 1:
            head = 0
        if inner != 1 or (address | token * t.itemsize | head * t.itemsize) & 15:
            raise ValueError("k / v / q need a contiguous innermost dim, and an address and "
                             "strides in whole 16 bytes")
        return address, token, head


def plan_append(indptr, indices: torch.Tensor, last_page_len, append_indptr, num_qo_heads: int,
                num_kv_heads: int, head_dim: int, page_size: int, *, q_data_type=torch.bfloat16,
                kv_data_type=None, rotary: RotaryTable | None = None, position_offset=None,
                positions: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                stream=None) -> AppendPlan:
    """Plan the append of append_indptr[i+1] - append_indptr[i] new tokens to
    request i.  indptr / indices / last_page_len describe the batch after the
    append, as plan takes them for the decode that follows; the new tokens are
    each request's last.  rotary: the rotation of k and q (None: none), at the
    token's index in its request plus position_offset[i]; with rotary.axes, at
    positions [axes, append_indptr[-1]], an int32 CUDA tensor that every run
    reads (it may be written between runs)."""
    kv_data_type = q_data_type if kv_data_type is None else kv_data_type
    indptr_h, indptr_p, n_indptr = _host_i32_ptr(indptr)
    last_h, last_p, n_last = _host_i32_ptr(last_page_len)
    app_h, app_p, n_app = _host_i32_ptr(append_indptr)
    B = n_indptr - 1
    if n_last < B or n_app != B + 1:
        raise ValueError("last_page_len shorter than the batch, or append_indptr not batch + 1 "
                         "long")
    off_p = None
    if position_offset is not None:
        off_h, off_p, n_off = _host_i32_ptr(position_offset)
        if n_off != B:
            raise ValueError("position_offset must have one value per request")
    _check_indices(indices, indptr_p, B)
    freq = None
    if rotary is not None:
        # the call reads rotary_dim / 2 doubles of it
        freq = np.ascontiguousarray(rotary.inv_freq, dtype=np.float64)
        if freq.shape != (rotary.rotary_dim // 2,):
            raise ValueError("rotary.inv_freq must have rotary_dim / 2 values")
    total = _i32_at(app_p, B) if B >= 0 else 0
    axes = None if rotary is None else rotary.axes
    if (axes is None) != (positions is None):
        raise ValueError("positions go with a RotaryTable of several axes")
    if axes is not None:
        if position_offset is not None:
            raise ValueError("positions are given: no position_offset")
        if (positions.dtype != torch.int32 or not _reachable(positions)
                or not positions.is_contiguous() or positions.dim() != 2
                or positions.shape[0] < rotary.num_axes or positions.shape[1] != total):
            raise ValueError(f"positions must be a contiguous int32 CUDA or page-locked tensor "
                             f"[{rotary.num_axes}, {total}]")
        axes = np.ascontiguousarray(axes, dtype=np.int32)
        if axes.shape != (rotary.rotary_dim // 2,):
            raise ValueError("rotary.axes must have rotary_dim / 2 values")
    device = torch.cuda.current_device()
    for t in (indices, positions):
        if t is not None and t.is_cuda and t.get_device() != device:
            raise ValueError("indices and positions must be on the current device")
    if workspace is not None and (workspace.get_device() != device
                                  or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on the current device")
    if workspace is None:
        workspace = _empty(append_workspace_size(max(B, 0), max(total, 0)), torch.uint8,
                           _cuda_device(indices), stream)
    handle = ctypes.c_void_p()
    first = (indptr_p, indices.data_ptr() if indices.numel() else None, last_p if B else None, app_p)
    rest = (B, num_qo_heads, num_kv_heads, head_dim, page_size, _dtype_code(q_data_type),
            _dtype_code(kv_data_type), freq.ctypes.data if rotary else None,
            rotary.rotary_dim if rotary else 0, int(rotary.interleaved) if rotary else 0,
            workspace.data_ptr(), workspace.numel() * workspace.element_size(),
            _stream_handle(stream), ctypes.byref(handle))
    if axes is None:
        _check(_L().fa_append_plan(*first, off_p, *rest), "fa_append_plan")
    else:
        _check(_L().fa_append_plan_axes(*first, positions.data_ptr() if total else None,
                                        positions.shape[0], axes.ctypes.data, *rest),
               "fa_append_plan_axes")
    return AppendPlan(handle.value, (indices, positions), workspace, q_data_type, kv_data_type,
                      (B, num_qo_heads, num_kv_heads, head_dim, page_size), total)


def _q_rows(q: torch.Tensor):
    """The fa_rows of a q [rows, heads, head_dim]."""
    address, (n, heads, _), (token, head, inner) = q.data_ptr(), q.shape, q.stride()
    # a stride that is never taken may be anything
    if n <= 1:
        token = 8
    if heads == 1:
        head = 8
    if n and (inner != 1 or (address | (token | head) * q.element_size()) & 15 or token <= 0
              or head <= 0):
        raise ValueError("q needs a contiguous innermost dim, and an address and strides in "
                         "whole 16 bytes")
    return _Rows(address, token, head)


class PrefillPlan:
    """Planned attention of packed query rows (prompts, chunks of prompts, single
    tokens) over their requests' pages.  Keeps the index tensor and the
    workspace alive."""

    def __init__(self, handle, indices, workspace, q_dtype, kv_dtype, shape, num_tokens):
        self._h = handle
        self._keep = (indices, workspace)
        self.q_dtype = q_dtype
        self.kv_dtype = kv_dtype
        self.batch, self.num_qo_heads, self.num_kv_heads, self.head_dim, self.page_size = shape
        self.num_tokens = num_tokens
        self._device = workspace.get_device()
        self._q_shape = (num_tokens, self.num_qo_heads, self.head_dim)
        self._nbytes = num_tokens * self.num_qo_heads * self.head_dim * q_dtype.itemsize
        self._lse_bytes = num_tokens * self.num_qo_heads * 4
        self._page_shape = (2, self.page_size, self.num_kv_heads, self.head_dim)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            _L().fa_prefill_plan_destroy(h)
            self._h = None

    def run(self, q: torch.Tensor, paged_kv: torch.Tensor, *, sm_scale: float | None = None,
            k_scale: float = 1.0, v_scale: float = 1.0, out: torch.Tensor | None = None,
            lse: torch.Tensor | None = None, return_lse: bool = True, stream=None):
        """Attention of q [qo_indptr[-1], Hq, D] (innermost dim contiguous, other
        strides free); returns (o, lse) (lse None if return_lse is False).
        k_scale / v_scale are an E4M3 cache's per-tensor scales."""
        rows, out, lse = self._outputs(q, paged_kv, out, lse, return_lse, stream)
        _check(_L().fa_prefill_run(
            self._h, ctypes.addressof(rows), paged_kv.data_ptr(), paged_kv.shape[0],
            0.0 if sm_scale is None else float(sm_scale), float(k_scale), float(v_scale),
            out.data_ptr(), lse.data_ptr() if lse is not None else None,
            _stream_handle(stream)), "fa_prefill_run")
        return out, lse

    def run_head_scales(self, q: torch.Tensor, paged_kv: torch.Tensor, k_scales: torch.Tensor,
                        v_scales: torch.Tensor, **kw):
        """As run, over an E4M3 cache with one scale per kv head: k_scales /
        v_scales [num_kv_heads] float32."""
        return self._run_scales("fa_prefill_run_head_scales", (self.num_kv_heads,), q, paged_kv,
                                k_scales, v_scales, **kw)

    def run_token_scales(self, q: torch.Tensor, paged_kv: torch.Tensor, k_scales: torch.Tensor,
                         v_scales: torch.Tensor, **kw):
        """As run, over an E4M3 cache with one scale per token and kv head:
        k_scales / v_scales [num_pages, num_kv_heads, page_size] float32."""
        shape = (paged_kv.shape[0], self.num_kv_heads, self.page_size)
        return self._run_scales("fa_prefill_run_token_scales", shape, q, paged_kv, k_scales,
                                v_scales, **kw)

    def run_block_scales(self, q: torch.Tensor, paged_kv: torch.Tensor, k_scales: torch.Tensor,
                         v_scales: torch.Tensor, **kw):
        """As run, over an E4M3 cache with one scale per page and kv head:
        k_scales / v_scales [num_pages, num_kv_heads] float32."""
        return self._run_scales("fa_prefill_run_block_scales",
                                (paged_kv.shape[0], self.num_kv_heads), q, paged_kv, k_scales,
                                v_scales, **kw)

    def _run_scales(self, name, shape, q, paged_kv, k_scales, v_scales, *, sm_scale=None, out=None,
                    lse=None, return_lse=True, stream=None):
        rows, out, lse = self._outputs(q, paged_kv, out, lse, return_lse, stream)
        _check_scales((k_scales, v_scales), shape, paged_kv)
        _check(getattr(_L(), name)(
            self._h, ctypes.addressof(rows), paged_kv.data_ptr(), paged_kv.shape[0],
            0.0 if sm_scale is None else float(sm_scale), k_scales.data_ptr(),
            v_scales.data_ptr(), out.data_ptr(), lse.data_ptr() if lse is not None else None,
            _stream_handle(stream)), name)
        return out, lse

    def _outputs(self, q, paged_kv, out, lse, return_lse, stream):
        """Check q / paged_kv against the plan; allocate missing outputs."""
        device = self._device
        if q.dtype is not self.q_dtype or paged_kv.dtype is not self.kv_dtype:
            raise TypeError("q / paged_kv dtype differs from the plan")
        if q.shape != self._q_shape or q.get_device() != device:
            raise ValueError(f"q must be a tensor {list(self._q_shape)} on the plan's device")
        rows = _q_rows(q)
        if (paged_kv.dim() != 5 or paged_kv.shape[1:] != self._page_shape
                or not paged_kv.is_contiguous() or paged_kv.get_device() != device):
            raise ValueError("paged_kv must be a contiguous tensor [num_pages, 2, page_size, "
                             "num_kv_heads, head_dim] on the plan's device")
        if out is None:
            out = (torch.empty_like(q) if stream is None and q.is_contiguous()
                   else _empty(self._q_shape, q.dtype, q.device, stream))
        else:
            nbytes, at, to = self._nbytes, q.data_ptr(), _room(out, self._nbytes).data_ptr()
            if out.dtype is not q.dtype or out.get_device() != device or not out.is_contiguous():
                raise ValueError("out must be contiguous, of q's dtype, on the plan's device")
            end = at + self._span(q)
            if nbytes and to < end and at < to + nbytes:
                raise ValueError("out must not overlap q")
        if lse is not None:
            _room(lse, self._lse_bytes)
            if (lse.dtype is not torch.float32 or lse.get_device() != device
                    or not lse.is_contiguous()):
                raise ValueError("lse must be contiguous float32, on the plan's device")
        elif return_lse:
            lse = _empty(self._q_shape[:2], torch.float32, q.device, stream)
        return rows, out, lse

    @staticmethod
    def _span(q) -> int:
        """Bytes from q's first element to past its last."""
        last = sum((n - 1) * st for n, st in zip(q.shape, q.stride()) if n)
        return (last + 1) * q.element_size()

    def check(self, stream=None) -> int:
        """Synchronise and return the device-check flags (0 = clean)."""
        flags = ctypes.c_int(0)
        st = _L().fa_prefill_check(self._h, _stream_handle(stream), ctypes.byref(flags))
        if st not in (FA_OK, -5):
            _check(st, "fa_prefill_check")
        return int(flags.value)


def plan_prefill(indptr, indices: torch.Tensor, last_page_len, qo_indptr, num_qo_heads: int,
                 num_kv_heads: int, head_dim: int, page_size: int, *, q_data_type=torch.bfloat16,
                 kv_data_type=None, workspace: torch.Tensor | None = None,
                 stream=None) -> PrefillPlan:
    """Plan causal attention of qo_indptr[i+1] - qo_indptr[i] query rows for request
    i, any number up to its length: the last positions of its cache (append them
    first).  run() takes q [qo_indptr[-1], Hq, D]."""
    kv_data_type = q_data_type if kv_data_type is None else kv_data_type
    indptr_h, indptr_p, n_indptr = _host_i32_ptr(indptr)
    last_h, last_p, n_last = _host_i32_ptr(last_page_len)
    qo_h, qo_p, n_qo = _host_i32_ptr(qo_indptr)
    B = n_indptr - 1
    if B < 0 or n_last < B or n_qo != B + 1:
        raise ValueError("last_page_len shorter than the batch, or qo_indptr not batch + 1 long")
    _check_indices(indices, indptr_p, B)
    q_code, kv_code = _dtype_code(q_data_type), _dtype_code(kv_data_type)
    workspace = _plan_workspace(
        workspace, indices, lambda: _L().fa_prefill_workspace_size(
            indptr_p, last_p if B else None, qo_p, B, num_qo_heads, num_kv_heads, head_dim, q_code,
            kv_code), stream)
    handle = ctypes.c_void_p()
    _check(_L().fa_prefill_plan(
        indptr_p, indices.data_ptr() if indices.numel() else None, last_p if B else None, qo_p, B,
        num_qo_heads, num_kv_heads, head_dim, page_size, q_code, kv_code, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_handle(stream),
        ctypes.byref(handle)), "fa_prefill_plan")
    return PrefillPlan(handle.value, indices, workspace, q_data_type, kv_data_type,
                       (B, num_qo_heads, num_kv_heads, head_dim, page_size), _i32_at(qo_p, B))


def plan_prefill_host(indptr, last_page_len, qo_indptr, group: int, num_kv_heads: int,
                      max_ctas: int):
    """Host-only work list of plan_prefill (fa_plan_prefill_host, no GPU): returns
    (cta_offsets, items [n, 8], merge [m, 8], num_slots)."""
    indptr_h, indptr_p, n_indptr = _host_i32_ptr(indptr)
    last_h, last_p, n_last = _host_i32_ptr(last_page_len)
    qo_h, qo_p, n_qo = _host_i32_ptr(qo_indptr)
    B = n_indptr - 1
    if B < 0 or n_last < B or n_qo != B + 1:
        raise ValueError("last_page_len shorter than the batch, or qo_indptr not batch + 1 long")
    cta = np.zeros(max_ctas + 1, np.int32)
    counts = [ctypes.c_int() for _ in range(4)]
    room = [0, 0]
    while True:
        items, merge = (np.zeros((n, 8), np.int32) for n in room)
        rc = _L().fa_plan_prefill_host(indptr_p, last_p if B else None, qo_p, B, group, num_kv_heads,
                                       max_ctas, cta.ctypes.data, items.ctypes.data, room[0],
                                       merge.ctypes.data, room[1],
                                       *(ctypes.byref(c) for c in counts))
        need = [counts[1].value, counts[2].value]
        if rc == -3 and need != room:
            room = need
            continue
        _check(rc, "fa_plan_prefill_host")
        return cta[:counts[0].value + 1], items[:need[0]], merge[:need[1]], counts[3].value


class WeightsPlan:
    """A planned accumulation of attention weights over a batch's cached tokens.
    Keeps the index tensor and the workspace alive."""

    def __init__(self, handle, indices, workspace, q_dtype, kv_dtype, shape, num_tokens):
        self._h = handle
        self._keep = (indices, workspace)
        self.q_dtype = q_dtype
        self.kv_dtype = kv_dtype
        self.batch, self.num_qo_heads, self.num_kv_heads, self.head_dim, self.page_size = shape
        self.num_tokens = num_tokens
        self._device = workspace.get_device()
        self._q_shape = (num_tokens, self.num_qo_heads, self.head_dim)
        self._page_shape = (2, self.page_size, self.num_kv_heads, self.head_dim)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            _L().fa_weights_plan_destroy(h)
            self._h = None

    def run(self, q: torch.Tensor, paged_kv: torch.Tensor, lse: torch.Tensor,
            weights: torch.Tensor, *, sm_scale: float | None = None, k_scale: float = 1.0,
            stream=None) -> torch.Tensor:
        """Add to weights [num_pages, num_kv_heads, page_size] float32 what the rows
        q [rows, Hq, D] gave each token; lse [rows, Hq] is what their attention
        returned.  Returns weights."""
        rows = self._checked(q, paged_kv, lse, weights)
        _check(_L().fa_weights_run(
            self._h, ctypes.addressof(rows), paged_kv.data_ptr(), paged_kv.shape[0],
            0.0 if sm_scale is None else float(sm_scale), float(k_scale), lse.data_ptr(),
            weights.data_ptr(), _stream_handle(stream)), "fa_weights_run")
        return weights

    def run_head_scales(self, q: torch.Tensor, paged_kv: torch.Tensor, lse: torch.Tensor,
                        weights: torch.Tensor, k_scales: torch.Tensor, **kw) -> torch.Tensor:
        """As run, over an E4M3 cache with one K scale per kv head [num_kv_heads]."""
        return self._run_scales("fa_weights_run_head_scales", (self.num_kv_heads,), q, paged_kv,
                                lse, weights, k_scales, **kw)

    def run_token_scales(self, q: torch.Tensor, paged_kv: torch.Tensor, lse: torch.Tensor,
                         weights: torch.Tensor, k_scales: torch.Tensor, **kw) -> torch.Tensor:
        """As run, over an E4M3 cache with one K scale per token and kv head
        [num_pages, num_kv_heads, page_size]."""
        shape = (paged_kv.shape[0], self.num_kv_heads, self.page_size)
        return self._run_scales("fa_weights_run_token_scales", shape, q, paged_kv, lse, weights,
                                k_scales, **kw)

    def run_block_scales(self, q: torch.Tensor, paged_kv: torch.Tensor, lse: torch.Tensor,
                         weights: torch.Tensor, k_scales: torch.Tensor, **kw) -> torch.Tensor:
        """As run, over an E4M3 cache with one K scale per page and kv head
        [num_pages, num_kv_heads]."""
        return self._run_scales("fa_weights_run_block_scales",
                                (paged_kv.shape[0], self.num_kv_heads), q, paged_kv, lse, weights,
                                k_scales, **kw)

    def _run_scales(self, name, shape, q, paged_kv, lse, weights, k_scales, *, sm_scale=None,
                    stream=None):
        rows = self._checked(q, paged_kv, lse, weights)
        _check_scales((k_scales,), shape, paged_kv)
        _check(getattr(_L(), name)(
            self._h, ctypes.addressof(rows), paged_kv.data_ptr(), paged_kv.shape[0],
            0.0 if sm_scale is None else float(sm_scale), k_scales.data_ptr(), lse.data_ptr(),
            weights.data_ptr(), _stream_handle(stream)), name)
        return weights

    def _checked(self, q, paged_kv, lse, weights):
        if q.dtype is not self.q_dtype or paged_kv.dtype is not self.kv_dtype:
            raise TypeError("q / paged_kv dtype differs from the plan")
        if q.shape != self._q_shape or q.get_device() != self._device:
            raise ValueError(f"q must be a tensor {list(self._q_shape)} on the plan's device")
        if (paged_kv.dim() != 5 or paged_kv.shape[1:] != self._page_shape
                or not paged_kv.is_contiguous() or paged_kv.get_device() != self._device):
            raise ValueError("paged_kv must be a contiguous tensor [num_pages, 2, page_size, "
                             "num_kv_heads, head_dim] on the plan's device")
        if (lse.dtype is not torch.float32 or lse.shape != self._q_shape[:2]
                or not lse.is_contiguous() or lse.get_device() != self._device):
            raise ValueError(f"lse must be a contiguous float32 tensor {list(self._q_shape[:2])} "
                             "on the plan's device")
        _check_weights(weights, paged_kv)
        return _q_rows(q)

    def check(self, stream=None) -> int:
        """Synchronise and return the device-check flags (0 = clean)."""
        flags = ctypes.c_int(0)
        st = _L().fa_weights_check(self._h, _stream_handle(stream), ctypes.byref(flags))
        if st not in (FA_OK, -5):
            _check(st, "fa_weights_check")
        return int(flags.value)


def _check_weights(weights, paged_kv) -> None:
    shape = (paged_kv.shape[0], paged_kv.shape[3], paged_kv.shape[2])
    if (weights.dtype is not torch.float32 or weights.shape != shape
            or not weights.is_contiguous() or weights.get_device() != paged_kv.get_device()):
        raise ValueError(f"weights must be a contiguous float32 tensor {list(shape)} on the device "
                         "of paged_kv")


def plan_weights(indptr, indices: torch.Tensor, last_page_len, qo_indptr, num_qo_heads: int,
                 num_kv_heads: int, head_dim: int, page_size: int, *, q_data_type=torch.bfloat16,
                 kv_data_type=None, workspace: torch.Tensor | None = None,
                 stream=None) -> WeightsPlan:
    """Plan the accumulation of the attention weights that qo_indptr[i+1] -
    qo_indptr[i] query rows of request i (its last positions) give its cached
    tokens; qo_indptr None: one row each, as after a decode step."""
    kv_data_type = q_data_type if kv_data_type is None else kv_data_type
    indptr_h, indptr_p, n_indptr = _host_i32_ptr(indptr)
    last_h, last_p, n_last = _host_i32_ptr(last_page_len)
    if qo_indptr is None:
        qo_indptr = np.arange(n_indptr, dtype=np.int32)
    qo_h, qo_p, n_qo = _host_i32_ptr(qo_indptr)
    B = n_indptr - 1
    if B < 0 or n_last < B or n_qo != B + 1:
        raise ValueError("last_page_len shorter than the batch, or qo_indptr not batch + 1 long")
    _check_indices(indices, indptr_p, B)
    workspace = _plan_workspace(
        workspace, indices, lambda: _L().fa_weights_workspace_size(B, max(_i32_at(indptr_p, B), 0)),
        stream)
    handle = ctypes.c_void_p()
    _check(_L().fa_weights_plan(
        indptr_p, indices.data_ptr() if indices.numel() else None, last_p if B else None, qo_p, B,
        num_qo_heads, num_kv_heads, head_dim, page_size, _dtype_code(q_data_type),
        _dtype_code(kv_data_type), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_handle(stream),
        ctypes.byref(handle)), "fa_weights_plan")
    return WeightsPlan(handle.value, indices, workspace, q_data_type, kv_data_type,
                       (B, num_qo_heads, num_kv_heads, head_dim, page_size), _i32_at(qo_p, B))


def _plan_workspace(workspace, indices, size, stream) -> torch.Tensor:
    """The caller's workspace, or one of size() bytes, on the current device."""
    device = torch.cuda.current_device()
    if indices.is_cuda and indices.get_device() != device:
        raise ValueError("indices must be on the current device")
    if workspace is None:
        # 0 for refused arguments, which the plan names
        return _empty(max(int(size()), 256), torch.uint8, _cuda_device(indices), stream)
    if workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the current device")
    return workspace


class EvictPlan:
    """A planned eviction.  indptr, indices and last_page_len describe the batch
    after it (indices where the plan's are), freed [n] the page ids that it no longer
    needs.  Both were taken from the page table as it was planned, on the plan's
    stream: writing the table later does not change them.  Keeps the index tensor
    and the workspace alive."""

    def __init__(self, handle, indices, workspace, kv_dtype, shape, after):
        self._h = handle
        self._keep = (indices, workspace)
        self.kv_dtype = kv_dtype
        self.batch, self.num_kv_heads, self.head_dim, self.page_size = shape
        self._device = workspace.get_device()
        self._page_shape = (2, self.page_size, self.num_kv_heads, self.head_dim)
        self.indptr, self.last_page_len = after

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            _L().fa_evict_plan_destroy(h)
            self._h = None

    def run(self, paged_kv: torch.Tensor, weights: torch.Tensor, *,
            k_scales: torch.Tensor | None = None, v_scales: torch.Tensor | None = None,
            stream=None) -> None:
        """Move each kv head's kept tokens to the front of its request's pages, in
        place; weights [num_pages, num_kv_heads, page_size] float32 go with them
        and are 0 behind them.  k_scales / v_scales: an E4M3 cache's scales per
        token, moved too."""
        if paged_kv.dtype is not self.kv_dtype:
            raise TypeError("paged_kv dtype differs from the plan")
        if (paged_kv.dim() != 5 or paged_kv.shape[1:] != self._page_shape
                or not paged_kv.is_contiguous() or paged_kv.get_device() != self._device):
            raise ValueError("paged_kv must be a contiguous tensor [num_pages, 2, page_size, "
                             "num_kv_heads, head_dim] on the plan's device")
        _check_weights(weights, paged_kv)
        if (k_scales is None) != (v_scales is None):
            raise ValueError("k_scales and v_scales go together")
        if k_scales is not None:
            _check_scales((k_scales, v_scales), weights.shape, paged_kv)
        _check(_L().fa_evict_run(
            self._h, paged_kv.data_ptr(), paged_kv.shape[0], weights.data_ptr(),
            None if k_scales is None else k_scales.data_ptr(),
            None if v_scales is None else v_scales.data_ptr(), _stream_handle(stream)),
            "fa_evict_run")

    def check(self, stream=None) -> int:
        """Synchronise and return the device-check flags (0 = clean)."""
        flags = ctypes.c_int(0)
        st = _L().fa_evict_check(self._h, _stream_handle(stream), ctypes.byref(flags))
        if st not in (FA_OK, -5):
            _check(st, "fa_evict_check")
        return int(flags.value)


def _pages_after(indptr, last, kept, page_size):
    """(indptr, last_page_len, entries that stay, entries that are freed) of a
    batch of which request i keeps the first `kept[i]` slots at most."""
    pages = np.diff(indptr).astype(np.int64)
    length = np.where(pages > 0, (pages - 1) * page_size + last, 0)
    length = np.minimum(length, kept)
    stay = -(-length // page_size)
    after = np.zeros(len(indptr), np.int64)
    np.cumsum(stay, out=after[1:])
    owner = np.repeat(np.arange(len(pages)), pages)
    at = np.arange(int(pages.sum())) - indptr[:-1].astype(np.int64)[owner]
    here = at < stay[owner]
    last_after = np.where(stay > 0, length - (stay - 1) * page_size, page_size)
    return (after.astype(np.int32), last_after.astype(np.int32), np.flatnonzero(here),
            np.flatnonzero(~here))


def _take_pages(table, stay, free, stream):
    """The page ids at the entries that stay and at those that are freed, where `table`
    is, as they stand when the work before on `stream` is done."""
    order = torch.from_numpy(np.concatenate([stay, free]).astype(np.int32))
    if not table.is_cuda:
        ids = table[order.long()].pin_memory()
    elif stream is None:
        ids = table.index_select(0, order.to(table.device))
    else:
        stream = _as_stream(stream)
        ids = _empty(order.shape, table.dtype, table.device, stream)
        with torch.cuda.stream(stream):
            torch.index_select(table, 0, order.to(table.device), out=ids)
    return ids[:len(stay)], ids[len(stay):]


def plan_evict(indptr, indices: torch.Tensor, last_page_len, keep, num_kv_heads: int,
               head_dim: int, page_size: int, *, recent=0, kv_data_type=torch.bfloat16,
               workspace: torch.Tensor | None = None, stream=None) -> EvictPlan:
    """Plan the eviction of each request's tokens beyond its budget: keep tokens stay
    (a number, or one per request), the last `recent` of them whatever their
    weight (likewise)."""
    indptr_h, indptr_p, n_indptr = _host_i32_ptr(indptr)
    last_h, last_p, n_last = _host_i32_ptr(last_page_len)
    B = n_indptr - 1
    if B < 0 or n_last < B:
        raise ValueError("last_page_len shorter than the batch")
    budgets = []
    for v in (keep, recent):
        a = _host_i32(np.full(B, v) if np.ndim(v) == 0 else v)
        if a.shape != (B,) or (a < 0).any():
            raise ValueError("keep and recent must be one number, or one per request, from 0")
        budgets.append(a)
    _check_indices(indices, indptr_p, B)
    total = max(_i32_at(indptr_p, B), 0) * page_size
    workspace = _plan_workspace(
        workspace, indices, lambda: _L().fa_evict_workspace_size(
            B, min(int(budgets[0].sum(dtype=np.int64)), total), num_kv_heads), stream)
    handle = ctypes.c_void_p()
    _check(_L().fa_evict_plan(
        indptr_p, indices.data_ptr() if indices.numel() else None, last_p if B else None,
        budgets[0].ctypes.data if B else None, budgets[1].ctypes.data if B else None, B,
        num_kv_heads, head_dim, page_size, _dtype_code(kv_data_type), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_handle(stream),
        ctypes.byref(handle)), "fa_evict_plan")
    ptr, last, stay, free = _pages_after(np.asarray(indptr_h), np.asarray(last_h)[:B], budgets[0],
                                         page_size)
    plan = EvictPlan(handle.value, indices, workspace, kv_data_type,
                     (B, num_kv_heads, head_dim, page_size),
                     (torch.from_numpy(ptr), torch.from_numpy(last)))
    plan.indices, plan.freed = _take_pages(indices.view(-1), stay, free, stream)
    return plan


class BatchDecodeWithPagedKVCacheWrapper:
    """plan/run wrapper in the shape the pages show: built once over a caller
    workspace with the "NHD" layout, planned per batch, run on the hot path."""

    def __init__(self, workspace_buffer: torch.Tensor, kv_layout: str = "NHD"):
        if kv_layout != "NHD":
            raise ValueError("only the NHD layout is supported")
        self._workspace = workspace_buffer
        self._plan: DecodePlan | None = None

    def plan(self, indptr, indices, last_page_len, num_qo_heads, num_kv_heads, head_dim,
             page_size, q_data_type=torch.bfloat16, kv_data_type=None, stream=None):
        self._plan = plan(indptr, indices, last_page_len, num_qo_heads, num_kv_heads, head_dim,
                          page_size, q_data_type=q_data_type, kv_data_type=kv_data_type,
                          workspace=self._workspace, stream=stream)
        return self._plan

    def run(self, q, paged_kv_cache, *, sm_scale=None, k_scale=1.0, v_scale=1.0,
            return_lse=False, out=None, lse=None, stream=None):
        if self._plan is None:
            raise RuntimeError("call plan() before run()")
        o, l = self._plan.run(q, paged_kv_cache, sm_scale=sm_scale, k_scale=k_scale,
                              v_scale=v_scale, out=out, lse=lse, return_lse=return_lse,
                              stream=stream)
        return (o, l) if return_lse else o
