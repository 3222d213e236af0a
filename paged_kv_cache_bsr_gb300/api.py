"""Thin ctypes binding of libpkvbsr.so (include/pkv_bsr.h).

Functions keep the C names without the ``pkv_`` prefix and only marshal
arguments: tensors become raw pointers, streams become cudaStream_t handles,
and a non-OK status becomes a ``PkvError``.  Every computation happens in the
library's CUDA kernels; there is no fallback path.  If the library has not
been built, loading raises.

``Plan`` bundles a plan handle with the device workspace and the pinned host
staging buffer it needs (allocated with torch, i.e. by the caller).
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional, Tuple

import torch

from . import build as _build

PKV_OK = 0
PKV_F16, PKV_BF16, PKV_F32 = 0, 1, 2
PLAN_DECODE, PLAN_PREFILL, PLAN_MIXED = 0, 1, 2
PLAN_DECODE_KV8, PLAN_PREFILL_KV8 = 3, 4  # over the 8-bit cache

_DTYPES = {torch.float16: PKV_F16, torch.bfloat16: PKV_BF16, torch.float32: PKV_F32}
_STORED = {PKV_F16: torch.float16, PKV_BF16: torch.bfloat16}


class PkvError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class Params(ctypes.Structure):
    _fields_ = [("num_qo_heads", ctypes.c_int), ("num_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("page_size", ctypes.c_int), ("dtype", ctypes.c_int), ("sm_scale", ctypes.c_float),
                ("logits_cap", ctypes.c_float), ("causal", ctypes.c_int)]


class Limits(ctypes.Structure):
    _fields_ = [("max_batch", ctypes.c_int), ("max_total_q", ctypes.c_int64), ("max_kv_pages", ctypes.c_int64)]


class RopeAxes(ctypes.Structure):
    _fields_ = [("theta", ctypes.c_double), ("rotary_dim", ctypes.c_int), ("num_axes", ctypes.c_int),
                ("sections", ctypes.c_int * 4), ("interleaved", ctypes.c_int)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("grid_ctas", ctypes.c_int), ("workers", ctypes.c_int), ("active_workers", ctypes.c_int),
                ("num_work", ctypes.c_int), ("num_merge", ctypes.c_int), ("num_slots", ctypes.c_int),
                ("max_cost", ctypes.c_int64), ("total_cost", ctypes.c_int64),
                ("prefill_ctas", ctypes.c_int), ("decode_ctas", ctypes.c_int)]


_lib = None
_lock = threading.Lock()

EXPORTS = [
    "pkv_status_string", "pkv_version", "pkv_plan_create", "pkv_plan_create_host", "pkv_plan_destroy",
    "pkv_plan_workspace_bytes", "pkv_plan_compute", "pkv_plan_run", "pkv_plan_get_info", "pkv_plan_get_work",
    "pkv_batch_decode_paged", "pkv_batch_prefill_paged", "pkv_merge_state", "pkv_merge_states",
    "pkv_get_device_error",
    "pkv_plan_set_timing_events", "pkv_batch_decode_paged_noalloc", "pkv_append_paged_kv",
    "pkv_batch_prefill_paged_masked", "pkv_batch_mixed_paged", "pkv_plan_set_pipelined",
    "pkv_plan_set_split_kv", "pkv_append_paged_kv_axes", "pkv_append_paged_kv8", "pkv_batch_decode_paged_kv8",
    "pkv_batch_prefill_paged_kv8",
]


def library_path() -> str:
    return _build.LIB_PATH


def load(path: Optional[str] = None):
    """Load libpkvbsr.so (raises if it is missing: there is no CPU path)."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or library_path()
        if not os.path.exists(p):
            raise RuntimeError(f"libpkvbsr.so is not built ({p}); run paged_kv_cache_bsr_gb300.build.build()")
        lib = ctypes.CDLL(p)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        sig = {
            "pkv_status_string": (ctypes.c_char_p, [i32]),
            "pkv_version": (i32, []),
            "pkv_plan_create": (i32, [ctypes.POINTER(vp), i32, ctypes.POINTER(Params), ctypes.POINTER(Limits), i32]),
            "pkv_plan_create_host": (i32, [ctypes.POINTER(vp), i32, ctypes.POINTER(Params), ctypes.POINTER(Limits), i32]),
            "pkv_plan_destroy": (i32, [vp]),
            "pkv_plan_workspace_bytes": (i32, [vp, ctypes.POINTER(sz), ctypes.POINTER(sz)]),
            "pkv_plan_compute": (i32, [vp, i32, vp, vp, vp, vp, i64, vp, sz]),
            "pkv_plan_run": (i32, [vp, i32, vp, vp, vp, vp, i64, vp, sz, vp, sz, vp]),
            "pkv_plan_get_info": (i32, [vp, ctypes.POINTER(PlanInfo)]),
            "pkv_plan_get_work": (i32, [vp, vp, i64, ctypes.POINTER(i64)]),
            "pkv_batch_decode_paged": (i32, [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
            "pkv_batch_prefill_paged": (i32, [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
            "pkv_merge_state": (i32, [vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, vp]),
            "pkv_merge_states": (i32, [vp, vp, i32, i64, vp, vp, i64, i32, i32, i32, vp]),
            "pkv_get_device_error": (i32, [vp, vp, ctypes.POINTER(i32), i32, vp]),
            "pkv_plan_set_timing_events": (i32, [vp, vp, vp]),
            "pkv_batch_decode_paged_noalloc": (i32, [vp, vp, sz, vp, vp, vp, vp, vp, vp, vp, vp]),
            "pkv_batch_prefill_paged_masked": (i32, [vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp, vp, vp]),
            "pkv_batch_mixed_paged": (i32, [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
            "pkv_plan_set_pipelined": (i32, [vp, i32]),
            "pkv_plan_set_split_kv": (i32, [vp, i32]),
            "pkv_append_paged_kv": (i32, [ctypes.POINTER(Params), i32, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp,
                                          vp, ctypes.c_double, vp, vp]),
            "pkv_append_paged_kv_axes": (i32, [ctypes.POINTER(Params), ctypes.POINTER(RopeAxes), i32, i64, i64, vp, vp,
                                               vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
            "pkv_append_paged_kv8": (i32, [ctypes.POINTER(Params), ctypes.POINTER(RopeAxes), i32, i64, i64, vp, vp, vp,
                                           vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
            "pkv_batch_decode_paged_kv8": (i32, [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
            "pkv_batch_prefill_paged_kv8": (i32, [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        if path is None:
            _lib = lib
        return lib


def status_string(status: int) -> str:
    try:
        return load().pkv_status_string(int(status)).decode()
    except RuntimeError:
        return "library not loaded"


def _check(st: int, what: str) -> None:
    if st != PKV_OK:
        raise PkvError(st, what)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libpkvbsr must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


# The current stream's handle without a Stream object around it (3 us a call on the host).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and torch.cuda.is_initialized():
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def dtype_code(dtype: torch.dtype) -> int:
    return _DTYPES[dtype]


def make_params(num_qo_heads, num_kv_heads, head_dim, page_size, dtype, sm_scale, logits_cap=0.0,
                causal=False) -> Params:
    return Params(int(num_qo_heads), int(num_kv_heads), int(head_dim), int(page_size),
                  dtype_code(dtype) if isinstance(dtype, torch.dtype) else int(dtype), float(sm_scale),
                  float(logits_cap), int(bool(causal)))


# ----------------------------------------------------------------------------- C names
def plan_create(kind: int, params: Params, limits: Limits, device: int) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    _check(load().pkv_plan_create(ctypes.byref(h), kind, ctypes.byref(params), ctypes.byref(limits), device),
           "pkv_plan_create")
    return h


def plan_create_host(kind: int, params: Params, limits: Limits, num_sms: int) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    _check(load().pkv_plan_create_host(ctypes.byref(h), kind, ctypes.byref(params), ctypes.byref(limits),
                                       num_sms), "pkv_plan_create_host")
    return h


def plan_destroy(h) -> None:
    _check(load().pkv_plan_destroy(h), "pkv_plan_destroy")


def plan_workspace_bytes(h) -> Tuple[int, int]:
    d, hb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().pkv_plan_workspace_bytes(h, ctypes.byref(d), ctypes.byref(hb)), "pkv_plan_workspace_bytes")
    return d.value, hb.value


def _host_i32(t):
    if t is None:
        return None
    t = torch.as_tensor(t, dtype=torch.int32)
    if t.is_cuda:
        raise ValueError("plan arrays must be host tensors")
    return t.contiguous()


def plan_compute(h, batch: int, qo_indptr_h, kv_indptr_h, kv_indices_h, kv_last_page_len_h, num_pages: int,
                 host_ws: torch.Tensor) -> None:
    qo, ip, ix, la = (_host_i32(x) for x in (qo_indptr_h, kv_indptr_h, kv_indices_h, kv_last_page_len_h))
    _check(load().pkv_plan_compute(h, int(batch), _ptr(qo), _ptr(ip), _ptr(ix), _ptr(la), int(num_pages),
                                   _ptr(host_ws), host_ws.numel() * host_ws.element_size()), "pkv_plan_compute")


def plan_run(h, batch: int, qo_indptr_h, kv_indptr_h, kv_indices_h, kv_last_page_len_h, num_pages: int,
             dev_ws: torch.Tensor, host_ws: torch.Tensor, stream=None) -> None:
    qo, ip, ix, la = (_host_i32(x) for x in (qo_indptr_h, kv_indptr_h, kv_indices_h, kv_last_page_len_h))
    _check(load().pkv_plan_run(h, int(batch), _ptr(qo), _ptr(ip), _ptr(ix), _ptr(la), int(num_pages),
                               _ptr(dev_ws), dev_ws.numel() * dev_ws.element_size(), _ptr(host_ws),
                               host_ws.numel() * host_ws.element_size(), _stream(stream)), "pkv_plan_run")


def plan_set_split_kv(h, on: bool) -> None:
    """Decode plans: split-KV on (default) or off (each page list whole on one worker)."""
    _check(load().pkv_plan_set_split_kv(h, int(bool(on))), "pkv_plan_set_split_kv")


def plan_get_info(h) -> PlanInfo:
    info = PlanInfo()
    _check(load().pkv_plan_get_info(h, ctypes.byref(info)), "pkv_plan_get_info")
    return info


def plan_get_work(h) -> torch.Tensor:
    n = ctypes.c_int64()
    lib = load()
    lib.pkv_plan_get_work(h, None, 0, ctypes.byref(n))
    out = torch.empty((n.value, 8), dtype=torch.int32)
    if n.value:
        _check(lib.pkv_plan_get_work(h, _ptr(out), n.value, ctypes.byref(n)), "pkv_plan_get_work")
    return out


def batch_decode_paged(h, q, kv_data, kv_indices, kv_indptr, kv_last_page_len, o, lse, dev_ws, stream=None) -> None:
    _check(load().pkv_batch_decode_paged(h, _ptr(q), _ptr(kv_data), _ptr(kv_indices), _ptr(kv_indptr),
                                         _ptr(kv_last_page_len), _ptr(o), _ptr(lse), _ptr(dev_ws),
                                         _stream(stream)), "pkv_batch_decode_paged")


def batch_decode_paged_noalloc(h, host_tables, q, kv_data, kv_indices, kv_indptr, kv_last_page_len, o, lse,
                               stream=None) -> None:
    """Decode with the library's static device scratch instead of a caller workspace.

    ``host_tables`` is the host buffer ``plan_compute`` filled for this plan.
    """
    _check(load().pkv_batch_decode_paged_noalloc(h, _ptr(host_tables),
                                                 host_tables.numel() * host_tables.element_size(), _ptr(q),
                                                 _ptr(kv_data), _ptr(kv_indices), _ptr(kv_indptr),
                                                 _ptr(kv_last_page_len), _ptr(o), _ptr(lse), _stream(stream)),
           "pkv_batch_decode_paged_noalloc")


def batch_prefill_paged(h, q, qo_indptr, kv_data, kv_indices, kv_indptr, kv_last_page_len, o, lse, dev_ws,
                        stream=None) -> None:
    _check(load().pkv_batch_prefill_paged(h, _ptr(q), _ptr(qo_indptr), _ptr(kv_data), _ptr(kv_indices),
                                          _ptr(kv_indptr), _ptr(kv_last_page_len), _ptr(o), _ptr(lse),
                                          _ptr(dev_ws), _stream(stream)), "pkv_batch_prefill_paged")


def batch_prefill_paged_masked(h, q, qo_indptr, kv_data, kv_indices, kv_indptr, kv_last_page_len, packed_mask,
                               o, lse, dev_ws, stream=None) -> None:
    """Prefill with a packed custom mask (uint8 device tensor, whole 32-bit words)."""
    _check(load().pkv_batch_prefill_paged_masked(h, _ptr(q), _ptr(qo_indptr), _ptr(kv_data), _ptr(kv_indices),
                                                 _ptr(kv_indptr), _ptr(kv_last_page_len), _ptr(packed_mask),
                                                 packed_mask.numel() * packed_mask.element_size(), _ptr(o),
                                                 _ptr(lse), _ptr(dev_ws), _stream(stream)),
           "pkv_batch_prefill_paged_masked")


def batch_mixed_paged(h, q, qo_indptr, kv_data, kv_indices, kv_indptr, kv_last_page_len, o, lse, dev_ws,
                      stream=None) -> None:
    _check(load().pkv_batch_mixed_paged(h, _ptr(q), _ptr(qo_indptr), _ptr(kv_data), _ptr(kv_indices),
                                        _ptr(kv_indptr), _ptr(kv_last_page_len), _ptr(o), _ptr(lse), _ptr(dev_ws),
                                        _stream(stream)), "pkv_batch_mixed_paged")


def merge_state(o_a, lse_a, o_b, lse_b, o_out, lse_out=None, stream=None) -> None:
    """merge_state over [n_rows, num_heads, head_dim] states (dtype fp16/bf16/fp32)."""
    if o_a.dim() != 3:
        raise ValueError("o must be [n_rows, num_heads, head_dim]")
    n, hh, d = o_a.shape
    _check(load().pkv_merge_state(_ptr(o_a), _ptr(lse_a), _ptr(o_b), _ptr(lse_b), _ptr(o_out), _ptr(lse_out),
                                  n, hh, d, dtype_code(o_a.dtype), _stream(stream)), "pkv_merge_state")


def merge_states(o_states, lse_states, num_states: int, o_out, lse_out=None, stream=None) -> None:
    """merge_state over ``num_states`` states laid out one after another: o_states is
    [num_states * n_rows, num_heads, head_dim] (fp16/bf16/fp32) and lse_states
    [num_states * n_rows, num_heads]; o_out [n_rows, num_heads, head_dim] may be the
    rows of one of the states."""
    if o_states.dim() != 3 or o_states.shape[0] % num_states:
        raise ValueError("o_states must be [num_states * n_rows, num_heads, head_dim]")
    rows, hh, d = o_states.shape
    n = rows // num_states
    _check(load().pkv_merge_states(_ptr(o_states), _ptr(lse_states), int(num_states), n, _ptr(o_out), _ptr(lse_out),
                                   n, hh, d, dtype_code(o_states.dtype), _stream(stream)), "pkv_merge_states")


def append_paged_kv(params: Params, append_indptr, kv_indptr, kv_indices, kv_last_page_len, k_new, v_new,
                    kv_data, q_in=None, q_out=None, rope_theta: float = 0.0, error=None, stream=None) -> None:
    """Write new tokens' K/V into their pages (page table already including them);
    with rope_theta > 0 rotate the keys and, when given, the queries (q_out may be q_in)."""
    batch = int(append_indptr.numel()) - 1
    nnz = int(k_new.shape[0])
    if q_in is not None and q_out is None:
        q_out = q_in
    _check(load().pkv_append_paged_kv(ctypes.byref(params), batch, nnz, int(kv_data.shape[0]), _ptr(append_indptr),
                                      _ptr(kv_indptr), _ptr(kv_indices), _ptr(kv_last_page_len), _ptr(k_new),
                                      _ptr(v_new), _ptr(kv_data), _ptr(q_in), _ptr(q_out), float(rope_theta),
                                      _ptr(error), _stream(stream)), "pkv_append_paged_kv")


def make_rope_axes(theta: float, rotary_dim: int, sections, interleaved: bool = False) -> RopeAxes:
    """A rotation by positions on len(sections) axes (1 to 4), sections[x] pairs of elements to axis x;
    the sections sum to rotary_dim / 2."""
    s = [int(x) for x in sections]
    if not 1 <= len(s) <= 4:
        raise ValueError("sections must name 1 to 4 axes")
    return RopeAxes(float(theta), int(rotary_dim), len(s), (ctypes.c_int * 4)(*s), int(bool(interleaved)))


def _ptrs(tensors):
    """The tensors' addresses (None for None): contiguous, and on the current CUDA device, where the
    kernels are launched."""
    dev, out = -2, []
    for x in tensors:
        if x is None:
            out.append(None)
            continue
        at = x.get_device()
        if at != dev:
            if dev != -2 or at < 0 or at != torch.cuda.current_device():
                raise ValueError("tensors must be on the current CUDA device")
            dev = at
        if not x.is_contiguous():
            raise ValueError("tensors passed to libpkvbsr must be contiguous")
        out.append(x.data_ptr())
    return out


_I32 = torch.int32


def _int32(*tensors) -> None:
    for x in tensors:
        if x is not None and x.dtype is not _I32:
            raise ValueError("page tables, row pointers, positions and error words must be int32")


_CODES = (torch.float8_e4m3fn, torch.uint8)


def _kv8_tensors(params: Params, kv8, kv8_scales) -> None:
    if kv8.dtype not in _CODES or kv8_scales.dtype is not torch.uint8:
        raise ValueError("kv8 must hold e4m3 codes (float8_e4m3fn or uint8) and kv8_scales be uint8")
    shape = kv8.shape
    if shape[1:] != (2, params.num_kv_heads, params.page_size, params.head_dim) or kv8_scales.shape != shape[:-1]:
        raise ValueError("kv8 must be [num_pages, 2, num_kv_heads, page_size, head_dim] and kv8_scales the same "
                         "without head_dim")


def _append_tensors(params: Params, rope, append_indptr, kv_indptr, kv_indices, kv_last_page_len, positions, k_new,
                    v_new, q_in, q_out, error):
    batch, nnz = append_indptr.numel() - 1, k_new.shape[0]
    _int32(append_indptr, kv_indptr, kv_indices, kv_last_page_len, positions, error)
    if batch < 0 or kv_indptr.numel() != batch + 1 or kv_last_page_len.numel() != batch:
        raise ValueError("append_indptr and kv_indptr must have batch + 1 entries, kv_last_page_len batch")
    dtype, dim = _STORED.get(params.dtype), params.head_dim
    kv_rows = (nnz, params.num_kv_heads, dim)
    fits = k_new.shape == kv_rows and v_new.shape == kv_rows and k_new.dtype is dtype and v_new.dtype is dtype
    if q_in is not None:
        q_rows = (nnz, params.num_qo_heads, dim)
        fits = fits and q_in.shape == q_rows and q_out.shape == q_rows and q_in.dtype is dtype and q_out.dtype is dtype
    if not fits:
        raise ValueError("k_new, v_new, q_in and q_out must be [nnz, heads, head_dim] of the params' dtype")
    if positions is not None and (rope is None or positions.shape != (rope.num_axes, nnz)):
        raise ValueError("positions go with a rotation and must be [num_axes, nnz]")
    return batch, nnz


def append_paged_kv_axes(params: Params, rope: Optional[RopeAxes], append_indptr, kv_indptr, kv_indices,
                         kv_last_page_len, positions, k_new, v_new, kv_data, q_in=None, q_out=None, error=None,
                         stream=None) -> None:
    """``append_paged_kv`` with the rotation's positions given ([num_axes, nnz] int32; None: each
    token's place in its request); rope None copies keys and queries.  q_out may be q_in (the default)."""
    if q_in is not None and q_out is None:
        q_out = q_in
    batch, nnz = _append_tensors(params, rope, append_indptr, kv_indptr, kv_indices, kv_last_page_len, positions, k_new,
                                 v_new, q_in, q_out, error)
    if kv_data.shape[1:] != (2, params.num_kv_heads, params.page_size, params.head_dim) or \
            kv_data.dtype is not k_new.dtype:
        raise ValueError("kv_data must be [num_pages, 2, num_kv_heads, page_size, head_dim] of the params' dtype")
    _check((_lib or load()).pkv_append_paged_kv_axes(
        ctypes.byref(params), None if rope is None else ctypes.byref(rope), batch, nnz, kv_data.shape[0],
        *_ptrs((append_indptr, kv_indptr, kv_indices, kv_last_page_len, positions, k_new, v_new, kv_data, q_in, q_out,
                error)), _stream(stream)), "pkv_append_paged_kv_axes")


def append_paged_kv8(params: Params, rope: Optional[RopeAxes], append_indptr, kv_indptr, kv_indices, kv_last_page_len,
                     positions, k_new, v_new, kv8, kv8_scales, q_in=None, q_out=None, error=None, stream=None) -> None:
    """``append_paged_kv_axes`` into the 8-bit cache: e4m3 codes ``kv8`` (float8_e4m3fn or uint8) and the
    exponent bytes ``kv8_scales`` (uint8) of their rows' power-of-two scales."""
    if q_in is not None and q_out is None:
        q_out = q_in
    batch, nnz = _append_tensors(params, rope, append_indptr, kv_indptr, kv_indices, kv_last_page_len, positions, k_new,
                                 v_new, q_in, q_out, error)
    _kv8_tensors(params, kv8, kv8_scales)
    _check((_lib or load()).pkv_append_paged_kv8(
        ctypes.byref(params), None if rope is None else ctypes.byref(rope), batch, nnz, kv8.shape[0],
        *_ptrs((append_indptr, kv_indptr, kv_indices, kv_last_page_len, positions, k_new, v_new, kv8, kv8_scales, q_in,
                q_out, error)), _stream(stream)), "pkv_append_paged_kv8")


def batch_decode_paged_kv8(h, q, kv8, kv8_scales, kv_indices, kv_indptr, kv_last_page_len, o, lse, dev_ws,
                           stream=None) -> None:
    """Decode over the 8-bit cache, on a plan of kind PLAN_DECODE_KV8."""
    _check((_lib or load()).pkv_batch_decode_paged_kv8(
        h, *_ptrs((q, kv8, kv8_scales, kv_indices, kv_indptr, kv_last_page_len, o, lse, dev_ws)), _stream(stream)),
        "pkv_batch_decode_paged_kv8")


def batch_prefill_paged_kv8(h, q, qo_indptr, kv8, kv8_scales, kv_indices, kv_indptr, kv_last_page_len, o, lse, dev_ws,
                            stream=None) -> None:
    """Prefill over the 8-bit cache, on a plan of kind PLAN_PREFILL_KV8."""
    _check((_lib or load()).pkv_batch_prefill_paged_kv8(
        h, *_ptrs((q, qo_indptr, kv8, kv8_scales, kv_indices, kv_indptr, kv_last_page_len, o, lse, dev_ws)),
        _stream(stream)), "pkv_batch_prefill_paged_kv8")


def plan_set_timing_events(h, start=None, stop=None) -> None:
    """Record torch.cuda.Event ``start``/``stop`` around the main kernel of later run calls."""
    def handle(ev):
        if ev is None:
            return None
        if not ev.cuda_event:
            ev.record()  # torch creates the event lazily
        return ctypes.c_void_p(ev.cuda_event)
    _check(load().pkv_plan_set_timing_events(h, handle(start), handle(stop)), "pkv_plan_set_timing_events")


def get_device_error(h, dev_ws, clear: bool = False, stream=None) -> int:
    code = ctypes.c_int()
    _check(load().pkv_get_device_error(h, _ptr(dev_ws), ctypes.byref(code), int(clear), _stream(stream)),
           "pkv_get_device_error")
    return code.value


# ----------------------------------------------------------------------------- convenience
class Plan:
    """A plan handle plus the caller-side buffers it needs.

    ``kind`` is PLAN_DECODE, PLAN_PREFILL, PLAN_MIXED, or PLAN_DECODE_KV8 / PLAN_PREFILL_KV8
    for the 8-bit cache (``run`` then takes its scales too).  The device workspace and the
    pinned host staging buffer are allocated once here, with torch, for the
    given limits; ``plan()`` re-plans a new batch into them and ``run()``
    launches the kernels.  The workspace comes from the pool of the stream that is
    current here: keep the plan until its runs on other streams are done.
    """

    def __init__(self, kind: int, *, num_qo_heads: int, num_kv_heads: int, head_dim: int, page_size: int,
                 dtype: torch.dtype, sm_scale: float, logits_cap: float = 0.0, causal: bool = False,
                 max_batch: int, max_total_q: Optional[int] = None, max_kv_pages: int,
                 device: Optional[int] = None, pipelined: bool = False, split_kv: bool = True):
        self.kind = kind
        self.device = torch.cuda.current_device() if device is None else int(device)
        self.params = make_params(num_qo_heads, num_kv_heads, head_dim, page_size, dtype, sm_scale, logits_cap,
                                  causal)
        self.limits = Limits(int(max_batch), int(max_batch if max_total_q is None else max_total_q),
                             int(max_kv_pages))
        self.handle = plan_create(kind, self.params, self.limits, self.device)
        dev_bytes, host_bytes = plan_workspace_bytes(self.handle)
        self.dev_ws = torch.empty(dev_bytes, dtype=torch.uint8, device=f"cuda:{self.device}")
        self.host_ws = torch.empty(host_bytes, dtype=torch.uint8, pin_memory=True)
        self.num_pages = 0
        self.batch = self.total_q = self.kv_pages = 0
        if pipelined:
            _check(load().pkv_plan_set_pipelined(self.handle, 1), "pkv_plan_set_pipelined")
        if not split_kv:
            plan_set_split_kv(self.handle, False)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value and _lib is not None:
            try:
                _lib.pkv_plan_destroy(h)
            except Exception:
                pass
            self.handle = None

    def plan(self, kv_indptr_h, kv_last_page_len_h, num_pages: int, *, qo_indptr_h=None, kv_indices_h=None,
             stream=None) -> None:
        batch = int(torch.as_tensor(kv_indptr_h).numel()) - 1
        plan_run(self.handle, batch, qo_indptr_h, kv_indptr_h, kv_indices_h, kv_last_page_len_h, num_pages,
                 self.dev_ws, self.host_ws, stream)
        self.num_pages = int(num_pages)
        if self.kind in (PLAN_DECODE_KV8, PLAN_PREFILL_KV8):  # what run() checks its tensors against
            self.batch = batch
            self.total_q = batch if self.kind == PLAN_DECODE_KV8 else int(torch.as_tensor(qo_indptr_h)[-1])
            self.kv_pages = int(torch.as_tensor(kv_indptr_h)[-1])

    def _check_kv8(self, q, kv8, kv8_scales, kv_indices, kv_indptr, kv_last_page_len, o, lse, qo_indptr) -> None:
        """The tensors of a run over the 8-bit cache against what the last plan() named."""
        p = self.params
        _kv8_tensors(p, kv8, kv8_scales)
        _int32(kv_indices, kv_indptr, kv_last_page_len, qo_indptr)
        if kv8.shape[0] < self.num_pages or kv_indices.numel() < self.kv_pages:
            raise ValueError("the pool or the page table is smaller than the plan's")
        if kv_indptr.numel() != self.batch + 1 or kv_last_page_len.numel() != self.batch:
            raise ValueError("kv_indptr must have batch + 1 entries, kv_last_page_len batch")
        if self.kind == PLAN_PREFILL_KV8 and (qo_indptr is None or qo_indptr.numel() != self.batch + 1):
            raise ValueError("a prefill takes qo_indptr with batch + 1 entries")
        shape, dtype = (self.total_q, p.num_qo_heads, p.head_dim), _STORED[p.dtype]
        if q.shape != shape or o.shape != shape or q.dtype is not dtype or o.dtype is not dtype:
            raise ValueError("q and o must be [rows of the plan, num_qo_heads, head_dim] of the plan's dtype")
        if lse is not None and (lse.shape != shape[:2] or lse.dtype is not torch.float32):
            raise ValueError("lse must be [rows of the plan, num_qo_heads] float32")

    def run(self, q, kv_data, kv_indices, kv_indptr, kv_last_page_len, o, lse=None, *, qo_indptr=None,
            mask=None, kv_scales=None, stream=None) -> None:
        if (kv_scales is not None) != (self.kind in (PLAN_DECODE_KV8, PLAN_PREFILL_KV8)):
            raise ValueError("kv_scales go with a plan for the 8-bit cache")
        if kv_scales is not None:
            if mask is not None:
                raise ValueError("a custom mask needs a prefill plan over the 16-bit cache")
            self._check_kv8(q, kv_data, kv_scales, kv_indices, kv_indptr, kv_last_page_len, o, lse, qo_indptr)
            if self.kind == PLAN_DECODE_KV8:
                batch_decode_paged_kv8(self.handle, q, kv_data, kv_scales, kv_indices, kv_indptr, kv_last_page_len, o,
                                       lse, self.dev_ws, stream)
            else:
                batch_prefill_paged_kv8(self.handle, q, qo_indptr, kv_data, kv_scales, kv_indices, kv_indptr,
                                        kv_last_page_len, o, lse, self.dev_ws, stream)
        elif mask is not None:
            if self.kind != PLAN_PREFILL:
                raise ValueError("a custom mask needs a prefill plan")
            batch_prefill_paged_masked(self.handle, q, qo_indptr, kv_data, kv_indices, kv_indptr, kv_last_page_len,
                                       mask, o, lse, self.dev_ws, stream)
        elif self.kind == PLAN_MIXED:
            batch_mixed_paged(self.handle, q, qo_indptr, kv_data, kv_indices, kv_indptr, kv_last_page_len, o, lse,
                              self.dev_ws, stream)
        elif self.kind == PLAN_DECODE:
            batch_decode_paged(self.handle, q, kv_data, kv_indices, kv_indptr, kv_last_page_len, o, lse,
                               self.dev_ws, stream)
        else:
            batch_prefill_paged(self.handle, q, qo_indptr, kv_data, kv_indices, kv_indptr, kv_last_page_len, o,
                                lse, self.dev_ws, stream)

    def info(self) -> PlanInfo:
        return plan_get_info(self.handle)

    def work(self) -> torch.Tensor:
        return plan_get_work(self.handle)

    def set_timing_events(self, start=None, stop=None) -> None:
        plan_set_timing_events(self.handle, start, stop)

    def device_error(self, clear: bool = False, stream=None) -> int:
        return get_device_error(self.handle, self.dev_ws, clear, stream)
