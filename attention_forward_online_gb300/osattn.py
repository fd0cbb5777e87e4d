"""ctypes binding for libosattn (argument marshalling only).

Every step of the forward pass, the backward pass and the row softmax runs
in the library's CUDA kernels, and the host-memory (offload) entry points
copy through the library's own streams; this module checks tensor shapes,
allocates outputs with torch (device and pinned host memory are torch's job
here), and passes raw pointers and the current stream through the C ABI
declared in include/osattn.h.  If libosattn.so is missing the calls raise:
there is no fallback implementation.

A call's `stream` defaults to torch's current one.  Given another, the call
works as if it were current: its kernels, and the copies, outputs and
workspaces it makes, are in that stream's order, where its inputs have to be
ready; the results are marked as used by the caller's current stream too.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct
import threading

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libosattn.so")

BF16 = 0
FP32 = 1
FP16 = 2
E4M3 = 3  # of a cache's pages only
OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED = 2
ERR_CUDA = 3
ERR_TIMEOUT = 4
ERR_SCRATCH_LIMIT = 5
NOALLOC_SCRATCH_BYTES = 32 << 20

EXPORTS = ("osattn_fwd", "osattn_fwd_strided", "osattn_fwd_splitkv",
           "osattn_splitkv_workspace_bytes", "osattn_fwd_splitkv_noalloc",
           "osattn_bwd", "osattn_bwd_strided", "osattn_bwd_workspace_bytes",
           "osattn_fwd_offload", "osattn_bwd_offload", "osattn_softmax_rows",
           "osattn_softmax_rows_offload",
           "osattn_status_string", "osattn_get_device_status",
           "osattn_version", "osattn_set_wait_limit_ns", "osattn_test_wait_timeout",
           "osattn_last_timeout_site", "osattn_step_trace_read",
           "osattn_mask_plan", "osattn_mask_plan_bytes", "osattn_fwd_mod", "osattn_bwd_mod",
           "osattn_bwd_mod_workspace_bytes", "osattn_tree_attn", "osattn_tree_workspace_bytes",
           "osattn_tree_attn_e4m3", "osattn_tree_e4m3_workspace_bytes", "osattn_rotary", "osattn_cache_append")

_lock = threading.Lock()
_lib = None


class _Score(ctypes.Structure):
    """struct osattn_score of include/osattn.h."""

    _fields_ = [("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p),
                ("rel_table", ctypes.c_void_p), ("rel_map", ctypes.c_void_p),
                ("rel_num", ctypes.c_int), ("rel_range", ctypes.c_int),
                ("q_offset", ctypes.c_int)]


class _Rotation(ctypes.Structure):
    """struct osattn_rotation of include/osattn.h."""

    _fields_ = [("freqs", ctypes.c_void_p), ("rot", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("amplitude", ctypes.c_float)]


_ROTATION = struct.Struct("@Piif4x")  # its bytes, which are made faster than the object
assert _ROTATION.size == ctypes.sizeof(_Rotation)


class OsattnError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


def lib():
    """Load libosattn.so (built in-tree by __graft_entry__.build())."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is not built; run `python -c \"import __graft_entry__ as g; "
                    "g.build()\"` (nvcc, sm_103a)")
            L = ctypes.CDLL(LIB_PATH)
            vp, i32 = ctypes.c_void_p, ctypes.c_int
            L.osattn_fwd.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                     ctypes.c_float, i32, vp, i32, vp]
            L.osattn_fwd.restype = i32
            i64p = ctypes.POINTER(ctypes.c_int64)
            L.osattn_fwd_strided.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                             i64p, i64p, i64p, i64p,
                                             ctypes.c_float, i32, vp, i32, vp]
            L.osattn_fwd_strided.restype = i32
            L.osattn_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                             ctypes.c_float, i32, vp, i32, i32, vp,
                                             ctypes.c_size_t, vp]
            L.osattn_fwd_splitkv.restype = i32
            L.osattn_fwd_splitkv_noalloc.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                                     ctypes.c_float, i32, vp, i32, i32, vp]
            L.osattn_fwd_splitkv_noalloc.restype = i32
            L.osattn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                     ctypes.c_float, i32, vp, i32, vp, ctypes.c_size_t, vp]
            L.osattn_bwd.restype = i32
            L.osattn_bwd_strided.argtypes = ([vp] * 9 + [i32] * 5 + [i64p] * 8 +
                                             [ctypes.c_float, i32, vp, i32, vp, ctypes.c_size_t, vp])
            L.osattn_bwd_strided.restype = i32
            L.osattn_fwd_offload.argtypes = ([vp] * 10 + [i32] * 5 + [ctypes.c_float, i32, vp, i32,
                                                                       i32, vp])
            L.osattn_fwd_offload.restype = i32
            L.osattn_bwd_offload.argtypes = ([vp] * 18 + [i32] * 5 + [ctypes.c_float, i32, vp, i32,
                                                                       vp, ctypes.c_size_t, i32, vp])
            L.osattn_bwd_offload.restype = i32
            L.osattn_softmax_rows_offload.argtypes = [vp] * 6 + [ctypes.c_int64, i32, i32,
                                                                 ctypes.c_int64, vp]
            L.osattn_softmax_rows_offload.restype = i32
            L.osattn_bwd_workspace_bytes.argtypes = [i32, i32, i32]
            L.osattn_bwd_workspace_bytes.restype = ctypes.c_size_t
            L.osattn_softmax_rows.argtypes = [vp, vp, vp, ctypes.c_int64, i32, i32, vp]
            L.osattn_softmax_rows.restype = i32
            L.osattn_splitkv_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
            L.osattn_splitkv_workspace_bytes.restype = ctypes.c_size_t
            L.osattn_status_string.argtypes = [i32]
            L.osattn_status_string.restype = ctypes.c_char_p
            L.osattn_get_device_status.argtypes = [vp]
            L.osattn_get_device_status.restype = i32
            L.osattn_version.argtypes = []
            L.osattn_version.restype = i32
            L.osattn_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
            L.osattn_set_wait_limit_ns.restype = ctypes.c_uint64
            L.osattn_test_wait_timeout.argtypes = [vp]
            L.osattn_test_wait_timeout.restype = i32
            L.osattn_last_timeout_site.argtypes = []
            L.osattn_last_timeout_site.restype = i32
            L.osattn_step_trace_read.argtypes = [vp, ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)]
            L.osattn_step_trace_read.restype = i32
            sz = ctypes.c_size_t
            L.osattn_mask_plan_bytes.argtypes = [i32, i32]
            L.osattn_mask_plan_bytes.restype = sz
            L.osattn_mask_plan.argtypes = [vp, sz] + [i32] * 6 + [vp] * 4
            L.osattn_mask_plan.restype = i32
            scp = ctypes.POINTER(_Score)
            L.osattn_fwd_mod.argtypes = ([vp] * 5 + [i32] * 6 + [i64p] * 4 +
                                         [ctypes.c_float, scp, vp, i32, vp])
            L.osattn_fwd_mod.restype = i32
            L.osattn_bwd_mod_workspace_bytes.argtypes = [i32] * 5
            L.osattn_bwd_mod_workspace_bytes.restype = sz
            L.osattn_bwd_mod.argtypes = ([vp] * 10 + [i32] * 6 + [i64p] * 8 +
                                         [ctypes.c_float, scp, vp, i32, vp, sz, vp])
            L.osattn_bwd_mod.restype = i32
            L.osattn_tree_workspace_bytes.argtypes = [i32] * 5
            L.osattn_tree_workspace_bytes.restype = sz
            L.osattn_tree_attn.argtypes = ([vp] * 8 + [i32] * 8 + [i64p] * 4 +
                                           [ctypes.c_float, ctypes.c_float, vp, i32, i32, vp, sz, vp])
            L.osattn_tree_attn.restype = i32
            L.osattn_tree_e4m3_workspace_bytes.argtypes = [i32] * 5
            L.osattn_tree_e4m3_workspace_bytes.restype = sz
            # (strides and the rotation as addresses: a ctypes pointer costs a call more to convert)
            L.osattn_tree_attn_e4m3.argtypes = ([vp] * 10 + [i32] * 9 + [vp] * 4 +
                                                [ctypes.c_float, ctypes.c_float, vp, i32, i32, vp, sz, vp])
            L.osattn_tree_attn_e4m3.restype = i32
            L.osattn_rotary.argtypes = [vp] * 4 + [i32] * 5 + [vp] * 4 + [vp, vp, i32, i32, i32, i32, vp]
            L.osattn_rotary.restype = i32
            L.osattn_cache_append.argtypes = [vp] * 12 + [i32] * 9 + [vp] * 6 + [vp, i32, i32, vp]
            L.osattn_cache_append.restype = i32
            _lib = L
        return _lib


def step_trace():
    """The clock stamps of a profiling build (OSATTN_STEP_TRACE=1; see
    include/osattn.h): (per-step stamps, a numpy int64 array [8, 7, 128, 4];
    per-CTA times, [4096, 6])."""
    import numpy as np

    need = ctypes.c_size_t(0)
    lib().osattn_step_trace_read(None, 0, ctypes.byref(need))
    buf = np.zeros(need.value // 8, dtype=np.int64)
    st = lib().osattn_step_trace_read(buf.ctypes.data, buf.nbytes, ctypes.byref(need))
    if st != OK:
        raise OsattnError(st, "osattn_step_trace_read")
    n = 8 * 7 * 128 * 4
    return buf[:n].reshape(8, 7, 128, 4), buf[n:].reshape(4096, 6)


def status_string(status: int) -> str:
    return lib().osattn_status_string(int(status)).decode()


def _stream_handle(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _raw_stream(index):
    """Handle of torch's current stream on device `index`."""
    return torch._C._cuda_getCurrentRawStream(index)


def _elsewhere_stream(stream, index):
    """Whether `stream` is given and is not torch's current one on device
    `index`."""
    if stream is None or stream.cuda_stream == _raw_stream(index):
        return False
    if getattr(stream, "device_index", index) != index:
        raise ValueError("stream is on another device than the tensors")
    return True


def _under(stream, index, call, *given):
    """call() with `stream` as torch's current one.  What a call makes (copies
    of views, outputs, workspaces) then comes from that stream's memory and is
    written in its order, behind whatever used the memory before; on the
    caller's stream a copy could come after the kernel that reads it.  The
    results are marked as used by the caller's stream too, and the tensors that
    the caller gave as used by `stream`."""
    import torch

    caller = torch.cuda.current_stream(index)
    if not hasattr(stream, "device_index"):  # another library's, known by its handle
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=index)
    with torch.cuda.stream(stream):
        results = call()
    for t in results if isinstance(results, tuple) else (results,):
        if isinstance(t, MaskPlan):
            t = t.buffer
        if t is not None and t.is_cuda:
            t.record_stream(caller)
    for t in given:
        if t is not None and t.is_cuda:
            t.record_stream(stream)
    return results


def fwd_raw(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, H, Nq, Nkv, d, scale, causal,
            key_len_ptr, dtype, stream_handle) -> int:
    """Direct call of osattn_fwd with integer pointers; returns the status."""
    return lib().osattn_fwd(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, int(B), int(H), int(Nq),
                            int(Nkv), int(d), float(scale), int(bool(causal)), key_len_ptr,
                            int(dtype), stream_handle)


def _dtype_code(t) -> int:
    import torch

    codes = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}
    if t.dtype not in codes:
        raise TypeError("q, k, v must all be bf16, all fp16 or all fp32")
    return codes[t.dtype]


def _shapes(q, k, v):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, H, N, d]")
    B, H, Nq, d = q.shape
    Nkv = k.shape[2]
    if tuple(k.shape) != (B, H, Nkv, d) or tuple(v.shape) != (B, H, Nkv, d):
        raise ValueError("k and v must be [B, H, Nkv, d] matching q")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share one dtype")
    for t in (q, k, v):
        if not t.is_cuda:
            raise ValueError("q, k, v must be CUDA tensors")
    return B, H, Nq, Nkv, d


def _key_len_ptr(key_len, B):
    import torch

    if key_len is None:
        return None, None
    if key_len.dtype != torch.int32 or not key_len.is_cuda or key_len.numel() != B:
        raise ValueError("key_len must be a CUDA int32 tensor with B entries")
    key_len = key_len.contiguous()
    return key_len, key_len.data_ptr()


def _bhn_strides(t):
    """(b, h, row) element strides of a [B, H, N, d] view whose d axis is
    contiguous, as a ctypes int64[3]."""
    if t.stride(3) != 1:
        raise ValueError("the last (d) axis must have stride 1")
    return (ctypes.c_int64 * 3)(t.stride(0), t.stride(1), t.stride(2))


def fwd(q, k, v, scale: float | None = None, causal: bool = False, key_len=None,
        out=None, lse=None, stream=None):
    """O, LSE = attention forward of CUDA tensors q [B,H,Nq,d], k/v [B,H,Nkv,d].

    dtype bf16, fp16 or fp32 (all three alike).  q, k, v and `out` may be any
    views whose last axis is contiguous (e.g. transposes of [B, N, H, d]);
    contiguous tensors go through osattn_fwd, others through
    osattn_fwd_strided with their strides.  key_len: None or a CUDA int32
    tensor [B].  `out` (q's shape and dtype) and `lse` (contiguous fp32
    [B, H, Nq]) may be given preallocated.  Enqueued on `stream` (default:
    torch's current stream); raises OsattnError if the library rejects the
    call."""
    import torch

    B, H, Nq, Nkv, d = _shapes(q, k, v)
    dtype = _dtype_code(q)
    index = q.get_device()
    if _elsewhere_stream(stream, index):
        return _under(stream, index, lambda: fwd(q, k, v, scale, causal, key_len, out, lse), out, lse)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    if out.shape != q.shape or out.dtype != q.dtype or not out.is_cuda:
        raise ValueError("out must be a CUDA tensor matching q")
    if tuple(lse.shape) != (B, H, Nq) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be fp32 [B, H, Nq]")
    kl, kl_ptr = _key_len_ptr(key_len, B)
    if all(t.is_contiguous() for t in (q, k, v, out)):
        st = fwd_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                     B, H, Nq, Nkv, d, scale, causal, kl_ptr, dtype, _stream_handle(stream))
        what = "osattn_fwd"
    else:
        qs, ks, vs, os_ = (_bhn_strides(t) for t in (q, k, v, out))
        st = lib().osattn_fwd_strided(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                      lse.data_ptr(), B, H, Nq, Nkv, d, qs, ks, vs, os_,
                                      float(scale), int(bool(causal)), kl_ptr, dtype,
                                      _stream_handle(stream))
        what = "osattn_fwd_strided"
    del kl
    if st != OK:
        raise OsattnError(st, what)
    return out, lse


MAX_SPLITS = 128


def splitkv_workspace_bytes(B: int, H: int, Nq: int, d: int, num_splits: int) -> int:
    return int(lib().osattn_splitkv_workspace_bytes(int(B), int(H), int(Nq), int(d),
                                                    int(num_splits)))


def _check_qkv(q, k, v):
    B, H, Nq, Nkv, d = _shapes(q, k, v)
    _dtype_code(q)
    for t in (q, k, v):
        if not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous")
    return B, H, Nq, Nkv, d


def fwd_offload(q_host, k_host, v_host, out_host=None, lse_host=None, q=None, k=None, v=None,
                out=None, lse=None, scale: float | None = None, causal: bool = False,
                key_len=None, heads_per_chunk: int = 0, stream=None):
    """Attention forward of host tensors through osattn_fwd_offload: q_host
    [B,H,Nq,d], k_host/v_host [B,H,Nkv,d] (contiguous CPU tensors, pinned for
    the copies to overlap the compute) are copied in chunks of heads to the
    device buffers q, k, v (allocated when not given), attended, and O/LSE are
    copied back into out_host/lse_host (pinned CPU tensors, allocated when not
    given).  Returns (out_host, lse_host); they are valid once `stream` has
    synchronised.  key_len is a CUDA int32 tensor with B entries or None;
    heads_per_chunk 0 lets the library size the chunks."""
    import torch

    for t in (q_host, k_host, v_host):
        if t.is_cuda or not t.is_contiguous() or t.dim() != 4:
            raise ValueError("q_host, k_host, v_host must be contiguous 4-D CPU tensors")
    B, H, Nq, d = q_host.shape
    Nkv = k_host.shape[2]
    if tuple(k_host.shape) != (B, H, Nkv, d) or tuple(v_host.shape) != (B, H, Nkv, d):
        raise ValueError("k_host and v_host must be [B, H, Nkv, d] matching q_host")
    if k_host.dtype != q_host.dtype or v_host.dtype != q_host.dtype:
        raise TypeError("q_host, k_host, v_host must share one dtype")
    dtype = _dtype_code(q_host)
    index = torch.cuda.current_device()
    if _elsewhere_stream(stream, index):
        return _under(stream, index, lambda: fwd_offload(q_host, k_host, v_host, out_host, lse_host, q, k, v, out,
                                                         lse, scale, causal, key_len, heads_per_chunk),
                      q, k, v, out, lse)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dev = torch.device("cuda", index)
    q = torch.empty(q_host.shape, dtype=q_host.dtype, device=dev) if q is None else q
    k = torch.empty(k_host.shape, dtype=k_host.dtype, device=dev) if k is None else k
    v = torch.empty(v_host.shape, dtype=v_host.dtype, device=dev) if v is None else v
    out = torch.empty(q_host.shape, dtype=q_host.dtype, device=dev) if out is None else out
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=dev) if lse is None else lse
    if out_host is None:
        out_host = torch.empty(q_host.shape, dtype=q_host.dtype).pin_memory()
    if lse_host is None:
        lse_host = torch.empty((B, H, Nq), dtype=torch.float32).pin_memory()
    for t, ref in ((q, q_host), (k, k_host), (v, v_host), (out, q_host), (out_host, q_host)):
        if tuple(t.shape) != tuple(ref.shape) or t.dtype != ref.dtype or not t.is_contiguous():
            raise ValueError("device buffers and out_host must be contiguous and match the inputs")
    for t in (lse, lse_host):
        if tuple(t.shape) != (B, H, Nq) or t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError("lse and lse_host must be contiguous fp32 [B, H, Nq]")
    if out_host.is_cuda or lse_host.is_cuda or not all(t.is_cuda for t in (q, k, v, out, lse)):
        raise ValueError("host tensors must be CPU tensors and staging buffers CUDA tensors")
    key_len, kl_ptr = _key_len_ptr(key_len, B)
    st = lib().osattn_fwd_offload(q_host.data_ptr(), k_host.data_ptr(), v_host.data_ptr(),
                                  out_host.data_ptr(), lse_host.data_ptr(), q.data_ptr(),
                                  k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H,
                                  Nq, Nkv, d, float(scale), int(bool(causal)), kl_ptr, dtype,
                                  int(heads_per_chunk), _stream_handle(stream))
    if st != OK:
        raise OsattnError(st, "osattn_fwd_offload")
    return out_host, lse_host


def fwd_splitkv(q, k, v, num_splits: int, scale: float | None = None, causal: bool = False,
                key_len=None, out=None, lse=None, workspace=None, stream=None):
    """Split-KV attention forward (bf16 or fp16): same result as fwd(), the key axis cut
    into num_splits ranges merged by the (m, l) combine.  `workspace` may be a
    preallocated CUDA uint8 tensor of at least splitkv_workspace_bytes(...)
    bytes; otherwise torch allocates one."""
    import torch

    B, H, Nq, Nkv, d = _check_qkv(q, k, v)
    index = q.get_device()
    if _elsewhere_stream(stream, index):
        return _under(stream, index, lambda: fwd_splitkv(q, k, v, num_splits, scale, causal, key_len, out, lse,
                                                         workspace), out, lse, workspace)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device) if lse is None else lse
    need = splitkv_workspace_bytes(B, H, Nq, d, max(int(num_splits), 1))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    key_len, kl_ptr = _key_len_ptr(key_len, B)
    dtype = _dtype_code(q)
    st = lib().osattn_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                  lse.data_ptr(), B, H, Nq, Nkv, d, float(scale),
                                  int(bool(causal)), kl_ptr, dtype, int(num_splits),
                                  workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                  _stream_handle(stream))
    if st != OK:
        raise OsattnError(st, "osattn_fwd_splitkv")
    return out, lse


def bwd_workspace_bytes(B: int, H: int, Nq: int) -> int:
    return int(lib().osattn_bwd_workspace_bytes(int(B), int(H), int(Nq)))


def bwd(q, k, v, o, lse, do, scale: float | None = None, causal: bool = False, key_len=None,
        dq=None, dk=None, dv=None, workspace=None, stream=None):
    """dQ, dK, dV of the attention forward for the upstream gradient `do`.

    q, k, v, o, do: CUDA bf16, fp16 or fp32 tensors ([B,H,Nq,d] for q, o, do;
    [B,H,Nkv,d] for k, v), any views whose last axis is contiguous; lse: the
    contiguous fp32 [B,H,Nq] LSE that fwd() returned for the same inputs.
    Contiguous tensors go through osattn_bwd, others through
    osattn_bwd_strided.  Outputs may be given preallocated (any such views);
    `workspace` (a CUDA uint8 tensor of at least bwd_workspace_bytes(B, H,
    Nq) bytes) too."""
    import torch

    B, H, Nq, Nkv, d = _shapes(q, k, v)
    dtype = _dtype_code(q)
    index = q.get_device()
    if _elsewhere_stream(stream, index):
        return _under(stream, index, lambda: bwd(q, k, v, o, lse, do, scale, causal, key_len, dq, dk, dv, workspace),
                      dq, dk, dv, workspace)
    for t in (o, do):
        if t.shape != q.shape or t.dtype != q.dtype or not t.is_cuda:
            raise ValueError("o and do must be CUDA tensors shaped and typed like q")
    if tuple(lse.shape) != (B, H, Nq) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be fp32 [B, H, Nq]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for t, ref in ((dq, q), (dk, k), (dv, v)):
        if t.shape != ref.shape or t.dtype != ref.dtype or not t.is_cuda:
            raise ValueError("dq, dk, dv must be CUDA tensors shaped and typed like q, k, v")
    need = bwd_workspace_bytes(B, H, Nq)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    key_len, kl_ptr = _key_len_ptr(key_len, B)
    ts = (q, k, v, o, do, dq, dk, dv)
    ptrs = [t.data_ptr() for t in ts]
    tail = (float(scale), int(bool(causal)), kl_ptr, dtype, workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if all(t.is_contiguous() for t in ts):
        st = lib().osattn_bwd(*ptrs[:5], lse.data_ptr(), *ptrs[5:], B, H, Nq, Nkv, d, *tail)
        what = "osattn_bwd"
    else:
        strides = [_bhn_strides(t) for t in ts]
        st = lib().osattn_bwd_strided(*ptrs[:5], lse.data_ptr(), *ptrs[5:], B, H, Nq, Nkv, d,
                                      *strides, *tail)
        what = "osattn_bwd_strided"
    if st != OK:
        raise OsattnError(st, what)
    return dq, dk, dv


def bwd_offload(q_host, k_host, v_host, o_host, lse_host, do_host, scale: float | None = None,
                causal: bool = False, key_len=None, dq_host=None, dk_host=None, dv_host=None,
                device_buffers=None, workspace=None, heads_per_chunk: int = 0, stream=None):
    """Gradients of host tensors through osattn_bwd_offload: inputs as for
    bwd() but contiguous CPU tensors (pinned for the copies to overlap the
    compute); dq_host, dk_host, dv_host are allocated (pinned) when not given.
    device_buffers, if given, is a tuple of the nine contiguous CUDA staging
    tensors (q, k, v, o, do, dq, dk, dv, lse); otherwise they are allocated.
    Returns (dq_host, dk_host, dv_host), valid once `stream` has
    synchronised."""
    import torch

    ins = (q_host, k_host, v_host, o_host, do_host)
    for t in ins + (lse_host,):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("host inputs must be contiguous CPU tensors")
    if q_host.dim() != 4:
        raise ValueError("q_host must be [B, H, Nq, d]")
    B, H, Nq, d = q_host.shape
    Nkv = k_host.shape[2]
    if tuple(k_host.shape) != (B, H, Nkv, d) or tuple(v_host.shape) != (B, H, Nkv, d):
        raise ValueError("k_host and v_host must be [B, H, Nkv, d] matching q_host")
    for t in (o_host, do_host):
        if tuple(t.shape) != tuple(q_host.shape):
            raise ValueError("o_host and do_host must be shaped like q_host")
    for t in ins[1:]:
        if t.dtype != q_host.dtype:
            raise TypeError("host inputs must share one dtype")
    if tuple(lse_host.shape) != (B, H, Nq) or lse_host.dtype != torch.float32:
        raise ValueError("lse_host must be fp32 [B, H, Nq]")
    dtype = _dtype_code(q_host)
    index = torch.cuda.current_device()
    if _elsewhere_stream(stream, index):
        return _under(stream, index, lambda: bwd_offload(q_host, k_host, v_host, o_host, lse_host, do_host, scale,
                                                         causal, key_len, dq_host, dk_host, dv_host, device_buffers,
                                                         workspace, heads_per_chunk),
                      *(device_buffers or ()), workspace)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dev = torch.device("cuda", index)
    if device_buffers is None:
        mk = lambda ref: torch.empty(ref.shape, dtype=ref.dtype, device=dev)  # noqa: E731
        device_buffers = (mk(q_host), mk(k_host), mk(v_host), mk(o_host), mk(do_host),
                          mk(q_host), mk(k_host), mk(v_host), mk(lse_host))
    qd, kd, vd, od, dod, dqd, dkd, dvd, lsed = device_buffers
    for t, ref in zip(device_buffers, (q_host, k_host, v_host, o_host, do_host, q_host, k_host,
                                       v_host, lse_host)):
        if (not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != tuple(ref.shape)
                or t.dtype != ref.dtype):
            raise ValueError("device buffers must be contiguous CUDA tensors matching the inputs")
    pin = lambda ref: torch.empty(ref.shape, dtype=ref.dtype).pin_memory()  # noqa: E731
    dq_host = pin(q_host) if dq_host is None else dq_host
    dk_host = pin(k_host) if dk_host is None else dk_host
    dv_host = pin(v_host) if dv_host is None else dv_host
    for t, ref in ((dq_host, q_host), (dk_host, k_host), (dv_host, v_host)):
        if t.is_cuda or not t.is_contiguous() or tuple(t.shape) != tuple(ref.shape) or t.dtype != ref.dtype:
            raise ValueError("dq_host, dk_host, dv_host must be contiguous CPU tensors matching the inputs")
    need = bwd_workspace_bytes(B, H, Nq)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    key_len, kl_ptr = _key_len_ptr(key_len, B)
    st = lib().osattn_bwd_offload(
        q_host.data_ptr(), k_host.data_ptr(), v_host.data_ptr(), o_host.data_ptr(),
        do_host.data_ptr(), lse_host.data_ptr(), dq_host.data_ptr(), dk_host.data_ptr(),
        dv_host.data_ptr(), qd.data_ptr(), kd.data_ptr(), vd.data_ptr(), od.data_ptr(),
        dod.data_ptr(), lsed.data_ptr(), dqd.data_ptr(), dkd.data_ptr(), dvd.data_ptr(), B, H, Nq,
        Nkv, d, float(scale), int(bool(causal)), kl_ptr, dtype, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), int(heads_per_chunk), _stream_handle(stream))
    if st != OK:
        raise OsattnError(st, "osattn_bwd_offload")
    return dq_host, dk_host, dv_host


def softmax_rows(x, out=None, lse=None, want_lse: bool = True, stream=None):
    """Row softmax of a contiguous CUDA [rows, N] bf16/fp16/fp32 tensor (online (m, l)
    normaliser).  Returns (y, lse or None); `out` may be `x` (in place)."""
    import torch

    if x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA [rows, N] tensor")
    codes = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}
    if x.dtype not in codes:
        raise TypeError("x must be bf16, fp16 or fp32")
    index = x.get_device()
    if _elsewhere_stream(stream, index):
        return _under(stream, index, lambda: softmax_rows(x, out, lse, want_lse), out, lse)
    rows, N = x.shape
    out = torch.empty_like(x) if out is None else out
    if want_lse and lse is None:
        lse = torch.empty(rows, dtype=torch.float32, device=x.device)
    dtype = codes[x.dtype]
    st = lib().osattn_softmax_rows(x.data_ptr(), out.data_ptr(),
                                   None if lse is None else lse.data_ptr(), rows, N, dtype,
                                   _stream_handle(stream))
    if st != OK:
        raise OsattnError(st, "osattn_softmax_rows")
    return out, lse


def softmax_rows_offload(x_host, out_host=None, lse_host=None, x=None, out=None, lse=None,
                         want_lse: bool = True, rows_per_chunk: int = 0, stream=None):
    """Row softmax of a contiguous CPU [rows, N] tensor (pinned for the copies
    to overlap) through osattn_softmax_rows_offload; x/out/lse are the device
    staging buffers (allocated when not given), out_host/lse_host the pinned
    results (allocated when not given).  Returns (out_host, lse_host or None),
    valid once `stream` has synchronised."""
    import torch

    if x_host.dim() != 2 or x_host.is_cuda or not x_host.is_contiguous():
        raise ValueError("x_host must be a contiguous CPU [rows, N] tensor")
    codes = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}
    if x_host.dtype not in codes:
        raise TypeError("x_host must be bf16, fp16 or fp32")
    rows, N = x_host.shape
    index = torch.cuda.current_device()
    if _elsewhere_stream(stream, index):
        return _under(stream, index, lambda: softmax_rows_offload(x_host, out_host, lse_host, x, out, lse, want_lse,
                                                                  rows_per_chunk), x, out, lse)
    dev = torch.device("cuda", index)
    x = torch.empty(x_host.shape, dtype=x_host.dtype, device=dev) if x is None else x
    out = torch.empty_like(x) if out is None else out
    out_host = torch.empty(x_host.shape, dtype=x_host.dtype).pin_memory() if out_host is None else out_host
    if want_lse:
        lse = torch.empty(rows, dtype=torch.float32, device=dev) if lse is None else lse
        lse_host = torch.empty(rows, dtype=torch.float32).pin_memory() if lse_host is None else lse_host
    else:
        lse = lse_host = None
    for t in (x, out):
        if not t.is_cuda or not t.is_contiguous() or t.shape != x_host.shape or t.dtype != x_host.dtype:
            raise ValueError("x and out must be contiguous CUDA tensors shaped like x_host")
    if out_host.is_cuda or not out_host.is_contiguous() or out_host.shape != x_host.shape:
        raise ValueError("out_host must be a contiguous CPU tensor shaped like x_host")
    st = lib().osattn_softmax_rows_offload(
        x_host.data_ptr(), out_host.data_ptr(), None if lse_host is None else lse_host.data_ptr(),
        x.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(), rows, N,
        codes[x_host.dtype], int(rows_per_chunk), _stream_handle(stream))
    if st != OK:
        raise OsattnError(st, "osattn_softmax_rows_offload")
    return out_host, lse_host


# ---------------------------------------------------------------- modified scores
_CODES = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}


class MaskPlan:
    """Which keys each query row sees: what mask_plan() returns and fwd_mod()
    and bwd_mod() take.  `buffer` is private to the library."""

    __slots__ = ("buffer", "B", "Nq", "Nkv", "q_offset", "stream")

    def __init__(self, buffer, B, Nq, Nkv, q_offset, stream=None):
        self.buffer, self.B, self.Nq, self.Nkv, self.q_offset = buffer, B, Nq, Nkv, q_offset
        self.stream = stream  # the one whose memory the buffer is

    def use(self, stream, index):
        """The buffer's address, for work on `stream`, the current one of
        device `index`: until that is done, the memory of a plan that is
        dropped is not handed out again."""
        if stream != self.stream:
            import torch

            self.buffer.record_stream(torch.cuda.current_stream(index))
        return self.buffer.data_ptr()


def _int32(t, shape, index, name):
    if t is None:
        return None
    if t.dtype != torch.int32 or not t.is_cuda or t.shape != shape:
        raise ValueError(f"{name} must be a CUDA int32 tensor of shape {list(shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on another device")
    return t.contiguous()


def _elsewhere(index):
    """Whether another device than `index` is current."""
    return torch.cuda.current_device() != index


def _address(strides):
    """Where the strides of _strides3() lie (as long as they are kept)."""
    return None if strides is None else ctypes.addressof(strides)


def _packed(t):
    """Whether the tensor of _of() `t` has no gaps and no repeats: torch.empty_like() then has its strides."""
    n = 1
    for stride, size in sorted(zip(t[1], t[0])):
        if size == 0 or (size != 1 and stride != n):
            return False
        n *= size
    return True


@functools.lru_cache(maxsize=256)
def _strides3(a, b, c):
    return (ctypes.c_int64 * 3)(a, b, c)


def _view_strides(t, name):
    """(b, h, row) element strides of a [B, H, N, d] view.  The stride of an
    axis of length 1 is never used to reach an element; one that the library
    would refuse is replaced."""
    b, h, n, one = t.stride()
    if one != 1:
        raise ValueError(f"the last (d) axis of {name} must have stride 1")
    shape = t.shape
    if 1 in shape:
        B, H, N, d = shape
        n = d if N == 1 else n
        h = max(n * N, 8) if H == 1 else h
        b = max(h * H, 8) if B == 1 else b
    return _strides3(b, h, n)


def mask_plan(B: int, Nq: int, Nkv: int, causal: bool = False, window: int = 0, q_offset: int = 0,
              key_len=None, prefix_len=None, doc_ids=None, device=None, out=None, stream=None):
    """The keys that each of B x Nq query rows sees, for fwd_mod() and
    bwd_mod(); one plan serves every layer and both passes of a step.

    Row i stands at position p = i + q_offset; key j is visible to it iff
    j < key_len[b]; with `causal` j <= p or j < prefix_len[b]; with a window
    |j - p| < window; with doc_ids ([B, Nkv] int32) j and p lie in one run of
    equal, non-negative ids.  key_len, prefix_len: CUDA int32 [B].  `out`: a
    MaskPlan of the same B and Nq to overwrite."""
    masks = (key_len, prefix_len, doc_ids)
    for t in masks:
        if t is not None and device is None:
            device = t.device
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise ValueError("a mask plan lives on a CUDA device")
    index = torch.cuda.current_device() if device.index is None else device.index
    if _elsewhere(index):
        with torch.cuda.device(index):
            return mask_plan(B, Nq, Nkv, causal, window, q_offset, *masks, device=f"cuda:{index}", out=out,
                             stream=stream)
    if _elsewhere_stream(stream, index):
        return _under(stream, index, lambda: mask_plan(B, Nq, Nkv, causal, window, q_offset, *masks,
                                                       device=f"cuda:{index}", out=out),
                      None if out is None else out.buffer)
    B, Nq, Nkv, window, q_offset = int(B), int(Nq), int(Nkv), int(window), int(q_offset)
    key_len = _int32(key_len, (B,), index, "key_len")
    prefix_len = _int32(prefix_len, (B,), index, "prefix_len")
    doc_ids = _int32(doc_ids, (B, Nkv), index, "doc_ids")
    handle = _raw_stream(index)
    if out is None:
        # tiles of 128 rows take 16 bytes each, rows 8
        need = max(B, 0) * ((max(Nq, 0) + 127) // 128 * 16 + max(Nq, 0) * 8)
        plan = MaskPlan(torch.empty(max(need, 16), dtype=torch.uint8, device=device), B, Nq, Nkv, q_offset, handle)
    else:
        plan = out
        if out.B != B or out.Nq != Nq or out.buffer.get_device() != index:
            raise ValueError("out must be a MaskPlan of the same B, Nq and device")
    st = (_lib or lib()).osattn_mask_plan(plan.use(handle, index), plan.buffer.numel(), B, Nq, Nkv, q_offset,
                                1 if causal else 0, window,
                                None if key_len is None else key_len.data_ptr(),
                                None if prefix_len is None else prefix_len.data_ptr(),
                                None if doc_ids is None else doc_ids.data_ptr(), handle)
    if st != OK:
        raise OsattnError(st, "osattn_mask_plan")
    plan.Nkv, plan.q_offset = Nkv, q_offset
    return plan


def rel_buckets(num_buckets: int, max_distance: int, bidirectional: bool = True):
    """A bucket map for fwd_mod()'s rel_map: int32 [2 * max_distance + 1], the
    bucket of each distance (key position less query position) from
    -max_distance to max_distance.  Small distances get a bucket each, the
    rest share buckets spaced by the logarithm up to max_distance; with
    `bidirectional` one half of the buckets is for keys behind the query,
    otherwise all such keys fall into bucket 0.  A CPU tensor."""
    num_buckets, max_distance = int(num_buckets), int(max_distance)
    n = num_buckets // 2 if bidirectional else num_buckets
    small = n // 2
    if small < 1 or max_distance <= small:
        raise ValueError("need at least 2 buckets a side and max_distance above the exact ones")
    out = []
    for rel in range(-max_distance, max_distance + 1):
        base = n if bidirectional and rel > 0 else 0
        dist = abs(rel) if bidirectional else max(-rel, 0)
        if dist >= small:
            dist = min(n - 1, small + int(math.log(dist / small) / math.log(max_distance / small)
                                          * (n - small)))
        out.append(base + dist)
    return torch.tensor(out, dtype=torch.int32)


def _mod_shapes(q, k, v):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q must be [B, H, Nq, d], k and v [B, Hkv, Nkv, d]")
    B, H, Nq, d = q.shape
    Hkv, Nkv = k.shape[1], k.shape[2]
    if k.shape != (B, Hkv, Nkv, d) or v.shape != k.shape:
        raise ValueError("k and v must be [B, Hkv, Nkv, d] matching q")
    if H < 1 or Hkv < 1 or H % Hkv or d < 1:
        raise ValueError("there must be heads, those of k and v dividing those of q, and d of at least 1")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share one dtype")
    if not q.is_cuda:
        raise ValueError("q, k, v must be CUDA tensors")
    index = q.get_device()
    if k.get_device() != index or v.get_device() != index:
        raise ValueError("q, k, v must be on one device")
    return B, H, Hkv, Nq, Nkv, d, index


def _slopes(slopes, H, index):
    if slopes.shape != (H,) or slopes.dtype != torch.float32 or slopes.get_device() != index:
        raise ValueError("slopes must be an fp32 tensor of shape [H] on q's device")
    return slopes.contiguous()


def _score(q, plan, index, H, B, Nq, Nkv, softcap, slopes, rel_table, rel_map):
    """struct osattn_score of a call, and the tensors it points into."""
    s = _Score(softcap)
    held = []
    if plan is not None:
        if (plan.B, plan.Nq, plan.Nkv) != (B, Nq, Nkv) or plan.buffer.get_device() != index:
            raise ValueError("plan was made for other sizes or another device")
        s.q_offset = plan.q_offset
    if slopes is not None:
        held.append(_slopes(slopes, H, index))
        s.slopes = held[-1].data_ptr()
    if (rel_table is None) != (rel_map is None):
        raise ValueError("rel_table and rel_map go together")
    if rel_table is not None:
        if (rel_table.dim() != 2 or rel_table.shape[1] != H or rel_table.dtype != q.dtype
                or rel_table.get_device() != index):
            raise ValueError("rel_table must be [buckets, H] with q's dtype and device")
        if (rel_map.dim() != 1 or rel_map.numel() % 2 == 0 or rel_map.dtype != torch.int32
                or rel_map.get_device() != index):
            raise ValueError("rel_map must be int32 [2 R + 1] on q's device")
        held += [rel_table.contiguous(), rel_map.contiguous()]
        s.rel_table, s.rel_map = held[-2].data_ptr(), held[-1].data_ptr()
        s.rel_num, s.rel_range = rel_table.shape[0], rel_map.numel() // 2
    return s, held


def _lse(lse, shape, index, like):
    """The caller's LSE tensor, or a new one."""
    if lse is None:
        return like.new_empty(shape, dtype=torch.float32)
    if (lse.shape != shape or lse.dtype != torch.float32 or not lse.is_contiguous()
            or lse.get_device() != index):
        raise ValueError(f"lse must be contiguous fp32 {list(shape)} on q's device")
    return lse


def fwd_mod(q, k, v, scale: float | None = None, plan=None, softcap: float = 0.0, slopes=None,
            rel_table=None, rel_map=None, out=None, lse=None, stream=None):
    """O, LSE = attention forward with modified scores: q [B,H,Nq,d], k/v
    [B,Hkv,Nkv,d] with Hkv dividing H, bf16 or fp16, any views whose last axis
    is contiguous.

    The scaled score y of query position p and key j becomes
    softcap * tanh(y / softcap) if softcap > 0 (0.001 .. 10000), then y - slopes[h] |j - p|
    (slopes: fp32 [H]) or y + rel_table[rel_map[clamp(j - p, -R, R) + R], h]
    (rel_table: [buckets, H] in q's dtype; rel_map: int32 [2 R + 1], see
    rel_buckets()).  plan: a MaskPlan, or None for no mask.  A row that sees
    no key gets O = 0 and LSE = -inf."""
    B, H, Hkv, Nq, Nkv, d, index = _mod_shapes(q, k, v)
    if _elsewhere(index):
        with torch.cuda.device(index):
            return fwd_mod(q, k, v, scale, plan, softcap, slopes, rel_table, rel_map, out, lse, stream)
    if _elsewhere_stream(stream, index):
        return _under(stream, index, lambda: fwd_mod(q, k, v, scale, plan, softcap, slopes, rel_table, rel_map, out,
                                                     lse), out, lse)
    dtype = _CODES.get(q.dtype)
    if dtype is None:
        raise TypeError("tensors must be bf16 or fp16")
    score, held = _score(q, plan, index, H, B, Nq, Nkv, softcap, slopes, rel_table, rel_map)
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or out.get_device() != index:
        raise ValueError("out must match q")
    lse = _lse(lse, (B, H, Nq), index, q)
    handle = _raw_stream(index)
    st = (_lib or lib()).osattn_fwd_mod(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, Hkv, Nq, Nkv, d,
        _view_strides(q, "q"), _view_strides(k, "k"), _view_strides(v, "v"), _view_strides(out, "out"),
        1.0 / math.sqrt(d) if scale is None else scale, ctypes.byref(score),
        None if plan is None else plan.use(handle, index), dtype, handle)
    if st != OK:
        raise OsattnError(st, "osattn_fwd_mod")
    return out, lse


def bwd_mod_workspace_bytes(B: int, H: int, Nq: int, Nkv: int, rel_range: int = 0) -> int:
    return int(lib().osattn_bwd_mod_workspace_bytes(int(B), int(H), int(Nq), int(Nkv), int(rel_range)))


def _bwd_mod_workspace(B, H, Nq, Nkv, rel_range):
    """bwd_mod_workspace_bytes() without a call into the library."""
    return 4 * B * H * (Nq + ((Nkv + 127) // 128 * (2 * rel_range + 1) if rel_range else 0))


def bwd_mod(q, k, v, o, lse, do, scale: float | None = None, plan=None, softcap: float = 0.0,
            slopes=None, rel_table=None, rel_map=None, dq=None, dk=None, dv=None, drel=None,
            workspace=None, stream=None):
    """dQ, dK, dV, and with a rel_table dRel [buckets, H], of fwd_mod() for the
    upstream gradient `do`, from its outputs o and lse.  Arguments as for
    fwd_mod(); dk and dv are summed over the query heads of a key head.
    Outputs and the workspace (a CUDA uint8 tensor of at least
    bwd_mod_workspace_bytes(B, H, Nq, Nkv, R or 0) bytes) may be given."""
    B, H, Hkv, Nq, Nkv, d, index = _mod_shapes(q, k, v)
    if _elsewhere(index):
        with torch.cuda.device(index):
            return bwd_mod(q, k, v, o, lse, do, scale, plan, softcap, slopes, rel_table, rel_map, dq, dk, dv,
                           drel, workspace, stream)
    if _elsewhere_stream(stream, index):
        return _under(stream, index, lambda: bwd_mod(q, k, v, o, lse, do, scale, plan, softcap, slopes, rel_table,
                                                     rel_map, dq, dk, dv, drel, workspace),
                      dq, dk, dv, drel, workspace)
    dtype = _CODES.get(q.dtype)
    if dtype is None:
        raise TypeError("tensors must be bf16 or fp16")
    for t in (o, do):
        if t.shape != q.shape or t.dtype != q.dtype or t.get_device() != index:
            raise ValueError("o and do must be shaped, typed and placed like q")
    if lse is None:
        raise ValueError("lse must be the one that fwd_mod() returned")
    _lse(lse, (B, H, Nq), index, None)
    score, held = _score(q, plan, index, H, B, Nq, Nkv, softcap, slopes, rel_table, rel_map)

    def grad(g, ref):
        if g is None:
            return torch.empty_like(ref)
        if g.shape != ref.shape or g.dtype != ref.dtype or g.get_device() != index:
            raise ValueError("gradients must be shaped, typed and placed like their tensors")
        return g

    dq, dk, dv = grad(dq, q), grad(dk, k), grad(dv, v)
    if rel_table is not None:
        drel = grad(drel, held[-2])  # the contiguous table
        if not drel.is_contiguous():
            raise ValueError("drel must be contiguous")
    elif drel is not None:
        raise ValueError("drel needs a rel_table")
    L = _lib or lib()
    if workspace is None:
        workspace = q.new_empty(_bwd_mod_workspace(B, H, Nq, Nkv, score.rel_range), dtype=torch.uint8)
    elif not workspace.is_contiguous() or workspace.get_device() != index:
        raise ValueError("workspace must be contiguous on q's device")
    handle = _raw_stream(index)
    st = L.osattn_bwd_mod(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), None if drel is None else drel.data_ptr(), B, H, Hkv,
        Nq, Nkv, d, _view_strides(q, "q"), _view_strides(k, "k"), _view_strides(v, "v"),
        _view_strides(o, "o"), _view_strides(do, "do"), _view_strides(dq, "dq"), _view_strides(dk, "dk"),
        _view_strides(dv, "dv"), 1.0 / math.sqrt(d) if scale is None else scale, ctypes.byref(score),
        None if plan is None else plan.use(handle, index), dtype, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), handle)
    if st != OK:
        raise OsattnError(st, "osattn_bwd_mod")
    return (dq, dk, dv) if drel is None else (dq, dk, dv, drel)


# ---------------------------------------------------------------- paged cache
def tree_workspace_bytes(B: int, H: int, Hkv: int, T: int, d: int) -> int:
    return int(lib().osattn_tree_workspace_bytes(int(B), int(H), int(Hkv), int(T), int(d)))


def _tree_workspace(B, group, T, d):
    """tree_workspace_bytes() without a call into the library (4 us of a step
    of 31, its code being cold after a launch)."""
    return (B + 4) // 4 * 16 + 1280 * min(T, max(128 // group, 1)) * group * (d + 1)


def tree_e4m3_workspace_bytes(B: int, H: int, Hkv: int, T: int, d: int) -> int:
    return int(lib().osattn_tree_e4m3_workspace_bytes(int(B), int(H), int(Hkv), int(T), int(d)))


def _tree_e4m3_workspace(B, group, T, d):
    """tree_e4m3_workspace_bytes() without a call into the library."""
    return (B + 4) // 4 * 16 + 1280 * min(T * group, 128) * (d + 1)


def _of(t):
    """What a call's plan asks of a tensor: shape, strides, type, device (None: there is no tensor)."""
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _flat(t):
    """The same, but whether it lies in one piece for its strides."""
    return None if t is None else (t.shape, t.is_contiguous(), t.dtype, t.get_device())


def _device_of(*tensors):
    """The device of _of() or _flat() `tensors`, the first of which is there."""
    index = tensors[0][3]
    if index < 0 or any(t is not None and t[3] != index for t in tensors):
        raise ValueError("the tensors of a call must be CUDA tensors on one device")
    return index


def _ints(t, shape, name):
    """Whether the int32 tensor of _flat() `t` has to be copied to lie in one piece."""
    if t is None:
        return False
    if t[2] != torch.int32 or tuple(t[0]) != shape:
        raise ValueError(f"{name} must be a CUDA int32 tensor of shape {list(shape)}")
    return not t[1]


def _strides_of(t, name):
    """(b, h, row) element strides of a [B, H, N, d] view (see _view_strides)."""
    (B, H, N, d), (b, h, n, one) = t[0], t[1]
    if one != 1:
        raise ValueError(f"the last (d) axis of {name} must have stride 1")
    n = d if N == 1 else n
    h = max(n * N, 16) if H == 1 else h
    b = max(h * H, 16) if B == 1 else b
    return _strides3(b, h, n)


def _scale_block(k_scale, v_scale, pages, Hkv, page_size):
    """The tokens that each scale of an e4m3 cache is for."""
    if k_scale is None or v_scale is None:
        raise ValueError("float8_e4m3fn pages need k_scale and v_scale")
    n = k_scale[0][-1] if len(k_scale[0]) == 3 else 0
    for t in (k_scale, v_scale):
        if tuple(t[0]) != (pages, Hkv, n) or t[2] != torch.float32 or not t[1]:
            raise ValueError("k_scale and v_scale must be contiguous fp32 [pages, Hkv, page_size / block] on the "
                             "pages' device")
    if n < 1 or page_size % n:
        raise ValueError("the scales of a page must divide its rows evenly")
    return page_size // n


# What the arguments' shapes, strides, types and devices say about a call, worked out once for
# each set of them: a step of a serving loop asks the same again and again (an append for 64
# sequences 24.5 -> 21.5 us of host time, one token over e4m3 pages 34 -> 29).  Of what is left
# the library's call takes 5 to 8 us, the first new output 5, others 2 to 3.
@functools.lru_cache(maxsize=256)
def _tree_e4m3_plan(q, k, v, ks, vs, table, ctx, mask):
    if len(q[0]) != 4 or len(k[0]) != 4 or v[0] != k[0]:
        raise ValueError("q must be [B, H, T, d], k_pages and v_pages [pages, Hkv, page_size, d]")
    B, H, T, d = q[0]
    pages, Hkv, page_size, dk = k[0]
    if dk != d or H < 1 or Hkv < 1 or H % Hkv or d < 1:
        raise ValueError("k_pages must have q's d and a number of heads that divides q's, none of them 0")
    if v[2] != k[2]:
        raise TypeError("k_pages and v_pages must share q's dtype, or be float8_e4m3fn")
    dtype = _CODES.get(q[2])
    if dtype is None:
        raise TypeError("tensors must be bf16 or fp16")
    block = _scale_block(ks, vs, pages, Hkv, page_size)
    if len(table[0]) != 2:
        raise ValueError("page_table must be [B, max_pages]")
    max_pages = table[0][1]
    copies = (_ints(table, (B, max_pages), "page_table"), _ints(ctx, (B,), "ctx_len"), False)
    if mask is not None:
        if mask[2] != torch.int64 or tuple(mask[0]) != (B, T):
            raise ValueError("tree_mask must be int64 [B, T] on q's device")
        copies = (*copies[:2], not mask[1])
    keep = (_strides_of(q, "q"), _strides_of(k, "k_pages"), _strides_of(v, "v_pages"))
    own = keep[0] if _packed(q) else None
    index = _device_of(q, k, v, ks, vs, table, ctx, mask)
    need = _tree_e4m3_workspace(B, H // Hkv, T, d)
    # (new tensors are made like these, which costs half of naming a size and a type)
    lse = torch.empty(1, dtype=torch.float32, device=torch.device("cuda", index)).expand(B, H, T)
    workspace = torch.empty(1, dtype=torch.uint8, device=lse.device).expand(need)
    return ((B, H, Hkv, T, d, pages, page_size, max_pages, block, *map(_address, keep)), copies, dtype,
            1.0 / math.sqrt(d), index, need, lse, workspace, own, keep)


def _tree_attn_e4m3(q, k_pages, v_pages, page_table, ctx_len, tree_mask, scale, softcap, slopes, window, out, lse,
                    workspace, stream, k_scale, v_scale):
    """tree_attn() over float8_e4m3fn pages."""
    args, copies, dtype, usual, index, need, lse_like, workspace_like, o_strides, _ = _tree_e4m3_plan(
        _of(q), _of(k_pages), _of(v_pages), _flat(k_scale), _flat(v_scale), _flat(page_table), _flat(ctx_len),
        _flat(tree_mask))
    if _elsewhere(index):
        with torch.cuda.device(index):
            return _tree_attn_e4m3(q, k_pages, v_pages, page_table, ctx_len, tree_mask, scale, softcap, slopes,
                                   window, out, lse, workspace, stream, k_scale, v_scale)
    if stream is not None and _elsewhere_stream(stream, index):
        return _under(stream, index, lambda: _tree_attn_e4m3(q, k_pages, v_pages, page_table, ctx_len, tree_mask,
                                                             scale, softcap, slopes, window, out, lse, workspace, None,
                                                             k_scale, v_scale), out, lse, workspace)
    if copies[0]:
        page_table = page_table.contiguous()
    if copies[1]:
        ctx_len = ctx_len.contiguous()
    if copies[2]:
        tree_mask = tree_mask.contiguous()
    if slopes is not None:
        slopes = _slopes(slopes, args[1], index)
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or out.get_device() != index:
        raise ValueError("out must match q")
    else:
        o_strides = None
    if o_strides is None:
        o_strides = _strides_of((q.shape, out.stride()), "out")
    lse = torch.empty_like(lse_like) if lse is None else _lse(lse, lse_like.shape, index, q)
    if workspace is None:
        workspace = torch.empty_like(workspace_like)
    else:
        if not workspace.is_contiguous() or workspace.get_device() != index:
            raise ValueError("workspace must be contiguous on q's device")
        need = workspace.numel() * workspace.element_size()
    st = (_lib or lib()).osattn_tree_attn_e4m3(
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        page_table.data_ptr(), ctx_len.data_ptr(), None if tree_mask is None else tree_mask.data_ptr(),
        out.data_ptr(), lse.data_ptr(), *args, o_strides,
        usual if scale is None else scale, softcap, None if slopes is None else slopes.data_ptr(), int(window), dtype,
        workspace.data_ptr(), need, _raw_stream(index))
    if st != OK:
        raise OsattnError(st, "osattn_tree_attn_e4m3")
    return out, lse


def tree_attn(q, k_pages, v_pages, page_table, ctx_len, tree_mask=None, scale: float | None = None,
              softcap: float = 0.0, slopes=None, window: int = 0, out=None, lse=None,
              workspace=None, stream=None, k_scale=None, v_scale=None):
    """O, LSE of T drafted tokens of every sequence (T = 1: a decode step) over
    its paged cache: q [B,H,T,d], k_pages/v_pages [pages,Hkv,page_size,d], bf16
    or fp16, any views whose last axis is contiguous; page_table int32
    [B,max_pages]; ctx_len int32 [B], the cached keys before the drafts, whose
    own keys follow them in the pages; tree_mask int64 [B,T], bit u of entry t
    set iff draft t sees draft u (None: u <= t; 0: padding, O = 0, LSE = -inf).

    softcap and slopes (fp32 [H]) as in fwd_mod(), with a window keys at a
    distance of at least `window` are hidden; draft t stands at ctx_len +
    (bits of its mask) - 1, which for a tree is its depth behind the context.

    Pages may be float8_e4m3fn, as cache_append() writes them: k_scale and
    v_scale (contiguous fp32 [pages,Hkv,page_size/block]) then hold the factor of
    each block of rows of a page, and q is bf16 or fp16.  They halve a decode step
    over long contexts; from 17 query rows a key head on (T H / Hkv) 16-bit pages are up
    to a third faster."""
    if k_pages.dtype is torch.float8_e4m3fn:
        return _tree_attn_e4m3(q, k_pages, v_pages, page_table, ctx_len, tree_mask, scale, softcap, slopes, window,
                               out, lse, workspace, stream, k_scale, v_scale)
    if k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale are for float8_e4m3fn pages")
    if q.dim() != 4 or k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
        raise ValueError("q must be [B, H, T, d], k_pages and v_pages [pages, Hkv, page_size, d]")
    B, H, T, d = q.shape
    pages, Hkv, page_size, dk = k_pages.shape
    if dk != d or H < 1 or Hkv < 1 or H % Hkv or d < 1:
        raise ValueError("k_pages must have q's d and a number of heads that divides q's, none of them 0")
    if k_pages.dtype != q.dtype or v_pages.dtype != q.dtype:
        raise TypeError("q, k_pages, v_pages must share one dtype (or the pages be float8_e4m3fn)")
    index = q.get_device()
    if not q.is_cuda or k_pages.get_device() != index or v_pages.get_device() != index:
        raise ValueError("q, k_pages, v_pages must be CUDA tensors on one device")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    if _elsewhere(index):
        with torch.cuda.device(index):
            return tree_attn(q, k_pages, v_pages, page_table, ctx_len, tree_mask, scale, softcap, slopes,
                             window, out, lse, workspace, stream)
    if _elsewhere_stream(stream, index):
        return _under(stream, index, lambda: tree_attn(q, k_pages, v_pages, page_table, ctx_len, tree_mask, scale,
                                                       softcap, slopes, window, out, lse, workspace),
                      out, lse, workspace)
    dtype = _CODES.get(q.dtype)
    if dtype is None:
        raise TypeError("tensors must be bf16 or fp16")
    max_pages = page_table.shape[1]
    page_table = _int32(page_table, (B, max_pages), index, "page_table")
    ctx_len = _int32(ctx_len, (B,), index, "ctx_len")
    if tree_mask is not None:
        if (tree_mask.dtype != torch.int64 or tree_mask.shape != (B, T)
                or tree_mask.get_device() != index):
            raise ValueError("tree_mask must be int64 [B, T] on q's device")
        tree_mask = tree_mask.contiguous()
    if slopes is not None:
        slopes = _slopes(slopes, H, index)
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or out.get_device() != index:
        raise ValueError("out must match q")
    lse = _lse(lse, (B, H, T), index, q)
    L = _lib or lib()
    if workspace is None:
        workspace = q.new_empty(_tree_workspace(B, H // Hkv, T, d), dtype=torch.uint8)
    elif not workspace.is_contiguous() or workspace.get_device() != index:
        raise ValueError("workspace must be contiguous on q's device")
    st = L.osattn_tree_attn(
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), ctx_len.data_ptr(),
        None if tree_mask is None else tree_mask.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, Hkv, T,
        d, pages, page_size, max_pages, _view_strides(q, "q"), _view_strides(k_pages, "k_pages"),
        _view_strides(v_pages, "v_pages"), _view_strides(out, "out"),
        1.0 / math.sqrt(d) if scale is None else scale, softcap,
        None if slopes is None else slopes.data_ptr(), int(window), dtype, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _raw_stream(index))
    if st != OK:
        raise OsattnError(st, "osattn_tree_attn")
    return out, lse


@functools.lru_cache(maxsize=256)
def _append_plan(k, v, kp, vp, ks, vs, table, ctx, count, q, freqs, at):
    if len(k[0]) != 4 or v[0] != k[0] or len(kp[0]) != 4 or vp[0] != kp[0]:
        raise ValueError("k and v must be [B, Hkv, T, d], k_pages and v_pages [pages, Hkv, page_size, d]")
    B, Hkv, T, d = k[0]
    pages, heads, page_size, dk = kp[0]
    if heads != Hkv or dk != d or Hkv < 1 or d < 1:
        raise ValueError("k_pages must have k's heads and d, none of them 0")
    dtype = _CODES.get(k[2])
    if dtype is None or v[2] != k[2]:
        raise TypeError("k and v must both be bf16 or both fp16")
    e4m3 = kp[2] == torch.float8_e4m3fn
    if vp[2] != kp[2] or not (e4m3 or kp[2] == k[2]):
        raise TypeError("k_pages and v_pages must share k's dtype, or be float8_e4m3fn")
    if not e4m3 and (ks is not None or vs is not None):
        raise ValueError("k_scale and v_scale are for float8_e4m3fn pages")
    block = _scale_block(ks, vs, pages, Hkv, page_size) if e4m3 else 0
    if len(table[0]) != 2:
        raise ValueError("page_table must be [B, max_pages]")
    max_pages = table[0][1]
    copies = [_ints(table, (B, max_pages), "page_table"), _ints(ctx, (B,), "ctx_len"), _ints(count, (B,), "new_len"),
              False, False]
    if freqs is None:
        if q is not None or at is not None:
            raise ValueError("q and positions are for a rotation: they need freqs")
    else:
        copies[3] = _freqs_of(freqs, d)
        copies[4] = _ints(at, (B, T), "positions")
    H, q_strides, own, rot = 0, None, None, 0 if freqs is None else 2 * freqs[0][0]
    if q is not None:
        H = q[0][1] if len(q[0]) == 4 else 0
        if tuple(q[0]) != (B, H, T, d) or H < 1 or q[2] != k[2]:
            raise ValueError("q must be [B, H, T, d] with k's dtype and device")
        q_strides = _strides_of(q, "q")
        own = q_strides if _packed(q) else None
    keep = (_strides_of(k, "k"), _strides_of(v, "v"), q_strides, _strides_of(kp, "k_pages"), _strides_of(vp, "v_pages"))
    return ((B, H, Hkv, T, d, pages, page_size, max_pages, block, *map(_address, keep)), any(copies), copies, dtype,
            E4M3 if e4m3 else dtype, rot, _device_of(k, v, kp, vp, ks, vs, table, ctx, count, q, freqs, at), own, keep)


def cache_append(k, v, k_pages, v_pages, page_table, ctx_len, new_len=None, q=None, freqs=None, positions=None,
                 interleaved: bool = False, amplitude: float = 1.0, q_out=None, k_scale=None, v_scale=None,
                 stream=None):
    """Writes the keys and values of T new tokens of every sequence, k/v
    [B,Hkv,T,d] in bf16 or fp16, into its pages (k_pages, v_pages
    [pages,Hkv,page_size,d], page_table int32 [B,max_pages]) behind the ctx_len
    (int32 [B]) tokens that are there; of sequence b the first new_len[b] of them
    (int32 [B]; None: T).  tree_attn() with the same ctx_len sees them.

    With freqs (see rotary()) the keys are rotated on the way, by positions
    (int32 [B,T]; None: ctx_len + t), and q [B,H,T,d] too: the result is q rotated
    (into q_out, which may be q), else None.

    Pages have k's dtype, or float8_e4m3fn with k_scale and v_scale (contiguous
    fp32 [pages,Hkv,page_size/block]): a block's scale is the least power of two
    with which its rows fit, grown, and its older rows rounded anew, when later
    rows need it.  A page that is written belongs to one sequence."""
    args, copy, copies, dtype, cache_dtype, rot, index, qo_strides, _ = _append_plan(
        _of(k), _of(v), _of(k_pages), _of(v_pages), _flat(k_scale), _flat(v_scale), _flat(page_table), _flat(ctx_len),
        _flat(new_len), _of(q), _flat(freqs), _flat(positions))
    if _elsewhere(index):
        with torch.cuda.device(index):
            return cache_append(k, v, k_pages, v_pages, page_table, ctx_len, new_len, q, freqs, positions,
                                interleaved, amplitude, q_out, k_scale, v_scale, stream)
    if stream is not None and _elsewhere_stream(stream, index):
        return _under(stream, index, lambda: cache_append(k, v, k_pages, v_pages, page_table, ctx_len, new_len, q,
                                                          freqs, positions, interleaved, amplitude, q_out, k_scale,
                                                          v_scale),
                      k_pages, v_pages, k_scale, v_scale, q_out)
    if copy:
        page_table, ctx_len, new_len, freqs, positions = (
            t.contiguous() if c else t for t, c in zip((page_table, ctx_len, new_len, freqs, positions), copies))
    if q is not None:
        if q_out is None:
            q_out = torch.empty_like(q)
        elif q_out.shape != q.shape or q_out.dtype != q.dtype or q_out.get_device() != index:
            raise ValueError("q_out must match q")
        else:
            qo_strides = None
        if qo_strides is None:
            qo_strides = _strides_of((q.shape, q_out.stride()), "q_out")
    elif q_out is not None:
        raise ValueError("q_out needs q")
    st = (_lib or lib()).osattn_cache_append(
        k.data_ptr(), v.data_ptr(), None if q is None else q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
        None if k_scale is None else k_scale.data_ptr(), None if v_scale is None else v_scale.data_ptr(),
        None if q is None else q_out.data_ptr(), page_table.data_ptr(), ctx_len.data_ptr(),
        None if new_len is None else new_len.data_ptr(), None if positions is None else positions.data_ptr(), *args,
        qo_strides, None if freqs is None else _rotation(freqs, rot, interleaved, amplitude), dtype, cache_dtype,
        _raw_stream(index))
    if st != OK:
        raise OsattnError(st, "osattn_cache_append")
    return q_out


# ---------------------------------------------------------------- rotary positions
def rotary_freqs(rot: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                 original: int = 4096, low: float = 1.0, high: float = 32.0):
    """Frequencies for rotary() and cache_append(): fp64 [rot / 2], radians a
    position, base^(-2 i / rot).  A CPU tensor.

    scaling stretches them for contexts `factor` times as long: "linear" divides
    all by factor; "base" raises the base so that the slowest is divided by it
    and the fastest stays; "ramp" keeps those that turn `high` times or more over
    `original` positions, divides those that turn `low` times or less, and
    blends in between (a context stretched so is often used with an amplitude of
    0.1 ln(factor) + 1).  The ramp is linear in the turns over `original`; for
    one that is linear in the pair's number instead, as some models have it, make the
    fp64 [rot / 2] tensor yourself: the calls take any frequencies."""
    rot = int(rot)
    if rot < 2 or rot % 2 or not base > 0 or not factor > 0:
        raise ValueError("rot must be even and at least 2, base and factor above 0")
    if scaling not in (None, "linear", "base", "ramp"):
        raise ValueError("scaling must be None, 'linear', 'base' or 'ramp'")
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = torch.tensor([float(base) ** (-i / rot) for i in range(0, rot, 2)], dtype=torch.float64)
    if scaling == "linear":
        f = f / factor
    elif scaling == "ramp":
        if not high > low or original < 1:
            raise ValueError("high must be above low, original at least 1")
        keep = ((original * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
    return f


def _freqs_of(freqs, d):
    """Whether the frequencies of _flat() `freqs` have to be copied to lie in one piece."""
    if len(freqs[0]) != 1 or freqs[2] != torch.float64:
        raise ValueError("freqs must be fp64 [rot / 2] on the tensors' device")
    if not 1 <= freqs[0][0] <= d // 2:
        raise ValueError("freqs must be for 2 .. d elements of a row")
    return not freqs[1]


def _rotation(freqs, rot, interleaved, amplitude):
    return _ROTATION.pack(freqs.data_ptr(), rot, 1 if interleaved else 0, amplitude)


@functools.lru_cache(maxsize=256)
def _rotary_plan(q, k, freqs, at):
    if len(q[0]) != 4 or (k is not None and len(k[0]) != 4):
        raise ValueError("q must be [B, H, N, d], k [B, Hkv, N, d]")
    B, H, N, d = q[0]
    dtype = _CODES.get(q[2])
    if dtype is None or (k is not None and k[2] != q[2]):
        raise TypeError("q and k must both be bf16, fp16 or fp32")
    if k is not None and (k[0][0] != B or k[0][2] != N or k[0][3] != d):
        raise ValueError("k must have q's batch, rows and d")
    if freqs is None:
        raise ValueError("freqs must be given")
    each = 1 if at is not None and len(at[0]) == 2 else 0
    copies = (_freqs_of(freqs, d), _ints(at, (B, N) if each else (N,), "positions"))

    def strides(t):
        if t is not None and t[1][3] != 1 and d != 1:
            raise ValueError("the last (d) axis must have stride 1")
        return None if t is None else _strides3(*t[1][:3])

    keep = (strides(q), strides(k))
    own = [x if t is not None and _packed(t) else None for t, x in zip((q, k), keep)]
    return ((B, H, 0 if k is None else k[0][1], N, d, *map(_address, keep)), copies, each, dtype, 2 * freqs[0][0],
            _device_of(q, k, freqs, at), *own, keep)


def _rotated(y, x, name, index):
    """The caller's output for x, or a new one (dense where x is broadcast)."""
    if y is None:
        return x.new_empty(x.shape) if 0 in x.stride() else torch.empty_like(x)
    if y.shape != x.shape or y.dtype != x.dtype or y.get_device() != index:
        raise ValueError(f"{name} must match its tensor")
    if y.stride(3) != 1 and y.shape[3] != 1:
        raise ValueError(f"the last (d) axis of {name} must have stride 1")
    return y


def rotary(q, k=None, freqs=None, positions=None, offset: int = 0, interleaved: bool = False,
           amplitude: float = 1.0, inverse: bool = False, out=None, k_out=None, stream=None):
    """q [B,H,N,d], and k [B,Hkv,N,d] if it is given, with their rows rotated by
    their positions: pair i of a row's first 2 len(freqs) elements turns by
    freqs[i] * position (freqs: CUDA fp64, see rotary_freqs()) and is multiplied
    by amplitude; the other elements stay.  Pairs are (i, i + len(freqs)), or
    (2 i, 2 i + 1) with `interleaved`.  positions: int32 [N] or [B,N]; None: row n
    stands at offset + n.

    With `inverse` by the negative angles: rotary(dy, ..., inverse=True) is the
    gradient of rotary(x, ...).  bf16, fp16 or fp32, any views whose last axis is
    contiguous (broadcast ones too); out and k_out may be given, and may be q and
    k.  Returns q's result, or the pair with k's."""
    args, copies, each, dtype, rot, index, o_strides, ko_strides, _ = _rotary_plan(_of(q), _of(k), _flat(freqs),
                                                                                  _flat(positions))
    if not -(1 << 31) <= offset < 1 << 31:
        raise ValueError("offset must be a 32-bit position")
    if _elsewhere(index):
        with torch.cuda.device(index):
            return rotary(q, k, freqs, positions, offset, interleaved, amplitude, inverse, out, k_out, stream)
    if stream is not None and _elsewhere_stream(stream, index):
        return _under(stream, index, lambda: rotary(q, k, freqs, positions, offset, interleaved, amplitude, inverse,
                                                    out, k_out), out, k_out)
    if copies[0]:
        freqs = freqs.contiguous()
    if copies[1]:
        positions = positions.contiguous()
    if out is None and o_strides is not None:
        out = torch.empty_like(q)
    else:
        out = _rotated(out, q, "out", index)
        o_strides = _strides3(*out.stride()[:3])
    k_ptr = ko_ptr = None
    if k is not None:
        if k_out is None and ko_strides is not None:
            k_out = torch.empty_like(k)
        else:
            k_out = _rotated(k_out, k, "k_out", index)
            ko_strides = _strides3(*k_out.stride()[:3])
        k_ptr, ko_ptr = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out needs k")
    st = (_lib or lib()).osattn_rotary(
        q.data_ptr(), k_ptr, out.data_ptr(), ko_ptr, *args, o_strides, ko_strides,
        _rotation(freqs, rot, interleaved, amplitude), None if positions is None else positions.data_ptr(), each,
        int(offset), 1 if inverse else 0, dtype, _raw_stream(index))
    if st != OK:
        raise OsattnError(st, "osattn_rotary")
    return out if k is None else (out, k_out)


def get_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return lib().osattn_get_device_status(_stream_handle(stream))


def version() -> int:
    return lib().osattn_version()
