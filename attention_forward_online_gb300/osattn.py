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
import threading

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libosattn.so")

BF16 = 0
FP32 = 1
FP16 = 2
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
           "osattn_bwd_mod_workspace_bytes", "osattn_tree_attn", "osattn_tree_workspace_bytes")

_lock = threading.Lock()
_lib = None


class _Score(ctypes.Structure):
    """struct osattn_score of include/osattn.h."""

    _fields_ = [("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p),
                ("rel_table", ctypes.c_void_p), ("rel_map", ctypes.c_void_p),
                ("rel_num", ctypes.c_int), ("rel_range", ctypes.c_int),
                ("q_offset", ctypes.c_int)]


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
    import torch

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


def tree_attn(q, k_pages, v_pages, page_table, ctx_len, tree_mask=None, scale: float | None = None,
              softcap: float = 0.0, slopes=None, window: int = 0, out=None, lse=None,
              workspace=None, stream=None):
    """O, LSE of T drafted tokens of every sequence (T = 1: a decode step) over
    its paged cache: q [B,H,T,d], k_pages/v_pages [pages,Hkv,page_size,d], bf16
    or fp16, any views whose last axis is contiguous; page_table int32
    [B,max_pages]; ctx_len int32 [B], the cached keys before the drafts, whose
    own keys follow them in the pages; tree_mask int64 [B,T], bit u of entry t
    set iff draft t sees draft u (None: u <= t; 0: padding, O = 0, LSE = -inf).

    softcap and slopes (fp32 [H]) as in fwd_mod(), with a window keys at a
    distance of at least `window` are hidden; draft t stands at ctx_len +
    (bits of its mask) - 1, which for a tree is its depth behind the context."""
    if q.dim() != 4 or k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
        raise ValueError("q must be [B, H, T, d], k_pages and v_pages [pages, Hkv, page_size, d]")
    B, H, T, d = q.shape
    pages, Hkv, page_size, dk = k_pages.shape
    if dk != d or H < 1 or Hkv < 1 or H % Hkv or d < 1:
        raise ValueError("k_pages must have q's d and a number of heads that divides q's, none of them 0")
    if k_pages.dtype != q.dtype or v_pages.dtype != q.dtype:
        raise TypeError("q, k_pages, v_pages must share one dtype")
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


def get_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return lib().osattn_get_device_status(_stream_handle(stream))


def version() -> int:
    return lib().osattn_version()
