"""Thin Python binding of the C ABI in ``include/fa.h`` (argument marshalling only).

Every entry point keeps the C name and takes torch CUDA tensors in place of
device pointers; shapes come from the tensors.  Nothing here computes: each
call checks the tensors, hands their pointers to ``libfa_gb300.so`` and turns a
non-OK status into ``FAError``.  If the library was not built the first call
raises: there is no fallback path.

``stream``: a torch stream or a handle; None is the current stream.  A call runs there without waiting for the current
stream: its inputs must be ready on it and stay until it is done.  Results that it allocates are ready on that stream and may be
used on the current one, too, once that has waited.
"""

from __future__ import annotations

import ctypes
import os
import threading
import warnings

import torch

__all__ = [
    "FAError", "library_path", "load_library", "DTYPE_CODES",
    "fa_fwd", "fa_bwd", "fa_bwd_workspace_size", "fa_bwd_preprocess", "fa_bwd_main", "fa_bwd_dq_convert",
    "fa_check_device_error", "fa_tile_counter", "fa_uses_tensor_cores", "fa_status_string",
    "fa_last_error_message", "fa_bwd_noalloc", "fa_fwd_gqa", "fa_bwd_gqa", "fa_decode", "fa_decode_workspace_size",
    "fa_quantize_fp8", "fa_fwd_fp8", "fa_fwd_fp8_gqa", "fa_fwd_masked", "fa_bwd_masked",
    "fa_selftest_bounded_wait", "fa_fwd_bwd_host", "fa_fwd_bwd_host_workspace_size",
    "attention_forward", "attention_backward", "attention_decode",
    "attention_forward_fp8", "quantize_fp8", "EXPORTED_SYMBOLS", "NOALLOC_SCRATCH_BYTES",
    "fa_sm_clock_sample", "kv4_cache", "fa_kv4_append", "fa_kv4_read", "kv4_read", "fa_decode_kv4",
    "fa_decode_kv4_workspace_size", "attention_decode_kv4", "fa_kv4_evict", "fa_fwd_varlen", "attention_forward_varlen",
    "fa_qk_norm_rope", "fa_qk_norm_rope_bwd", "fa_qk_norm_rope_bwd_workspace_size", "rope_table", "qk_norm_rope",
    "qk_norm_rope_backward", "fa_fwd_window", "fa_bwd_window", "fa_fwd_varlen_window",
    "fa_decode_window", "fa_decode_window_workspace_size", "fa_decode_prefix", "fa_decode_prefix_workspace_size",
    "attention_decode_window", "attention_decode_prefix",
]

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_FILE = "libfa_gb300.so"

FA_OK = 0
NOALLOC_SCRATCH_BYTES = 64 << 20  # FA_BWD_NOALLOC_SCRATCH_BYTES in include/fa.h
DTYPE_CODES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
EXPORTED_SYMBOLS = (
    "fa_fwd", "fa_bwd_workspace_size", "fa_bwd", "fa_bwd_preprocess", "fa_bwd_main", "fa_bwd_dq_convert",
    "fa_check_device_error", "fa_tile_counter", "fa_uses_tensor_cores", "fa_status_string",
    "fa_last_error_message", "fa_bwd_noalloc", "fa_fwd_gqa", "fa_bwd_gqa", "fa_decode", "fa_decode_workspace_size",
    "fa_quantize_fp8", "fa_fwd_fp8", "fa_fwd_fp8_gqa", "fa_fwd_masked", "fa_bwd_masked",
    "fa_selftest_bounded_wait", "fa_fwd_bwd_host", "fa_fwd_bwd_host_workspace_size", "fa_sm_clock_sample",
    "fa_debug_build", "fa_selftest_debug_check", "fa_kv4_append", "fa_kv4_read", "fa_decode_kv4",
    "fa_decode_kv4_workspace_size", "fa_kv4_evict", "fa_fwd_varlen", "fa_qk_norm_rope", "fa_qk_norm_rope_bwd",
    "fa_qk_norm_rope_bwd_workspace_size", "fa_fwd_window", "fa_bwd_window", "fa_fwd_varlen_window", "fa_decode_window",
    "fa_decode_window_workspace_size", "fa_decode_prefix", "fa_decode_prefix_workspace_size",
)

_lib = None
_lock = threading.Lock()


class FAError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


def library_path() -> str:
    return os.path.join(HERE, LIB_FILE)


def load_library(path=None):
    """Load ``libfa_gb300.so`` (built by ``exact_tiled_attention_07_gb300.build``); raises if absent.

    With ``path``, load that build of the library instead (for instance the FA_DEBUG build,
    ``build.build(debug=True)``) and make it the one every entry point here calls.
    """
    global _lib
    if path is None and _lib is not None:
        return _lib
    with _lock:
        if path is None and _lib is not None:
            return _lib
        path = path or library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"the CUDA library {path} is not built; run __graft_entry__.build() first")
        lib = ctypes.CDLL(path)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp]
        lib.fa_bwd_workspace_size.argtypes = [i, i, i, i]
        lib.fa_bwd_workspace_size.restype = sz
        lib.fa_bwd.argtypes = [vp] * 10 + [sz, i, i, i, i, f, i, i, vp]
        lib.fa_bwd_preprocess.argtypes = [vp, vp, vp, vp, sz, i, i, i, i, i, vp]
        lib.fa_bwd_main.argtypes = [vp] * 7 + [sz, i, i, i, i, f, i, i, vp]
        lib.fa_bwd_dq_convert.argtypes = [vp, sz, vp, i, i, i, i, f, i, vp]
        lib.fa_bwd_noalloc.argtypes = [vp] * 9 + [i, i, i, i, f, i, i, vp]
        lib.fa_fwd_gqa.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
        lib.fa_bwd_gqa.argtypes = [vp] * 10 + [sz, i, i, i, i, i, f, i, i, vp]
        lib.fa_decode_workspace_size.argtypes = [i] * 7
        lib.fa_decode_workspace_size.restype = sz
        lib.fa_decode.argtypes = [vp] * 5 + [i] * 6 + [f, i, i, vp, sz, vp]
        lib.fa_quantize_fp8.argtypes = [vp, vp, vp, i, i, i, i, i, vp]
        lib.fa_fwd_masked.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, i, i, vp]
        lib.fa_bwd_masked.argtypes = [vp] * 10 + [sz, i, i, i, i, i, f, i, i, vp, i, i, vp]
        lib.fa_fwd_fp8.argtypes = [vp] * 8 + [i, i, i, i, f, i, i, vp]
        lib.fa_fwd_fp8_gqa.argtypes = [vp] * 8 + [i, i, i, i, i, f, i, i, vp]
        lib.fa_selftest_bounded_wait.argtypes = [i, i, vp]
        lib.fa_fwd_bwd_host_workspace_size.argtypes = [i, i, i, i, i, i, i]
        lib.fa_fwd_bwd_host_workspace_size.restype = sz
        lib.fa_fwd_bwd_host.argtypes = [vp] * 10 + [sz, i, i, i, i, i, f, i, i, i, vp]
        i64 = ctypes.c_int64
        lib.fa_fwd_varlen.argtypes = [vp] * 6 + [i] * 5 + [i64] * 8 + [f, i, i, vp]
        lib.fa_kv4_append.argtypes = [vp] * 6 + [i] * 5 + [i64] * 4 + [i, vp]
        lib.fa_kv4_read.argtypes = [vp] * 5 + [i] * 5 + [i64] * 4 + [i, vp]
        lib.fa_decode_kv4_workspace_size.argtypes = [i] * 7
        lib.fa_decode_kv4_workspace_size.restype = sz
        lib.fa_decode_kv4.argtypes = [vp] * 7 + [i] * 6 + [f, i, i, vp, sz, vp]
        lib.fa_kv4_evict.argtypes = [vp] * 3 + [i, i] + [vp] * 4 + [i] * 5 + [vp]
        lib.fa_fwd_window.argtypes = [vp] * 5 + [i] * 5 + [f, i, i, i, vp]
        lib.fa_bwd_window.argtypes = [vp] * 10 + [sz] + [i] * 5 + [f, i, i, i, vp]
        lib.fa_fwd_varlen_window.argtypes = [vp] * 6 + [i] * 5 + [i64] * 8 + [f, i, i, i, vp]
        lib.fa_decode_window_workspace_size.argtypes = [i] * 6
        lib.fa_decode_window_workspace_size.restype = sz
        lib.fa_decode_window.argtypes = [vp] * 6 + [i] * 6 + [f, i, i, i, vp, sz, vp]
        lib.fa_decode_prefix_workspace_size.argtypes = [i] * 7
        lib.fa_decode_prefix_workspace_size.restype = sz
        lib.fa_decode_prefix.argtypes = [vp] * 8 + [i] * 7 + [f, i, vp, sz, vp]
        lib.fa_qk_norm_rope.argtypes = [vp] * 9 + [i] * 8 + [f, i, i, vp]
        lib.fa_qk_norm_rope_bwd_workspace_size.argtypes = [i]
        lib.fa_qk_norm_rope_bwd_workspace_size.restype = sz
        lib.fa_qk_norm_rope_bwd.argtypes = [vp] * 13 + [sz, vp] + [i] * 8 + [f, i, i, vp]
        lib.fa_check_device_error.argtypes = [vp]
        lib.fa_sm_clock_sample.argtypes = [vp, i, vp]
        lib.fa_debug_build.argtypes = []
        lib.fa_debug_build.restype = ctypes.c_int
        lib.fa_selftest_debug_check.argtypes = [i, i, vp]
        lib.fa_tile_counter.argtypes = [vp, ctypes.POINTER(ctypes.c_ulonglong), i]
        lib.fa_uses_tensor_cores.argtypes = [i, i, i]
        lib.fa_status_string.argtypes = [i]
        lib.fa_status_string.restype = ctypes.c_char_p
        lib.fa_last_error_message.argtypes = []
        lib.fa_last_error_message.restype = ctypes.c_char_p
        for name in ("fa_fwd", "fa_bwd", "fa_fwd_gqa", "fa_bwd_gqa", "fa_decode", "fa_quantize_fp8", "fa_fwd_fp8",
                     "fa_fwd_fp8_gqa",
                     "fa_fwd_masked", "fa_bwd_masked", "fa_selftest_bounded_wait", "fa_fwd_bwd_host",
                     "fa_bwd_noalloc", "fa_bwd_preprocess",
                     "fa_bwd_main", "fa_bwd_dq_convert",
                     "fa_check_device_error", "fa_tile_counter", "fa_uses_tensor_cores", "fa_sm_clock_sample",
                     "fa_selftest_debug_check", "fa_kv4_append", "fa_kv4_read", "fa_decode_kv4", "fa_kv4_evict",
                     "fa_fwd_varlen", "fa_qk_norm_rope", "fa_qk_norm_rope_bwd", "fa_fwd_window", "fa_bwd_window",
                     "fa_fwd_varlen_window", "fa_decode_window", "fa_decode_prefix"):
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
        return lib


def _check(status: int):
    if status != FA_OK:
        lib = load_library()
        msg = lib.fa_last_error_message().decode() or lib.fa_status_string(status).decode()
        raise FAError(status, msg)


def _stream(stream):
    if stream is None:
        # the handle alone: torch.cuda.current_stream() takes about 10 us of host time
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _p(t):
    return t.data_ptr() if t is not None else None


def _c_int(x):
    """x for a C int of the library, one that does not fit as the nearest that does: a window or a count of that size is
    past every length, or refused, either way.  (ctypes takes the low 32 bits: 2^32 sinks would be none.)"""
    x = int(x)
    return max(-0x80000000, min(x, 0x7FFFFFFF))


def _shape4(t):
    if t.dim() != 4:
        raise ValueError(f"expected a [B, H, N, d] tensor, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous [B, H, N, d]")
    return tuple(int(s) for s in t.shape)


def _dt(t):
    try:
        return DTYPE_CODES[t.dtype]
    except KeyError:
        raise ValueError(f"unsupported dtype {t.dtype}") from None


def _on_device(*ts, strided=()):
    """Every tensor given (None is skipped) is a contiguous CUDA tensor on the current device:
    the library takes raw device pointers and launches on the current device, so a host tensor
    or one on another GPU would hand the kernels an address they cannot use.  Those in `strided`
    (the first ones, checked by _packed) need not be contiguous."""
    dev = None
    for n, t in enumerate((*strided, *ts)):
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("device arguments must be CUDA tensors (the library takes device pointers)")
        if n >= len(strided) and not t.is_contiguous():
            raise ValueError("device arguments must be contiguous")
        if dev is None:
            dev, cur = t.device.index, torch.cuda.current_device()
            if dev != cur:
                raise ValueError(f"tensors are on cuda:{dev} but the current device is cuda:{cur}; "
                                 f"call within torch.cuda.device({dev})")
        elif t.device.index != dev:
            raise ValueError("all device arguments must be on one GPU")


def _ready(*ts, strided=()):
    """_on_device for the calls of a generation step, whose checks cost more than their kernels: one
    query a tensor; where something is not as it should be, _on_device says what."""
    first = strided[0] if strided else ts[0]
    dev = first.get_device()
    ok = dev >= 0 and dev == torch._C._cuda_getDevice()
    for t in strided:
        ok = ok and t.get_device() == dev
    for t in ts:
        ok = ok and (t is None or (t.get_device() == dev and t.is_contiguous()))
    if not ok:
        _on_device(*ts, strided=strided)


def _current(stream):
    """_stream after _ready (CUDA is up)."""
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()) if stream is None else _stream(stream)


def _new(shape, dtype, device, stream, scratch=False):
    """A tensor for a call on `stream` (None: the current one) to fill.  It comes from that stream's memory: a block of the current
    stream's may have been freed with kernels queued that still use it, which a call on another stream does not wait for.  What
    is returned (all but scratch) is the current stream's to use as well, so its memory is not handed out again before
    what that stream has queued by then."""
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if not scratch:
        t.record_stream(torch.cuda.current_stream())
    return t


def _new_workspace(nbytes, device, stream):
    return _new(nbytes, torch.uint8, device, stream, scratch=True)


def _rows(L, n, what="L"):
    """L (or another per-row vector) is an fp32 tensor of n elements."""
    if L.dtype != torch.float32 or L.numel() != n:
        raise ValueError(f"{what} must be an fp32 tensor of {n} elements")


def _same(ref, *ts):
    for t in ts:
        if t.shape != ref.shape or t.dtype != ref.dtype or t.device != ref.device or not t.is_contiguous():
            raise ValueError("Q, K, V, O, dO, dQ, dK, dV must share shape, dtype and device and be contiguous")


def fa_fwd(Q, K, V, O, L, scale, causal, stream=None):
    B, H, N, d = _shape4(Q)
    _on_device(Q, K, V, O, L)
    _same(Q, K, V, O)
    if L.dtype != torch.float32 or L.numel() != B * H * N or not L.is_contiguous():
        raise ValueError("L must be a contiguous fp32 tensor of B*H*N elements")
    _check(load_library().fa_fwd(_p(Q), _p(K), _p(V), _p(O), _p(L), B, H, N, d, float(scale), int(bool(causal)),
                                 _dt(Q), _stream(stream)))


def _kv_heads(Q, K, V, *kv_like):
    """Key/value head count of K (grouped-query attention) after checking the shapes agree."""
    B, H, N, d = _shape4(Q)
    Bk, Hkv, Nk, dk = _shape4(K)
    if (Bk, Nk, dk) != (B, N, d) or Hkv < 1 or H % Hkv:
        raise ValueError("K must be [B, Hkv, N, d] with H a multiple of Hkv")
    for t in (V,) + kv_like:
        if t.shape != K.shape or t.dtype != Q.dtype or t.device != Q.device or not t.is_contiguous():
            raise ValueError("K, V (and dK, dV) must share shape, dtype and device and be contiguous")
    return Hkv


def fa_fwd_gqa(Q, K, V, O, L, scale, causal, stream=None):
    B, H, N, d = _shape4(Q)
    _on_device(Q, K, V, O, L)
    Hkv = _kv_heads(Q, K, V)
    _same(Q, O)
    if L.dtype != torch.float32 or L.numel() != B * H * N or not L.is_contiguous():
        raise ValueError("L must be a contiguous fp32 tensor of B*H*N elements")
    _check(load_library().fa_fwd_gqa(_p(Q), _p(K), _p(V), _p(O), _p(L), B, H, Hkv, N, d, float(scale),
                                     int(bool(causal)), _dt(Q), _stream(stream)))


def fa_bwd_gqa(Q, K, V, O, dO, L, dQ, dK, dV, workspace, scale, causal, stream=None):
    B, H, N, d = _shape4(Q)
    _on_device(Q, K, V, O, dO, L, dQ, dK, dV, workspace)
    Hkv = _kv_heads(Q, K, V, dK, dV)
    _same(Q, O, dO, dQ)
    _rows(L, B * H * N)
    _check(load_library().fa_bwd_gqa(_p(Q), _p(K), _p(V), _p(O), _p(dO), _p(L), _p(dQ), _p(dK), _p(dV),
                                     _p(workspace), workspace.numel() * workspace.element_size(), B, H, Hkv, N, d,
                                     float(scale), int(bool(causal)), _dt(Q), _stream(stream)))


def fa_bwd_workspace_size(B, H, N, d) -> int:
    return int(load_library().fa_bwd_workspace_size(B, H, N, d))


def fa_bwd(Q, K, V, O, dO, L, dQ, dK, dV, workspace, scale, causal, stream=None):
    B, H, N, d = _shape4(Q)
    _on_device(Q, K, V, O, dO, L, dQ, dK, dV, workspace)
    _same(Q, K, V, O, dO, dQ, dK, dV)
    _rows(L, B * H * N)
    _check(load_library().fa_bwd(_p(Q), _p(K), _p(V), _p(O), _p(dO), _p(L), _p(dQ), _p(dK), _p(dV), _p(workspace),
                                 workspace.numel() * workspace.element_size(), B, H, N, d, float(scale),
                                 int(bool(causal)), _dt(Q), _stream(stream)))


def fa_bwd_preprocess(O, dO, L, workspace, stream=None):
    B, H, N, d = _shape4(O)
    _on_device(O, dO, L, workspace)
    _same(O, dO)
    _rows(L, B * H * N)
    _check(load_library().fa_bwd_preprocess(_p(O), _p(dO), _p(L), _p(workspace),
                                            workspace.numel() * workspace.element_size(), B, H, N, d, _dt(O),
                                            _stream(stream)))


def fa_bwd_main(Q, K, V, dO, dK, dV, workspace, scale, causal, stream=None):
    B, H, N, d = _shape4(Q)
    _on_device(Q, K, V, dO, dK, dV, workspace)
    _same(Q, K, V, dO, dK, dV)
    _check(load_library().fa_bwd_main(_p(Q), _p(K), _p(V), _p(dO), _p(dK), _p(dV), _p(workspace),
                                      workspace.numel() * workspace.element_size(), B, H, N, d, float(scale),
                                      int(bool(causal)), _dt(Q), _stream(stream)))


def fa_bwd_dq_convert(workspace, dQ, scale, stream=None):
    B, H, N, d = _shape4(dQ)
    _on_device(workspace, dQ)
    _check(load_library().fa_bwd_dq_convert(_p(workspace), workspace.numel() * workspace.element_size(), _p(dQ),
                                            B, H, N, d, float(scale), _dt(dQ), _stream(stream)))


def fa_bwd_noalloc(Q, K, V, O, dO, L, dQ, dK, dV, scale, causal, stream=None):
    """fa_bwd with the library's static device scratch instead of a workspace (no allocation)."""
    B, H, N, d = _shape4(Q)
    _on_device(Q, K, V, O, dO, L, dQ, dK, dV)
    _same(Q, K, V, O, dO, dQ, dK, dV)
    _rows(L, B * H * N)
    _check(load_library().fa_bwd_noalloc(_p(Q), _p(K), _p(V), _p(O), _p(dO), _p(L), _p(dQ), _p(dK), _p(dV), B, H, N,
                                         d, float(scale), int(bool(causal)), _dt(Q), _stream(stream)))


def fa_fwd_bwd_host_workspace_size(B, H, Hkv, N, d, dtype, chunk=0) -> int:
    return int(load_library().fa_fwd_bwd_host_workspace_size(B, H, Hkv, N, d, DTYPE_CODES[dtype], _c_int(chunk)))


def fa_fwd_bwd_host(Q, K, V, dO, O, L, dQ, dK, dV, workspace, scale, causal, chunk=0, stream=None):
    """Forward + backward with CPU tensors in and out (page-locked for the copies to overlap) and
    a device workspace of fa_fwd_bwd_host_workspace_size bytes."""
    B, H, N, d = _shape4(Q)
    Bk, Hkv, Nk, dk = _shape4(K)
    if (Bk, Nk, dk) != (B, N, d) or Hkv < 1 or H % Hkv:
        raise ValueError("K must be [B, Hkv, N, d] with H a multiple of Hkv")
    for t in (Q, K, V, dO, O, L, dQ, dK, dV):
        if t.device.type != "cpu" or not t.is_contiguous():
            raise ValueError("fa_fwd_bwd_host takes contiguous host (CPU) tensors")
    for t in (V, dK, dV):
        if t.shape != K.shape or t.dtype != Q.dtype:
            raise ValueError("V, dK, dV must be [B, Hkv, N, d] of Q's dtype")
    for t in (dO, O, dQ):
        if t.shape != Q.shape or t.dtype != Q.dtype:
            raise ValueError("dO, O, dQ must be [B, H, N, d] of Q's dtype")
    if L.dtype != torch.float32 or L.numel() != B * H * N:
        raise ValueError("L must be an fp32 tensor of B*H*N elements")
    if workspace.device.type != "cuda":
        raise ValueError("the workspace is device memory")
    _on_device(workspace)
    _check(load_library().fa_fwd_bwd_host(_p(Q), _p(K), _p(V), _p(dO), _p(O), _p(L), _p(dQ), _p(dK), _p(dV),
                                          _p(workspace), workspace.numel() * workspace.element_size(), B, H, Hkv, N,
                                          d, float(scale), int(bool(causal)), _dt(Q), _c_int(chunk), _stream(stream)))


def fa_decode_workspace_size(B, H, Hkv, Nq, Nk, d, splits=0) -> int:
    return int(load_library().fa_decode_workspace_size(B, H, Hkv, Nq, Nk, d, _c_int(splits)))


def fa_decode(Q, K, V, O, L, scale, splits=0, workspace=None, stream=None):
    """Decode: Q, O [B, H, Nq, d] against the cache K, V [B, Hkv, Nk, d]; L [B, H, Nq]."""
    B, H, Nq, d = _shape4(Q)
    Bk, Hkv, Nk, dk = _shape4(K)
    _on_device(Q, K, V, O, L, workspace)
    if (Bk, dk) != (B, d) or V.shape != K.shape or V.dtype != Q.dtype or K.dtype != Q.dtype or not V.is_contiguous():
        raise ValueError("K, V must be [B, Hkv, Nk, d] of Q's dtype")
    _same(Q, O)
    if L.dtype != torch.float32 or L.numel() != B * H * Nq or not L.is_contiguous():
        raise ValueError("L must be a contiguous fp32 tensor of B*H*Nq elements")
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().fa_decode(_p(Q), _p(K), _p(V), _p(O), _p(L), B, H, Hkv, Nq, Nk, d, float(scale), _c_int(splits),
                                    _dt(Q), _p(workspace), nbytes, _stream(stream)))


def fa_quantize_fp8(X, X8, scales, stream=None):
    """Block quantisation of X [B, H, N, d] to E4M3 codes X8 (uint8, same shape) and
    scales [B, H, ceil(N / 128)] fp32."""
    B, H, N, d = _shape4(X)
    _on_device(X, X8, scales)
    if X8.dtype != torch.uint8 or tuple(X8.shape) != (B, H, N, d) or not X8.is_contiguous():
        raise ValueError("X8 must be a contiguous uint8 tensor of X's shape")
    nb = (N + 127) // 128
    if scales.dtype != torch.float32 or scales.numel() != B * H * nb or not scales.is_contiguous():
        raise ValueError(f"scales must be a contiguous fp32 tensor of B*H*ceil(N/128) = {B * H * nb} elements")
    _check(load_library().fa_quantize_fp8(_p(X), _p(X8), _p(scales), B, H, N, d, _dt(X), _stream(stream)))


def fa_fwd_fp8(Q8, K8, V8, q_scales, k_scales, v_scales, O, L, scale, causal, stream=None):
    """Forward on E4M3 codes with block scales; O [B, H, N, d] bf16 or fp16, L [B, H, N] fp32.
    K8, V8 (and their scales) may have fewer heads than Q8 (grouped-query: fa_fwd_fp8_gqa)."""
    B, H, N, d = _shape4(Q8)
    Hkv = _shape4(K8)[1]
    _on_device(Q8, K8, V8, q_scales, k_scales, v_scales, O, L)
    nb = (N + 127) // 128
    for t, heads in ((Q8, H), (K8, Hkv), (V8, Hkv)):
        if t.dtype != torch.uint8 or tuple(t.shape) != (B, heads, N, d) or not t.is_contiguous():
            raise ValueError("Q8 [B, H, N, d] and K8, V8 [B, Hkv, N, d] must be contiguous uint8 tensors")
    if Hkv < 1 or H % Hkv:
        raise ValueError("H must be a multiple of the key/value heads Hkv")
    for t, heads in ((q_scales, H), (k_scales, Hkv), (v_scales, Hkv)):
        if t.dtype != torch.float32 or t.numel() != B * heads * nb or not t.is_contiguous():
            raise ValueError("block scales must be contiguous fp32 tensors of B*heads*ceil(N/128) elements")
    if tuple(O.shape) != (B, H, N, d) or not O.is_contiguous():
        raise ValueError("O must be a contiguous [B, H, N, d] tensor")
    if L.dtype != torch.float32 or L.numel() != B * H * N or not L.is_contiguous():
        raise ValueError("L must be a contiguous fp32 tensor of B*H*N elements")
    if Hkv != H:
        _check(load_library().fa_fwd_fp8_gqa(_p(Q8), _p(K8), _p(V8), _p(q_scales), _p(k_scales), _p(v_scales), _p(O),
                                             _p(L), B, H, Hkv, N, d, float(scale), int(bool(causal)), _dt(O),
                                             _stream(stream)))
        return
    _check(load_library().fa_fwd_fp8(_p(Q8), _p(K8), _p(V8), _p(q_scales), _p(k_scales), _p(v_scales), _p(O), _p(L),
                                     B, H, N, d, float(scale), int(bool(causal)), _dt(O), _stream(stream)))


def fa_fwd_fp8_gqa(Q8, K8, V8, q_scales, k_scales, v_scales, O, L, scale, causal, stream=None):
    """fa_fwd_fp8 with K8, V8 of Hkv heads (H a multiple of Hkv); the same checks."""
    fa_fwd_fp8(Q8, K8, V8, q_scales, k_scales, v_scales, O, L, scale, causal, stream)


def _mask_args(block_mask, H):
    """(pointer, mask_heads) of a uint8 block mask [nb, nb] (shared) or [H, nb, nb] (per head)."""
    if block_mask is None:
        return ctypes.c_void_p(0), 0
    if block_mask.dtype != torch.uint8 or not block_mask.is_contiguous() or not block_mask.is_cuda:
        raise ValueError("block_mask must be a contiguous uint8 CUDA tensor")
    heads = 1 if block_mask.dim() == 2 else block_mask.shape[0]
    return _p(block_mask), heads


def fa_fwd_masked(Q, K, V, O, L, scale, causal, window=0, block_mask=None, stream=None):
    """Forward with a sliding window and/or a block mask over 128 x 128 score blocks."""
    B, H, N, d = _shape4(Q)
    _on_device(Q, K, V, O, L, block_mask)
    Hkv = _kv_heads(Q, K, V)
    _same(Q, O)
    _rows(L, B * H * N)
    mp, mh = _mask_args(block_mask, H)
    _check(load_library().fa_fwd_masked(_p(Q), _p(K), _p(V), _p(O), _p(L), B, H, Hkv, N, d, float(scale),
                                        int(bool(causal)), _c_int(window), mp, mh, _dt(Q), _stream(stream)))


def fa_bwd_masked(Q, K, V, O, dO, L, dQ, dK, dV, workspace, scale, causal, window=0, block_mask=None, stream=None):
    """Backward of fa_fwd_masked (same mask)."""
    B, H, N, d = _shape4(Q)
    _on_device(Q, K, V, O, dO, L, dQ, dK, dV, workspace, block_mask)
    Hkv = _kv_heads(Q, K, V, dK, dV)
    _same(Q, O, dO, dQ)
    _rows(L, B * H * N)
    mp, mh = _mask_args(block_mask, H)
    nbytes = workspace.numel() * workspace.element_size()
    _check(load_library().fa_bwd_masked(_p(Q), _p(K), _p(V), _p(O), _p(dO), _p(L), _p(dQ), _p(dK), _p(dV),
                                        _p(workspace), nbytes, B, H, Hkv, N, d, float(scale), int(bool(causal)),
                                        _c_int(window), mp, mh, _dt(Q), _stream(stream)))


def _window_shape(Q, K, V, q_like=(), kv_like=(), rows=(), more=()):
    """(B, H, Hkv, N, d) of a call with a window and sinks, after checking its tensors: q_like shaped as Q, kv_like as K, rows fp32
    vectors of a number a query."""
    qs, ks, dt = Q.shape, K.shape, Q.dtype
    if len(qs) != 4 or len(ks) != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    B, H, N, d = qs
    if ks[0] != B or ks[2:] != qs[2:] or ks[1] < 1 or H % ks[1]:
        raise ValueError("K must be [B, Hkv, N, d] with H a multiple of Hkv")
    for t in q_like:
        if t.shape != qs or t.dtype != dt:
            raise ValueError("Q, O, dO and dQ must share shape and dtype")
    for t in (K, V, *kv_like):
        if t.shape != ks or t.dtype != dt:
            raise ValueError("K, V, dK and dV must share shape, and dtype with Q")
    for t in rows:
        _rows(t, B * H * N)
    _ready(Q, K, V, *q_like, *kv_like, *rows, *more)
    return B, H, ks[1], N, d


def fa_fwd_window(Q, K, V, O, L, scale, window, sinks=0, stream=None):
    """Causal forward with a sliding window and the first `sinks` keys always visible."""
    shape = _window_shape(Q, K, V, (O,), (), (L,))
    _check(load_library().fa_fwd_window(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), L.data_ptr(), *shape,
                                        float(scale), _c_int(window), _c_int(sinks), _dt(Q), _current(stream)))


def fa_bwd_window(Q, K, V, O, dO, L, dQ, dK, dV, workspace, scale, window, sinks=0, stream=None):
    """Backward of fa_fwd_window."""
    shape = _window_shape(Q, K, V, (O, dO, dQ), (dK, dV), (L,), (workspace,))
    _check(load_library().fa_bwd_window(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), dO.data_ptr(), L.data_ptr(),
                                        dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), workspace.data_ptr(),
                                        workspace.numel() * workspace.element_size(), *shape, float(scale), _c_int(window),
                                        _c_int(sinks), _dt(Q), _current(stream)))


def _packed(t, what):
    """(T, heads, d, token stride, head stride) of a packed [T, heads, d] tensor whose rows are
    contiguous; strides of one-sized dimensions, which torch leaves open, as if contiguous."""
    if t.dim() != 3:
        raise ValueError(f"{what}: expected a packed [T, heads, d] tensor, got shape {tuple(t.shape)}")
    T, h, d = t.shape
    ts, hs, es = t.stride()
    if d > 1 and es != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return T, h, d, (ts if T > 1 else h * d), (hs if h > 1 else d)


def _int32(t, n, what):
    if t.dtype != torch.int32 or t.numel() != n:
        raise ValueError(f"{what} must be an int32 tensor of {n} elements")


def _varlen_args(Q, K, V, O, L, cu_seqlens):
    """What the calls over packed sequences take up to their scale, after checking it."""
    T, H, d, q_ts, q_hs = _packed(Q, "Q")
    Tk, Hkv, dk, k_ts, k_hs = _packed(K, "K")
    _, _, _, v_ts, v_hs = _packed(V, "V")
    _, _, _, o_ts, o_hs = _packed(O, "O")
    _ready(L, cu_seqlens, strided=(Q, K, V, O))
    if (Tk, dk) != (T, d) or Hkv < 1 or H % Hkv:
        raise ValueError("K must be [T, Hkv, d] with H a multiple of Hkv")
    if V.shape != K.shape or O.shape != Q.shape or not (Q.dtype == K.dtype == V.dtype == O.dtype):
        raise ValueError("V must have K's shape, O must have Q's, and all four one dtype")
    _rows(L, H * T)
    n = cu_seqlens.numel()
    if cu_seqlens.dim() != 1 or n < 1:
        raise ValueError("cu_seqlens must be an int32 tensor of S + 1 elements")
    _int32(cu_seqlens, n, "cu_seqlens")
    return (Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), L.data_ptr(), cu_seqlens.data_ptr(), _c_int(n - 1), T, H, Hkv,
            d, q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs)


def fa_fwd_varlen(Q, K, V, O, L, cu_seqlens, scale, causal, stream=None):
    """Forward over packed sequences: Q, O [T, H, d], K, V [T, Hkv, d] (rows of contiguous d, any
    strides between them), L [H, T]; sequence s is rows cu_seqlens[s] .. cu_seqlens[s + 1] (int32)."""
    args = _varlen_args(Q, K, V, O, L, cu_seqlens)
    _check(load_library().fa_fwd_varlen(*args, scale, bool(causal), _dt(Q), _current(stream)))


def fa_fwd_varlen_window(Q, K, V, O, L, cu_seqlens, scale, window, sinks=0, stream=None):
    """fa_fwd_varlen, causal, with a sliding window and the first `sinks` rows of each sequence always visible."""
    args = _varlen_args(Q, K, V, O, L, cu_seqlens)
    _check(load_library().fa_fwd_varlen_window(*args, scale, _c_int(window), _c_int(sinks), _dt(Q), _current(stream)))


def _kv4_shape(cache):
    """(B, Hkv, capacity, d) of a 4-bit cache tensor (kv4_cache)."""
    if cache.dtype != torch.uint8 or cache.dim() != 4 or cache.shape[3] % 72:
        raise ValueError("a 4-bit cache is a uint8 tensor [B, Hkv, capacity / 64, 72 d]")
    B, Hkv, nb, nbytes = cache.shape
    return B, Hkv, nb * 64, nbytes // 72


def _kv4_weights(t, B, Hkv, capacity, what):
    if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != (B, Hkv, capacity)):
        raise ValueError(f"{what} must be an fp32 tensor [{B}, {Hkv}, {capacity}]")


def kv4_cache(B, Hkv, capacity, d, device="cuda"):
    """An empty 4-bit key/value cache for B sequences of up to `capacity` tokens (rounded up to a
    multiple of 64): a uint8 tensor [B, Hkv, capacity / 64, 72 d] (block layout: include/fa.h)."""
    if d not in (64, 128, 256):
        raise ValueError(f"the 4-bit cache supports d in {{64, 128, 256}}, got {d}")
    return torch.zeros((B, Hkv, (capacity + 63) // 64, 72 * d), dtype=torch.uint8, device=device)


def _kv4_rows(K, V, cu_seqlens, lens, cache, weights):
    B, Hkv, capacity, d = _kv4_shape(cache)
    T, hk, dk, k_ts, k_hs = _packed(K, "K")
    _, _, _, v_ts, v_hs = _packed(V, "V")
    _ready(cu_seqlens, lens, cache, weights, strided=(K, V))
    if (hk, dk) != (Hkv, d) or V.shape != K.shape or V.dtype != K.dtype:
        raise ValueError("K, V must be [T, Hkv, d] of one dtype with the cache's heads and head dimension")
    _int32(cu_seqlens, B + 1, "cu_seqlens")
    _int32(lens, B, "lens")
    _kv4_weights(weights, B, Hkv, capacity, "weights")
    return (B, T, Hkv, capacity, d, k_ts, k_hs, v_ts, v_hs, _dt(K))


def fa_kv4_append(K, V, cu_seqlens, lens, cache, weights=None, stream=None):
    """Packed rows K, V [T, Hkv, d] (rows cu_seqlens[b] .. cu_seqlens[b + 1] of sequence b) into the
    newest slots of a 4-bit cache; lens [B] counts them already. weights [B, Hkv, capacity]: set
    to 0 at the new slots."""
    args = _kv4_rows(K, V, cu_seqlens, lens, cache, weights)
    _check(load_library().fa_kv4_append(_p(K), _p(V), _p(cu_seqlens), _p(lens), _p(cache), _p(weights), *args,
                                        _current(stream)))


def fa_kv4_read(cache, cu_seqlens, lens, K, V, stream=None):
    """The values of the newest slots into packed K, V [T, Hkv, d]: the inverse of fa_kv4_append."""
    args = _kv4_rows(K, V, cu_seqlens, lens, cache, None)
    _check(load_library().fa_kv4_read(_p(cache), _p(cu_seqlens), _p(lens), _p(K), _p(V), *args, _current(stream)))


def fa_decode_kv4_workspace_size(B, H, Hkv, Nq, capacity, d, weights=False) -> int:
    return int(load_library().fa_decode_kv4_workspace_size(B, H, Hkv, Nq, capacity, d, int(bool(weights))))


def fa_decode_kv4(Q, cache, lens, O, L, scale, causal=False, weights_in=None, weights_out=None, workspace=None,
                  stream=None):
    """Decode: Q, O [B, H, Nq, d] over a 4-bit cache with lens [B] slots in use; L [B, H, Nq].
    weights_out [B, Hkv, capacity] = weights_in + the attention each slot got (slots in use). workspace: of
    fa_decode_kv4_workspace_size bytes; where none is given, one is allocated with torch."""
    shape = _kv4_decode_shape(Q, cache, lens, weights_in, weights_out)
    _ready(O, L, Q, workspace)
    _same(Q, O)
    _rows(L, O.numel() // O.shape[3])
    if workspace is None:
        workspace = _new_workspace(fa_decode_kv4_workspace_size(*shape, weights_out is not None), Q.device, stream)
    nbytes = workspace.numel() * workspace.element_size()
    _check(load_library().fa_decode_kv4(_p(Q), _p(cache), _p(lens), _p(O), _p(L), _p(weights_in), _p(weights_out),
                                        *shape, float(scale), int(bool(causal)), _dt(Q), _p(workspace), nbytes,
                                        _current(stream)))


def _kv4_decode_shape(Q, cache, lens, weights_in, weights_out):
    """(B, H, Hkv, Nq, capacity, d) of a decode over a 4-bit cache, after checking what it reads."""
    if Q.dim() != 4 or not Q.is_contiguous():
        _shape4(Q)
    B, H, Nq, d = Q.shape
    Bc, Hkv, capacity, dc = _kv4_shape(cache)
    _ready(Q, cache, lens, weights_in, weights_out)
    if (Bc, dc) != (B, d):
        raise ValueError("the cache must have Q's batch and head dimension")
    _int32(lens, B, "lens")
    _kv4_weights(weights_in, B, Hkv, capacity, "weights_in")
    _kv4_weights(weights_out, B, Hkv, capacity, "weights_out")
    return B, H, Hkv, Nq, capacity, d


def fa_kv4_evict(cache, weights, lens, keep, recent, out_cache, out_weights, out_lens, kept, stream=None):
    """The `recent` newest and the heaviest other slots of each sequence and head, `keep` in all, in
    their order into another cache (with weights and lens); kept [B, Hkv, keep]: where they were."""
    B, Hkv, capacity, d = _kv4_shape(cache)
    Bo, ho, out_capacity, do = _kv4_shape(out_cache)
    _ready(cache, weights, lens, out_cache, out_weights, out_lens, kept)
    if (Bo, ho, do) != (B, Hkv, d):
        raise ValueError("out_cache must have the cache's batch, heads and head dimension")
    if weights is None or out_weights is None:
        raise ValueError("eviction needs weights and out_weights")
    _kv4_weights(weights, B, Hkv, capacity, "weights")
    _kv4_weights(out_weights, B, Hkv, out_capacity, "out_weights")
    _int32(lens, B, "lens")
    _int32(out_lens, B, "out_lens")
    _int32(kept, B * Hkv * int(keep), "kept")
    _check(load_library().fa_kv4_evict(_p(cache), _p(weights), _p(lens), _c_int(keep), _c_int(recent), _p(out_cache),
                                       _p(out_weights), _p(out_lens), _p(kept), B, Hkv, capacity, out_capacity, d,
                                       _current(stream)))


def _cache_shape(Q, K, V, lens):
    """(B, H, Hkv, Nq, capacity, d) of a decode over 16-bit caches of different lengths, after checking what it reads."""
    if Q.dim() != 4 or K.dim() != 4:
        raise ValueError("expected Q [B, H, Nq, d] and caches [B, Hkv, capacity, d]")
    B, H, Nq, d = Q.shape
    Bk, Hkv, capacity, dk = K.shape
    _ready(Q, K, V, lens)
    if (Bk, dk) != (B, d) or V.shape != K.shape or not (Q.dtype == K.dtype == V.dtype):
        raise ValueError("K, V must be [B, Hkv, capacity, d] of Q's batch, head dimension and dtype")
    _int32(lens, B, "lens")
    return B, H, Hkv, Nq, capacity, d


def _prefix_shape(shape, Q, KP, VP):
    """shape with the prefix' length behind Nq, after checking KP, VP [Hkv, P, d]."""
    B, H, Hkv, Nq, capacity, d = shape
    if KP.dim() != 3 or (KP.shape[0], KP.shape[2]) != (Hkv, d) or VP.shape != KP.shape or not (
            KP.dtype == VP.dtype == Q.dtype):
        raise ValueError("the prefix must be [Hkv, P, d] of the caches' heads, head dimension and dtype")
    _ready(Q, KP, VP)
    return B, H, Hkv, Nq, KP.shape[1], capacity, d


def fa_decode_window_workspace_size(B, H, Hkv, Nq, capacity, d) -> int:
    return int(load_library().fa_decode_window_workspace_size(B, H, Hkv, Nq, capacity, d))


def fa_decode_prefix_workspace_size(B, H, Hkv, Nq, P, capacity, d) -> int:
    return int(load_library().fa_decode_prefix_workspace_size(B, H, Hkv, Nq, P, capacity, d))


def fa_decode_window(Q, K, V, lens, O, L, scale, window=0, sinks=0, workspace=None, stream=None):
    """Decode: Q, O [B, H, Nq, d] over caches K, V [B, Hkv, capacity, d] with lens [B] slots in use, the newest of them
    the Nq rows' own; window > 0: each row sees its `window` newest slots and the first `sinks`. L [B, H, Nq]. workspace: of
    fa_decode_window_workspace_size bytes; where none is given, one is allocated with torch."""
    shape = _cache_shape(Q, K, V, lens)
    _ready(O, L, Q, workspace)
    _same(Q, O)
    _rows(L, O.numel() // max(1, O.shape[3]))
    ws = workspace if workspace is not None else _new_workspace(fa_decode_window_workspace_size(*shape), Q.device, stream)
    _check(load_library().fa_decode_window(_p(Q), _p(K), _p(V), _p(lens), _p(O), _p(L), *shape, float(scale), _c_int(window),
                                           _c_int(sinks), _dt(Q), _p(ws), ws.numel() * ws.element_size(), _current(stream)))


def fa_decode_prefix(Q, KP, VP, K, V, lens, O, L, scale, workspace=None, stream=None):
    """Decode behind a shared prefix: as fa_decode_window without a window, and each row sees all of KP, VP [Hkv, P, d] too."""
    shape = _prefix_shape(_cache_shape(Q, K, V, lens), Q, KP, VP)
    _ready(O, L, Q, workspace)
    _same(Q, O)
    _rows(L, O.numel() // max(1, O.shape[3]))
    ws = workspace if workspace is not None else _new_workspace(fa_decode_prefix_workspace_size(*shape), Q.device, stream)
    _check(load_library().fa_decode_prefix(_p(Q), _p(KP), _p(VP), _p(K), _p(V), _p(lens), _p(O), _p(L), *shape, float(scale),
                                           _dt(Q), _p(ws), ws.numel() * ws.element_size(), _current(stream)))


def _token_rows(t):
    """(batch, token, head stride) of a [B, N, heads, d] tensor, or of a packed [T, heads, d] one (one batch); 0 where there
    is one step only (torch leaves the strides of one-sized dimensions open)."""
    sh, st = t.shape, t.stride()
    if st[-1] != 1 and sh[-1] > 1:
        raise ValueError("the last dimension must be contiguous")
    if len(sh) == 3:
        return 0, (st[0] if sh[0] > 1 else 0), (st[1] if sh[1] > 1 else 0)
    return (st[0] if sh[0] > 1 else 0), (st[1] if sh[1] > 1 else 0), (st[2] if sh[2] > 1 else 0)


def _norm_rope_sizes(q, k, wq, wk, table, positions, eps, interleaved, more=()):
    """What fa_qk_norm_rope and its backward are called with behind their strides, after checking all but the
    outputs; more: gradients, shaped as q and k by turns."""
    shape, dt = q.shape, q.dtype
    if len(shape) == 4:
        B, N, H, d = shape
    elif len(shape) == 3:
        B, (N, H, d) = 1, shape
    else:
        raise ValueError(f"expected [B, N, H, d] or packed [T, H, d] queries, got shape {tuple(shape)}")
    ks = k.shape
    if len(ks) != len(shape) or ks[-1] != d or ks[:-2] != shape[:-2] or k.dtype != dt:
        raise ValueError("the keys must have the queries' batch, tokens, head dimension and dtype")
    if max(B, N, H, ks[-2]) > 0x7FFFFFFF:
        raise ValueError(f"too many rows for one call: {tuple(shape)} and {tuple(ks)}")
    for n, t in enumerate(more):
        if t.shape != (ks if n & 1 else shape) or t.dtype != dt:
            raise ValueError("outputs and gradients must have their rows' heads, shape and dtype")
    wdt = wq.dtype if wq is not None else dt if wk is None else wk.dtype
    if (wq is not None and wq.numel() != d) or (wk is not None and (wk.numel() != d or wk.dtype != wdt)):
        raise ValueError("weights must be [d] tensors of one dtype, fp32 or the rows'")
    if table is None:
        length = rotary = 0
    else:
        if table.dtype != torch.float32 or table.dim() != 2:
            raise ValueError("the rotation table must be an fp32 tensor [positions, rotary] (rope_table)")
        length, rotary = table.shape
    if positions is not None:
        _int32(positions, B * N, "positions")
    _ready(wq, wk, table, positions, strided=(q, k, *more))
    if wdt not in DTYPE_CODES or dt not in DTYPE_CODES:
        raise ValueError(f"unsupported dtype {dt} or {wdt}")
    return (B, N, H, ks[-2], d, rotary, bool(interleaved), _c_int(length), float(eps), DTYPE_CODES[dt], DTYPE_CODES[wdt])


_Strides4, _Strides6 = ctypes.c_int64 * 12, ctypes.c_int64 * 18


def fa_qk_norm_rope(Q, K, wq, wk, table, Qo, Ko, positions=None, eps=1e-6, interleaved=False, stream=None):
    """Qo, Ko = the heads of Q [B, N, H, d] and K [B, N, Hkv, d] (or packed [T, heads, d]; any strides between rows)
    normed with the weights wq, wk [d] (None: ones) and rotated by position with table [positions, rotary] (None: not
    rotated). positions: int32, one a token; None: 0 .. N - 1."""
    strides = _Strides4(*_token_rows(Q), *_token_rows(K), *_token_rows(Qo), *_token_rows(Ko))
    sizes = _norm_rope_sizes(Q, K, wq, wk, table, positions, eps, interleaved, (Qo, Ko))
    _check(load_library().fa_qk_norm_rope(Q.data_ptr(), K.data_ptr(), _p(wq), _p(wk), _p(table), _p(positions), Qo.data_ptr(),
                                          Ko.data_ptr(), strides, *sizes, _current(stream)))


def fa_qk_norm_rope_bwd_workspace_size(d) -> int:
    return int(load_library().fa_qk_norm_rope_bwd_workspace_size(int(d)))


def fa_qk_norm_rope_bwd(dQo, dKo, Q, K, wq, wk, table, dQ, dK, dwq, dwk, positions=None, eps=1e-6, interleaved=False,
                        workspace=None, stream=None):
    """Gradients of fa_qk_norm_rope: dQ, dK (as Q, K) and dwq, dwk ([d] of the weights' dtype, or None; where one
    weight is None, of the other's) from dQo, dKo."""
    weight = wk if wq is None else wq
    for dw in (dwq, dwk):
        if dw is None:
            continue
        if weight is None:
            raise ValueError("a weight gradient without weights")
        if dw.numel() != Q.shape[-1] or dw.dtype != weight.dtype:  # (the library takes one dtype for both weights)
            raise ValueError("weight gradients must be [d] tensors of the weights' dtype")
    sizes = _norm_rope_sizes(Q, K, wq, wk, table, positions, eps, interleaved, (dQo, dKo, dQ, dK))
    _ready(dwq, dwk, workspace, strided=(Q,))
    _norm_rope_bwd(dQo, dKo, Q, K, wq, wk, table, positions, dQ, dK, dwq, dwk, workspace,
                   (*_token_rows(dQo), *_token_rows(dKo), *_token_rows(Q), *_token_rows(K), *_token_rows(dQ),
                    *_token_rows(dK)), sizes, stream)


def _norm_rope_bwd(dQo, dKo, Q, K, wq, wk, table, positions, dQ, dK, dwq, dwk, workspace, strides, sizes, stream):
    lib = load_library()
    if workspace is None:
        workspace = _new_workspace(lib.fa_qk_norm_rope_bwd_workspace_size(sizes[4]), Q.device, stream)
    _check(lib.fa_qk_norm_rope_bwd(dQo.data_ptr(), dKo.data_ptr(), Q.data_ptr(), K.data_ptr(), _p(wq), _p(wk), _p(table),
                                   _p(positions), dQ.data_ptr(), dK.data_ptr(), _p(dwq), _p(dwk), workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size(), _Strides6(*strides), *sizes,
                                   _current(stream)))


def fa_selftest_bounded_wait(timeout_ms=20, arrive=False, stream=None):
    """Launch the bounded-wait self-test (see include/fa.h); read the outcome with fa_check_device_error."""
    _check(load_library().fa_selftest_bounded_wait(int(timeout_ms), int(bool(arrive)), _stream(stream)))


def fa_sm_clock_sample(out, stream=None):
    """Enqueue one reading of every SM's cycle counter and the global timer into ``out``, a CUDA
    uint64 (or int64) tensor of 3 x blocks elements, blocks <= the SM count (see include/fa.h)."""
    _on_device(out)
    if out.element_size() != 8 or out.numel() % 3 != 0:
        raise ValueError("out must hold 3 x blocks 64-bit words")
    _check(load_library().fa_sm_clock_sample(_p(out), out.numel() // 3, _stream(stream)))


def fa_debug_build() -> bool:
    """Whether the loaded library was built with FA_DEBUG (device-side index checks)."""
    return bool(load_library().fa_debug_build())


def fa_selftest_debug_check(index, limit, stream=None):
    """Launch one device index check of index against [0, limit) (debug builds; see include/fa.h)."""
    _check(load_library().fa_selftest_debug_check(int(index), int(limit), _stream(stream)))


def fa_check_device_error(stream=None):
    _check(load_library().fa_check_device_error(_stream(stream)))


def fa_tile_counter(stream=None, reset=False) -> int:
    v = ctypes.c_ulonglong(0)
    _check(load_library().fa_tile_counter(_stream(stream), ctypes.byref(v), int(bool(reset))))
    return int(v.value)


def fa_uses_tensor_cores(pass_: str, dtype, d: int) -> bool:
    code = DTYPE_CODES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return bool(load_library().fa_uses_tensor_cores(0 if pass_ == "fwd" else 1, code, int(d)))


def fa_status_string(status: int) -> str:
    return load_library().fa_status_string(int(status)).decode()


def fa_last_error_message() -> str:
    return load_library().fa_last_error_message().decode()


# ---------------------------------------------------------------------------
# conveniences: allocate outputs with torch, then call the entry points above
# ---------------------------------------------------------------------------


def _warn_cuda_core(pass_, t, d):
    """A 16-bit pass with no tensor-core kernel runs on the CUDA-core kernels: say so."""
    if t.dtype != torch.float32 and not fa_uses_tensor_cores(pass_, t.dtype, d):
        warnings.warn(f"{t.dtype} {'forward' if pass_ == 'fwd' else 'backward'} at d={d} runs on the CUDA-core "
                      f"kernels (fp32 arithmetic): no tensor-core kernel for this head dimension", stacklevel=3)


def _sinks_allowed(causal, window, sinks, block_mask=None):
    """Whether a call is one of a window with sinks (fa_fwd_window and its kind): sinks given, 0 as well where it is such a window."""
    good = causal and window >= 1 and block_mask is None
    if not sinks:
        return sinks is not None and good
    if not good:
        raise ValueError("sinks go with causal attention and a window, without a block mask")
    return True


def attention_forward(q, k, v, causal=False, scale=None, stream=None, window=0, block_mask=None, sinks=None):
    """O, L = fa_fwd(q, k, v) (fa_fwd_gqa when k, v have fewer heads than q; fa_fwd_masked with a
    window or a block mask; fa_fwd_window with a window, causal, and sinks given, which may be 0); outputs on q's
    device. sinks=None: the kernels that a window took before there were sinks, so that results stay as they were to the
    bit; 0 is the same mask on the faster ones (the same O, L and dV; dK and dQ by unrounded probabilities, and d = 256 too)."""
    if _sinks_allowed(causal, window, sinks, block_mask):
        shape = _window_shape(q, k, v)
        o = _new(q.shape, q.dtype, q.device, stream)
        lse = _new(q.shape[:3], torch.float32, q.device, stream)
        _check(load_library().fa_fwd_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), *shape,
                                            shape[4] ** -0.5 if scale is None else float(scale), _c_int(window), _c_int(sinks),
                                            _dt(q), _current(stream)))
        return o, lse
    B, H, N, d = _shape4(q)
    _warn_cuda_core("fwd", q, d)
    scale = d ** -0.5 if scale is None else scale
    o = _new(q.shape, q.dtype, q.device, stream)
    lse = _new((B, H, N), torch.float32, q.device, stream)
    if window or block_mask is not None:
        fa_fwd_masked(q, k, v, o, lse, scale, causal, window, block_mask, stream)
    elif k.shape[1] != H:
        fa_fwd_gqa(q, k, v, o, lse, scale, causal, stream)
    else:
        fa_fwd(q, k, v, o, lse, scale, causal, stream)
    return o, lse


def attention_backward(q, k, v, o, do, lse, causal=False, scale=None, workspace=None, stream=None, window=0,
                       block_mask=None, sinks=None):
    """dQ, dK, dV = fa_bwd(...) (fa_bwd_masked with a window or a block mask; fa_bwd_window with a window
    and sinks, which may be 0: see attention_forward); outputs (and workspace, unless given) allocated with torch."""
    if _sinks_allowed(causal, window, sinks, block_mask):
        lib, dt, dev = load_library(), q.dtype, q.device
        B, H, Hkv, N, d = _window_shape(q, k, v, (o, do), (), (lse,), (workspace,))
        dq = _new(q.shape, dt, dev, stream)
        dk, dv = _new(k.shape, dt, dev, stream), _new(k.shape, dt, dev, stream)
        ws = workspace
        if ws is None:
            ws = _new_workspace(max(lib.fa_bwd_workspace_size(B, H, N, d), 16), dev, stream)
        _check(lib.fa_bwd_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
                                 dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(),
                                 ws.numel() * ws.element_size(), B, H, Hkv, N, d,
                                 d ** -0.5 if scale is None else float(scale), _c_int(window), _c_int(sinks), _dt(q),
                                 _current(stream)))
        return dq, dk, dv
    B, H, N, d = _shape4(q)
    _warn_cuda_core("bwd", q, d)
    scale = d ** -0.5 if scale is None else scale
    dq, dk, dv = (_new(t.shape, t.dtype, t.device, stream) for t in (q, k, v))
    if workspace is None:
        workspace = _new_workspace(max(fa_bwd_workspace_size(B, H, N, d), 16), q.device, stream)
    if window or block_mask is not None:
        fa_bwd_masked(q, k, v, o, do, lse, dq, dk, dv, workspace, scale, causal, window, block_mask, stream)
    elif k.shape[1] != H:
        fa_bwd_gqa(q, k, v, o, do, lse, dq, dk, dv, workspace, scale, causal, stream)
    else:
        fa_bwd(q, k, v, o, do, lse, dq, dk, dv, workspace, scale, causal, stream)
    return dq, dk, dv


def attention_decode(q, k, v, scale=None, splits=0, stream=None):
    """O, L = fa_decode(q, k, v) for q [B, H, Nq, d] over the cache k, v [B, Hkv, Nk, d]."""
    B, H, Nq, d = _shape4(q)
    _, Hkv, Nk, _ = _shape4(k)
    scale = d ** -0.5 if scale is None else scale
    o = _new(q.shape, q.dtype, q.device, stream)
    lse = _new((B, H, Nq), torch.float32, q.device, stream)
    nbytes = fa_decode_workspace_size(B, H, Hkv, Nq, Nk, d, splits)
    ws = _new_workspace(nbytes, q.device, stream) if nbytes else None
    fa_decode(q, k, v, o, lse, scale, splits, ws, stream)
    return o, lse


def attention_forward_varlen(q, k, v, cu_seqlens, causal=False, scale=None, stream=None, window=0, sinks=0):
    """O [T, H, d], L [H, T] = fa_fwd_varlen(...) for packed q [T, H, d], k, v [T, Hkv, d]; fa_fwd_varlen_window with a
    window (causal), and sinks."""
    if window and not causal:
        raise ValueError("a window over packed sequences is causal")
    _sinks_allowed(causal, window, sinks)
    T, H, d, _, _ = _packed(q, "Q")
    scale = d ** -0.5 if scale is None else scale
    o = _new((T, H, d), q.dtype, q.device, stream)
    lse = _new((H, T), torch.float32, q.device, stream)
    if window:
        fa_fwd_varlen_window(q, k, v, o, lse, cu_seqlens, scale, window, sinks, stream)
    else:
        fa_fwd_varlen(q, k, v, o, lse, cu_seqlens, scale, causal, stream)
    return o, lse


def attention_decode_window(q, k, v, lens, window=0, sinks=0, scale=None, stream=None):
    """O, L = fa_decode_window(...) for q [B, H, Nq, d] over caches k, v [B, Hkv, capacity, d]; outputs and workspace
    allocated with torch."""
    shape = _cache_shape(q, k, v, lens)
    lib = load_library()
    B, H, _, Nq, _, d = shape
    dev = q.device
    o = _new((B, H, Nq, d), q.dtype, dev, stream)
    lse = _new((B, H, Nq), torch.float32, dev, stream)
    nbytes = lib.fa_decode_window_workspace_size(*shape)
    ws = _new_workspace(nbytes, dev, stream)
    _check(lib.fa_decode_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), lens.data_ptr(), o.data_ptr(), lse.data_ptr(), *shape,
                                d ** -0.5 if scale is None else float(scale), _c_int(window), _c_int(sinks), _dt(q),
                                ws.data_ptr(), nbytes, _current(stream)))
    return o, lse


def attention_decode_prefix(q, k_prefix, v_prefix, k, v, lens, scale=None, stream=None):
    """O, L = fa_decode_prefix(...) for q [B, H, Nq, d] behind a prefix k_prefix, v_prefix [Hkv, P, d] and over caches
    k, v [B, Hkv, capacity, d]; outputs and workspace allocated with torch."""
    shape = _prefix_shape(_cache_shape(q, k, v, lens), q, k_prefix, v_prefix)
    lib = load_library()
    B, H, _, Nq, _, _, d = shape
    dev = q.device
    o = _new((B, H, Nq, d), q.dtype, dev, stream)
    lse = _new((B, H, Nq), torch.float32, dev, stream)
    nbytes = lib.fa_decode_prefix_workspace_size(*shape)
    ws = _new_workspace(nbytes, dev, stream)
    _check(lib.fa_decode_prefix(q.data_ptr(), k_prefix.data_ptr(), v_prefix.data_ptr(), k.data_ptr(), v.data_ptr(),
                                lens.data_ptr(), o.data_ptr(), lse.data_ptr(), *shape,
                                d ** -0.5 if scale is None else float(scale), _dt(q), ws.data_ptr(), nbytes,
                                _current(stream)))
    return o, lse


def rope_table(positions, rotary, base=10000.0, device="cuda"):
    """The fp32 rotation table [positions, rotary] of qk_norm_rope: cos of the angles p base^(-2 i / rotary), i < rotary / 2,
    then their sin; angles in 64 bits (in 32, far positions' angles are off by more than the table's rounding)."""
    freq = float(base) ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device=device) / max(int(rotary), 1))
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat((angle.cos(), angle.sin()), -1).float()


def qk_norm_rope(q, k, q_weight, k_weight, table, positions=None, eps=1e-6, interleaved=False, stream=None):
    """fa_qk_norm_rope into new tensors: from q [B, N, H, d], k [B, N, Hkv, d] (slices of a fused projection's output, say)
    [B, H, N, d] and [B, Hkv, N, d], what attention_forward takes; from packed [T, heads, d] the same, packed, what
    attention_forward_varlen takes."""
    sizes = _norm_rope_sizes(q, k, q_weight, k_weight, table, positions, eps, interleaved)
    B, N, H, Hkv, d = sizes[:5]
    dt, dev = q.dtype, q.device
    if q.dim() == 4:
        qo, ko = _new((B, H, N, d), dt, dev, stream), _new((B, Hkv, N, d), dt, dev, stream)
        out = (H * N * d, d, N * d, Hkv * N * d, d, N * d)
    else:
        qo, ko = _new((N, H, d), dt, dev, stream), _new((N, Hkv, d), dt, dev, stream)
        out = (0, H * d, d, 0, Hkv * d, d)
    _check(load_library().fa_qk_norm_rope(q.data_ptr(), k.data_ptr(), _p(q_weight), _p(k_weight), _p(table), _p(positions),
                                          qo.data_ptr(), ko.data_ptr(), _Strides4(*_token_rows(q), *_token_rows(k), *out),
                                          *sizes, _current(stream)))
    return qo, ko


def qk_norm_rope_backward(dqo, dko, q, k, q_weight, k_weight, table, positions=None, eps=1e-6, interleaved=False,
                          stream=None, out=None):
    """dq, dk, dq_weight, dk_weight = the gradients of qk_norm_rope from those of its results (dqo, dko as it returns them). dq
    and dk have q's and k's shapes; out: tensors (slices of a fused gradient, say) that take them. A weight's gradient
    has its dtype and is None where there is no weight."""
    if out is not None:
        dq, dk = out
    else:
        dt, dev = q.dtype, q.device
        dq, dk = _new(q.shape, dt, dev, stream), _new(k.shape, dt, dev, stream)
    dwq = None if q_weight is None else _new(q_weight.shape, q_weight.dtype, q.device, stream)
    dwk = None if k_weight is None else _new(k_weight.shape, k_weight.dtype, q.device, stream)
    if dqo.dim() == 4 and dko.dim() == 4:  # [B, heads, N, d]
        sizes = _norm_rope_sizes(q, k, q_weight, k_weight, table, positions, eps, interleaved, (dq, dk))
        B, N, H, Hkv, d = sizes[:5]
        if (dqo.shape, dko.shape) != ((B, H, N, d), (B, Hkv, N, d)) or not (dqo.dtype == dko.dtype == q.dtype):
            raise ValueError("the gradients must be [B, H, N, d] and [B, Hkv, N, d] of the rows' dtype")
        _ready(q_weight, strided=(q, dqo, dko))
        (b0, h0, t0), (b1, h1, t1) = _token_rows(dqo), _token_rows(dko)
        outer = (b0, t0, h0, b1, t1, h1)
    else:
        sizes = _norm_rope_sizes(q, k, q_weight, k_weight, table, positions, eps, interleaved, (dqo, dko, dq, dk))
        outer = (*_token_rows(dqo), *_token_rows(dko))
    _norm_rope_bwd(dqo, dko, q, k, q_weight, k_weight, table, positions, dq, dk, dwq, dwk, None,
                   (*outer, *_token_rows(q), *_token_rows(k), *_token_rows(dq), *_token_rows(dk)), sizes, stream)
    return dq, dk, dwq, dwk


def kv4_read(cache, cu_seqlens, lens, total, dtype=torch.bfloat16, stream=None):
    """k, v [total, Hkv, d] = fa_kv4_read(...): the values of the newest slots, packed."""
    _, Hkv, _, d = _kv4_shape(cache)
    k, v = (_new((total, Hkv, d), dtype, cache.device, stream) for _ in range(2))
    fa_kv4_read(cache, cu_seqlens, lens, k, v, stream)
    return k, v


def attention_decode_kv4(q, cache, lens, causal=False, scale=None, weights_in=None, weights_out=None, stream=None):
    """O, L = fa_decode_kv4(...) for q [B, H, Nq, d] over a 4-bit cache; outputs and workspace
    allocated with torch."""
    shape = B, H, Hkv, Nq, capacity, d = _kv4_decode_shape(q, cache, lens, weights_in, weights_out)
    lib = load_library()
    dev = q.device
    o = _new((B, H, Nq, d), q.dtype, dev, stream)
    lse = _new((B, H, Nq), torch.float32, dev, stream)
    nbytes = lib.fa_decode_kv4_workspace_size(*shape, weights_out is not None)
    ws = _new_workspace(nbytes, dev, stream) if nbytes else None
    _check(lib.fa_decode_kv4(q.data_ptr(), cache.data_ptr(), lens.data_ptr(), o.data_ptr(), lse.data_ptr(),
                             _p(weights_in), _p(weights_out), *shape,
                             d ** -0.5 if scale is None else float(scale), int(bool(causal)), _dt(q), _p(ws), nbytes,
                             _current(stream)))
    return o, lse


def quantize_fp8(x, stream=None):
    """(codes, scales) = block quantisation of x [B, H, N, d] (one scale per 128 rows of a head)."""
    B, H, N, d = _shape4(x)
    x8 = _new((B, H, N, d), torch.uint8, x.device, stream)
    sc = _new((B, H, (N + 127) // 128), torch.float32, x.device, stream)
    fa_quantize_fp8(x, x8, sc, stream)
    return x8, sc


def attention_forward_fp8(q8, k8, v8, q_scales, k_scales, v_scales, scale=None, causal=False,
                          out_dtype=torch.bfloat16, stream=None):
    """O, L = fa_fwd_fp8(...) on E4M3 codes and their block scales."""
    B, H, N, d = _shape4(q8)
    scale = d ** -0.5 if scale is None else scale
    o = _new((B, H, N, d), out_dtype, q8.device, stream)
    lse = _new((B, H, N), torch.float32, q8.device, stream)
    fa_fwd_fp8(q8, k8, v8, q_scales, k_scales, v_scales, o, lse, scale, causal, stream)
    return o, lse
