"""Thin Python binding of the C ABI in include/llattn.h (argument marshalling only).

Every step of the forward runs in libllattn.so's CUDA kernels; this module
only checks tensors, passes raw device pointers, sizes and the current CUDA
stream, and turns status codes into exceptions.  There is no CPU fallback:
if the library is missing, ``lib()`` raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libllattn.so")

F32, BF16 = 0, 1
NORMS = {"l2": 0, "rms": 1}
LAYOUTS = {"half": 0, "interleaved": 1}
PATHS = {"auto": 0, "simt": 1, "tcgen05": 2, "tcgen05_serial": 3}

# Every symbol include/llattn.h declares.
EXPORTS = (
    "llattn_abi_version", "llattn_status_str", "llattn_num_levels", "llattn_fwd",
    "llattn_fwd_f32", "llattn_workspace_bytes", "llattn_fwd_ex", "llattn_device_status",
    "llattn_last_cuda_error", "llattn_fwd_host", "llattn_profile", "llattn_profile_read",
    "llattn_fwd_noalloc", "llattn_decode_state_bytes", "llattn_decode_step",
    "llattn_bwd_workspace_bytes", "llattn_bwd", "llattn_fwd_bf16", "llattn_stream_status",
    "llattn_segment_plan", "llattn_set_segment_chunks", "llattn_gdn_fwd",
    "llattn_prefill_state", "llattn_qk_norm_rope", "llattn_qk_norm_rope_bwd_workspace_bytes",
    "llattn_qk_norm_rope_bwd", "llattn_glr_workspace_bytes",
    "llattn_glr_packed_workspace_bytes", "llattn_glr_fwd", "llattn_glr_bwd",
    "llattn_decode_q8_state_bytes", "llattn_decode_step_q8",
    "llattn_prefill_q8_workspace_bytes", "llattn_prefill_state_q8",
    "llattn_read_state_q8",
)

NOALLOC_SCRATCH_BYTES = 32 << 20  # LLATTN_NOALLOC_SCRATCH_BYTES

_lib = None


class LLAttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib().llattn_status_str(status).decode()
        if status == 5:
            msg += f" (cudaError {lib().llattn_last_cuda_error()})"
        super().__init__(f"{where}: {msg} [status {status}]")


def lib():
    """Load libllattn.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m hierarchical_fenwick_state_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i, f_p, i_p = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p
    L.llattn_abi_version.restype = i
    L.llattn_status_str.restype = ctypes.c_char_p
    L.llattn_status_str.argtypes = [i]
    L.llattn_num_levels.restype = i
    L.llattn_num_levels.argtypes = [i]
    L.llattn_fwd.restype = i
    L.llattn_fwd.argtypes = [vp, vp, vp, f_p, f_p, f_p, i, i, i, i, i, i_p, vp]
    L.llattn_fwd_f32.restype = i
    L.llattn_fwd_f32.argtypes = [vp, vp, vp, f_p, f_p, f_p, i, i, i, i, i, i_p, vp]
    L.llattn_workspace_bytes.restype = i
    L.llattn_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i, i, ctypes.POINTER(ctypes.c_size_t)]
    L.llattn_fwd_ex.restype = i
    L.llattn_fwd_ex.argtypes = [i, i, i, vp, vp, vp, f_p, f_p, f_p, i, i, i, i, i, i_p, vp,
                                ctypes.c_size_t, vp]
    L.llattn_device_status.restype = i
    L.llattn_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint), i]
    L.llattn_last_cuda_error.restype = i
    L.llattn_fwd_host.restype = i
    L.llattn_fwd_host.argtypes = [i, vp, vp, vp, f_p, f_p, f_p, i, i, i, i, i, i_p, vp]
    L.llattn_fwd_noalloc.restype = i
    L.llattn_fwd_noalloc.argtypes = [i, vp, vp, vp, f_p, f_p, f_p, i, i, i, i, i, i_p, vp]
    L.llattn_decode_state_bytes.restype = i
    L.llattn_decode_state_bytes.argtypes = [i, i, i, i, i, ctypes.POINTER(ctypes.c_size_t)]
    L.llattn_decode_step.restype = i
    L.llattn_decode_step.argtypes = [i, vp, vp, vp, f_p, f_p, i_p, f_p, f_p, i, i, i, i, i, vp]
    L.llattn_prefill_state.restype = i
    L.llattn_prefill_state.argtypes = [i, vp, vp, f_p, f_p, i, i, i, i, i, i, i_p, vp]
    L.llattn_bwd_workspace_bytes.restype = i
    L.llattn_bwd_workspace_bytes.argtypes = [i, i, i, i, i, ctypes.POINTER(ctypes.c_size_t)]
    L.llattn_bwd.restype = i
    L.llattn_bwd.argtypes = [i, vp, vp, vp, f_p, f_p, vp, f_p, f_p, f_p, f_p, f_p, i, i, i, i, i,
                             i_p, vp, ctypes.c_size_t, vp]
    L.llattn_fwd_bf16.restype = i
    L.llattn_fwd_bf16.argtypes = [vp, vp, vp, f_p, f_p, f_p, i, i, i, i, i, i_p, vp]
    L.llattn_stream_status.restype = i
    L.llattn_stream_status.argtypes = [ctypes.POINTER(ctypes.c_uint), i, vp]
    L.llattn_gdn_fwd.restype = i
    L.llattn_gdn_fwd.argtypes = [i, vp, vp, vp, f_p, f_p, f_p, f_p, i, i, i, i, i, i_p, vp]
    L.llattn_segment_plan.restype = i
    L.llattn_segment_plan.argtypes = [i, i, i, i, i, i, ctypes.POINTER(ctypes.c_int)]
    L.llattn_set_segment_chunks.restype = i
    L.llattn_set_segment_chunks.argtypes = [i]
    ll, sz, fl, szp = ctypes.c_longlong, ctypes.c_size_t, ctypes.c_float, ctypes.POINTER(ctypes.c_size_t)
    L.llattn_qk_norm_rope.restype = i
    L.llattn_qk_norm_rope.argtypes = [i, vp, vp, ll, ll, f_p, f_p, i_p, f_p, vp, vp, ll, i, i, i, i,
                                      i, i, i, fl, vp]
    L.llattn_qk_norm_rope_bwd_workspace_bytes.restype = i
    L.llattn_qk_norm_rope_bwd_workspace_bytes.argtypes = [i, i, szp]
    L.llattn_qk_norm_rope_bwd.restype = i
    L.llattn_qk_norm_rope_bwd.argtypes = [i, vp, vp, ll, ll, f_p, f_p, i_p, f_p, f_p, f_p, f_p, f_p,
                                          ll, ll, f_p, f_p, ll, i, i, i, i, i, i, i, fl, vp, sz, vp]
    L.llattn_glr_workspace_bytes.restype = i
    L.llattn_glr_workspace_bytes.argtypes = [i, i, i, szp]
    L.llattn_glr_packed_workspace_bytes.restype = i
    L.llattn_glr_packed_workspace_bytes.argtypes = [i, i, ll, i, szp]
    L.llattn_glr_fwd.restype = i
    L.llattn_glr_fwd.argtypes = [i, vp, f_p, f_p, f_p, f_p, i, i, i, i_p, vp, sz, vp]
    L.llattn_glr_bwd.restype = i
    L.llattn_glr_bwd.argtypes = [f_p] * 8 + [i, i, i, i_p, vp, sz, vp]
    L.llattn_decode_q8_state_bytes.restype = i
    L.llattn_decode_q8_state_bytes.argtypes = [i, i, i, i, i, szp]
    L.llattn_decode_step_q8.restype = i
    L.llattn_decode_step_q8.argtypes = [i, vp, vp, vp, f_p, f_p, i_p, vp, f_p, i, i, i, i, i, vp]
    L.llattn_prefill_q8_workspace_bytes.restype = i
    L.llattn_prefill_q8_workspace_bytes.argtypes = [i, i, i, i, i, i, szp]
    L.llattn_prefill_state_q8.restype = i
    L.llattn_prefill_state_q8.argtypes = [i, vp, vp, f_p, vp, i, i, i, i, i, i, i_p, vp, sz, vp]
    L.llattn_read_state_q8.restype = i
    L.llattn_read_state_q8.argtypes = [vp, i_p, vp, i, i, i, i, i, i, vp]
    L.llattn_profile.restype = i
    L.llattn_profile.argtypes = [i]
    L.llattn_profile_read.restype = i
    L.llattn_profile_read.argtypes = [ctypes.POINTER(ctypes.c_double),
                                      ctypes.POINTER(ctypes.c_longlong),
                                      ctypes.POINTER(ctypes.c_longlong), i]
    _lib = L
    return L


def num_levels(T: int) -> int:
    return int(lib().llattn_num_levels(int(T)))


def _check(st: int, where: str):
    if st != 0:
        raise LLAttnError(st, where)


def workspace_bytes(in_dtype: int, path: str, chunk: int, B: int, H: int, T: int, dk: int,
                    dv: int, varlen: bool) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().llattn_workspace_bytes(in_dtype, PATHS[path], chunk, B, H, T, dk, dv,
                                        int(varlen), ctypes.byref(n)), "llattn_workspace_bytes")
    return int(n.value)


def _stream_handle(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def forward(q, k, v, log_a, lam, *, cu_seqlens=None, T: Optional[int] = None, out=None,
            path: str = "auto", chunk: int = 0, workspace=None, stream=None):
    """o = llattn forward on device tensors (torch).  Returns out (fp32).

    Dense: q,k [B,T,H,dk], v [B,T,H,dv], log_a [B,T,H], lam [B,T,H,L].
    Packed: q,k [total,H,dk] ..., cu_seqlens int32 [B+1] on the device, and T
    the bound on every sequence length.
    """
    import torch
    dtype = q.dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("q/k/v must be bf16 or fp32")
    for t in (q, k, v, log_a, lam):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("inputs must be contiguous CUDA tensors")
    if k.dtype != dtype or v.dtype != dtype:
        raise TypeError("q, k, v must share a dtype")
    if log_a.dtype != torch.float32 or lam.dtype != torch.float32:
        raise TypeError("log_a and lam must be fp32")
    if cu_seqlens is None:
        B, Tq, H, dk = q.shape
        T = Tq
    else:
        if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda:
            raise TypeError("cu_seqlens must be an int32 CUDA tensor")
        B = cu_seqlens.numel() - 1
        _, H, dk = q.shape
        if T is None:
            raise ValueError("varlen needs T (max sequence length bound)")
    dv = v.shape[-1]
    if out is None:
        out = torch.empty(v.shape, dtype=torch.float32, device=v.device)
    ws_ptr, ws_n = None, 0
    if workspace is not None:
        ws_ptr, ws_n = ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size()
    in_dtype = BF16 if dtype == torch.bfloat16 else F32
    cu_ptr = ctypes.c_void_p(cu_seqlens.data_ptr()) if cu_seqlens is not None else None
    st = lib().llattn_fwd_ex(in_dtype, PATHS[path], int(chunk), ctypes.c_void_p(q.data_ptr()),
                             ctypes.c_void_p(k.data_ptr()), ctypes.c_void_p(v.data_ptr()),
                             ctypes.c_void_p(log_a.data_ptr()), ctypes.c_void_p(lam.data_ptr()),
                             ctypes.c_void_p(out.data_ptr()), int(B), int(H), int(T), int(dk),
                             int(dv), cu_ptr, ws_ptr, ws_n, _stream_handle(stream))
    _check(st, "llattn_fwd_ex")
    return out


def fwd(q, k, v, log_a, lam, out, B, H, T, dk, dv, cu_seqlens=None, stream=None):
    """Direct call of llattn_fwd (bf16 inputs, default path) on raw tensors."""
    st = lib().llattn_fwd(ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
                          ctypes.c_void_p(v.data_ptr()), ctypes.c_void_p(log_a.data_ptr()),
                          ctypes.c_void_p(lam.data_ptr()), ctypes.c_void_p(out.data_ptr()),
                          int(B), int(H), int(T), int(dk), int(dv),
                          ctypes.c_void_p(cu_seqlens.data_ptr()) if cu_seqlens is not None else None,
                          _stream_handle(stream))
    _check(st, "llattn_fwd")
    return out


def fwd_bf16(q, k, v, log_a, lam, out, B, H, T, dk, dv, cu_seqlens=None, stream=None):
    """Direct call of llattn_fwd_bf16 (the same call as llattn_fwd)."""
    st = lib().llattn_fwd_bf16(ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
                               ctypes.c_void_p(v.data_ptr()), ctypes.c_void_p(log_a.data_ptr()),
                               ctypes.c_void_p(lam.data_ptr()), ctypes.c_void_p(out.data_ptr()),
                               int(B), int(H), int(T), int(dk), int(dv),
                               ctypes.c_void_p(cu_seqlens.data_ptr()) if cu_seqlens is not None else None,
                               _stream_handle(stream))
    _check(st, "llattn_fwd_bf16")
    return out


def fwd_f32(q, k, v, log_a, lam, out, B, H, T, dk, dv, cu_seqlens=None, stream=None):
    st = lib().llattn_fwd_f32(ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
                              ctypes.c_void_p(v.data_ptr()), ctypes.c_void_p(log_a.data_ptr()),
                              ctypes.c_void_p(lam.data_ptr()), ctypes.c_void_p(out.data_ptr()),
                              int(B), int(H), int(T), int(dk), int(dv),
                              ctypes.c_void_p(cu_seqlens.data_ptr()) if cu_seqlens is not None else None,
                              _stream_handle(stream))
    _check(st, "llattn_fwd_f32")
    return out


def fwd_host(in_dtype: int, q, k, v, log_a, lam, out, B, H, T, dk, dv, cu_seqlens=None,
             stream=None):
    """llattn_fwd_host on host buffers (numpy arrays or pinned CPU tensors; q/k/v as
    uint16 bf16 bit patterns for in_dtype=BF16).  Copies in, computes, copies out."""
    def ptr(x):
        if x is None:
            return None
        if hasattr(x, "data_ptr"):
            return ctypes.c_void_p(x.data_ptr())
        return ctypes.c_void_p(x.ctypes.data)
    st = lib().llattn_fwd_host(in_dtype, ptr(q), ptr(k), ptr(v), ptr(log_a), ptr(lam), ptr(out),
                               int(B), int(H), int(T), int(dk), int(dv), ptr(cu_seqlens),
                               _stream_handle(stream) if stream is not None else None)
    _check(st, "llattn_fwd_host")
    return out


def fwd_noalloc(q, k, v, log_a, lam, out, B, H, T, dk, dv, cu_seqlens=None, stream=None):
    """Direct call of llattn_fwd_noalloc on raw device tensors (bf16 or fp32 q/k/v):
    the forward with no device allocation, scratch from the library's fixed array."""
    in_dtype = BF16 if str(q.dtype) == "torch.bfloat16" else F32
    st = lib().llattn_fwd_noalloc(in_dtype, ctypes.c_void_p(q.data_ptr()),
                                  ctypes.c_void_p(k.data_ptr()), ctypes.c_void_p(v.data_ptr()),
                                  ctypes.c_void_p(log_a.data_ptr()),
                                  ctypes.c_void_p(lam.data_ptr()), ctypes.c_void_p(out.data_ptr()),
                                  int(B), int(H), int(T), int(dk), int(dv),
                                  ctypes.c_void_p(cu_seqlens.data_ptr()) if cu_seqlens is not None
                                  else None, _stream_handle(stream))
    _check(st, "llattn_fwd_noalloc")
    return out


def decode_state_bytes(B: int, H: int, L: int, dk: int, dv: int) -> int:
    """Bytes of the decoding state buffer (llattn_decode_state_bytes)."""
    n = ctypes.c_size_t(0)
    _check(lib().llattn_decode_state_bytes(int(B), int(H), int(L), int(dk), int(dv),
                                           ctypes.byref(n)), "llattn_decode_state_bytes")
    return int(n.value)


def decode_step(q, k, v, log_a, lam, pos, state, out, B, H, L, dk, dv, stream=None):
    """Direct call of llattn_decode_step on raw device tensors: one new token per sequence.

    q, k [B,H,dk] and v [B,H,dv] (bf16 or fp32), log_a [B,H] and lam [B,H,L] fp32, pos int32
    [B] (tokens each sequence has absorbed; read only), state fp32 of decode_state_bytes()
    bytes (kept between steps), out fp32 [B,H,dv]."""
    in_dtype = BF16 if str(q.dtype) == "torch.bfloat16" else F32
    st = lib().llattn_decode_step(in_dtype, ctypes.c_void_p(q.data_ptr()),
                                  ctypes.c_void_p(k.data_ptr()), ctypes.c_void_p(v.data_ptr()),
                                  ctypes.c_void_p(log_a.data_ptr()),
                                  ctypes.c_void_p(lam.data_ptr()), ctypes.c_void_p(pos.data_ptr()),
                                  ctypes.c_void_p(state.data_ptr()),
                                  ctypes.c_void_p(out.data_ptr()), int(B), int(H), int(L),
                                  int(dk), int(dv), _stream_handle(stream))
    _check(st, "llattn_decode_step")
    return out


def prefill_state(k, v, log_a, state, B, H, T, L, dk, dv, cu_seqlens=None, stream=None):
    """Direct call of llattn_prefill_state: the decoding state of every sequence at the
    position equal to its length (a prompt's hand-off to decode_step).

    k, v dense [B,T,H,d] or packed [total,H,d] (bf16 or fp32) as the forward takes them,
    log_a fp32 [..,H], state fp32 of decode_state_bytes(B,H,L,dk,dv) bytes (written),
    cu_seqlens int32 [B+1] or None."""
    in_dtype = BF16 if str(k.dtype) == "torch.bfloat16" else F32
    st = lib().llattn_prefill_state(in_dtype, ctypes.c_void_p(k.data_ptr()),
                                    ctypes.c_void_p(v.data_ptr()),
                                    ctypes.c_void_p(log_a.data_ptr()),
                                    ctypes.c_void_p(state.data_ptr()), int(B), int(H), int(T),
                                    int(L), int(dk), int(dv),
                                    ctypes.c_void_p(cu_seqlens.data_ptr())
                                    if cu_seqlens is not None else None,
                                    _stream_handle(stream))
    _check(st, "llattn_prefill_state")
    return state


def bwd_workspace_bytes(B: int, H: int, T: int, dk: int, dv: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().llattn_bwd_workspace_bytes(int(B), int(H), int(T), int(dk), int(dv),
                                            ctypes.byref(n)), "llattn_bwd_workspace_bytes")
    return int(n.value)


def backward(q, k, v, log_a, lam, dout, *, cu_seqlens=None, T: Optional[int] = None,
             grads=None, workspace=None, stream=None):
    """Gradients of sum(dout * out) through llattn_bwd, on device tensors (torch).

    Shapes as in forward(); dout like out, in the dtype of q.  Returns a dict of fp32 tensors
    q, k, v, log_a, lam (or fills `grads`, a dict of preallocated ones)."""
    import torch
    in_dtype = BF16 if q.dtype == torch.bfloat16 else F32
    for t in (q, k, v, log_a, lam, dout):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("inputs must be contiguous CUDA tensors")
    if k.dtype != q.dtype or v.dtype != q.dtype or dout.dtype != q.dtype:
        raise TypeError("q, k, v and dout must share a dtype")
    if cu_seqlens is None:
        B, T, H, dk = q.shape
    else:
        B = cu_seqlens.numel() - 1
        _, H, dk = q.shape
        if T is None:
            raise ValueError("varlen needs T (max sequence length bound)")
    dv = v.shape[-1]
    if grads is None:
        grads = {n: torch.empty(x.shape, dtype=torch.float32, device=x.device)
                 for n, x in (("q", q), ("k", k), ("v", v), ("log_a", log_a), ("lam", lam))}
    ws_ptr, ws_n = None, 0
    if workspace is not None:
        ws_ptr, ws_n = ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size()
    P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    st = lib().llattn_bwd(in_dtype, P(q), P(k), P(v), P(log_a), P(lam), P(dout), P(grads["q"]),
                          P(grads["k"]), P(grads["v"]), P(grads["log_a"]), P(grads["lam"]),
                          int(B), int(H), int(T), int(dk), int(dv),
                          P(cu_seqlens) if cu_seqlens is not None else None, ws_ptr, ws_n,
                          _stream_handle(stream))
    _check(st, "llattn_bwd")
    return grads


def profile(enable: bool):
    _check(lib().llattn_profile(int(enable)), "llattn_profile")


def profile_read(reset: bool = True):
    """(main-kernel device ms summed, main-kernel launches timed, total kernel launches)."""
    ms, n, tot = ctypes.c_double(0), ctypes.c_longlong(0), ctypes.c_longlong(0)
    _check(lib().llattn_profile_read(ctypes.byref(ms), ctypes.byref(n), ctypes.byref(tot),
                                     int(reset)), "llattn_profile_read")
    return float(ms.value), int(n.value), int(tot.value)


def device_status(clear: bool = True) -> int:
    flags = ctypes.c_uint(0)
    st = lib().llattn_device_status(ctypes.byref(flags), int(clear))
    if st not in (0, 6):
        _check(st, "llattn_device_status")
    return int(flags.value)


def gdn_forward(q, k, v, log_alpha, beta, lam, *, cu_seqlens=None, T: Optional[int] = None,
                out=None, stream=None):
    """Log-Linear Gated DeltaNet forward (llattn_gdn_fwd) on device tensors; returns out (fp32).
    Layouts as ``forward``; log_alpha and beta are [.., H] fp32."""
    import torch
    if q.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("q/k/v must be bf16 or fp32")
    for t in (q, k, v, log_alpha, beta, lam):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("inputs must be contiguous CUDA tensors")
    H, dk, dv = q.shape[-2], q.shape[-1], v.shape[-1]
    if cu_seqlens is None:
        B, T = q.shape[0], q.shape[1]
    else:
        B = cu_seqlens.numel() - 1
        if T is None:
            raise ValueError("packed inputs need T (the bound on every length)")
    if out is None:
        out = torch.empty(v.shape, dtype=torch.float32, device=v.device)
    in_dtype = BF16 if q.dtype == torch.bfloat16 else F32
    cu_ptr = ctypes.c_void_p(cu_seqlens.data_ptr()) if cu_seqlens is not None else None
    st = lib().llattn_gdn_fwd(in_dtype, ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
                              ctypes.c_void_p(v.data_ptr()), ctypes.c_void_p(log_alpha.data_ptr()),
                              ctypes.c_void_p(beta.data_ptr()), ctypes.c_void_p(lam.data_ptr()),
                              ctypes.c_void_p(out.data_ptr()), int(B), int(H), int(T), int(dk),
                              int(dv), cu_ptr, _stream_handle(stream))
    _check(st, "llattn_gdn_fwd")
    return out


def segment_plan(B: int, H: int, T: int, dk: int, dv: int, varlen: bool = False) -> int:
    """Chunks per segment of a tensor-core call of this shape (0: whole sequences per CTA)."""
    n = ctypes.c_int(0)
    _check(lib().llattn_segment_plan(B, H, T, dk, dv, int(varlen), ctypes.byref(n)),
           "llattn_segment_plan")
    return int(n.value)


def set_segment_chunks(chunks: int) -> None:
    """Force the tensor-core path's segment length (0: automatic)."""
    _check(lib().llattn_set_segment_chunks(int(chunks)), "llattn_set_segment_chunks")


def stream_status(clear: bool = True, stream=None) -> int:
    """llattn_stream_status: the status word, read in order on one stream (no device sync)."""
    flags = ctypes.c_uint(0)
    st = lib().llattn_stream_status(ctypes.byref(flags), int(clear), _stream_handle(stream))
    if st not in (0, 6):
        _check(st, "llattn_stream_status")
    return int(flags.value)


def _on_device(fn, dev, stream, where, args):
    """The C call `fn(*args, stream)` with `dev`, the tensors' device, current."""
    import torch
    C = torch._C
    if stream is None:   # (torch.cuda.current_stream() builds a Stream object, 4 us of a 10 us call)
        raw = C._cuda_getCurrentRawStream(dev.index)
    elif stream.device != dev:
        raise ValueError(f"stream must be on {dev}")
    else:
        raw = stream.cuda_stream
    if dev.index == C._cuda_getDevice():
        st = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, raw)
    if st != 0:
        raise LLAttnError(st, where)


def _in_dtype(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError("inputs must be bf16 or fp32")


def _expect(t, name, dtype, shape, dev, contiguous=True):
    """Type, device, shape (None: any) and contiguity of an argument that may be absent; its
    address (None where it is absent)."""
    if t is None:
        return None
    if (t.dtype == dtype and t.device == dev and (shape is None or t.shape == shape)
            and (not contiguous or t.is_contiguous())):
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _new(like, shape, stream, dtype=None):
    """An uninitialised result, which torch hands on in the order of the stream that writes it."""
    import torch
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _like(t, stream):
    """The same, shaped as the contiguous tensor t (a third of new_empty's host time)."""
    import torch
    if stream is None:
        return torch.empty_like(t)
    with torch.cuda.stream(stream):
        return torch.empty_like(t)


def _expect_state(t, name, n, dev):
    """The address of a contiguous fp32 tensor of n values that may be absent."""
    import torch
    p = _expect(t, name, torch.float32, None, dev)
    if t is not None and t.numel() != n:
        raise ValueError(f"{name} must hold one value for each sequence and channel ({n})")
    return p


def _token_rows(t, name):
    """(tokens, rows per token, d, stride of a token) of a tensor [..., rows, d] whose rows lie
    side by side and whose tokens are one stride apart."""
    shape, stride = t.shape, t.stride()
    if len(shape) < 3:
        raise ValueError(f"{name} must be [..., rows, d]")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    G, d = shape[-2], shape[-1]
    if len(shape) == 3:
        n, step = shape[0], stride[0]
    else:
        n, step, span = 1, None, 1   # of the dimensions with more than one entry, the inner ones so far
        for x, st in zip(reversed(shape[:-2]), reversed(stride[:-2])):
            n *= x
            if x == 1:
                continue
            if step is None:
                step = st
            elif x and st != step * span:
                raise ValueError(f"{name}'s tokens must be one stride apart")
            span *= x
    if n * G * d and (stride[-1] != 1 or (G > 1 and stride[-2] != d)):
        raise ValueError(f"{name}'s rows must lie side by side")
    return n, G, d, step if n > 1 else G * d


def _qk_args(q, k, wq, wk, pos, inv_freq, norm, layout):
    """What both directions check and pass: dtype code, tokens, groups, sizes, strides, addresses."""
    import torch
    dt, dev, f32 = _in_dtype(q), q.device, torch.float32
    n, Gq, d, qs = _token_rows(q, "q")
    _, Gk, dk, ks = _token_rows(k, "k")
    if k.dtype != q.dtype:
        raise TypeError("q and k must share a dtype")
    if k.shape[:-2] != q.shape[:-2] or dk != d:
        raise ValueError("q and k must have the same tokens and row length")
    if k.device != dev:
        raise ValueError(f"k must be on {dev}")
    w = (None if wq is None else _expect(wq, "wq", f32, (d,), dev),
         None if wk is None else _expect(wk, "wk", f32, (d,), dev))
    rot, at, freq = 0, None, None
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        freq = _expect(inv_freq, "inv_freq", f32, (rot // 2,), dev)
        if pos is None:
            raise ValueError("a rotation needs pos")
        if pos.numel() != n:
            raise ValueError("pos must have one entry for each token")
        at = _expect(pos, "pos", torch.int32, None, dev)
    if norm not in NORMS or layout not in LAYOUTS:
        raise ValueError(f"norm is one of {tuple(NORMS)}, layout one of {tuple(LAYOUTS)}")
    return dt, dev, n, Gq, Gk, d, rot, (q.data_ptr(), k.data_ptr(), qs, ks, *w, at, freq)


def qk_norm_rope(q, k, *, wq=None, wk=None, pos=None, inv_freq=None, heads: Optional[int] = None,
                 norm: str = "l2", layout: str = "half", eps: float = 1e-6, out=None, stream=None):
    """Norms of q and k rows with the position rotation (llattn_qk_norm_rope): returns (qo, ko).

    q [..., Gq, d], k [..., Gk, d] bf16 or fp32; rows of a token side by side, tokens one stride
    apart (slices of a projection's output do).  heads: rows each token has in the outputs
    [..., heads, d] (default: the larger of Gq, Gk); each group is written to heads / G of them.
    wq, wk fp32 [d]; inv_freq fp32 [rot/2] with pos int32, one entry per token, or None."""
    dt, dev, n, Gq, Gk, d, rot, args = _qk_args(q, k, wq, wk, pos, inv_freq, norm, layout)
    H = max(Gq, Gk) if heads is None else heads
    shape = q.shape if H == Gq else q.shape[:-2] + (H, d)
    if out is None:
        out = _new(q, shape, stream)
        out = (out, _like(out, stream))
        o = (out[0].data_ptr(), out[1].data_ptr())
    else:
        o = (_expect(out[0], "out[0]", q.dtype, shape, dev), _expect(out[1], "out[1]", q.dtype, shape, dev))
    _on_device(lib().llattn_qk_norm_rope, dev, stream, "llattn_qk_norm_rope",
               (dt, *args, *o, n, Gq, Gk, H, d, rot, LAYOUTS[layout], NORMS[norm], eps))
    return out


def qk_norm_rope_backward(q, k, dqo, dko, *, wq=None, wk=None, pos=None, inv_freq=None,
                          norm: str = "l2", layout: str = "half", eps: float = 1e-6, grads=None,
                          workspace=None, stream=None):
    """Gradients of qk_norm_rope from those at its outputs (llattn_qk_norm_rope_bwd).

    q, k, wq, wk, pos, inv_freq, norm, layout, eps as in the forward; dqo, dko fp32
    [..., heads, d].  Returns a dict of fp32 tensors q, k and, where weights are given, wq, wk (or
    fills `grads`, a dict of preallocated ones; its q and k may be strided as the inputs may).
    workspace: qk_norm_rope_bwd_workspace_bytes(d) bytes, or None for torch's."""
    import torch
    dt, dev, n, Gq, Gk, d, rot, args = _qk_args(q, k, wq, wk, pos, inv_freq, norm, layout)
    if dqo.dim() < 3:
        raise ValueError("dqo must be [..., heads, d]")
    f32, H = torch.float32, dqo.shape[-2]
    shape = q.shape if H == Gq else q.shape[:-2] + (H, d)
    dy = (_expect(dqo, "dqo", f32, shape, dev), _expect(dko, "dko", f32, shape, dev))
    if grads is None:
        grads = {"q": _like(dqo, stream) if H == Gq else _new(dqo, q.shape, stream),
                 "k": _like(dko, stream) if H == Gk else _new(dqo, k.shape, stream)}
        if wq is not None:
            grads["wq"] = _like(wq, stream)
        if wk is not None:
            grads["wk"] = _like(wk, stream)
        dqs, dks = Gq * d, Gk * d
    else:
        _expect(grads["q"], "grads['q']", f32, q.shape, dev, contiguous=False)
        _expect(grads["k"], "grads['k']", f32, k.shape, dev, contiguous=False)
        dqs, dks = _token_rows(grads["q"], "grads['q']")[3], _token_rows(grads["k"], "grads['k']")[3]
    dw = (_expect(grads.get("wq"), "grads['wq']", f32, (d,), dev),
          _expect(grads.get("wk"), "grads['wk']", f32, (d,), dev))
    need = 148 * 2 * 2 * d * 4 if dw[0] or dw[1] else 0   # as qk_norm_rope_bwd_workspace_bytes
    ws, at, size = _workspace(workspace, need, dqo, stream)
    _on_device(lib().llattn_qk_norm_rope_bwd, dev, stream, "llattn_qk_norm_rope_bwd",
               (dt, *args, *dy, grads["q"].data_ptr(), grads["k"].data_ptr(), dqs, dks, *dw, n, Gq,
                Gk, H, d, rot, LAYOUTS[layout], NORMS[norm], eps, at, size))
    return grads


def qk_norm_rope_bwd_workspace_bytes(d: int, weights: bool = True) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().llattn_qk_norm_rope_bwd_workspace_bytes(int(d), int(weights), ctypes.byref(n)),
           "llattn_qk_norm_rope_bwd_workspace_bytes")
    return int(n.value)


def _glr_shape(t, cu_seqlens, T):
    """(B, T, D) of [B, T, ...channels], or [total, ...channels] with cu_seqlens."""
    if not t.is_cuda:
        raise ValueError("inputs must be CUDA tensors")
    shape = t.shape
    if cu_seqlens is None:
        if len(shape) < 3:
            raise ValueError("dense inputs are [B, T, ...channels]")
        B, T, D = shape[0], shape[1], shape[2]
        rest = shape[3:]
    else:
        if T is None:
            raise ValueError("packed inputs need T (the bound on every length)")
        if len(shape) < 2 or cu_seqlens.numel() < 1:
            raise ValueError("packed inputs are [total, ...channels] with cu_seqlens [B + 1]")
        B, D, rest = cu_seqlens.numel() - 1, shape[1], shape[2:]
        T = min(T, shape[0])       # (no sequence is longer than all rows)
    for x in rest:
        D *= x
    return B, T, D


def glr_workspace_bytes(B: int, T: int, D: int) -> int:
    """Bytes of scratch of glr_forward and of glr_backward (llattn_glr_workspace_bytes)."""
    n = ctypes.c_size_t(0)
    _check(lib().llattn_glr_workspace_bytes(int(B), int(T), int(D), ctypes.byref(n)),
           "llattn_glr_workspace_bytes")
    return int(n.value)


def glr_packed_workspace_bytes(B: int, T: int, rows: int, D: int) -> int:
    """The same for a packed batch of that many rows (llattn_glr_packed_workspace_bytes)."""
    n = ctypes.c_size_t(0)
    _check(lib().llattn_glr_packed_workspace_bytes(int(B), int(T), int(rows), int(D), ctypes.byref(n)),
           "llattn_glr_packed_workspace_bytes")
    return int(n.value)


def _glr_need(B, T, D, rows=None):
    """Either without the call (sizes that they refuse are refused by the operator)."""
    if T <= 64 or B == 0 or D == 0:
        return 0
    slots = -(-T // 64) * B
    return 256 + (slots if rows is None else min(slots, rows // 64 + B)) * -(-D // 32) * 512


def _workspace(workspace, need, like, stream):
    """A call's scratch: the caller's, or torch's for this call alone (none where none is needed):
    (tensor, address, bytes).  like: an fp32 tensor on the call's device."""
    if workspace is not None:
        if workspace.device != like.device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {like.device}")
        return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if need == 0:
        return None, None, 0
    ws = _new(like, need // 4, stream)
    return ws, ws.data_ptr(), need


def glr_forward(x, log_a, *, h0=None, h_last=None, cu_seqlens=None, T: Optional[int] = None,
                out=None, workspace=None, stream=None):
    """The gated linear recurrence h_t = exp(log_a_t) h_{t-1} + x_t (llattn_glr_fwd): returns h (fp32).

    x bf16 or fp32 and log_a fp32, both [B, T, ...channels], or [total, ...channels] with
    cu_seqlens and T.  h0 [B, ...channels] fp32 is the state carried in; h_last, a preallocated
    tensor of the same shape (h0 itself will do), receives the state after the last token.
    workspace: glr_workspace_bytes() bytes (packed: glr_packed_workspace_bytes() will do), or None
    for torch's."""
    import torch
    dt, (B, T, D) = _in_dtype(x), _glr_shape(x, cu_seqlens, T)
    dev, f32 = x.device, torch.float32
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    la = _expect(log_a, "log_a", f32, x.shape, dev)
    states = _expect_state(h0, "h0", B * D, dev), _expect_state(h_last, "h_last", B * D, dev)
    cu = _expect(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
    if out is None:
        out = _like(log_a, stream)
    h = _expect(out, "out", f32, x.shape, dev)
    ws, at, size = _workspace(workspace, _glr_need(B, T, D, None if cu is None else log_a.shape[0]), log_a, stream)
    _on_device(lib().llattn_glr_fwd, dev, stream, "llattn_glr_fwd",
               (dt, x.data_ptr(), la, states[0], h, states[1], B, T, D, cu, at, size))
    return out


def glr_backward(log_a, h, dh, *, h0=None, dh_last=None, cu_seqlens=None, T: Optional[int] = None,
                 grads=None, workspace=None, stream=None):
    """Gradients of glr_forward from dh (and dh_last) through llattn_glr_bwd.

    log_a, h (the forward's output), dh fp32, shaped as in the forward; h0, dh_last fp32
    [B, ...channels] or None.  Returns a dict of fp32 tensors x, log_a and, where h0 is given, h0
    (or fills `grads`, a dict of preallocated ones)."""
    import torch
    B, T, D = _glr_shape(log_a, cu_seqlens, T)
    dev, f32 = log_a.device, torch.float32
    shape = log_a.shape
    ins = (_expect(log_a, "log_a", f32, None, dev), _expect(h, "h", f32, shape, dev),
           _expect_state(h0, "h0", B * D, dev), _expect(dh, "dh", f32, shape, dev),
           _expect_state(dh_last, "dh_last", B * D, dev))
    cu = _expect(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
    if grads is None:
        grads = {"x": _like(log_a, stream), "log_a": _like(log_a, stream)}
        if h0 is not None:
            grads["h0"] = _like(h0, stream)
    outs = (_expect(grads["x"], "grads['x']", f32, shape, dev),
            _expect(grads["log_a"], "grads['log_a']", f32, shape, dev),
            _expect_state(grads.get("h0"), "grads['h0']", B * D, dev))
    ws, at, size = _workspace(workspace, _glr_need(B, T, D, None if cu is None else log_a.shape[0]), log_a, stream)
    _on_device(lib().llattn_glr_bwd, dev, stream, "llattn_glr_bwd",
               (*ins, *outs, B, T, D, cu, at, size))
    return grads


def decode_q8_state_bytes(B: int, H: int, L: int, dk: int, dv: int) -> int:
    """Bytes of the 8-bit decoding state buffer (llattn_decode_q8_state_bytes)."""
    n = ctypes.c_size_t(0)
    _check(lib().llattn_decode_q8_state_bytes(int(B), int(H), int(L), int(dk), int(dv),
                                              ctypes.byref(n)), "llattn_decode_q8_state_bytes")
    return int(n.value)


def _q8_state(state, B, H, L, dk, dv):
    if not state.is_cuda or not state.is_contiguous():
        raise ValueError("state must be a contiguous CUDA tensor")
    need = B * H * (L - 1) * (dk * dv + 8 + dk * (dv // 32))   # as llattn_decode_q8_state_bytes
    if state.numel() * state.element_size() < need:
        raise ValueError(f"state must hold {need} bytes")
    return state.device


def decode_step_q8(q, k, v, log_a, lam, pos, state, out, B, H, L, dk, dv, stream=None):
    """llattn_decode_step_q8: decode_step on the 8-bit state (a buffer of decode_q8_state_bytes()
    bytes, of any dtype).  q, k [B,H,dk] and v [B,H,dv] bf16 or fp32, log_a [B,H] and lam [B,H,L]
    fp32, pos int32 [B], out fp32 [B,H,dv]."""
    import torch
    dt, dev, f32 = _in_dtype(q), _q8_state(state, B, H, L, dk, dv), torch.float32
    t, key, val = q.dtype, (B, H, dk), (B, H, dv)
    args = (_expect(q, "q", t, key, dev), _expect(k, "k", t, key, dev), _expect(v, "v", t, val, dev),
            _expect(log_a, "log_a", f32, (B, H), dev), _expect(lam, "lam", f32, (B, H, L), dev),
            _expect(pos, "pos", torch.int32, (B,), dev), state.data_ptr(), _expect(out, "out", f32, val, dev))
    _on_device(lib().llattn_decode_step_q8, dev, stream, "llattn_decode_step_q8",
               (dt, *args, B, H, L, dk, dv))
    return out


def prefill_q8_workspace_bytes(B: int, H: int, T: int, L: int, dk: int, dv: int) -> int:
    """Bytes of scratch of prefill_state_q8 (llattn_prefill_q8_workspace_bytes)."""
    n = ctypes.c_size_t(0)
    _check(lib().llattn_prefill_q8_workspace_bytes(int(B), int(H), int(T), int(L), int(dk), int(dv),
                                                   ctypes.byref(n)),
           "llattn_prefill_q8_workspace_bytes")
    return int(n.value)


_prefill_q8_need = functools.lru_cache(maxsize=1024)(prefill_q8_workspace_bytes)   # (of the sizes alone)


def prefill_state_q8(k, v, log_a, state, B, H, T, L, dk, dv, cu_seqlens=None, workspace=None,
                     stream=None):
    """llattn_prefill_state_q8: prefill_state into the 8-bit state.  k, v dense [B,T,H,d] or packed
    [total,H,d] (bf16 or fp32), log_a fp32 [..,H], cu_seqlens int32 [B+1] or None.  workspace:
    prefill_q8_workspace_bytes() bytes, or None for torch's."""
    import torch
    dt, dev, t = _in_dtype(k), _q8_state(state, B, H, L, dk, dv), k.dtype
    lead = (B, T) if cu_seqlens is None else (k.shape[0],)
    args = (_expect(k, "k", t, lead + (H, dk), dev), _expect(v, "v", t, lead + (H, dv), dev),
            _expect(log_a, "log_a", torch.float32, lead + (H,), dev), state.data_ptr())
    cu = _expect(cu_seqlens, "cu_seqlens", torch.int32, (B + 1,), dev)
    if cu is not None and k.shape[0] == 0:
        T = 0                        # no rows at all: every sequence is empty
    ws, at, size = _workspace(workspace, _prefill_q8_need(B, H, T, L, dk, dv), log_a, stream)
    _on_device(lib().llattn_prefill_state_q8, dev, stream, "llattn_prefill_state_q8",
               (dt, *args, B, H, T, L, dk, dv, cu, at, size))
    return state


def read_state_q8(state, B, H, L, dk, dv, slot=None, out=None, dtype=None, stream=None):
    """llattn_read_state_q8: the values an 8-bit state holds, [B,H,L-1,dk,dv], or with slot (int32
    [B]) those of one slot of each sequence, [B,H,dk,dv]; bf16 (the default) and fp32 are exact."""
    import torch
    dev = _q8_state(state, B, H, L, dk, dv)
    at = _expect(slot, "slot", torch.int32, (B,), dev)
    shape = (B, H, dk, dv) if slot is not None else (B, H, L - 1, dk, dv)
    if out is None:
        out = _new(state, shape, stream, dtype or torch.bfloat16)
    o = _expect(out, "out", out.dtype, shape, dev)
    _on_device(lib().llattn_read_state_q8, dev, stream, "llattn_read_state_q8",
               (state.data_ptr(), at, o, _in_dtype(out), B, H, L, dk, dv))
    return out
