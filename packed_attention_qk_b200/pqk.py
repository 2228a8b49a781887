"""Thin Python binding of libpqk's C ABI (include/pqk.h).

Argument marshalling only: every step of the hot path runs in the CUDA
kernels behind the C ABI. PyTorch supplies device memory (``data_ptr``) and
the current CUDA stream, or the caller's choice of one (``stream``: a torch
stream or a raw handle). Ordering such a call behind the work that makes its
inputs, and the readers of its outputs behind it, is the caller's part, as with
torch's own operations. There is no fallback: if ``libpqk.so`` has not been
built, loading fails with an error.
"""

from __future__ import annotations

import ctypes as C
import functools
import math
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libpqk.so")

PQK_OK = 0
STATUS = {0: "PQK_OK", -1: "PQK_ERR_INVALID_ARG", -2: "PQK_ERR_UNSUPPORTED", -3: "PQK_ERR_MISALIGNED",
          -4: "PQK_ERR_CUDA", -5: "PQK_ERR_WORKSPACE", -6: "PQK_ERR_TIMEOUT", -7: "PQK_ERR_BAD_SEQLENS"}
ROPE_INTERLEAVED, ROPE_HALF = 0, 1
NORM_RMS, NORM_LAYER, NORM_NONE = 0, 1, 2

# every symbol include/pqk.h declares
EXPORTS = ("pqk_qk_norm_rope", "pqk_qk_norm_rope_e4m3", "pqk_qk_norm_rope_3axis", "pqk_qk_fullc_norm_rope", "pqk_varlen_attn_workspace_size", "pqk_varlen_attn_fwd",
           "pqk_varlen_attn_fwd_skip", "pqk_quantize_qk_e4m3", "pqk_varlen_attn_fwd_fp8qk", "pqk_quantize_e4m3",
           "pqk_varlen_attn_fwd_fp8",
           "pqk_varlen_attn_fwd_noalloc", "pqk_modulate_swiglu", "pqk_linear_gated_residual", "pqk_linear_swiglu",
           "pqk_norm_modulate_i8", "pqk_quantize_i8", "pqk_linear_i8_gated_residual", "pqk_linear_i8_swiglu",
           "pqk_varlen_cross_attn_workspace_size", "pqk_varlen_cross_attn_fwd",
           "pqk_get_device_status", "pqk_set_wait_timeout_ns", "pqk_set_attn_cta_pairs", "pqk_selftest_wait_timeout",
           "pqk_status_string",
           "pqk_version")


class PqkError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} returned {code} ({STATUS.get(code, 'unknown')}: {status_string(code)})")
        self.code = code


_lib = None


def lib(path: str | None = None) -> C.CDLL:
    """Load libpqk.so (built by packed_attention_qk_b200.build) and declare
    its signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libpqk.so not found at {p}: build it with `python -m packed_attention_qk_b200.build`")
    L = C.CDLL(p)
    vp, i64, i32, f32, sz = C.c_void_p, C.c_int64, C.c_int, C.c_float, C.c_size_t
    L.pqk_qk_norm_rope.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, vp, vp, vp, i64, i32, i32, f32, f32, i32, vp]
    L.pqk_qk_norm_rope.restype = i32
    L.pqk_qk_norm_rope_e4m3.argtypes = [vp, vp, vp, vp, i64, i64, vp, vp, vp, i64, i32, i32, f32, f32, i32, vp, vp]
    L.pqk_qk_norm_rope_e4m3.restype = i32
    L.pqk_qk_norm_rope_3axis.argtypes = [vp, vp, vp, vp, i64, i64, vp, vp, vp, i32, i32, i32, i64, i32, i32, f32, f32,
                                         i32, vp]
    L.pqk_qk_norm_rope_3axis.restype = i32
    L.pqk_qk_fullc_norm_rope.argtypes = [vp, vp, vp, vp, i64, i64, vp, vp, vp, i64, i32, i32, f32, f32, i32, vp]
    L.pqk_qk_fullc_norm_rope.restype = i32
    L.pqk_varlen_attn_workspace_size.argtypes = [i32]
    L.pqk_varlen_attn_workspace_size.restype = sz
    L.pqk_varlen_attn_fwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, i32, i64, i32, i32, f32, vp, sz,
                                      vp]
    L.pqk_varlen_attn_fwd.restype = i32
    L.pqk_varlen_attn_fwd_skip.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, i32, i64, i32, i32, f32, f32,
                                           vp, vp, sz, vp]
    L.pqk_varlen_attn_fwd_skip.restype = i32
    L.pqk_quantize_qk_e4m3.argtypes = [vp, vp, i64, i64, i64, i32, i32, vp, vp, vp, vp]
    L.pqk_quantize_qk_e4m3.restype = i32
    L.pqk_varlen_attn_fwd_fp8qk.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, vp, i32, i64, i32, i32, f32, f32, vp,
                                            vp, sz, vp]
    L.pqk_varlen_attn_fwd_fp8qk.restype = i32
    L.pqk_quantize_e4m3.argtypes = [vp, i64, i64, i32, i32, vp, vp, vp]
    L.pqk_quantize_e4m3.restype = i32
    L.pqk_varlen_attn_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, vp, i64, vp, i32, i64, i32, i32, f32, f32, vp, vp, sz,
                                          vp]
    L.pqk_varlen_attn_fwd_fp8.restype = i32
    L.pqk_varlen_attn_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, i32, i64, i32, i32, f32,
                                              vp]
    L.pqk_varlen_attn_fwd_noalloc.restype = i32
    L.pqk_modulate_swiglu.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, f32, vp, vp, i64, vp,
                                      i32, vp]
    L.pqk_modulate_swiglu.restype = i32
    L.pqk_linear_gated_residual.argtypes = [vp, i64, vp, vp, i64, vp, vp, i32, vp, i64, i64, i32, i32, vp]
    L.pqk_linear_gated_residual.restype = i32
    L.pqk_linear_swiglu.argtypes = [vp, i64, vp, vp, i64, i64, i32, i32, vp]
    L.pqk_linear_swiglu.restype = i32
    L.pqk_norm_modulate_i8.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32,
                                       f32, vp]
    L.pqk_norm_modulate_i8.restype = i32
    L.pqk_quantize_i8.argtypes = [vp, i64, i64, i32, vp, i64, vp, vp]
    L.pqk_quantize_i8.restype = i32
    L.pqk_linear_i8_gated_residual.argtypes = [vp, i64, vp, vp, i64, vp, vp, i64, vp, vp, i32, vp, i64, i64, i32, i32,
                                               vp]
    L.pqk_linear_i8_gated_residual.restype = i32
    L.pqk_linear_i8_swiglu.argtypes = [vp, i64, vp, vp, i64, vp, vp, i64, i64, i32, i32, vp]
    L.pqk_linear_i8_swiglu.restype = i32
    L.pqk_varlen_cross_attn_workspace_size.argtypes = [i32, i32]
    L.pqk_varlen_cross_attn_workspace_size.restype = sz
    L.pqk_varlen_cross_attn_fwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, vp, i32, i64, i64, i32, i32,
                                            i32, f32, vp, sz, vp]
    L.pqk_varlen_cross_attn_fwd.restype = i32
    L.pqk_get_device_status.argtypes = [vp]
    L.pqk_get_device_status.restype = i32
    L.pqk_set_wait_timeout_ns.argtypes = [i64]
    L.pqk_set_wait_timeout_ns.restype = None
    L.pqk_set_attn_cta_pairs.argtypes = [C.c_int]
    L.pqk_set_attn_cta_pairs.restype = None
    L.pqk_selftest_wait_timeout.argtypes = [i64, vp]
    L.pqk_selftest_wait_timeout.restype = i32
    L.pqk_status_string.argtypes = [i32]
    L.pqk_status_string.restype = C.c_char_p
    L.pqk_version.argtypes = []
    L.pqk_version.restype = C.c_char_p
    if path is None:
        _lib = L
    return L


def status_string(code: int) -> str:
    return lib().pqk_status_string(code).decode()


def _check(fn: str, rc: int) -> None:
    if rc != PQK_OK:
        raise PqkError(fn, rc)


def _stream(stream) -> int | None:
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    torch = _torch or _load_torch()
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _token_stride(t, ndim: int) -> int:
    assert t.dim() == ndim, f"expected a {ndim}-d tensor, got {tuple(t.shape)}"
    for d in range(1, ndim):
        want = 1
        for e in range(d + 1, ndim):
            want *= t.shape[e]
        assert t.stride(d) == want, "only the token (first) dimension may be strided"
    return t.stride(0)


_torch = None


def _load_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _stream_object(stream):
    """The torch stream of a call's `stream`: None, a stream or a raw handle."""
    if not isinstance(stream, int):
        return stream
    cuda = (_torch or _load_torch()).cuda
    # ExternalStream(0) is a new stream, not the default one
    return cuda.ExternalStream(stream) if stream != 0 else cuda.default_stream()


def _new(stream, shape, dtype, device):
    """A new tensor for a call on `stream`, on that stream's account (see
    _Args), and for the caller's current stream to read."""
    torch = _torch or _load_torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_stream_object(stream)):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


class _Args:
    """Checks of one call's tensors: type, shape, unit stride inside a row,
    and the current CUDA device (the library launches on it). What a call
    usually gets, a contiguous tensor of the right shape, passes in one
    comparison: the checks of a call cost about as much as its launch.

    What the call allocates belongs to the stream that it runs on: memory
    that the current stream freed may still be read or written by work queued
    there, and a call on another stream is not ordered behind that work."""

    __slots__ = ("fn", "torch", "dev", "device", "side")

    def __init__(self, fn: str, stream=None):
        self.fn, self.torch, self.dev, self.device = fn, _torch or _load_torch(), None, None
        self.side = _stream_object(stream)

    def fail(self, name: str, why: str):
        raise ValueError(f"{self.fn}: {name} {why}")

    def first(self, name: str, t, dtype, ndim: int):
        """The call's first tensor: its shape and row stride (see rows), once
        it is a CUDA tensor of the current device with `ndim` dimensions."""
        if not isinstance(t, self.torch.Tensor):
            self.fail(name, "is not a tensor")
        shape = t.shape
        if t.dtype is not dtype:
            self.fail(name, f"is {t.dtype}, not {str(dtype)[6:]}")
        if len(shape) != ndim:
            self.fail(name, f"has shape {tuple(shape)}, not {ndim} dimensions")
        dev = t.get_device()
        if dev < 0:
            self.fail(name, f"is on {t.device}, not on a CUDA device")
        if dev != self.torch._C._cuda_getDevice():
            self.fail(name, f"is on {t.device}, not on the current device")
        self.dev, self.device = dev, t.device
        return shape, self._row_stride(name, t, shape)

    def whole(self, name: str, t, dtype, shape) -> None:
        """t must be `dtype`, of `shape` and contiguous."""
        try:
            if t.dtype is dtype and t.shape == shape and t.get_device() == self.dev and t.is_contiguous():
                return
        except AttributeError:
            self.fail(name, "is not a tensor")
        self._kind(name, t, dtype, shape)
        self.fail(name, f"is not contiguous (strides {t.stride()})")

    def rows(self, name: str, t, dtype, shape) -> int:
        """t must be `dtype`, of `shape` and contiguous inside a row (all
        dimensions but the first). Returns the row stride; for at most one row,
        whose stride means nothing, its length in whole 16-byte units."""
        try:
            same = t.dtype is dtype and t.shape == shape and t.get_device() == self.dev
        except AttributeError:
            self.fail(name, "is not a tensor")
        if not same:
            self._kind(name, t, dtype, shape)
        return self._row_stride(name, t, shape)

    def _row_stride(self, name: str, t, shape) -> int:
        strides = t.stride()
        if shape[0] > 1 and strides[-1] == 1 and (len(shape) == 2 or strides[1] == shape[2]):
            return strides[0]
        want = 1
        for d in range(len(shape) - 1, 0, -1):
            if strides[d] != want and shape[d] > 1 and t.numel() > 0:
                self.fail(name, f"is not contiguous inside a row (strides {strides})")
            want *= shape[d]
        if shape[0] <= 1:
            unit = 16 // t.element_size()
            return -(-want // unit) * unit
        return strides[0]

    def _kind(self, name: str, t, dtype, shape) -> None:
        if not isinstance(t, self.torch.Tensor):
            self.fail(name, "is not a tensor")
        if t.dtype is not dtype:
            self.fail(name, f"is {t.dtype}, not {str(dtype)[6:]}")
        if t.shape != shape:
            self.fail(name, f"has shape {tuple(t.shape)}, not {tuple(shape)}")
        if t.get_device() != self.dev:
            self.fail(name, f"is on {t.device}, not on cuda:{self.dev}")

    def new(self, dtype, *shape):
        """A new contiguous tensor on the call's device (with the strides given
        an allocation takes 1.5 us instead of 2.0), for the call's stream to
        write and the caller's current stream to read."""
        if len(shape) == 1:
            strides = (1,)
        elif len(shape) == 2:
            strides = (shape[1], 1)
        else:
            strides = (shape[1] * shape[2], shape[2], 1)
        if self.side is None:
            return self.torch.empty_strided(shape, strides, dtype=dtype, device=self.device)
        with self.torch.cuda.stream(self.side):
            t = self.torch.empty_strided(shape, strides, dtype=dtype, device=self.device)
        t.record_stream(self.torch.cuda.current_stream())
        return t

    def stream(self) -> int:
        """The handle of the caller's stream, or the current one's."""
        if self.side is None:
            return self.torch._C._cuda_getCurrentRawStream(self.dev)
        return self.side.cuda_stream

    def used(self, *tensors) -> None:
        """The caller's own outputs and workspace, written on a stream of its
        choice: their memory is not handed out again before that stream is
        through with it."""
        if self.side is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.side)


def _requests(a: _Args, cu_seqlens, name: str = "cu_seqlens") -> int:
    """The number of requests of a cu_seqlens (0 for None)."""
    if cu_seqlens is None:
        return 0
    if not isinstance(cu_seqlens, a.torch.Tensor) or cu_seqlens.dim() != 1:
        a.fail(name, "is not a one-dimensional tensor")
    n = cu_seqlens.shape[0]
    a.whole(name, cu_seqlens, a.torch.int32, (n,))
    return n - 1


def _rows_i8(a: _Args, name: str, t, T: int, C: int):
    """The int8 [T, C] tensor t, or a new one whose rows start on 16-byte
    boundaries, and its row stride."""
    if t is not None:
        return t, a.rows(name, t, a.torch.int8, (T, C))
    wide = (C + 15) // 16 * 16
    t = a.new(a.torch.int8, T, wide)
    return (t if wide == C else t[:, :C]), wide


def _floats(a: _Args, name: str, t, n: int):
    """The fp32 [n] tensor t, or a new one."""
    if t is None:
        return a.new(a.torch.float32, n)
    a.whole(name, t, a.torch.float32, (n,))
    return t


def _rows_bf16(a: _Args, name: str, t, shape):
    """The bf16 tensor t of `shape`, or a new one, and its row stride."""
    if t is not None:
        return t, a.rows(name, t, a.torch.bfloat16, shape)
    t = a.new(a.torch.bfloat16, *shape)
    return t, math.prod(shape[1:])


# ---------------------------------------------------------------- calls

def qk_norm_rope(q, k, w_q, w_k, pos, *, eps: float = 1e-6, rope_base: float = 10000.0,
                 style: int = ROPE_INTERLEAVED, q_out=None, k_out=None, stream=None):
    """Fused Q/K RMSNorm + RoPE. q, k: bf16 [T, H, D] (token dim may be
    strided); q_out, k_out: [T, H, D] views with their own token strides
    (default: in place)."""
    q_out = q if q_out is None else q_out
    k_out = k if k_out is None else k_out
    T, H, D = q.shape
    assert tuple(q_out.shape) == (T, H, D) and tuple(k_out.shape) == (T, H, D)
    _check("pqk_qk_norm_rope", lib().pqk_qk_norm_rope(
        _ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), _token_stride(q, 3), _token_stride(k, 3), _token_stride(q_out, 3),
        _token_stride(k_out, 3), _ptr(w_q), _ptr(w_k), _ptr(pos), T, H, D, eps, rope_base, style, _stream(stream)))
    return q_out, k_out


def qk_norm_rope_e4m3(q, k, w_q, w_k, pos, *, eps: float = 1e-6, rope_base: float = 10000.0,
                      style: int = ROPE_INTERLEAVED, q8=None, k8=None, deq=None, stream=None):
    """Fused Q/K RMSNorm + RoPE with e4m3 output at the per-tensor bound
    scale sqrt(D) max|w| -> 448. Returns (q8, k8 uint8 [T, H, D], deq fp32 [2H])."""
    import torch
    T, H, D = q.shape
    if q8 is None:
        q8 = _new(stream, (T, H, D), torch.uint8, q.device)
    if k8 is None:
        k8 = _new(stream, (T, H, D), torch.uint8, q.device)
    if deq is None:
        deq = _new(stream, 2 * H, torch.float32, q.device)
    assert q8.is_contiguous() and k8.is_contiguous() and deq.numel() >= 2 * H
    _check("pqk_qk_norm_rope_e4m3", lib().pqk_qk_norm_rope_e4m3(
        _ptr(q), _ptr(k), _ptr(q8), _ptr(k8), _token_stride(q, 3), _token_stride(k, 3), _ptr(w_q), _ptr(w_k),
        _ptr(pos), T, H, D, eps, rope_base, style, _ptr(deq), _stream(stream)))
    return q8, k8, deq


def qk_norm_rope_3axis(q, k, w_q, w_k, pos3, sections, *, eps: float = 1e-6, rope_base: float = 10000.0,
                       style: int = ROPE_INTERLEAVED, q_out=None, k_out=None, stream=None):
    """Fused Q/K RMSNorm + RoPE with (t, h, w) ids per token (pos3: int32
    [T, 3]); sections: pairs per axis, summing to D/2."""
    q_out = q if q_out is None else q_out
    k_out = k if k_out is None else k_out
    T, H, D = q.shape
    qs, ks = _token_stride(q, 3), _token_stride(k, 3)
    assert _token_stride(q_out, 3) == qs and _token_stride(k_out, 3) == ks
    st, sh, sw = (int(v) for v in sections)
    _check("pqk_qk_norm_rope_3axis", lib().pqk_qk_norm_rope_3axis(
        _ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), qs, ks, _ptr(w_q), _ptr(w_k), _ptr(pos3), st, sh, sw, T, H, D,
        eps, rope_base, style, _stream(stream)))
    return q_out, k_out


def qk_fullc_norm_rope(q, k, w_q, w_k, pos, *, eps: float = 1e-6, rope_base: float = 10000.0,
                       style: int = ROPE_INTERLEAVED, q_out=None, k_out=None, stream=None):
    """Fused Q/K RMSNorm over all H*D elements of a token (weights [H*D]) +
    RoPE per head."""
    q_out = q if q_out is None else q_out
    k_out = k if k_out is None else k_out
    T, H, D = q.shape
    qs, ks = _token_stride(q, 3), _token_stride(k, 3)
    assert _token_stride(q_out, 3) == qs and _token_stride(k_out, 3) == ks
    _check("pqk_qk_fullc_norm_rope", lib().pqk_qk_fullc_norm_rope(
        _ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), qs, ks, _ptr(w_q), _ptr(w_k), _ptr(pos), T, H, D, eps,
        rope_base, style, _stream(stream)))
    return q_out, k_out


def varlen_attn_workspace_size(B: int) -> int:
    return int(lib().pqk_varlen_attn_workspace_size(B))


def varlen_attn_fwd(q, k, v, cu_seqlens, *, softmax_scale: float | None = None, o=None, lse=None,
                    workspace=None, want_lse: bool = False, stream=None):
    """Packed varlen attention. q, k, v: bf16 [T, H, D]; cu_seqlens: int32
    [B+1] on the device. Returns (o, lse or None)."""
    import torch
    T, H, D = q.shape
    B = cu_seqlens.shape[0] - 1
    scale = softmax_scale if softmax_scale is not None else D ** -0.5
    if o is None:
        o = _new(stream, (T, H, D), q.dtype, q.device)
    if lse is None and want_lse:
        lse = _new(stream, (H, T), torch.float32, q.device)
    ws_bytes = varlen_attn_workspace_size(B)
    if workspace is None:
        workspace = _new(stream, ws_bytes, torch.uint8, q.device)
    _check("pqk_varlen_attn_fwd", lib().pqk_varlen_attn_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _token_stride(q, 3), _token_stride(k, 3),
        _token_stride(v, 3), _token_stride(o, 3), _ptr(cu_seqlens), B, T, H, D, scale, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return o, lse


def varlen_attn_fwd_skip(q, k, v, cu_seqlens, skip_threshold_log2: float, *, softmax_scale: float | None = None,
                         o=None, lse=None, workspace=None, want_lse: bool = False, skip_counts=None, stream=None):
    """Packed varlen attention that drops key blocks whose scores lie more
    than skip_threshold_log2 (log2 units) below the earlier blocks' maximum
    for every row of a 32-row query block. skip_counts: None or a device
    int64 tensor of 2 elements that the call adds to (dropped 32-row blocks,
    left-out 128-row P x V products). Returns (o, lse or None)."""
    import torch
    T, H, D = q.shape
    B = cu_seqlens.shape[0] - 1
    scale = softmax_scale if softmax_scale is not None else D ** -0.5
    if o is None:
        o = _new(stream, (T, H, D), q.dtype, q.device)
    if lse is None and want_lse:
        lse = _new(stream, (H, T), torch.float32, q.device)
    ws_bytes = varlen_attn_workspace_size(B)
    if workspace is None:
        workspace = _new(stream, ws_bytes, torch.uint8, q.device)
    if skip_counts is not None:
        assert skip_counts.dtype == torch.int64 and skip_counts.numel() >= 2 and skip_counts.is_contiguous()
    _check("pqk_varlen_attn_fwd_skip", lib().pqk_varlen_attn_fwd_skip(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _token_stride(q, 3), _token_stride(k, 3),
        _token_stride(v, 3), _token_stride(o, 3), _ptr(cu_seqlens), B, T, H, D, scale, float(skip_threshold_log2),
        _ptr(skip_counts), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    return o, lse


def quantize_qk_e4m3(q, k, *, q8=None, k8=None, scales=None, stream=None):
    """Per-head absmax e4m3 quantisation of Q and K (bf16 [T, H, D]).
    Returns (q8, k8 uint8 [T, H, D], deq fp32 [2H] view of ``scales``)."""
    import torch
    T, H, D = q.shape
    if q8 is None:
        q8 = _new(stream, (T, H, D), torch.uint8, q.device)
    if k8 is None:
        k8 = _new(stream, (T, H, D), torch.uint8, q.device)
    if scales is None:
        scales = _new(stream, 4 * H, torch.float32, q.device)
    assert q8.is_contiguous() and k8.is_contiguous() and scales.numel() >= 4 * H
    _check("pqk_quantize_qk_e4m3", lib().pqk_quantize_qk_e4m3(
        _ptr(q), _ptr(k), _token_stride(q, 3), _token_stride(k, 3), T, H, D, _ptr(q8), _ptr(k8), _ptr(scales),
        _stream(stream)))
    return q8, k8, scales[2 * H:4 * H]


def varlen_attn_fwd_fp8qk(q8, k8, v, deq, cu_seqlens, *, softmax_scale: float | None = None, o=None, lse=None,
                          workspace=None, want_lse: bool = False, skip_threshold_log2: float = math.inf,
                          skip_counts=None, stream=None):
    """Packed varlen attention with Q K^T on the FP8 tensor cores: q8, k8
    e4m3 bytes [T, H, D] (quantize_qk_e4m3), deq fp32 [2H], v bf16; block
    skipping as varlen_attn_fwd_skip when skip_threshold_log2 is finite.
    Returns (o, lse or None)."""
    import torch
    T, H, D = v.shape
    B = cu_seqlens.shape[0] - 1
    scale = softmax_scale if softmax_scale is not None else D ** -0.5
    if o is None:
        o = _new(stream, (T, H, D), v.dtype, v.device)
    if lse is None and want_lse:
        lse = _new(stream, (H, T), torch.float32, v.device)
    if workspace is None:
        workspace = _new(stream, varlen_attn_workspace_size(B), torch.uint8, v.device)
    assert q8.is_contiguous() and k8.is_contiguous() and tuple(q8.shape) == (T, H, D) == tuple(k8.shape)
    _check("pqk_varlen_attn_fwd_fp8qk", lib().pqk_varlen_attn_fwd_fp8qk(
        _ptr(q8), _ptr(k8), _ptr(v), _ptr(deq), _ptr(o), _ptr(lse), _token_stride(v, 3), _token_stride(o, 3),
        _ptr(cu_seqlens), B, T, H, D, scale, float(skip_threshold_log2), _ptr(skip_counts), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return o, lse


def quantize_e4m3(x, *, x8=None, scales=None, stream=None):
    """Per-head absmax e4m3 quantisation of one bf16 [T, H, D] tensor.
    Returns (x8 uint8 [T, H, D], deq fp32 [H] view of ``scales``)."""
    import torch
    T, H, D = x.shape
    if x8 is None:
        x8 = _new(stream, (T, H, D), torch.uint8, x.device)
    if scales is None:
        scales = _new(stream, 2 * H, torch.float32, x.device)
    assert x8.is_contiguous() and scales.numel() >= 2 * H
    _check("pqk_quantize_e4m3", lib().pqk_quantize_e4m3(_ptr(x), _token_stride(x, 3), T, H, D, _ptr(x8),
                                                         _ptr(scales), _stream(stream)))
    return x8, scales[H:2 * H]


def varlen_attn_fwd_fp8(q8, k8, v8, deq, cu_seqlens, *, softmax_scale: float | None = None, o=None, lse=None,
                        workspace=None, want_lse: bool = False, skip_threshold_log2: float = math.inf,
                        skip_counts=None, stream=None):
    """The attention with Q K^T and P V on the FP8 tensor cores: q8, k8, v8
    e4m3 bytes [T, H, D]; deq fp32 [3H] (Q's, K's, V's factors). A finite
    skip_threshold_log2 adds block skipping (skip_counts as in
    varlen_attn_fwd_skip). Returns (o bf16 [T, H, D], lse or None)."""
    import torch
    T, H, D = q8.shape
    B = cu_seqlens.shape[0] - 1
    scale = softmax_scale if softmax_scale is not None else D ** -0.5
    if o is None:
        o = _new(stream, (T, H, D), torch.bfloat16, q8.device)
    if lse is None and want_lse:
        lse = _new(stream, (H, T), torch.float32, q8.device)
    if workspace is None:
        workspace = _new(stream, varlen_attn_workspace_size(B), torch.uint8, q8.device)
    for t in (q8, k8, v8):
        assert t.is_contiguous() and tuple(t.shape) == (T, H, D)
    assert deq.is_contiguous() and deq.numel() >= 3 * H
    if skip_counts is not None:
        assert skip_counts.dtype == torch.int64 and skip_counts.numel() >= 2 and skip_counts.is_contiguous()
    _check("pqk_varlen_attn_fwd_fp8", lib().pqk_varlen_attn_fwd_fp8(
        _ptr(q8), _ptr(k8), _ptr(v8), _ptr(deq), _ptr(o), _ptr(lse), _token_stride(o, 3), _ptr(cu_seqlens), B, T, H,
        D, scale, float(skip_threshold_log2), _ptr(skip_counts), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return o, lse


def varlen_attn_fwd_noalloc(q, k, v, cu_seqlens, *, softmax_scale: float | None = None, o=None, lse=None,
                            want_lse: bool = False, stream=None):
    """Packed varlen attention for callers that cannot allocate device
    memory: the tile schedule lives in the library's own fixed device array
    (at most 4096 requests; calls must not overlap on the GPU). The outputs
    are allocated here only when not passed in."""
    import torch
    T, H, D = q.shape
    B = cu_seqlens.shape[0] - 1
    scale = softmax_scale if softmax_scale is not None else D ** -0.5
    if o is None:
        o = _new(stream, (T, H, D), q.dtype, q.device)
    if lse is None and want_lse:
        lse = _new(stream, (H, T), torch.float32, q.device)
    _check("pqk_varlen_attn_fwd_noalloc", lib().pqk_varlen_attn_fwd_noalloc(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _token_stride(q, 3), _token_stride(k, 3),
        _token_stride(v, 3), _token_stride(o, 3), _ptr(cu_seqlens), B, T, H, D, scale, _stream(stream)))
    return o, lse


def modulate_swiglu(x, shift, scale, cu_seqlens, *, gate_res=None, branch=None, gate=None, up=None,
                    norm_type: int = NORM_RMS, eps: float = 1e-6, x_out=None, h=None, act=None, stream=None):
    """Fused gated residual + norm + adaLN modulation, and SwiGLU.
    Returns (x_out or None, h, act or None)."""
    T, Cdim = x.shape
    B = cu_seqlens.shape[0] - 1
    if h is None:
        h = _new(stream, x.shape, x.dtype, x.device)
    F, gu_stride = 0, 0
    if gate is not None:
        F = gate.shape[1]
        gu_stride = _token_stride(gate, 2)
        assert _token_stride(up, 2) == gu_stride
        if act is None:
            act = _new(stream, (T, F), x.dtype, x.device)
    _check("pqk_modulate_swiglu", lib().pqk_modulate_swiglu(
        _ptr(x), _ptr(branch), _ptr(x_out), _ptr(h), _ptr(shift), _ptr(scale), _ptr(gate_res), _ptr(cu_seqlens),
        B, T, Cdim, norm_type, eps, _ptr(gate), _ptr(up), gu_stride, _ptr(act), F, _stream(stream)))
    return x_out, h, act


def linear_gated_residual(a, w, *, x=None, gate_res=None, cu_seqlens=None, out=None, stream=None):
    """out = x + gate_res[request] * (a @ w.T) on the tensor cores (the
    residual add in the GEMM's epilogue); with x None the product alone.
    a: [T, K] bf16 (rows may be strided), w: [N, K] bf16, x: [T, N] bf16,
    gate_res: [B, N] fp32. out may be x (in place)."""
    T, K = a.shape
    N = w.shape[0]
    assert w.shape == (N, K) and w.is_contiguous()
    if out is None:
        out = _new(stream, (T, N), a.dtype, a.device)
    B = 0 if cu_seqlens is None else cu_seqlens.shape[0] - 1
    x_stride = 0 if x is None else _token_stride(x, 2)
    _check("pqk_linear_gated_residual", lib().pqk_linear_gated_residual(
        _ptr(a), _token_stride(a, 2), _ptr(w), _ptr(x), x_stride, _ptr(gate_res), _ptr(cu_seqlens), B, _ptr(out),
        _token_stride(out, 2), T, K, N, _stream(stream)))
    return out


def linear_swiglu(a, w1, *, act=None, stream=None):
    """act = silu(a @ w1[:F].T) * (a @ w1[F:].T) on the tensor cores (SwiGLU
    in the GEMM's epilogue). a: [T, K] bf16, w1: [2F, K] bf16."""
    T, K = a.shape
    F = w1.shape[0] // 2
    assert w1.shape == (2 * F, K) and w1.is_contiguous()
    if act is None:
        act = _new(stream, (T, F), a.dtype, a.device)
    _check("pqk_linear_swiglu", lib().pqk_linear_swiglu(
        _ptr(a), _token_stride(a, 2), _ptr(w1), _ptr(act), _token_stride(act, 2), T, K, F, _stream(stream)))
    return act


def norm_modulate_i8(x, *, branch=None, gate_res=None, weight=None, shift=None, scale=None, cu_seqlens=None,
                     norm_type: int = NORM_RMS, eps: float = 1e-6, x_out=None, h8=None, h_scale=None, stream=None):
    """Gated residual + norm + adaLN modulation with an int8 output and one
    scale per token: x' = x + gate_res[request] * branch (without gate_res:
    x + branch), h = norm(x') * weight * (1 + scale[request]) +
    shift[request], h8 = round(127 h / max |h|), ties to even, h_scale =
    max |h| / 127.
    x, branch, x_out: bf16 [T, C] (rows may be strided; x_out may be x);
    weight bf16 [C]; gate_res, shift, scale fp32 [B, C]; cu_seqlens int32
    [B+1]. Returns (x_out or None, h8 int8 [T, C], h_scale fp32 [T])."""
    a = _Args("norm_modulate_i8", stream)
    bf16, f32 = a.torch.bfloat16, a.torch.float32
    shape, x_stride = a.first("x", x, bf16, 2)
    T, Cdim = shape
    br_stride = 0 if branch is None else a.rows("branch", branch, bf16, shape)
    xo_stride = 0 if x_out is None else a.rows("x_out", x_out, bf16, shape)
    B = _requests(a, cu_seqlens)
    if gate_res is not None:
        a.whole("gate_res", gate_res, f32, (B, Cdim))
    if shift is not None:
        a.whole("shift", shift, f32, (B, Cdim))
    if scale is not None:
        a.whole("scale", scale, f32, (B, Cdim))
    if weight is not None:
        a.whole("weight", weight, bf16, (Cdim,))
    h8, h8_stride = _rows_i8(a, "h8", h8, T, Cdim)
    h_scale = _floats(a, "h_scale", h_scale, T)
    _check("pqk_norm_modulate_i8", lib().pqk_norm_modulate_i8(
        x.data_ptr(), x_stride, _ptr(branch), br_stride, _ptr(x_out), xo_stride, h8.data_ptr(), h8_stride,
        h_scale.data_ptr(), _ptr(weight), _ptr(shift), _ptr(scale), _ptr(gate_res), _ptr(cu_seqlens), B, T, Cdim,
        norm_type, eps, a.stream()))
    a.used(x_out, h8, h_scale)
    return x_out, h8, h_scale


def quantize_i8(x, *, x8=None, scales=None, stream=None):
    """The rows of a bf16 tensor [T, C] as int8 codes with one scale per row
    (max |x| / 127). Returns (x8 int8 [T, C], scales fp32 [T])."""
    a = _Args("quantize_i8", stream)
    bf16 = a.torch.bfloat16
    (T, Cdim), x_stride = a.first("x", x, bf16, 2)
    x8, x8_stride = _rows_i8(a, "x8", x8, T, Cdim)
    scales = _floats(a, "scales", scales, T)
    _check("pqk_quantize_i8", lib().pqk_quantize_i8(x.data_ptr(), x_stride, T, Cdim, x8.data_ptr(), x8_stride,
                                                    scales.data_ptr(), a.stream()))
    a.used(x8, scales)
    return x8, scales


def _i8_operands(a: _Args, a8, a_scale, w8, w_scale):
    i8, f32 = a.torch.int8, a.torch.float32
    (T, K), a_stride = a.first("a8", a8, i8, 2)
    if not isinstance(w8, a.torch.Tensor) or w8.dim() != 2:
        a.fail("w8", "is not a two-dimensional tensor")
    N = w8.shape[0]
    w_stride = a.rows("w8", w8, i8, (N, K))
    a.whole("a_scale", a_scale, f32, (T,))
    a.whole("w_scale", w_scale, f32, (N,))
    return T, K, N, a_stride, w_stride


def linear_i8_gated_residual(a8, a_scale, w8, w_scale, *, x=None, gate_res=None, cu_seqlens=None, out=None,
                             stream=None):
    """out = x + gate_res[request] * y with y = a_scale * w_scale * (a8 @
    w8.T), the product in 8-bit integers; with x None y alone. a8: int8
    [T, K], w8: int8 [N, K] (rows on 16-byte boundaries, as quantize_i8 and
    norm_modulate_i8 give them), a_scale fp32 [T], w_scale fp32 [N], x bf16
    [T, N], gate_res fp32 [B, N]. out (bf16) may be x (in place)."""
    a = _Args("linear_i8_gated_residual", stream)
    T, K, N, a_stride, w_stride = _i8_operands(a, a8, a_scale, w8, w_scale)
    B = _requests(a, cu_seqlens)
    x_stride = 0 if x is None else a.rows("x", x, a.torch.bfloat16, (T, N))
    if gate_res is not None:
        a.whole("gate_res", gate_res, a.torch.float32, (B, N))
    out, out_stride = _rows_bf16(a, "out", out, (T, N))
    _check("pqk_linear_i8_gated_residual", lib().pqk_linear_i8_gated_residual(
        a8.data_ptr(), a_stride, a_scale.data_ptr(), w8.data_ptr(), w_stride, w_scale.data_ptr(), _ptr(x), x_stride,
        _ptr(gate_res), _ptr(cu_seqlens), B, out.data_ptr(), out_stride, T, K, N, a.stream()))
    a.used(out)
    return out


def linear_i8_swiglu(a8, a_scale, w8, w_scale, *, act=None, stream=None):
    """act = silu(y[:, :F]) * y[:, F:] with y = a_scale * w_scale * (a8 @
    w8.T), the product in 8-bit integers. a8: int8 [T, K], w8: int8 [2F, K],
    a_scale fp32 [T], w_scale fp32 [2F]. Returns act bf16 [T, F]."""
    a = _Args("linear_i8_swiglu", stream)
    T, K, rows, a_stride, w_stride = _i8_operands(a, a8, a_scale, w8, w_scale)
    F, odd = divmod(rows, 2)
    if odd:
        a.fail("w8", "has an odd number of rows")
    act, act_stride = _rows_bf16(a, "act", act, (T, F))
    _check("pqk_linear_i8_swiglu", lib().pqk_linear_i8_swiglu(
        a8.data_ptr(), a_stride, a_scale.data_ptr(), w8.data_ptr(), w_stride, w_scale.data_ptr(), act.data_ptr(),
        act_stride, T, K, F, a.stream()))
    a.used(act)
    return act


@functools.lru_cache(maxsize=64)
def varlen_cross_attn_workspace_size(B: int, D: int) -> int:
    return int(lib().pqk_varlen_cross_attn_workspace_size(B, D))


def varlen_cross_attn_fwd(q, k, v, cu_seqlens_q, cu_seqlens_k, *, softmax_scale: float | None = None, o=None,
                          lse=None, workspace=None, want_lse: bool = False, stream=None):
    """Packed attention of each request's queries to its own keys of another
    packed sequence. q: bf16 [Tq, H, D]; k, v: bf16 [Tk, Hkv, D], Hkv a
    divisor of H; cu_seqlens_q, cu_seqlens_k: int32 [B+1] on the device, from
    0 to at most Tq and Tk (rows behind the last request are left as they
    are). A request without keys gives o = 0, lse = -inf. Returns (o, lse
    fp32 [H, Tq] or None)."""
    a = _Args("varlen_cross_attn_fwd", stream)
    torch, bf16 = a.torch, a.torch.bfloat16
    shape, q_stride = a.first("q", q, bf16, 3)
    Tq, H, D = shape
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        a.fail("k", "is not a three-dimensional tensor")
    Tk, Hkv = k.shape[:2]
    kv_shape = (Tk, Hkv, D)
    k_stride = a.rows("k", k, bf16, kv_shape)
    v_stride = a.rows("v", v, bf16, kv_shape)
    if cu_seqlens_q is None:
        a.fail("cu_seqlens_q", "is not a one-dimensional tensor")
    B = _requests(a, cu_seqlens_q, "cu_seqlens_q")
    a.whole("cu_seqlens_k", cu_seqlens_k, torch.int32, (B + 1,))
    scale = softmax_scale if softmax_scale is not None else D ** -0.5
    o, o_stride = _rows_bf16(a, "o", o, shape)
    if lse is not None:
        a.whole("lse", lse, torch.float32, (H, Tq))
    elif want_lse:
        lse = a.new(torch.float32, H, Tq)
    if workspace is None:
        workspace = a.new(torch.uint8, varlen_cross_attn_workspace_size(B, D))
    elif not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous() or workspace.device != a.device:
        a.fail("workspace", f"is not a contiguous tensor on {a.device}")
    _check("pqk_varlen_cross_attn_fwd", lib().pqk_varlen_cross_attn_fwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _ptr(lse), q_stride, k_stride, v_stride, o_stride,
        cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), B, Tq, Tk, H, Hkv, D, scale, workspace.data_ptr(),
        workspace.nbytes, a.stream()))
    a.used(o, lse, workspace)
    return o, lse


def get_device_status(stream=None) -> int:
    return int(lib().pqk_get_device_status(_stream(stream)))


def set_wait_timeout_ns(ns: int) -> None:
    lib().pqk_set_wait_timeout_ns(int(ns))


def set_attn_cta_pairs(enable: bool) -> None:
    """The bf16, head_dim 128 attention on CTA pairs (bit-identical results)."""
    lib().pqk_set_attn_cta_pairs(1 if enable else 0)


def selftest_wait_timeout(timeout_ns: int, stream=None) -> None:
    _check("pqk_selftest_wait_timeout", lib().pqk_selftest_wait_timeout(int(timeout_ns), _stream(stream)))


def version() -> str:
    return lib().pqk_version().decode()
