"""Thin PyTorch-facing binding of the C ABI in include/mate.h.

Each function marshals torch CUDA tensors into the pointers and sizes of the
C entry point of the same name and raises ``MateError`` on a non-zero status.
PyTorch supplies device memory and the current stream; every step of the
computation runs in libmate.so. The ``bissd`` / ``tesa`` helpers read the
dims off the tensor shapes and allocate the output and workspace with torch.
"""
from __future__ import annotations

import ctypes
from contextlib import contextmanager
from typing import NamedTuple, Optional, Sequence

import torch

from . import _lib
from ._lib import (MATE_BF16, MATE_DIR_BI, MATE_F32, MATE_I8, MATE_NORM_LAYER, MATE_NORM_NONE, MATE_NORM_RMS, check,
                   mate_attn_dims, mate_block_norm_dims, mate_compose_dims, mate_frontend_dims, mate_gate_norm_dims,
                   mate_linear_i8_dims, mate_quant_dims, mate_ssd_dims)

_DT = {torch.float32: MATE_F32, torch.bfloat16: MATE_BF16}


def _stream_handle(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _handle(stream):
    return stream if type(stream) is int else _stream_handle(stream)


def _ptr(t: Optional[torch.Tensor]) -> ctypes.c_void_p:
    if t is None:
        return ctypes.c_void_p(0)
    return ctypes.c_void_p(t.data_ptr())


def _int3(v: Optional[Sequence[int]]):
    if v is None:
        return None
    return (ctypes.c_int * 3)(*[_lib.Int.from_param(int(u)) for u in v])


def _require(t: torch.Tensor, name: str, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _holds(t: torch.Tensor, name: str, n: int):
    """A tensor holds the `n` elements that the call reads or writes through its address."""
    if t.numel() < n:
        raise ValueError(f"{name} must hold {n} elements, got {tuple(t.shape)}")


def _matrix(w: torch.Tensor, name: str, rows: int, cols: int):
    if w.numel() != rows * cols:
        raise ValueError(f"{name} must be ({rows}, {cols}), got {tuple(w.shape)}")


class Codes(NamedTuple):
    """Rows held as 8-bit codes: value[..., k] is about q[..., k] * scale[...]."""
    q: torch.Tensor      # (..., K) int8
    scale: torch.Tensor  # (...) fp32


@contextmanager
def _on(t: torch.Tensor, stream):
    """`t`'s device and `stream` made current, so that outputs and temporaries belong to
    the stream that writes them. Yields the stream handle of the call."""
    with torch.cuda.device(t.device):
        if stream is None:
            yield torch.cuda.current_stream(t.device)
            return
        if not isinstance(stream, torch.cuda.Stream):
            handle = int(getattr(stream, "cuda_stream", stream))
            stream = torch.cuda.ExternalStream(handle, device=t.device) if handle else torch.cuda.default_stream(t.device)
        if stream.device != t.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
        with torch.cuda.stream(stream):
            yield stream


def _current(dev: int) -> int:
    """Handle of the current stream of device `dev`, without making a stream object."""
    return torch._C._cuda_getCurrentRawStream(dev)


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _same_device(first: torch.Tensor, *others):
    dev = first.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"all tensors of a call must be on one device, got {first.device} and {t.device}")


def _rows(shape) -> int:
    n = 1
    for s in shape:
        n *= s
    return n


def _out(out: Optional[torch.Tensor], name: str, shape, dtype, like: torch.Tensor) -> torch.Tensor:
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    _require(out, name, dtype)
    if out.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(out.shape)}")
    _same_device(like, out)
    return out


def ssd_dims(batch, nheads, headdim, dstate, ngroups, chunk, dtype, directions=MATE_DIR_BI) -> mate_ssd_dims:
    return mate_ssd_dims(batch, nheads, headdim, dstate, ngroups, chunk,
                         _DT[dtype] if isinstance(dtype, torch.dtype) else int(dtype), directions)


def attn_dims(batch, nheads, headdim, dtype) -> mate_attn_dims:
    return mate_attn_dims(batch, nheads, headdim, _DT[dtype] if isinstance(dtype, torch.dtype) else int(dtype))


# ---------------------------------------------------------------------------
# the C entry points, one to one
# ---------------------------------------------------------------------------
def mate_bissd_workspace_bytes(T: int, H: int, W: int, review_pool, dims: mate_ssd_dims) -> int:
    return int(_lib.load().mate_bissd_workspace_bytes(T, H, W, _int3(review_pool), ctypes.byref(dims)))


def mate_bissd_fwd(x, dt, A, B, C, D, T, H, W, scan_mode, review_pool, out, dims: mate_ssd_dims,
                   workspace: torch.Tensor, stream=None) -> None:
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = _lib.load().mate_bissd_fwd(_ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), T, H, W, scan_mode,
                                    _int3(review_pool), _ptr(out), ctypes.byref(dims), _ptr(workspace),
                                    ctypes.c_size_t(ws_bytes), _stream_handle(stream))
    check("mate_bissd_fwd", rc)


def mate_bissd_fwd_noalloc(x, dt, A, B, C, D, T, H, W, scan_mode, review_pool, out, dims: mate_ssd_dims,
                           stream=None) -> None:
    """mate_bissd_fwd with the library's fixed scratch array instead of a caller workspace."""
    rc = _lib.load().mate_bissd_fwd_noalloc(_ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), T, H, W,
                                            scan_mode, _int3(review_pool), _ptr(out), ctypes.byref(dims),
                                            _stream_handle(stream))
    check("mate_bissd_fwd_noalloc", rc)


def tesa_fwd(q, k, v, T, H, W, Tw, Sw, shift, out, dims: mate_attn_dims, stream=None) -> None:
    rc = _lib.load().tesa_fwd(_ptr(q), _ptr(k), _ptr(v), T, H, W, Tw, Sw, _int3(shift), _ptr(out),
                              ctypes.byref(dims), _stream_handle(stream))
    check("tesa_fwd", rc)


def mate_compose_fwd(y_ma, y_te, w_ma, w_te, out, dims: mate_compose_dims, stream=None) -> None:
    rc = _lib.load().mate_compose_fwd(_ptr(y_ma), _ptr(y_te), _ptr(w_ma), _ptr(w_te), _ptr(out), ctypes.byref(dims),
                                      _stream_handle(stream))
    check("mate_compose_fwd", rc)


def mate_gate_norm_fwd(y, z, w, eps: float, out, dims: mate_gate_norm_dims, stream=None) -> None:
    rc = _lib.load().mate_gate_norm_fwd(_ptr(y), _ptr(z), _ptr(w), float(eps), _ptr(out), ctypes.byref(dims),
                                        _stream_handle(stream))
    check("mate_gate_norm_fwd", rc)


def mate_quant_rows_fwd(x, q, scale, dims: mate_quant_dims, stream=None) -> None:
    rc = _lib.load().mate_quant_rows_fwd(_addr(x), _addr(q), _addr(scale), ctypes.byref(dims), _handle(stream))
    check("mate_quant_rows_fwd", rc)


def mate_linear_i8_fwd(x, x_scale, w, w_scale, bias, addend, out, dims: mate_linear_i8_dims, stream=None) -> None:
    rc = _lib.load().mate_linear_i8_fwd(_addr(x), _addr(x_scale), _addr(w), _addr(w_scale), _addr(bias), _addr(addend),
                                        _addr(out), ctypes.byref(dims), _handle(stream))
    check("mate_linear_i8_fwd", rc)


def mate_gate_norm_i8_fwd(y, z, w, eps: float, q, scale, dims: mate_gate_norm_dims, stream=None) -> None:
    rc = _lib.load().mate_gate_norm_i8_fwd(_addr(y), _addr(z), _addr(w), float(eps), _addr(q), _addr(scale),
                                           ctypes.byref(dims), _handle(stream))
    check("mate_gate_norm_i8_fwd", rc)


def mate_block_norm_fwd(x, y, w_post, gate, w_pre, scale, shift, x_out, h, h_scale, dims: mate_block_norm_dims,
                        stream=None) -> None:
    rc = _lib.load().mate_block_norm_fwd(_addr(x), _addr(y), _addr(w_post), _addr(gate), _addr(w_pre), _addr(scale),
                                         _addr(shift), _addr(x_out), _addr(h), _addr(h_scale), ctypes.byref(dims),
                                         _handle(stream))
    check("mate_block_norm_fwd", rc)


def mate_debug_rms_map(T, H, W, scan_mode, flip, out, stream=None) -> None:
    check("mate_debug_rms_map",
          _lib.load().mate_debug_rms_map(T, H, W, scan_mode, int(flip), _ptr(out), _stream_handle(stream)))


def mate_debug_tesa_map(T, H, W, Tw, Sw, shift, out, stream=None) -> None:
    check("mate_debug_tesa_map",
          _lib.load().mate_debug_tesa_map(T, H, W, Tw, Sw, _int3(shift), _ptr(out), _stream_handle(stream)))


def mate_last_error(stream=None) -> int:
    return int(_lib.load().mate_last_error(_stream_handle(stream)))


def mate_version() -> int:
    return int(_lib.load().mate_version())


# ---------------------------------------------------------------------------
# shape-reading helpers
# ---------------------------------------------------------------------------
def bissd_workspace(x: torch.Tensor, B: torch.Tensor, review_pool=None, chunk: int = 256,
                    directions: int = MATE_DIR_BI) -> torch.Tensor:
    b, T, H, W, nh, P = x.shape
    G, Ns = B.shape[4:]
    dims = ssd_dims(b, nh, P, Ns, G, chunk, x.dtype, directions)
    n = mate_bissd_workspace_bytes(T, H, W, review_pool, dims)
    if n == 0:
        raise ValueError("unsupported bi-SSD dims")
    return torch.empty(n, dtype=torch.uint8, device=x.device)


def bissd(x, dt, A, B, C, D, scan_mode: int, review_pool=None, chunk: int = 256, directions: int = MATE_DIR_BI,
          out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """MA-branch token mix. x: (batch, T, H, W, nh, P); dt: (batch, T, H, W, nh) fp32;
    A, D: (nh,) fp32; B, C: (batch, T, H, W, G, Ns). Returns out shaped like x."""
    for t, n in ((x, "x"), (B, "B"), (C, "C")):
        _require(t, n, x.dtype)
    for t, n in ((dt, "dt"), (A, "A"), (D, "D")):
        _require(t, n, torch.float32)
    b, T, H, W, nh, P = x.shape
    G, Ns = B.shape[4:]
    tokens = b * T * H * W
    for t, n, size in ((dt, "dt", tokens * nh), (A, "A", nh), (D, "D", nh), (B, "B", tokens * G * Ns),
                       (C, "C", tokens * G * Ns)):
        _holds(t, n, size)
    if out is None:
        out = torch.empty_like(x)
    else:
        _require(out, "out", x.dtype)
        _holds(out, "out", x.numel())
    if workspace is None:
        workspace = bissd_workspace(x, B, review_pool, chunk, directions)
    dims = ssd_dims(b, nh, P, Ns, G, chunk, x.dtype, directions)
    mate_bissd_fwd(x, dt, A, B, C, D, T, H, W, scan_mode, review_pool, out, dims, workspace, stream)
    return out


def tesa(q, k, v, Tw: int, Sw: int, shift=(0, 0, 0), out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """TE-branch window attention. q, k, v: (batch, T, H, W, nh, d). Returns out shaped like q."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, n, q.dtype)
    b, T, H, W, nh, d = q.shape
    _holds(k, "k", q.numel())
    _holds(v, "v", q.numel())
    if out is None:
        out = torch.empty_like(q)
    else:
        _require(out, "out", q.dtype)
        _holds(out, "out", q.numel())
    tesa_fwd(q, k, v, T, H, W, Tw, Sw, shift, out, attn_dims(b, nh, d, q.dtype), stream)
    return out


def compose(y_ma, y_te, w_ma, w_te, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """MATE composition: out = y_ma w_ma^T + y_te w_te^T (bf16). y_ma: (..., k_ma), the bi-SSD
    output with its heads flattened; y_te: (..., k_te), the TESA output likewise; w_ma: (d_model,
    k_ma), w_te: (d_model, k_te). Returns (..., d_model)."""
    for t, n in ((y_ma, "y_ma"), (y_te, "y_te"), (w_ma, "w_ma"), (w_te, "w_te")):
        _require(t, n, torch.bfloat16)
    lead = y_ma.shape[:-1]
    if y_te.shape[:-1] != lead:
        raise ValueError("y_ma and y_te must cover the same tokens")
    M = 1
    for s in lead:
        M *= int(s)
    N = int(w_ma.shape[0])
    _matrix(w_ma, "w_ma", N, int(y_ma.shape[-1]))
    _matrix(w_te, "w_te", N, int(y_te.shape[-1]))
    if out is None:
        out = torch.empty(*lead, N, dtype=torch.bfloat16, device=y_ma.device)
    else:
        _require(out, "out", torch.bfloat16)
        _holds(out, "out", M * N)
    dims = mate_compose_dims(M, int(y_ma.shape[-1]), int(y_te.shape[-1]), N, MATE_BF16)
    mate_compose_fwd(y_ma, y_te, w_ma, w_te, out, dims, stream)
    return out


def gate_norm(y, z, w, group: int, eps: float = 1e-5, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """MA-branch output side: out = y SiLU(z) / sqrt(mean over each group of `group` channels
    of (y SiLU(z))^2 + eps) * w (bf16). y: (..., C), the bi-SSD output with its heads flattened;
    z: (..., C), the front-end's z; w: (C,) fp32. Returns (..., C)."""
    _require(y, "y", torch.bfloat16)
    _require(z, "z", torch.bfloat16)
    _require(w, "w", torch.float32)
    if z.shape != y.shape or w.shape != (y.shape[-1],):
        raise ValueError("y and z must have one shape and w one entry per channel")
    M = 1
    for s in y.shape[:-1]:
        M *= int(s)
    if out is None:
        out = torch.empty_like(y)
    else:
        _require(out, "out", torch.bfloat16)
        _holds(out, "out", y.numel())
    dims = mate_gate_norm_dims(M, int(y.shape[-1]), int(group), MATE_BF16)
    mate_gate_norm_fwd(y, z, w, eps, out, dims, stream)
    return out


def linear(x, w, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x w^T on the tensor cores (bf16): the composition GEMM with one input part.
    x: (..., K); w: (N, K) in the nn.Linear layout. Returns (..., N)."""
    _require(x, "x", torch.bfloat16)
    _require(w, "w", torch.bfloat16)
    M = 1
    for s in x.shape[:-1]:
        M *= int(s)
    N = int(w.shape[0])
    _matrix(w, "w", N, int(x.shape[-1]))
    if out is None:
        out = torch.empty(*x.shape[:-1], N, dtype=torch.bfloat16, device=x.device)
    else:
        _require(out, "out", torch.bfloat16)
        _holds(out, "out", M * N)
    mate_compose_fwd(x, None, w, None, out, mate_compose_dims(M, int(x.shape[-1]), 0, N, MATE_BF16), stream)
    return out


def quantize_rows(x, stream=None) -> Codes:
    """8-bit codes and the scale of every row. x: (..., K) bf16, tokens or the rows of an
    nn.Linear weight. Returns Codes(q (..., K) int8, scale (...) fp32) with
    scale = max|x| / 127 and q = rint(127 x / max|x|)."""
    _require(x, "x", torch.bfloat16)
    if x.dim() < 1:
        raise ValueError("x must be (..., K)")
    dev = x.get_device()
    if stream is not None or dev != torch._C._cuda_getDevice():
        with _on(x, stream):
            return quantize_rows(x)
    dims = mate_quant_dims.of(_rows(x.shape[:-1]), x.shape[-1], MATE_BF16)
    q, scale = torch.empty_like(x, dtype=torch.int8), x.new_empty(x.shape[:-1], dtype=torch.float32)
    rc = _lib.load().mate_quant_rows_fwd(x.data_ptr(), q.data_ptr(), scale.data_ptr(), ctypes.byref(dims), _current(dev))
    check("mate_quant_rows_fwd", rc)
    return Codes(q, scale)


def _check_linear_i8(x_q, x_scale, w_q, w_scale, bias, addend, out_dtype):
    """Every argument check of linear_i8 with its message; linear_i8 itself asks the same in one
    expression and comes here when it does not hold."""
    if out_dtype not in _DT:
        raise ValueError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    _require(x_q, "x_q", torch.int8)
    _require(w_q, "w_q", torch.int8)
    _require(x_scale, "x_scale", torch.float32)
    _require(w_scale, "w_scale", torch.float32)
    if w_q.dim() != 2 or x_q.dim() < 1 or x_q.shape[-1] != w_q.shape[1]:
        raise ValueError("x_q must be (..., K) and w_q (N, K)")
    N = w_q.shape[0]
    if x_q.shape[:-1] != x_scale.shape or w_scale.shape != (N,):
        raise ValueError("x_scale must have one entry per token and w_scale one per row of w_q")
    if bias is not None:
        _require(bias, "bias", torch.float32)
        if bias.shape != (N,):
            raise ValueError("bias must have one entry per row of w_q")
    if addend is not None:
        _require(addend, "addend", out_dtype)
        if addend.shape != x_scale.shape + (N,):
            raise ValueError(f"addend must have shape {tuple(x_scale.shape) + (N,)}")
    _same_device(x_q, x_scale, w_q, w_scale, bias, addend)


def linear_i8(x_q, x_scale, w_q, w_scale, bias=None, addend=None, out_dtype=torch.bfloat16,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """8-bit linear layer: x_scale w_scale (x_q w_q^T) + bias + addend, the sum exact (of any int8 codes)
    and one rounding to out_dtype (bf16 or fp32). x_q: (..., K) int8; x_scale: (...) fp32; w_q: (N, K)
    int8; w_scale: (N,) fp32; bias: (N,) fp32; addend: (..., N) out_dtype, and may be `out`.
    Returns (..., N)."""
    try:
        dev, (N, K) = x_q.get_device(), w_q.shape
        fine = (dev >= 0 and out_dtype in _DT
                and x_q.dtype is torch.int8 and w_q.dtype is torch.int8
                and x_scale.dtype is torch.float32 and w_scale.dtype is torch.float32
                and w_q.get_device() == dev and x_scale.get_device() == dev and w_scale.get_device() == dev
                and x_q.is_contiguous() and w_q.is_contiguous() and x_scale.is_contiguous() and w_scale.is_contiguous()
                and x_q.shape == (*x_scale.shape, K) and w_scale.shape == (N,)
                and (bias is None or (bias.dtype is torch.float32 and bias.get_device() == dev and bias.is_contiguous()
                                      and bias.shape == (N,)))
                and (addend is None or (addend.dtype is out_dtype and addend.get_device() == dev
                                        and addend.is_contiguous() and addend.shape == (*x_scale.shape, N))))
    except (AttributeError, TypeError, ValueError):
        fine = False
    if not fine:
        _check_linear_i8(x_q, x_scale, w_q, w_scale, bias, addend, out_dtype)
        dev, (N, K) = x_q.get_device(), w_q.shape
    if stream is not None or dev != torch._C._cuda_getDevice():
        with _on(x_q, stream):
            return linear_i8(x_q, x_scale, w_q, w_scale, bias, addend, out_dtype, out)
    dims = mate_linear_i8_dims.of(x_scale.numel(), K, N, _DT[out_dtype])
    shape = (*x_scale.shape, N)
    out = x_q.new_empty(shape, dtype=out_dtype) if out is None else _out(out, "out", shape, out_dtype, x_q)
    rc = _lib.load().mate_linear_i8_fwd(x_q.data_ptr(), x_scale.data_ptr(), w_q.data_ptr(), w_scale.data_ptr(),
                                        _addr(bias), _addr(addend), out.data_ptr(), ctypes.byref(dims), _current(dev))
    check("mate_linear_i8_fwd", rc)
    return out


def gate_norm_i8(y, z, w, group: int, eps: float = 1e-5, stream=None) -> Codes:
    """gate_norm with its output as 8-bit codes and one scale per row (not rounded to bf16
    between). Arguments as for gate_norm. Returns Codes(q (..., C), scale (...))."""
    _require(y, "y", torch.bfloat16)
    _require(z, "z", torch.bfloat16)
    _require(w, "w", torch.float32)
    if z.shape != y.shape or w.shape != (y.shape[-1],):
        raise ValueError("y and z must have one shape and w one entry per channel")
    _same_device(y, z, w)
    dev = y.get_device()
    if stream is not None or dev != torch._C._cuda_getDevice():
        with _on(y, stream):
            return gate_norm_i8(y, z, w, group, eps)
    dims = mate_gate_norm_dims.of(_rows(y.shape[:-1]), y.shape[-1], int(group), MATE_BF16)
    q, scale = torch.empty_like(y, dtype=torch.int8), y.new_empty(y.shape[:-1], dtype=torch.float32)
    rc = _lib.load().mate_gate_norm_i8_fwd(y.data_ptr(), z.data_ptr(), w.data_ptr(), float(eps), q.data_ptr(),
                                           scale.data_ptr(), ctypes.byref(dims), _current(dev))
    check("mate_gate_norm_i8_fwd", rc)
    return Codes(q, scale)


_NORMS = {"rms": MATE_NORM_RMS, "layer": MATE_NORM_LAYER}


def _check_vec(t, name, C, dev):
    """A weight of block_norm: its address."""
    if t is None:
        return None
    _require(t, name, torch.float32)
    if t.shape != (C,):
        raise ValueError(f"{name} must have one entry per channel")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    return t.data_ptr()


def _check_mod(t, name, batch, C, dev):
    """A modulation vector of block_norm: its address and its stride between batch elements."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or t.get_device() != dev:
        raise ValueError(f"{name} must be a float32 CUDA tensor on cuda:{dev}")
    n = t.dim()
    if t.shape != ((batch, C) if n == 2 else (C,)) or (C > 1 and t.stride(n - 1) != 1):
        raise ValueError(f"{name} must be (batch, C) or (C,), its channels contiguous")
    return t.data_ptr(), t.stride(0) if n == 2 and batch > 1 else 0


def block_norm(x, y=None, *, w_post=None, gate=None, residual_scale: float = 1.0, post_norm: bool = True, w_pre=None,
               scale=None, shift=None, norm: str = "rms", eps: float = 1e-6, h_dtype=torch.bfloat16,
               x_out: Optional[torch.Tensor] = None, stream=None):
    """The norms before and after a block with its modulation, gate and residual scale, in
    one pass over the residual stream:
        x_out = residual_scale x + gate (N(y) w_post)     with y, the block's output
        h     = N(x_out) w_pre (1 + scale) + shift        the next block's input
    (h from x itself without y). x: (batch, ..., C) bf16 or fp32; y: like x, bf16; w_post,
    w_pre: (C,) fp32; gate, scale, shift: (batch, C) fp32 (or (C,) for all batch elements), which
    may be column ranges of one wider tensor. norm: "rms" or "layer", for both norms;
    post_norm=False leaves y as it is. h_dtype: torch.bfloat16, torch.int8 (h is Codes) or None
    (no h). x_out may be x. Returns (x_out or None, h or None)."""
    if norm not in _NORMS:
        raise ValueError(f"norm must be one of {sorted(_NORMS)}, got {norm!r}")
    if h_dtype is None:
        if w_pre is not None or scale is not None or shift is not None:
            raise ValueError("w_pre, scale and shift go with h")
        if y is None:
            raise ValueError("nothing to compute: neither y nor h")
    elif h_dtype is not torch.bfloat16 and h_dtype is not torch.int8:
        raise ValueError(f"h_dtype must be bfloat16, int8 or None, got {h_dtype}")
    if y is None and (w_post is not None or gate is not None or x_out is not None or residual_scale != 1.0):
        raise ValueError("w_post, gate, residual_scale and x_out go with y")
    _require(x, "x")
    if x.dtype not in _DT or x.dim() < 2:
        raise ValueError(f"x must be (batch, ..., C) bfloat16 or float32, got {x.dtype}")
    dev, shape = x.get_device(), x.shape
    batch, C = shape[0], shape[-1]
    if y is not None:
        _require(y, "y", torch.bfloat16)
        if y.shape != shape or y.get_device() != dev:
            raise ValueError("x and y must have one shape and be on one device")
        if w_post is not None and not post_norm:
            raise ValueError("w_post goes with post_norm")
    p_post, p_pre = _check_vec(w_post, "w_post", C, dev), _check_vec(w_pre, "w_pre", C, dev)
    p_gate, s_gate = _check_mod(gate, "gate", batch, C, dev)
    p_scale, s_scale = _check_mod(scale, "scale", batch, C, dev)
    p_shift, s_shift = _check_mod(shift, "shift", batch, C, dev)
    if stream is not None or dev != torch._C._cuda_getDevice():
        with _on(x, stream):
            return block_norm(x, y, w_post=w_post, gate=gate, residual_scale=residual_scale, post_norm=post_norm,
                              w_pre=w_pre, scale=scale, shift=shift, norm=norm, eps=eps, h_dtype=h_dtype, x_out=x_out)
    kind, rows = _NORMS[norm], _rows(shape[1:-1])
    dims = mate_block_norm_dims.of(batch, rows, C, kind if post_norm else MATE_NORM_NONE, kind, _DT[x.dtype],
                                   MATE_I8 if h_dtype is torch.int8 else MATE_BF16, s_gate, s_scale, s_shift,
                                   residual_scale, eps)
    if y is not None:
        x_out = torch.empty_like(x) if x_out is None else _out(x_out, "x_out", shape, x.dtype, x)
    h = None if h_dtype is None else torch.empty_like(x, dtype=h_dtype)
    h_scale = x.new_empty(shape[:-1], dtype=torch.float32) if h_dtype is torch.int8 else None
    rc = _lib.load().mate_block_norm_fwd(x.data_ptr(), _addr(y), p_post, p_gate, p_pre, p_scale, p_shift, _addr(x_out),
                                         _addr(h), _addr(h_scale), ctypes.byref(dims), _current(dev))
    check("mate_block_norm_fwd", rc)
    return x_out, (h if h_scale is None else Codes(h, h_scale))


# the block's weights that its matrix products read
_PROJECTIONS = ("w_in", "w_q", "w_k", "w_v", "w_ma", "w_te")


def quantize_block(weights, stream=None):
    """A block's weights with those of its matrix products as 8-bit codes (a scale per output
    channel), for block() and stack(). The others are kept as they are."""
    out = dict(weights)
    for n in _PROJECTIONS:
        out[n] = quantize_rows(weights[n], stream=stream)
    return out


def modulation(c, w: Codes, bias=None, stream=None) -> torch.Tensor:
    """A layer's modulation vectors from its conditioning, as an 8-bit linear layer with fp32
    output. c: (batch, K) bf16; w: Codes of (3 d_model, K); bias: (3 d_model,) fp32. Returns
    (batch, 3 d_model): shift, scale and gate, as stack() takes them."""
    _require(c, "c", torch.bfloat16)
    with _on(c, stream):
        return linear_i8(*quantize_rows(c), *w, bias=bias, out_dtype=torch.float32)


def block(u, weights, *, scan_mode: int, review_pool, chunk: int, nheads: int, headdim: int, ngroups: int,
          dstate: int, attn_heads: int, attn_dim: int, Tw: int, Sw: int, shift, eps: float = 1e-5, stream=None,
          keep: bool = False):
    """One MATE token mixer, every step in the library's kernels. u: (batch, T, H, W, d_model) bf16.
        MA-branch: z, x, dt, B, C = front-end(u); y = bi-SSD(x, dt, A, B, C, D) in the RMS order
                   `scan_mode` with review tokens; y_ma = gated norm(y, z)
        TE-branch: q, k, v = u w_q^T, u w_k^T, u w_v^T; y_te = TESA(q, k, v)
        out = y_ma w_ma^T + y_te w_te^T
    weights: w_in, conv_w, conv_b, dt_bias, A, D, norm_w, w_q, w_k, w_v, w_ma, w_te (as
    workloads.generate_block draws them). Returns out (batch, T, H, W, d_model), and with
    `keep` also a dict of the intermediate tensors.
    With weights from quantize_block every matrix product runs in 8 bits: u may then be Codes (a
    block_norm's h) and is quantised per token otherwise, the gated norm and the TESA output
    become Codes too, and the scan and the attention run in bf16 as above."""
    w = weights
    eight = [isinstance(w[n], Codes) for n in _PROJECTIONS]
    if any(eight):
        if not all(eight):
            raise ValueError("the weights of all the block's matrix products must be Codes, or none (quantize_block)")
        with _on(u.q if isinstance(u, Codes) else u, stream):
            return _block_i8(u, w, scan_mode, review_pool, chunk, nheads, headdim, ngroups, dstate, attn_heads, attn_dim,
                             Tw, Sw, shift, eps, keep)
    if isinstance(u, Codes):
        raise ValueError("u is Codes: the weights must be 8-bit too (quantize_block)")
    b, T, H, W, _ = u.shape
    z, x, dt, B, C = frontend(u, w["w_in"], w["conv_w"], w["conv_b"], w["dt_bias"], scan_mode, nheads, headdim,
                              ngroups, dstate, stream=stream)
    y = bissd(x, dt, w["A"], B, C, w["D"], scan_mode, review_pool, chunk=chunk, stream=stream)
    d_inner = nheads * headdim
    y_ma = gate_norm(y.view(b, T, H, W, d_inner), z, w["norm_w"], d_inner // ngroups, eps, stream=stream)
    q, k, v = (linear(u, w[n], stream=stream).view(b, T, H, W, attn_heads, attn_dim) for n in ("w_q", "w_k", "w_v"))
    y_te = tesa(q, k, v, Tw, Sw, shift, stream=stream)
    out = compose(y_ma, y_te.view(b, T, H, W, attn_heads * attn_dim), w["w_ma"], w["w_te"], stream=stream)
    if keep:
        return out, dict(z=z, x=x, dt=dt, B=B, C=C, y=y, y_ma=y_ma, q=q, k=k, v=v, y_te=y_te)
    return out


def _block_i8(u, w, scan_mode, review_pool, chunk, nheads, headdim, ngroups, dstate, attn_heads, attn_dim, Tw, Sw, shift,
              eps, keep):
    if not isinstance(u, Codes):
        u = quantize_rows(u)
    b, T, H, W, _ = u.q.shape
    z, x, dt, B, C = frontend_i8(u, w["w_in"], w["conv_w"], w["conv_b"], w["dt_bias"], scan_mode, nheads, headdim,
                                 ngroups, dstate)
    y = bissd(x, dt, w["A"], B, C, w["D"], scan_mode, review_pool, chunk=chunk)
    d_inner = nheads * headdim
    y_ma = gate_norm_i8(y.view(b, T, H, W, d_inner), z, w["norm_w"], d_inner // ngroups, eps)
    q, k, v = (linear_i8(*u, *w[n]).view(b, T, H, W, attn_heads, attn_dim) for n in ("w_q", "w_k", "w_v"))
    y_te = tesa(q, k, v, Tw, Sw, shift)
    c_te = quantize_rows(y_te.view(b, T, H, W, attn_heads * attn_dim))
    # the branches' codes have scales of their own: the second product adds the first, which is rounded to
    # bf16 on the way (by at most 2^-8 of itself; the codes leave it off by about 1%)
    te = linear_i8(*c_te, *w["w_te"])
    if keep:
        out = linear_i8(*y_ma, *w["w_ma"], addend=te)
        return out, dict(u=u, z=z, x=x, dt=dt, B=B, C=C, y=y, y_ma=y_ma, q=q, k=k, v=v, y_te=y_te, c_te=c_te, te=te)
    return linear_i8(*y_ma, *w["w_ma"], addend=te, out=te)


def stack(x, layers, *, norm: str = "rms", residual_scale: float = 1.0, norm_eps: float = 1e-6, stream=None, **spec):
    """Residual layers around the token mixer (adaLN form). For each layer in turn, with N the
    norm and (shift, scale, gate) its modulation:
        h = N(x) w_pre (1 + scale) + shift;  y = block(h);  x = residual_scale x + gate N(y) w_post
    x: (batch, T, H, W, d_model) bf16 or fp32, not written. layers: a sequence of (weights, mod) or
    (weights, mod, overrides): weights as block() takes them (8-bit ones run the layer in 8 bits), with
    w_pre and w_post (d_model,) fp32 where the norms have weights; mod (batch, 3 d_model) fp32, the
    shift, scale and gate of every batch element (see modulation()); overrides a dict of block()
    arguments of that layer alone (scan_mode and shift alternate between layers). spec: block()'s
    arguments (but for keep, and the stream is the stack's). The norm after a layer and the one before the next are one pass. Returns x."""
    layers = [tuple(ly) + ({},) * (3 - len(ly)) for ly in layers]
    if not layers:
        return x
    C = int(x.shape[-1])
    for _, mod, over in layers:
        if "keep" in spec or "keep" in over or "stream" in over:
            raise ValueError("stack() keeps no layer's intermediate tensors (keep) and has one stream for all layers")
        if tuple(mod.shape) != (x.shape[0], 3 * C):
            raise ValueError(f"mod must be (batch, 3 d_model) = {(int(x.shape[0]), 3 * C)}, got {tuple(mod.shape)}")
    kw = dict(norm=norm, eps=norm_eps)

    def before(w, mod, _):
        return dict(w_pre=w.get("w_pre"), shift=mod[:, :C], scale=mod[:, C:2 * C],
                    h_dtype=torch.int8 if isinstance(w["w_in"], Codes) else torch.bfloat16)

    with _on(x, stream):
        _, h = block_norm(x, **before(*layers[0]), **kw)
        for i, (w, mod, over) in enumerate(layers):
            y = block(h, w, **{**spec, **over})
            after = before(*layers[i + 1]) if i + 1 < len(layers) else dict(h_dtype=None)
            x, h = block_norm(x, y, w_post=w.get("w_post"), gate=mod[:, 2 * C:], residual_scale=residual_scale, **after,
                              **kw)
    return x


def mate_frontend_workspace_bytes(T: int, H: int, W: int, dims: mate_frontend_dims) -> int:
    return int(_lib.load().mate_frontend_workspace_bytes(T, H, W, ctypes.byref(dims)))


def mate_frontend_fwd(u, w_in, conv_w, conv_b, dt_bias, T, H, W, scan_mode, z, x, dt, B, C,
                      dims: mate_frontend_dims, workspace, stream=None) -> None:
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = _lib.load().mate_frontend_fwd(_ptr(u), _ptr(w_in), _ptr(conv_w), _ptr(conv_b), _ptr(dt_bias), T, H, W,
                                       scan_mode, _ptr(z), _ptr(x), _ptr(dt), _ptr(B), _ptr(C), ctypes.byref(dims),
                                       _ptr(workspace), nbytes, _stream_handle(stream))
    check("mate_frontend_fwd", rc)


def frontend(u, w_in, conv_w, conv_b, dt_bias, scan_mode: int, nheads: int, headdim: int, ngroups: int, dstate: int,
             stream=None):
    """MA-branch front-end. u: (batch, T, H, W, d_model) bf16; w_in: (d_inner + dc + nheads, d_model)
    bf16; conv_w: (dc, 4), conv_b: (dc), dt_bias: (nheads) fp32. Returns z, x, dt, B, C shaped as
    mate_bissd_fwd and the gate take them."""
    _require(u, "u", torch.bfloat16)
    _require(w_in, "w_in", torch.bfloat16)
    for t, n in ((conv_w, "conv_w"), (conv_b, "conv_b"), (dt_bias, "dt_bias")):
        _require(t, n, torch.float32)
    b, T, H, W, dm = u.shape
    dc = nheads * headdim + 2 * ngroups * dstate
    _matrix(w_in, "w_in", nheads * headdim + dc + nheads, dm)
    for t, n, size in ((conv_w, "conv_w", dc * 4), (conv_b, "conv_b", dc), (dt_bias, "dt_bias", nheads)):
        _holds(t, n, size)
    dims = mate_frontend_dims(b, dm, nheads, headdim, ngroups, dstate, MATE_BF16)
    nbytes = mate_frontend_workspace_bytes(T, H, W, dims)
    if nbytes == 0:
        raise ValueError("unsupported front-end dims")
    ws = torch.empty(nbytes, dtype=torch.uint8, device=u.device)
    kw = dict(dtype=torch.bfloat16, device=u.device)
    z = torch.empty(b, T, H, W, nheads * headdim, **kw)
    x = torch.empty(b, T, H, W, nheads, headdim, **kw)
    dt = torch.empty(b, T, H, W, nheads, dtype=torch.float32, device=u.device)
    Bm = torch.empty(b, T, H, W, ngroups, dstate, **kw)
    Cm = torch.empty(b, T, H, W, ngroups, dstate, **kw)
    mate_frontend_fwd(u, w_in, conv_w, conv_b, dt_bias, T, H, W, scan_mode, z, x, dt, Bm, Cm, dims, ws, stream)
    return z, x, dt, Bm, Cm


def mate_frontend_i8_fwd(u, u_scale, w_in, w_scale, conv_w, conv_b, dt_bias, T, H, W, scan_mode, z, x, dt, B, C,
                         dims: mate_frontend_dims, workspace, stream=None) -> None:
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = _lib.load().mate_frontend_i8_fwd(_ptr(u), _ptr(u_scale), _ptr(w_in), _ptr(w_scale), _ptr(conv_w),
                                          _ptr(conv_b), _ptr(dt_bias), T, H, W, scan_mode, _ptr(z), _ptr(x), _ptr(dt),
                                          _ptr(B), _ptr(C), ctypes.byref(dims), _ptr(workspace), nbytes,
                                          _stream_handle(stream))
    check("mate_frontend_i8_fwd", rc)


def frontend_i8(u: Codes, w_in: Codes, conv_w, conv_b, dt_bias, scan_mode: int, nheads: int, headdim: int, ngroups: int,
                dstate: int, stream=None):
    """frontend with in_proj in 8 bits. u: Codes of (batch, T, H, W, d_model); w_in: Codes of
    (d_inner + dc + nheads, d_model); the rest and the results as for frontend."""
    _require(u.q, "u.q", torch.int8)
    _require(w_in.q, "w_in.q", torch.int8)
    for t, n in ((u.scale, "u.scale"), (w_in.scale, "w_in.scale"), (conv_w, "conv_w"), (conv_b, "conv_b"),
                 (dt_bias, "dt_bias")):
        _require(t, n, torch.float32)
    b, T, H, W, dm = u.q.shape
    d_inner, dc = nheads * headdim, nheads * headdim + 2 * ngroups * dstate
    for t, n, shape in ((u.scale, "u.scale", (b, T, H, W)), (w_in.q, "w_in.q", (d_inner + dc + nheads, dm)),
                        (w_in.scale, "w_in.scale", (d_inner + dc + nheads,)), (conv_w, "conv_w", (dc, 4)),
                        (conv_b, "conv_b", (dc,)), (dt_bias, "dt_bias", (nheads,))):
        if tuple(t.shape) != shape:
            raise ValueError(f"{n} must have shape {shape}, got {tuple(t.shape)}")
    _same_device(u.q, u.scale, w_in.q, w_in.scale, conv_w, conv_b, dt_bias)
    dims = mate_frontend_dims(b, dm, nheads, headdim, ngroups, dstate, MATE_BF16)
    nbytes = mate_frontend_workspace_bytes(T, H, W, dims)
    if nbytes == 0:
        raise ValueError("unsupported front-end dims")
    with _on(u.q, stream) as st:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=u.q.device)
        kw = dict(dtype=torch.bfloat16, device=u.q.device)
        z = torch.empty(b, T, H, W, d_inner, **kw)
        x = torch.empty(b, T, H, W, nheads, headdim, **kw)
        dt = torch.empty(b, T, H, W, nheads, dtype=torch.float32, device=u.q.device)
        Bm = torch.empty(b, T, H, W, ngroups, dstate, **kw)
        Cm = torch.empty(b, T, H, W, ngroups, dstate, **kw)
        mate_frontend_i8_fwd(u.q, u.scale, w_in.q, w_in.scale, conv_w, conv_b, dt_bias, T, H, W, scan_mode, z, x, dt,
                             Bm, Cm, dims, ws, st)
    return z, x, dt, Bm, Cm


def rms_map(T: int, H: int, W: int, scan_mode: int, flip: bool = False, device="cuda") -> torch.Tensor:
    out = torch.empty(T * H * W, dtype=torch.int32, device=device)
    mate_debug_rms_map(T, H, W, scan_mode, flip, out)
    return out


def tesa_map(T: int, H: int, W: int, Tw: int, Sw: int, shift, device="cuda") -> torch.Tensor:
    out = torch.empty(T * H * W, dtype=torch.int32, device=device)
    mate_debug_tesa_map(T, H, W, Tw, Sw, shift, out)
    return out
