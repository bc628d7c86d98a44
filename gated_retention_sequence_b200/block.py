"""The selective state space block's operators as calls on torch CUDA tensors.

``short_conv``, ``selective_scan`` and ``residual_norm`` (with their forms for
packed batches and single tokens, and their gradients) check types and shapes, allocate
outputs and scratch with torch's allocator and call the C ABI of
``include/gret.h``; all arithmetic runs in the CUDA library.

Activations may be columns of a wider tensor (a slice of a joint projection):
the last dimension is dense and the rows are equally far apart.  Parameters and
states are contiguous fp32, tails have the activations' dtype.  A call runs on
``stream`` (default: the current stream of the tensors' device), and what it
allocates belongs to that stream.
"""
from __future__ import annotations

import contextlib
import enum
from typing import Optional

from . import gret as _g
from .gret import Dtype, GretError, _check, _io_of, _ptr


class Activation(enum.IntEnum):
    NONE = 0
    SWISH = 1


def _lib():
    return _g._lib or _g.load()


# ---------------------------------------------------------------- raw C calls
def gret_short_conv(x, ldx, w, bias, tail0, y, tail, B, N, D, K, io_dtype, act, stream) -> int:
    return _lib().gret_short_conv(x, ldx, w, bias, tail0, y, tail, B, N, D, K, int(io_dtype), int(act), stream)


def gret_short_conv_varlen(x, ldx, w, bias, tail0, cu_seqlens, num_seqs, total_tokens, max_seqlen, y, tail, D, K,
                           io_dtype, act, stream) -> int:
    return _lib().gret_short_conv_varlen(x, ldx, w, bias, tail0, cu_seqlens, num_seqs, total_tokens, max_seqlen, y,
                                            tail, D, K, int(io_dtype), int(act), stream)


def gret_short_conv_step(x, ldx, w, bias, tail_in, tail_out, y, num_seqs, D, K, io_dtype, act, stream) -> int:
    return _lib().gret_short_conv_step(x, ldx, w, bias, tail_in, tail_out, y, num_seqs, D, K, int(io_dtype),
                                          int(act), stream)


def gret_selective_scan(u, ldu, dt, lddt, A, Bm, ldb, Cm, ldc, skip, z, ldz, dt_bias, h0, o, h_final, B, N, D, n,
                        io_dtype, workspace, workspace_bytes, stream) -> int:
    return _lib().gret_selective_scan(u, ldu, dt, lddt, A, Bm, ldb, Cm, ldc, skip, z, ldz, dt_bias, h0, o, h_final,
                                         B, N, D, n, int(io_dtype), workspace, workspace_bytes, stream)


def gret_selective_scan_workspace_size(B, N, D, n, io_dtype) -> int:
    return _lib().gret_selective_scan_workspace_size(B, N, D, n, int(io_dtype))


def gret_selective_scan_varlen(u, ldu, dt, lddt, A, Bm, ldb, Cm, ldc, skip, z, ldz, dt_bias, h0, cu_seqlens, num_seqs,
                               total_tokens, max_seqlen, o, h_final, D, n, io_dtype, workspace, workspace_bytes,
                               stream) -> int:
    return _lib().gret_selective_scan_varlen(u, ldu, dt, lddt, A, Bm, ldb, Cm, ldc, skip, z, ldz, dt_bias, h0,
                                                cu_seqlens, num_seqs, total_tokens, max_seqlen, o, h_final, D, n,
                                                int(io_dtype), workspace, workspace_bytes, stream)


def gret_selective_scan_varlen_workspace_size(num_seqs, total_tokens, max_seqlen, D, n, io_dtype) -> int:
    return _lib().gret_selective_scan_varlen_workspace_size(num_seqs, total_tokens, max_seqlen, D, n, int(io_dtype))


def gret_selective_step(u, ldu, dt, lddt, A, Bm, ldb, Cm, ldc, skip, z, ldz, dt_bias, h_in, h_out, o, num_seqs, D, n,
                        io_dtype, stream) -> int:
    return _lib().gret_selective_step(u, ldu, dt, lddt, A, Bm, ldb, Cm, ldc, skip, z, ldz, dt_bias, h_in, h_out, o,
                                         num_seqs, D, n, int(io_dtype), stream)


def gret_residual_norm(x, ldx, y, ldy, gate, ldg, scale, w_post, w_next, r, n, T, D, eps, stream_dtype, io_dtype,
                       stream) -> int:
    return _lib().gret_residual_norm(x, ldx, y, ldy, gate, ldg, scale, w_post, w_next, r, n, T, D, eps,
                                        int(stream_dtype), int(io_dtype), stream)


def gret_short_conv_backward_workspace_size(B, N, D, K, io_dtype) -> int:
    return _lib().gret_short_conv_backward_workspace_size(B, N, D, K, int(io_dtype))


def gret_short_conv_backward(x, ldx, w, bias, tail0, dy, dtail, dx, dw, dbias, dtail0, B, N, D, K, io_dtype, act,
                             workspace, workspace_bytes, stream) -> int:
    return _lib().gret_short_conv_backward(x, ldx, w, bias, tail0, dy, dtail, dx, dw, dbias, dtail0, B, N, D, K,
                                              int(io_dtype), int(act), workspace, workspace_bytes, stream)


def gret_selective_scan_backward_workspace_size(B, N, D, n, io_dtype) -> int:
    return _lib().gret_selective_scan_backward_workspace_size(B, N, D, n, int(io_dtype))


def gret_selective_scan_backward(u, ldu, dt, lddt, A, Bm, ldb, Cm, ldc, skip, z, ldz, dt_bias, h0, dout, dh_final, du,
                                 ddt, dA, dBm, dCm, dskip, dz, ddt_bias, dh0, B, N, D, n, io_dtype, workspace,
                                 workspace_bytes, stream) -> int:
    return _lib().gret_selective_scan_backward(u, ldu, dt, lddt, A, Bm, ldb, Cm, ldc, skip, z, ldz, dt_bias, h0,
                                                  dout, dh_final, du, ddt, dA, dBm, dCm, dskip, dz, ddt_bias, dh0, B,
                                                  N, D, n, int(io_dtype), workspace, workspace_bytes, stream)


def gret_residual_norm_backward_workspace_size(T, D) -> int:
    return _lib().gret_residual_norm_backward_workspace_size(T, D)


def gret_residual_norm_backward(x, ldx, y, ldy, gate, ldg, scale, w_post, w_next, dr, dn, dx, dy, dgate, dscale, dw_post,
                                dw_next, T, D, eps, stream_dtype, io_dtype, workspace, workspace_bytes, stream) -> int:
    return _lib().gret_residual_norm_backward(x, ldx, y, ldy, gate, ldg, scale, w_post, w_next, dr, dn, dx, dy,
                                                 dgate, dscale, dw_post, dw_next, T, D, eps, int(stream_dtype),
                                                 int(io_dtype), workspace, workspace_bytes, stream)


# ---------------------------------------------------------------- helpers
def _rows(t, name, dtype, shape, dev) -> int:
    """Check an activation and return its row stride."""
    if not (t.is_cuda and t.dtype is dtype and t.device == dev and t.shape == shape):
        if not t.is_cuda or t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}" if t.is_cuda else f"{name} must be a CUDA tensor")
        if t.dtype != dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.is_contiguous():
        return shape[-1]
    # the dimensions with more than one entry lie `ld` rows apart, in order; one broadcast (a stride of 0) has no such rows
    strides = t.stride()
    ld, rows = None, 1
    for i in range(len(shape) - 2, -1, -1):
        size = shape[i]
        if size != 1:
            if ld is None:
                ld = strides[i]
            elif strides[i] != rows * ld:
                ld = -1
                break
            rows *= size
    if ld is None:
        ld = shape[-1]
    if strides[-1] != 1 or ld < shape[-1]:
        raise ValueError(f"the rows of {name} must be dense and equally far apart (strides {strides})")
    if (ld * t.element_size()) % 16:
        raise ValueError(f"the rows of {name} must lie on 16-byte boundaries (row stride {ld})")
    return ld


def _first(t) -> Dtype:
    """The io dtype of a call's first activation, whose sizes have to fit the library's 31-bit counts."""
    if t.numel() >> 31 and max(t.shape) >> 31:
        raise GretError(_g.Status.ERR_UNSUPPORTED, f"sizes {tuple(t.shape)}")
    return _io_of(t)


def _longest(max_seqlen, T) -> int:
    """The longest sequence of T packed rows, given an upper bound."""
    return max(min(int(max_seqlen), T), 0)


def _dense(t, name, dtype, shape, dev):
    """``_check``, quick where all is well."""
    if not (t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous() and t.is_cuda):
        _check(t, name, dtype, shape, dev)


def _opt(t, name, dtype, shape, dev):
    if t is not None:
        _dense(t, name, dtype, shape, dev)


def _act(activation) -> Activation:
    if activation in (None, "none"):
        return Activation.NONE
    if activation == "swish":
        return Activation.SWISH
    raise ValueError(f"activation is 'swish' or 'none', got {activation!r}")


class _Here:
    """A call on the current stream of the current device: nothing to switch."""
    __slots__ = ("handle",)

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self):
        return self.handle

    def __exit__(self, *exc):
        return False


@contextlib.contextmanager
def _elsewhere(dev, stream):
    torch = _g._torch()
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        yield stream.cuda_stream


def _on(dev, stream):
    """The device and stream a call runs on, made current while it allocates and launches; gives the raw stream."""
    torch = _g._torch()
    if stream is None:
        if torch.cuda.current_device() == dev.index:
            return _Here(torch._C._cuda_getCurrentRawStream(dev.index))
        stream = torch.cuda.current_stream(dev)
    elif stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, expected {dev}")
    return _elsewhere(dev, stream)


def _like(t):
    """A dense tensor of t's shape and type (torch's quicker allocation where t is dense itself)."""
    return _g._torch().empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _raise_if(status, what):
    if status:
        raise GretError(status, what)


def _workspace(workspace, need, dev):
    """The caller's workspace when it is large enough, else one that belongs to the current stream."""
    if not need:
        return None
    if workspace is not None and workspace.numel() * workspace.element_size() >= need:
        if not workspace.is_cuda or workspace.device != dev:
            raise ValueError(f"the workspace is on {workspace.device}, expected {dev}")
        if not workspace.is_contiguous():
            raise ValueError("the workspace must be contiguous")
        return workspace
    return _g._torch().empty(need, dtype=_g._torch().uint8, device=dev)


def _conv_weights(w, bias, D, dev):
    torch = _g._torch()
    if w.dim() != 2:
        raise ValueError(f"w has shape {tuple(w.shape)}, expected ({D}, taps)")
    _dense(w, "w", torch.float32, (D, w.shape[1]), dev)
    _opt(bias, "bias", torch.float32, (D,), dev)
    return w.shape[1]


# ---------------------------------------------------------------- short convolution
def short_conv(x, w, bias=None, tail0=None, activation: Optional[str] = "swish", y=None, tail=None,
               want_tail: bool = True, stream=None):
    """Short causal convolution of prompts (gret_short_conv).

    x [B,N,D] bf16 or fp32; w [D,K] fp32, K of 2 to 4 (the last tap takes the token itself); bias [D] fp32 or None;
    tail0 [B,K-1,D], the last inputs of the piece before, or None.  Returns (y [B,N,D], tail [B,K-1,D] or None)."""
    B, N, D = x.shape
    dev, io = x.device, _first(x)
    ldx = _rows(x, "x", x.dtype, x.shape, dev)
    K = _conv_weights(w, bias, D, dev)
    _opt(tail0, "tail0", x.dtype, (B, K - 1, D), dev)
    _opt(y, "y", x.dtype, (B, N, D), dev)
    _opt(tail, "tail", x.dtype, (B, K - 1, D), dev)
    act = _act(activation)
    with _on(dev, stream) as st:
        if y is None:
            y = _like(x)
        if tail is None and want_tail:
            tail = x.new_empty((B, K - 1, D))
        _raise_if(_lib().gret_short_conv(_ptr(x), ldx, _ptr(w), _ptr(bias), _ptr(tail0), _ptr(y), _ptr(tail), B, N, D, K, io,
                                  act, st), "gret_short_conv")
    return y, tail


def short_conv_varlen(x, w, bias, cu_seqlens, max_seqlen: int, tail0=None, activation: Optional[str] = "swish",
                      y=None, tail=None, want_tail: bool = True, stream=None):
    """Short causal convolution of a packed batch (gret_short_conv_varlen).

    x [T,D]; cu_seqlens int32 [S+1] on the device; tail0 [S,K-1,D] or None; the rest as for ``short_conv``.
    Returns (y [T,D], tail [S,K-1,D] or None)."""
    torch = _g._torch()
    T, D = x.shape
    S, longest = cu_seqlens.numel() - 1, _longest(max_seqlen, T)
    dev, io = x.device, _first(x)
    ldx = _rows(x, "x", x.dtype, x.shape, dev)
    K = _conv_weights(w, bias, D, dev)
    _dense(cu_seqlens, "cu_seqlens", torch.int32, (S + 1,), dev)
    _opt(tail0, "tail0", x.dtype, (S, K - 1, D), dev)
    _opt(y, "y", x.dtype, (T, D), dev)
    _opt(tail, "tail", x.dtype, (S, K - 1, D), dev)
    act = _act(activation)
    with _on(dev, stream) as st:
        if y is None:
            y = _like(x)
        if tail is None and want_tail:
            tail = x.new_empty((S, K - 1, D))
        _raise_if(_lib().gret_short_conv_varlen(_ptr(x), ldx, _ptr(w), _ptr(bias), _ptr(tail0), _ptr(cu_seqlens), S, T,
                                         longest, _ptr(y), _ptr(tail), D, K, io, act, st),
                  "gret_short_conv_varlen")
    return y, tail


def short_conv_step(x, w, bias, tail, activation: Optional[str] = "swish", y=None, tail_out=None, stream=None):
    """One token per sequence (gret_short_conv_step): x [S,D], tail [S,K-1,D].

    The new tail goes to ``tail_out``, or over ``tail`` where that is None.  Returns (y [S,D], the new tail)."""
    S, D = x.shape
    dev, io = x.device, _first(x)
    ldx = _rows(x, "x", x.dtype, x.shape, dev)
    K = _conv_weights(w, bias, D, dev)
    _dense(tail, "tail", x.dtype, (S, K - 1, D), dev)
    _opt(tail_out, "tail_out", x.dtype, (S, K - 1, D), dev)
    _opt(y, "y", x.dtype, (S, D), dev)
    act = _act(activation)
    if tail_out is None:
        tail_out = tail
    with _on(dev, stream) as st:
        if y is None:
            y = _like(x)
        _raise_if(_lib().gret_short_conv_step(_ptr(x), ldx, _ptr(w), _ptr(bias), _ptr(tail), _ptr(tail_out), _ptr(y), S, D, K,
                                       io, act, st), "gret_short_conv_step")
    return y, tail_out


def short_conv_backward(x, w, bias, dy, tail0=None, dtail=None, activation: Optional[str] = "swish", workspace=None,
                        stream=None):
    """Gradients of <y, dy> + <tail, dtail> (gret_short_conv_backward).

    Shapes as for ``short_conv``.  Returns a dict: dx (x's dtype), dw [D,K] fp32, dbias [D] fp32 (None without a bias),
    dtail0 (x's dtype; None without a tail0)."""
    torch = _g._torch()
    B, N, D = x.shape
    dev, io = x.device, _first(x)
    ldx = _rows(x, "x", x.dtype, x.shape, dev)
    K = _conv_weights(w, bias, D, dev)
    _dense(dy, "dy", x.dtype, (B, N, D), dev)
    _opt(tail0, "tail0", x.dtype, (B, K - 1, D), dev)
    _opt(dtail, "dtail", x.dtype, (B, K - 1, D), dev)
    act = _act(activation)
    with _on(dev, stream) as st:
        g = {"dx": _like(x), "dw": torch.empty_like(w),
             "dbias": None if bias is None else torch.empty_like(bias),
             "dtail0": None if tail0 is None else torch.empty_like(tail0)}
        need = gret_short_conv_backward_workspace_size(B, N, D, K, io)
        workspace = _workspace(workspace, need, dev)
        _raise_if(_lib().gret_short_conv_backward(_ptr(x), ldx, _ptr(w), _ptr(bias), _ptr(tail0), _ptr(dy), _ptr(dtail),
                                           _ptr(g["dx"]), _ptr(g["dw"]), _ptr(g["dbias"]), _ptr(g["dtail0"]), B, N, D,
                                           K, io, act, _ptr(workspace), need, st), "gret_short_conv_backward")
    return g


# ---------------------------------------------------------------- selective scan
def _scan_inputs(u, dt, A, B, C, skip, z, dt_bias):
    """Check the scan's inputs; returns (device, io dtype, D, n, row strides)."""
    torch = _g._torch()
    dev, D, rows = u.device, u.shape[-1], u.shape[:-1]
    if A.dim() != 2:
        raise ValueError(f"A has shape {tuple(A.shape)}, expected ({D}, states)")
    n = A.shape[1]
    io = _first(u)
    ld = (_rows(u, "u", u.dtype, u.shape, dev), _rows(dt, "dt", u.dtype, u.shape, dev),
          _rows(B, "B", u.dtype, rows + (n,), dev), _rows(C, "C", u.dtype, rows + (n,), dev),
          _rows(z, "z", u.dtype, u.shape, dev) if z is not None else 0)
    _dense(A, "A", torch.float32, (D, n), dev)
    _opt(skip, "skip", torch.float32, (D,), dev)
    _opt(dt_bias, "dt_bias", torch.float32, (D,), dev)
    return dev, io, D, n, ld


def selective_scan(u, dt, A, B, C, skip=None, z=None, dt_bias=None, h0=None, o=None, h_final=None,
                   want_state: bool = True, workspace=None, stream=None):
    """Selective state space scan of prompts (gret_selective_scan).

    u, dt, z [b,N,D] and B, C [b,N,n] in bf16 or fp32; A [D,n], skip [D], dt_bias [D] fp32; h0 [b,D,n] fp32 or None;
    skip, z and dt_bias may be None.  Returns (o [b,N,D], h_final [b,D,n] fp32 or None)."""
    torch = _g._torch()
    b, N, D = u.shape
    dev, io, D, n, ld = _scan_inputs(u, dt, A, B, C, skip, z, dt_bias)
    _opt(h0, "h0", torch.float32, (b, D, n), dev)
    _opt(o, "o", u.dtype, (b, N, D), dev)
    _opt(h_final, "h_final", torch.float32, (b, D, n), dev)
    with _on(dev, stream) as st:
        if o is None:
            o = _like(u)
        if h_final is None and want_state:
            h_final = torch.empty((b, D, n), dtype=torch.float32, device=dev)
        need = gret_selective_scan_workspace_size(b, N, D, n, io)
        workspace = _workspace(workspace, need, dev)
        _raise_if(_lib().gret_selective_scan(_ptr(u), ld[0], _ptr(dt), ld[1], _ptr(A), _ptr(B), ld[2], _ptr(C), ld[3],
                                      _ptr(skip), _ptr(z), ld[4], _ptr(dt_bias), _ptr(h0), _ptr(o), _ptr(h_final), b, N,
                                      D, n, io, _ptr(workspace), need, st), "gret_selective_scan")
    return o, h_final


def selective_scan_varlen(u, dt, A, B, C, cu_seqlens, max_seqlen: int, skip=None, z=None, dt_bias=None, h0=None,
                          o=None, h_final=None, want_state: bool = True, workspace=None, stream=None):
    """Selective state space scan of a packed batch (gret_selective_scan_varlen).

    u, dt, z [T,D]; B, C [T,n]; cu_seqlens int32 [S+1] on the device; h0 [S,D,n] fp32 or None; the rest as for
    ``selective_scan``.  Returns (o [T,D], h_final [S,D,n] fp32 or None)."""
    torch = _g._torch()
    T, D = u.shape
    S, longest = cu_seqlens.numel() - 1, _longest(max_seqlen, T)
    dev, io, D, n, ld = _scan_inputs(u, dt, A, B, C, skip, z, dt_bias)
    _dense(cu_seqlens, "cu_seqlens", torch.int32, (S + 1,), dev)
    _opt(h0, "h0", torch.float32, (S, D, n), dev)
    _opt(o, "o", u.dtype, (T, D), dev)
    _opt(h_final, "h_final", torch.float32, (S, D, n), dev)
    with _on(dev, stream) as st:
        if o is None:
            o = _like(u)
        if h_final is None and want_state:
            h_final = torch.empty((S, D, n), dtype=torch.float32, device=dev)
        need = gret_selective_scan_varlen_workspace_size(S, T, longest, D, n, io)
        workspace = _workspace(workspace, need, dev)
        _raise_if(_lib().gret_selective_scan_varlen(_ptr(u), ld[0], _ptr(dt), ld[1], _ptr(A), _ptr(B), ld[2], _ptr(C), ld[3],
                                             _ptr(skip), _ptr(z), ld[4], _ptr(dt_bias), _ptr(h0), _ptr(cu_seqlens), S,
                                             T, longest, _ptr(o), _ptr(h_final), D, n, io, _ptr(workspace),
                                             need, st), "gret_selective_scan_varlen")
    return o, h_final


def selective_step(u, dt, A, B, C, h, skip=None, z=None, dt_bias=None, h_out=None, o=None, stream=None):
    """One token per sequence (gret_selective_step): u, dt, z [S,D]; B, C [S,n]; h [S,D,n] fp32.

    The new state goes to ``h_out``, or over ``h`` where that is None.  Returns (o [S,D], the new state)."""
    torch = _g._torch()
    S, D = u.shape
    dev, io, D, n, ld = _scan_inputs(u, dt, A, B, C, skip, z, dt_bias)
    _dense(h, "h", torch.float32, (S, D, n), dev)
    _opt(h_out, "h_out", torch.float32, (S, D, n), dev)
    _opt(o, "o", u.dtype, (S, D), dev)
    if h_out is None:
        h_out = h
    with _on(dev, stream) as st:
        if o is None:
            o = _like(u)
        _raise_if(_lib().gret_selective_step(_ptr(u), ld[0], _ptr(dt), ld[1], _ptr(A), _ptr(B), ld[2], _ptr(C), ld[3],
                                      _ptr(skip), _ptr(z), ld[4], _ptr(dt_bias), _ptr(h), _ptr(h_out), _ptr(o), S, D, n,
                                      io, st), "gret_selective_step")
    return o, h_out


def selective_scan_backward(u, dt, A, B, C, do, skip=None, z=None, dt_bias=None, h0=None, dh_final=None,
                            want_dh0: bool = False, workspace=None, stream=None):
    """Gradients of <o, do> + <h_final, dh_final> (gret_selective_scan_backward).

    Shapes as for ``selective_scan``.  Returns a dict: du, ddt, dB, dC, dz (u's dtype) and dA, dskip, ddt_bias, dh0
    (fp32); dz, dskip and ddt_bias are None where their input is, dh0 without h0 unless ``want_dh0``."""
    torch = _g._torch()
    b, N, D = u.shape
    dev, io, D, n, ld = _scan_inputs(u, dt, A, B, C, skip, z, dt_bias)
    _dense(do, "do", u.dtype, (b, N, D), dev)
    _opt(h0, "h0", torch.float32, (b, D, n), dev)
    _opt(dh_final, "dh_final", torch.float32, (b, D, n), dev)
    with _on(dev, stream) as st:
        g = {"du": _like(u), "ddt": _like(dt), "dA": torch.empty_like(A), "dB": _like(B), "dC": _like(C),
             "dz": None if z is None else _like(z), "dskip": None if skip is None else torch.empty_like(skip),
             "ddt_bias": None if dt_bias is None else torch.empty_like(dt_bias),
             "dh0": torch.empty((b, D, n), dtype=torch.float32, device=dev) if h0 is not None or want_dh0 else None}
        need = gret_selective_scan_backward_workspace_size(b, N, D, n, io)
        workspace = _workspace(workspace, need, dev)
        _raise_if(_lib().gret_selective_scan_backward(_ptr(u), ld[0], _ptr(dt), ld[1], _ptr(A), _ptr(B), ld[2], _ptr(C), ld[3],
                                               _ptr(skip), _ptr(z), ld[4], _ptr(dt_bias), _ptr(h0), _ptr(do),
                                               _ptr(dh_final), _ptr(g["du"]), _ptr(g["ddt"]), _ptr(g["dA"]),
                                               _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dskip"]), _ptr(g["dz"]),
                                               _ptr(g["ddt_bias"]), _ptr(g["dh0"]), b, N, D, n, io, _ptr(workspace),
                                               need, st), "gret_selective_scan_backward")
    return g


# ---------------------------------------------------------------- residual norm
def _norm_inputs(x, y, gate, scale, w_post, w_next, n=None):
    """Check the norm's inputs; returns (device, stream dtype, io dtype, T, D, row strides).  Without y an fp32 stream's n
    may be bf16: its given buffer says so."""
    torch = _g._torch()
    shape = x.shape
    dev, D = x.device, shape[-1]
    if y is None:
        if gate is not None or scale is not None or w_post is not None:
            raise ValueError("gate, scale and w_post go with y")
        if w_next is None:
            raise ValueError("y or w_next is required")
        like = x if n is None else n
    else:
        like = y
    stream_dtype = io = _first(x)
    if like.dtype is not x.dtype:
        io = _io_of(like)
        if io == Dtype.F32:
            raise TypeError(f"x has dtype {x.dtype}, expected {like.dtype} or torch.float32")
    ld = (_rows(x, "x", x.dtype, shape, dev),
          _rows(y, "y", y.dtype, shape, dev) if y is not None else 0,
          _rows(gate, "gate", like.dtype, shape, dev) if gate is not None else 0)
    par = (D,)
    _opt(scale, "scale", torch.float32, par, dev)
    _opt(w_post, "w_post", torch.float32, par, dev)
    _opt(w_next, "w_next", torch.float32, par, dev)
    return dev, stream_dtype, io, x.numel() // D if D else 0, D, ld


def residual_norm(x, y=None, gate=None, scale=None, w_post=None, w_next=None, eps: float = 1e-5, r=None, n=None,
                  stream=None):
    """A block's output into the residual stream and the norm before the next block (gret_residual_norm).

    r = x + scale * rms(y) * w_post * swish(gate);  n = rms(r) * w_next, with rms(v) = v / sqrt(mean(v^2) + eps).
    x [...,D] bf16 or fp32 (the residual stream); y, gate [...,D] in x's dtype, or bf16 beside an fp32 x; scale, w_post,
    w_next [D] fp32.  Each of gate, scale, w_post and w_next may be None; without y the call is the norm alone.
    Returns (r in x's dtype, n in y's dtype or None); ``r=x`` updates the stream in place.  Without y, r is x itself and n
    has x's dtype unless a buffer for it is given (bf16 beside an fp32 stream)."""
    torch = _g._torch()
    dev, sd, io, T, D, ld = _norm_inputs(x, y, gate, scale, w_post, w_next, n)
    io_torch = torch.float32 if io == Dtype.F32 else torch.bfloat16
    _opt(r, "r", x.dtype, x.shape, dev)
    _opt(n, "n", io_torch, x.shape, dev)
    if n is not None and w_next is None:
        raise ValueError("n goes with w_next")
    if r is not None and y is None and r.data_ptr() != x.data_ptr():
        raise ValueError("r goes with y")
    with _on(dev, stream) as st:
        if y is None:
            r = x
        elif r is None:
            r = _like(x)
        if n is None and w_next is not None:
            n = _like(x) if x.dtype == io_torch else x.new_empty(x.shape, dtype=io_torch)
        _raise_if(_lib().gret_residual_norm(_ptr(x), ld[0], _ptr(y), ld[1], _ptr(gate), ld[2], _ptr(scale), _ptr(w_post),
                                     _ptr(w_next), _ptr(r) if y is not None else None, _ptr(n), T, D, float(eps), sd,
                                     io, st), "gret_residual_norm")
    return r, n


def residual_norm_backward(x, y=None, dr=None, dn=None, gate=None, scale=None, w_post=None, w_next=None,
                           eps: float = 1e-5, workspace=None, stream=None):
    """Gradients of <r, dr> + <n, dn> (gret_residual_norm_backward).

    Shapes as for ``residual_norm``; dr has x's dtype and may be None, dn goes with w_next.  Returns a dict: dx (x's
    dtype), dy, dgate (y's dtype), dscale, dw_post, dw_next (fp32), None where the input is None."""
    torch = _g._torch()
    if (dn is None) != (w_next is None):
        raise ValueError("dn goes with w_next")
    if dr is None and dn is None:
        raise ValueError("dr or dn is required")
    dev, sd, io, T, D, ld = _norm_inputs(x, y, gate, scale, w_post, w_next, dn)
    io_torch = torch.float32 if io == Dtype.F32 else torch.bfloat16
    _opt(dr, "dr", x.dtype, x.shape, dev)
    _opt(dn, "dn", io_torch, x.shape, dev)
    with _on(dev, stream) as st:
        row = lambda t: None if t is None else _like(t)  # noqa: E731
        par = lambda w: None if w is None else torch.empty_like(w)  # noqa: E731
        g = {"dx": _like(x), "dy": row(y), "dgate": row(gate), "dscale": par(scale), "dw_post": par(w_post),
             "dw_next": par(w_next)}
        need = gret_residual_norm_backward_workspace_size(T, D)
        workspace = _workspace(workspace, need, dev)
        _raise_if(_lib().gret_residual_norm_backward(_ptr(x), ld[0], _ptr(y), ld[1], _ptr(gate), ld[2], _ptr(scale),
                                              _ptr(w_post), _ptr(w_next), _ptr(dr), _ptr(dn), _ptr(g["dx"]),
                                              _ptr(g["dy"]), _ptr(g["dgate"]), _ptr(g["dscale"]), _ptr(g["dw_post"]),
                                              _ptr(g["dw_next"]), T, D, float(eps), sd, io, _ptr(workspace), need, st),
                  "gret_residual_norm_backward")
    return g
