"""Python entry points of what stands around and beside the TTT scans: the
RMS norm, the input projection from 8-bit operands, the short causal
convolution and the selective state space scan.  As ops.py: names of the C
ABI (include/ttt.h holds the semantics), arguments checked and marshalled,
outputs and workspaces allocated with torch, kernels launched asynchronously
on the current stream of the tensors' device.  With ``stream`` the call is
made under that stream: its outputs and workspace belong to it too."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from . import _lib
from .ops import HEAD_DIM, _dev_tensor

__all__ = ["ttt_rms_norm_forward", "ttt_rms_norm_forward_f8", "ttt_rms_norm_backward",
           "ttt_input_projection_f8", "ttt_conv_forward", "ttt_conv_decode_step",
           "ttt_conv_backward", "ttt_ssm_forward", "ttt_ssm_decode_step", "ttt_ssm_backward"]

F8 = torch.float8_e4m3fn

# the current device, and the handle of its current stream without a Stream
# object around it, where this torch has them directly
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)


# The host side of a call is what a launch of a few microseconds waits for, so
# a good argument costs one line of comparisons; only one that fails them goes
# through _dev_tensor, which finds out why and raises.

def _check(name, t, dtype, shape, device):
    try:
        if (t.dtype is dtype and t.shape == shape and t.device == device
                and t.is_contiguous()):
            return t
    except AttributeError:
        pass
    return _dev_tensor(name, t, dtype, shape, device)


def _io(name, t) -> int:
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous()):
        _dev_tensor(name, t)
    if t.dtype is torch.bfloat16:
        return _lib.TTT_BF16
    if t.dtype is torch.float32:
        return _lib.TTT_F32
    raise ValueError("%s must be bfloat16 or float32 (got %s)" % (name, t.dtype))


def _optional(name, t, dtype, shape, device):
    if t is not None:
        _check(name, t, dtype, shape, device)


def _given(name, t, shape, dtype, device):
    """An output: the caller's tensor, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _check(name, t, dtype, shape, device)


def _like(name, t, x):
    """As _given, of x's shape and type."""
    return torch.empty_like(x) if t is None else _check(name, t, x.dtype, x.shape, x.device)


def _workspace(ws, need, device):
    if ws is None:
        return torch.empty(need or 1, dtype=torch.uint8, device=device)
    return _dev_tensor("workspace", ws, torch.uint8, device=device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _on_stream(func):
    @functools.wraps(func)
    def call(*args, stream=None, **kw):
        if stream is None:
            return func(*args, **kw)
        data = args[0] if args else kw.get("x", kw.get("r"))
        if isinstance(data, torch.Tensor) and data.device != stream.device:
            raise ValueError("stream must be on %s, like the data (got %s)"
                             % (data.device, stream.device))
        with torch.cuda.stream(stream):
            return func(*args, **kw)
    return call


def _call(func, device, *args):
    """The library's function on the device's current stream; it launches on
    the current device."""
    index = device.index
    if index == _current_device():
        rc = getattr(_lib.lib(), func)(*args, _current_stream(index))
    else:
        with torch.cuda.device(device):
            rc = getattr(_lib.lib(), func)(*args, _current_stream(index))
    if rc:
        _lib.check(func, rc)


# ---- RMS norm ---------------------------------------------------------------

def _norm_args(x, weight, residual, res_out):
    io = _io("x", x)
    if x.dim() < 1:
        raise ValueError("x must be [..., width]")
    width = x.shape[-1]
    rows = x.numel() // width if width else 0
    dev = x.device
    _check("weight", weight, torch.float32, (width,), dev)
    _optional("residual", residual, x.dtype, x.shape, dev)
    if residual is None:
        if res_out is not None:
            raise ValueError("res_out is given without a residual")
    else:
        res_out = _like("res_out", res_out, x)
    return io, rows, width, res_out


@_on_stream
def ttt_rms_norm_forward(x: torch.Tensor, weight: torch.Tensor,
                         residual: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
                         y: Optional[torch.Tensor] = None,
                         res_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """RMS norm over the last dimension of x [..., width] (bf16 or fp32) after
    adding residual; returns (y, r) with r = x + residual in x's type, or None
    without a residual.  weight [width] fp32; width a multiple of 8.
    res_out: where to write r (may be residual itself)."""
    io, rows, width, res_out = _norm_args(x, weight, residual, res_out)
    y = _like("y", y, x)
    _call("ttt_rms_norm_forward", x.device, rows, width, io, float(eps), _ptr(x), _ptr(residual),
          _ptr(weight), _ptr(y), _ptr(res_out))
    return y, res_out


@_on_stream
def ttt_rms_norm_forward_f8(x: torch.Tensor, weight: torch.Tensor,
                            residual: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
                            y: Optional[torch.Tensor] = None,
                            scale: Optional[torch.Tensor] = None,
                            res_out: Optional[torch.Tensor] = None, stream=None
                            ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """ttt_rms_norm_forward with an 8-bit output: returns (y8 [..., width]
    float8_e4m3fn, scale [...] fp32, r); y8 * scale stands for the norm's
    output.  The x and x_scale of ttt_input_projection_f8."""
    io, rows, width, res_out = _norm_args(x, weight, residual, res_out)
    y = torch.empty_like(x, dtype=F8) if y is None else _check("y", y, F8, x.shape, x.device)
    scale = _given("scale", scale, x.shape[:-1], torch.float32, x.device)
    _call("ttt_rms_norm_forward_f8", x.device, rows, width, io, float(eps), _ptr(x),
          _ptr(residual), _ptr(weight), _ptr(y), _ptr(scale), _ptr(res_out))
    return y, scale, res_out


@_on_stream
def ttt_rms_norm_backward(r: torch.Tensor, weight: torch.Tensor, dy: torch.Tensor,
                          dr: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
                          dx: Optional[torch.Tensor] = None,
                          dweight: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None
                          ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Gradients of the RMS norm; returns (dx, dweight).  r: the norm's input
    (the forward's r, or x where there was no residual); dy: cotangent of y;
    dr: cotangent of r past the norm, or None.  dx is the gradient of x and of
    the residual alike.  workspace: a uint8 GPU tensor of at least
    ttt_rms_norm_backward_workspace_bytes bytes to use instead of a fresh one."""
    io = _io("r", r)
    if r.dim() < 1:
        raise ValueError("r must be [..., width]")
    dev, width = r.device, r.shape[-1]
    rows = r.numel() // width if width else 0
    _check("weight", weight, torch.float32, (width,), dev)
    _check("dy", dy, r.dtype, r.shape, dev)
    _optional("dr", dr, r.dtype, r.shape, dev)
    dx = _like("dx", dx, r)
    dweight = _given("dweight", dweight, (width,), torch.float32, dev)
    need = int(_lib.lib().ttt_rms_norm_backward_workspace_bytes(rows, width))
    workspace = _workspace(workspace, need, dev)
    _call("ttt_rms_norm_backward", dev, rows, width, io, float(eps), _ptr(r), _ptr(weight),
          _ptr(dy), _ptr(dr), _ptr(dx), _ptr(dweight), _ptr(workspace), workspace.numel())
    return dx, dweight


# ---- input projection from 8-bit operands -----------------------------------

@_on_stream
def ttt_input_projection_f8(x: torch.Tensor, x_scale: torch.Tensor, w_in: torch.Tensor,
                            w_scale: torch.Tensor, b_eta: torch.Tensor, *, heads: int,
                            eta_base: float, head_dim: int = HEAD_DIM, out=None, stream=None
                            ) -> Tuple[torch.Tensor, ...]:
    """ttt_input_projection from 8-bit operands: x [B,T,D] and w_in
    [3*H*d + H, D] float8_e4m3fn with x_scale [B,T] and w_scale [3*H*d + H]
    fp32, a scale per row (x and x_scale as ttt_rms_norm_forward_f8 gives
    them; a weight's scale is its row's largest magnitude / 448).  Returns
    (q, k, v, eta): q, k, v [B,H,T,d] bf16, eta [B,H,T] fp32.  out: an
    optional tuple of four tensors to write instead."""
    if not (isinstance(x, torch.Tensor) and x.dtype is F8 and x.is_cuda and x.is_contiguous()):
        _dev_tensor("x", x, F8)
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    B, T, D = x.shape
    H, d, dev = int(heads), int(head_dim), x.device
    n = 3 * H * d + H
    _check("x_scale", x_scale, torch.float32, (B, T), dev)
    _check("w_in", w_in, F8, (n, D), dev)
    _check("w_scale", w_scale, torch.float32, (n,), dev)
    _check("b_eta", b_eta, torch.float32, (H,), dev)
    if out is None:
        q = torch.empty((B, H, T, d), dtype=torch.bfloat16, device=dev)
        k, v = torch.empty_like(q), torch.empty_like(q)
        eta = torch.empty((B, H, T), dtype=torch.float32, device=dev)
    else:
        q, k, v, eta = out
        for name, t in (("q", q), ("k", k), ("v", v)):
            _check(name, t, torch.bfloat16, (B, H, T, d), dev)
        _check("eta", eta, torch.float32, (B, H, T), dev)
    p = _lib.TTTParams(B, H, T, d, 16, _lib.TTT_BF16, 0, 0.0, 0)
    _call("ttt_input_projection_f8", dev, ctypes.byref(p), D, _ptr(x), _ptr(x_scale), _ptr(w_in),
          _ptr(w_scale), _ptr(b_eta), float(eta_base), _ptr(q), _ptr(k), _ptr(v), _ptr(eta))
    return q, k, v, eta


# ---- short causal convolution -----------------------------------------------

def _conv_args(x, w, bias, dims):
    io = _io("x", x)
    if x.dim() != dims:
        raise ValueError("x must be %s" % ("[B, H, T, d]" if dims == 4 else "[B, H, d]"))
    B, H, d = x.shape[0], x.shape[1], x.shape[-1]
    T = x.shape[2] if dims == 4 else 1
    dev = x.device
    if not (isinstance(w, torch.Tensor) and w.dtype is torch.float32 and w.device == dev
            and w.is_contiguous()):
        _dev_tensor("w", w, torch.float32, device=dev)
    if w.dim() != 3 or w.shape[0] != H or w.shape[2] != d:
        raise ValueError("w must have shape (%d, taps, %d) (got %s)" % (H, d, tuple(w.shape)))
    _optional("bias", bias, torch.float32, (H, d), dev)
    taps = w.shape[1]
    return _lib.TTTParams(B, H, T, d, 16, io, 0, 0.0, 0), taps, (B, H, max(taps - 1, 0), d)


@_on_stream
def ttt_conv_forward(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
                     state0: Optional[torch.Tensor] = None, silu: bool = True,
                     y: Optional[torch.Tensor] = None, state_out: Optional[torch.Tensor] = None,
                     return_state: bool = False, stream=None
                     ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Short causal convolution of x [B,H,T,d] (bf16 or fp32) along T with one
    filter of 2 to 4 taps per head and feature, w [H,taps,d] (the last tap
    meets the token itself) and bias [H,d] fp32, then SiLU if silu; returns
    (y, the last taps-1 inputs [B,H,taps-1,d] or None).  state0: the inputs
    before the first token (zeros if None)."""
    p, taps, tail = _conv_args(x, w, bias, 4)
    _optional("state0", state0, x.dtype, tail, x.device)
    y = _like("y", y, x)
    if state_out is not None or return_state:
        state_out = _given("state_out", state_out, tail, x.dtype, x.device)
    _call("ttt_conv_forward", x.device, ctypes.byref(p), taps, _lib.TTT_CONV_SILU if silu else 0,
          _ptr(x), _ptr(w), _ptr(bias), _ptr(state0), _ptr(y), _ptr(state_out))
    return y, state_out


@_on_stream
def ttt_conv_decode_step(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor],
                         state: torch.Tensor, *, silu: bool = True,
                         y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token of ttt_conv_forward: x [B,H,d]; state [B,H,taps-1,d] in x's
    type holds the inputs before it and is moved on in place.  Returns y."""
    p, taps, tail = _conv_args(x, w, bias, 3)
    _check("state", state, x.dtype, tail, x.device)
    y = _like("y", y, x)
    _call("ttt_conv_decode_step", x.device, ctypes.byref(p), taps,
          _lib.TTT_CONV_SILU if silu else 0, _ptr(x), _ptr(w), _ptr(bias), _ptr(state), _ptr(y))
    return y


@_on_stream
def ttt_conv_backward(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor],
                      dy: torch.Tensor, *, state0: Optional[torch.Tensor] = None,
                      dstate: Optional[torch.Tensor] = None, silu: bool = True,
                      workspace: Optional[torch.Tensor] = None, stream=None
                      ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor,
                                 Optional[torch.Tensor]]:
    """Gradients of ttt_conv_forward; returns (dx, dw, dbias, dstate0), the
    last None without a state0.  dy: cotangent of y; dstate: of the final
    state, or None.  workspace: a uint8 GPU tensor of at least
    ttt_conv_backward_workspace_bytes bytes to use instead of a fresh one."""
    p, taps, tail = _conv_args(x, w, bias, 4)
    dev = x.device
    _optional("state0", state0, x.dtype, tail, dev)
    _check("dy", dy, x.dtype, x.shape, dev)
    _optional("dstate", dstate, x.dtype, tail, dev)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    dbias = torch.empty((w.shape[0], w.shape[2]), dtype=torch.float32, device=dev)
    dstate0 = None if state0 is None else torch.empty_like(state0)
    need = int(_lib.lib().ttt_conv_backward_workspace_bytes(ctypes.byref(p), taps))
    workspace = _workspace(workspace, need, dev)
    _call("ttt_conv_backward", dev, ctypes.byref(p), taps, _lib.TTT_CONV_SILU if silu else 0,
          _ptr(x), _ptr(w), _ptr(bias), _ptr(state0), _ptr(dy), _ptr(dstate), _ptr(dx), _ptr(dw),
          _ptr(dbias), _ptr(dstate0), _ptr(workspace), workspace.numel())
    return dx, dw, dbias, dstate0


# ---- selective state space scan ---------------------------------------------

def _ssm_args(x, dt, a, b, c, d_skip, dims):
    io = _io("x", x)
    if x.dim() != dims:
        raise ValueError("x must be %s" % ("[B, H, T, d]" if dims == 4 else "[B, H, d]"))
    B, H, d = x.shape[0], x.shape[1], x.shape[-1]
    t = x.shape[2:-1]
    dev = x.device
    _check("dt", dt, torch.float32, (B, H) + tuple(t), dev)
    _check("a", a, torch.float32, (H,), dev)
    if not (isinstance(b, torch.Tensor) and b.dtype is x.dtype and b.device == dev
            and b.is_contiguous()):
        _dev_tensor("b", b, x.dtype, device=dev)
    if b.dim() != dims or b.shape[0] != B or b.shape[2:-1] != t:
        raise ValueError("b must be [B, groups, T, N] beside x (got %s)" % (tuple(b.shape),))
    _check("c", c, x.dtype, b.shape, dev)
    _optional("d_skip", d_skip, torch.float32, (H,), dev)
    G, N = b.shape[1], b.shape[-1]
    p = _lib.TTTParams(B, H, t[0] if dims == 4 else 1, d, 16, io, 0, 0.0, 0)
    return p, G, N, (B, H, N, d)


@_on_stream
def ttt_ssm_forward(x: torch.Tensor, dt: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                    c: torch.Tensor, d_skip: Optional[torch.Tensor] = None, *,
                    state0: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                    state_out: Optional[torch.Tensor] = None, return_state: bool = True,
                    workspace: Optional[torch.Tensor] = None, stream=None
                    ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Selective state space scan: with S_t = exp(a dt_t) S_{t-1} + dt_t b_t^T x_t,
    returns (y [B,H,T,d], y_t = c_t S_t + d_skip x_t, and the final state
    [B,H,N,d] fp32 or None).  x [B,H,T,d] and b, c [B,G,T,N] (G dividing H;
    N = 32, 64 or 128) bf16 or fp32; dt [B,H,T], a [H], d_skip [H] fp32;
    state0 [B,H,N,d] fp32 (zeros if None; state_out may be the same tensor).
    q, k, v and eta of ttt_input_projection fit as c, b, x and dt.
    workspace: a uint8 GPU tensor of at least ttt_ssm_forward_workspace_bytes
    bytes to use instead of a fresh one."""
    p, G, N, state = _ssm_args(x, dt, a, b, c, d_skip, 4)
    dev = x.device
    _optional("state0", state0, torch.float32, state, dev)
    y = _like("y", y, x)
    if state_out is not None or return_state:
        state_out = _given("state_out", state_out, state, torch.float32, dev)
    if workspace is None:
        need = int(_lib.lib().ttt_ssm_forward_workspace_bytes(ctypes.byref(p), G, N))
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    else:
        _dev_tensor("workspace", workspace, torch.uint8, device=dev)
    _call("ttt_ssm_forward", dev, ctypes.byref(p), G, N, _ptr(x), _ptr(dt), _ptr(a), _ptr(b),
          _ptr(c), _ptr(d_skip), _ptr(state0), _ptr(y), _ptr(state_out), _ptr(workspace),
          0 if workspace is None else workspace.numel())
    return y, state_out


@_on_stream
def ttt_ssm_decode_step(x: torch.Tensor, dt: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                        c: torch.Tensor, state: torch.Tensor,
                        d_skip: Optional[torch.Tensor] = None, *,
                        y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token of ttt_ssm_forward: x [B,H,d], dt [B,H], b, c [B,G,N]; state
    [B,H,N,d] fp32 is moved on in place.  Returns y [B,H,d]."""
    p, G, N, shape = _ssm_args(x, dt, a, b, c, d_skip, 3)
    _check("state", state, torch.float32, shape, x.device)
    y = _like("y", y, x)
    _call("ttt_ssm_decode_step", x.device, ctypes.byref(p), G, N, _ptr(x), _ptr(dt), _ptr(a),
          _ptr(b), _ptr(c), _ptr(d_skip), _ptr(state), _ptr(y))
    return y


@_on_stream
def ttt_ssm_backward(x: torch.Tensor, dt: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                     c: torch.Tensor, dy: torch.Tensor, d_skip: Optional[torch.Tensor] = None, *,
                     state0: Optional[torch.Tensor] = None,
                     dstate: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None
                     ) -> Tuple[Optional[torch.Tensor], ...]:
    """Gradients of ttt_ssm_forward; returns (dx, ddt, da, db, dc, dd, dstate0),
    dd None without a d_skip and dstate0 without a state0.  dy: cotangent of
    y; dstate: of the final state, or None.  Nothing of the forward call has
    to be kept.  workspace: a uint8 GPU tensor of at least
    ttt_ssm_backward_workspace_bytes bytes to use instead of a fresh one."""
    p, G, N, state = _ssm_args(x, dt, a, b, c, d_skip, 4)
    dev = x.device
    _check("dy", dy, x.dtype, x.shape, dev)
    _optional("state0", state0, torch.float32, state, dev)
    _optional("dstate", dstate, torch.float32, state, dev)
    dx, db, dc = torch.empty_like(x), torch.empty_like(b), torch.empty_like(c)
    ddt, da = torch.empty_like(dt), torch.empty_like(a)
    dd = None if d_skip is None else torch.empty_like(d_skip)
    dstate0 = None if state0 is None else torch.empty_like(state0)
    need = int(_lib.lib().ttt_ssm_backward_workspace_bytes(ctypes.byref(p), G, N))
    workspace = _workspace(workspace, need, dev)
    _call("ttt_ssm_backward", dev, ctypes.byref(p), G, N, _ptr(x), _ptr(dt), _ptr(a), _ptr(b),
          _ptr(c), _ptr(d_skip), _ptr(state0), _ptr(dy), _ptr(dstate), _ptr(dx), _ptr(ddt),
          _ptr(da), _ptr(db), _ptr(dc), _ptr(dd), _ptr(dstate0), _ptr(workspace),
          workspace.numel())
    return dx, ddt, da, db, dc, dd, dstate0
