"""Operators around the recurrence: short causal convolution, selective state
space scan, gated group norm.

A layer built on ``chunk_gated_delta_rule`` runs a short convolution on its
inputs and a gated norm on its outputs; ``selective_scan`` is the state space
recurrence that takes the delta rule's place in its sibling layer.  As in
``binding.py`` only arguments are marshalled here: every step of the
computation runs in the kernels behind ``include/gdn.h``, and there is no
fallback.

``short_conv``, ``selective_scan`` and ``gated_group_norm`` are differentiable;
``gdn_conv_step`` and ``gdn_scan_step`` advance a serving loop's state slots by
one token.  Inputs may be slices of a wider row (the output of one projection,
say): every entry of a token has to be contiguous, the distance between tokens
is free; for the scan's x, B and C, and the scan step's x, both start and distance
have to be whole 16 bytes (``.contiguous()`` makes them so).  Tensors of a call share one device, whose current stream it uses.

Calls can be captured into a graph, a backward pass too, provided that no eager
graph of the same leaves is alive then: autograd would synchronise with the
stream that one was made on, which a capture cannot.

Reverse mode only: forward-mode derivatives are refused.  No derivative passes
through the ``gdn_*`` calls; the two steps refuse inputs that ask for one.
Tracers that would record a call without its kernels are refused as well
(``torch.jit.trace`` keeps the three operators as one operation each, and a
function compiled by ``torch.compile`` leaves its graph for a call).
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from .binding import GDNError, _check, _compiling, _dtype_code, _gradient, _outside, _ptr, _vp, lib as _load

__all__ = ["short_conv", "selective_scan", "gated_group_norm", "gdn_conv_fwd", "gdn_conv_bwd", "gdn_conv_step",
           "gdn_scan_fwd", "gdn_scan_bwd", "gdn_scan_step", "gdn_norm_fwd", "gdn_norm_bwd"]

_NO_SWITCH = contextlib.nullcontext()
_i32, _i64, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class ConvArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("B", _i32), ("T", _i32), ("D", _i32), ("W", _i32), ("x", _vp), ("x_stride", _i64),
                ("w", _vp), ("bias", _vp), ("init", _vp), ("cu_seqlens", _vp), ("num_seqs", _i32), ("silu", _i32)]


class ConvFwdArgs(ctypes.Structure):
    _fields_ = [("a", ConvArgs), ("y", _vp), ("final_state", _vp)]


class ConvBwdArgs(ctypes.Structure):
    _fields_ = [("a", ConvArgs), ("dy", _vp), ("dfinal", _vp), ("dx", _vp), ("dw", _vp), ("dbias", _vp),
                ("dinit", _vp), ("workspace", _vp), ("workspace_bytes", _sz)]


class ConvStepArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("N", _i32), ("D", _i32), ("W", _i32), ("x", _vp), ("x_stride", _i64),
                ("state", _vp), ("state_idx", _vp), ("num_slots", _i32), ("w", _vp), ("bias", _vp), ("silu", _i32),
                ("y", _vp)]


class ScanArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("dt_dtype", _i32), ("B", _i32), ("T", _i32), ("H", _i32), ("G", _i32), ("Dk", _i32),
                ("Dv", _i32), ("x", _vp), ("dt", _vp), ("b", _vp), ("c", _vp), ("x_stride", _i64),
                ("dt_stride", _i64), ("b_stride", _i64), ("c_stride", _i64), ("A", _vp), ("D", _vp), ("dt_bias", _vp),
                ("dt_softplus", _i32), ("round_once", _i32), ("h0", _vp), ("cu_seqlens", _vp), ("cu_seqlens_host", _vp),
                ("num_seqs", _i32), ("seg_mode", _i32), ("workspace", _vp), ("workspace_bytes", _sz)]


class ScanFwdArgs(ctypes.Structure):
    _fields_ = [("a", ScanArgs), ("y", _vp), ("hT", _vp), ("h_save", _vp)]


class ScanBwdArgs(ctypes.Structure):
    _fields_ = [("a", ScanArgs), ("h_saved", _vp), ("dy", _vp), ("dhT", _vp), ("dx", _vp), ("ddt", _vp), ("db", _vp),
                ("dc", _vp), ("dA", _vp), ("dD", _vp), ("ddt_bias", _vp), ("dh0", _vp)]


class ScanStepArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("dt_dtype", _i32), ("N", _i32), ("H", _i32), ("G", _i32), ("Dk", _i32),
                ("Dv", _i32), ("x", _vp), ("dt", _vp), ("b", _vp), ("c", _vp), ("x_stride", _i64),
                ("dt_stride", _i64), ("b_stride", _i64), ("c_stride", _i64), ("A", _vp), ("D", _vp), ("dt_bias", _vp),
                ("dt_softplus", _i32), ("state", _vp), ("state_idx", _vp), ("num_slots", _i32), ("y", _vp)]


class NormArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("R", _i64), ("G", _i32), ("D", _i32), ("x", _vp), ("x_stride", _i64), ("z", _vp),
                ("z_stride", _i64), ("w", _vp), ("bias", _vp), ("shared", _i32), ("center", _i32),
                ("gate_first", _i32), ("eps", ctypes.c_float)]


class NormFwdArgs(ctypes.Structure):
    _fields_ = [("a", NormArgs), ("y", _vp)]


class NormBwdArgs(ctypes.Structure):
    _fields_ = [("a", NormArgs), ("dy", _vp), ("dx", _vp), ("dz", _vp), ("dw", _vp), ("dbias", _vp),
                ("workspace", _vp), ("workspace_bytes", _sz)]


_SIGNATURES = [("gdn_conv_fwd", ConvFwdArgs), ("gdn_conv_bwd", ConvBwdArgs), ("gdn_conv_step", ConvStepArgs),
               ("gdn_scan_fwd", ScanFwdArgs), ("gdn_scan_bwd", ScanBwdArgs), ("gdn_scan_step", ScanStepArgs),
               ("gdn_norm_fwd", NormFwdArgs), ("gdn_norm_bwd", NormBwdArgs)]
_SIZES = [("gdn_conv_bwd_workspace_size", ConvBwdArgs), ("gdn_scan_fwd_workspace_size", ScanFwdArgs),
          ("gdn_scan_bwd_workspace_size", ScanBwdArgs), ("gdn_scan_states_bytes", ScanArgs),
          ("gdn_norm_bwd_workspace_size", NormBwdArgs)]
_lib = None


def lib():
    """libgdn.so with these operators' signatures set."""
    global _lib
    if _lib is None:
        L = _load()
        for name, st in _SIGNATURES:
            getattr(L, name).argtypes, getattr(L, name).restype = [ctypes.POINTER(st), _vp], ctypes.c_int
        for name, st in _SIZES:
            getattr(L, name).argtypes, getattr(L, name).restype = [ctypes.POINTER(st)], _sz
        _lib = L
    return _lib


# ------------------------------------------------------------------ argument checks
def _t(name, t, shape, dtype, dev, optional=False):
    """A contiguous tensor of this shape, dtype and device (or None)."""
    if t is not None and t.shape == shape and t.dtype is dtype and t.device == dev and t.is_contiguous():
        return t
    if t is None:
        if optional:
            return None
        raise GDNError(f"{name} is missing")
    if tuple(t.shape) != tuple(shape):
        raise GDNError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != dtype:
        raise GDNError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise GDNError(f"{name} must be on {dev}, got {t.device}")
    if not t.is_contiguous():
        raise GDNError(f"{name} must be contiguous")
    return t


def _rows(name, t, shape, inner, dtype, dev):
    """The token stride of a tensor of this shape whose last `inner` dimensions are
    contiguous and whose tokens (the dimensions before) lie evenly apart."""
    if t.shape != shape:
        raise GDNError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype != dtype:
        raise GDNError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise GDNError(f"{name} must be on {dev}, got {t.device}")
    nd, width = t.dim(), 1
    if t.is_contiguous():
        for n in shape[nd - inner:]:
            width *= n
        return width
    for d in range(nd - 1, nd - 1 - inner, -1):
        if t.shape[d] != 1 and t.stride(d) != width:
            raise GDNError(f"the entries of one token of {name} must be contiguous")
        width *= t.shape[d]
    if t.numel() == 0:
        return width
    stride = span = None
    for d in range(nd - 1 - inner, -1, -1):
        if t.shape[d] == 1:
            continue
        if stride is None:
            stride, span = t.stride(d), t.stride(d) * t.shape[d]
        elif t.stride(d) != span:
            raise GDNError(f"the tokens of {name} must lie evenly apart")
        else:
            span *= t.shape[d]
    return width if stride is None else stride


def _past_32_bits():
    """The library's sizes are 32 bits; a larger one would be cut to its low half."""
    raise GDNError("problem too large: a size of 2^31 or more")


def _seqs(cu, cu_host, B, T, dev, need_host):
    """(device pointer, host tensor or None, number of sequences)."""
    if cu is None:
        if cu_host is not None:
            raise GDNError("cu_seqlens_host given without cu_seqlens")
        return None, None, B
    if B != 1:
        raise GDNError(f"cu_seqlens needs batch size 1 (packed sequences), got {B}")
    if cu.dim() != 1 or cu.numel() < 2:
        raise GDNError("cu_seqlens must be [N + 1]")
    _t("cu_seqlens", cu, cu.shape, torch.int32, dev)
    if cu_host is None and need_host:
        cu_host = cu.cpu()  # synchronises; pass the host copy to avoid it
    if cu_host is not None:
        cu_host = torch.as_tensor(cu_host, dtype=torch.int32).contiguous()
        if cu_host.is_cuda or cu_host.numel() != cu.numel():
            raise GDNError("cu_seqlens_host must be a host copy of cu_seqlens")
        if int(cu_host[0]) != 0 or int(cu_host[-1]) != T or bool((cu_host[1:] < cu_host[:-1]).any()):
            raise GDNError(f"cu_seqlens must rise from 0 to {T}")
    return cu, cu_host, cu.numel() - 1


def _own_lengths(cu_host):
    """A copy of the host lengths, kept for the backward pass: the caller may reuse its own."""
    return None if cu_host is None else torch.as_tensor(cu_host, dtype=torch.int32).clone()


def _workspace(nbytes, dev):
    if nbytes == 0:
        _check(1)
    return torch.empty(nbytes, dtype=torch.uint8, device=dev)


def _on_gpu(name, t):
    if not t.is_cuda:
        raise GDNError(f"{name} must be on a GPU")
    return t.device


def _on(dev):
    """The device made current for a call, where it is not already."""
    return _NO_SWITCH if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


# The current stream's handle; without building a Stream object around it (1.7 us,
# a fifth of a single-token call) where this PyTorch has the call for that.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


# The library's calls are invisible to tracers, which would keep the outputs' allocation
# and drop what fills them: such a call is refused.  An autograd function is one
# operation to torch.jit.trace, and its replay calls the library; what it runs inside
# is not traced.
_is_tracing, _dispatch_modes = torch._C._is_tracing, torch._C._len_torch_dispatch_stack
_MODES = [torch._C._TorchDispatchModeKey.PROXY, torch._C._TorchDispatchModeKey.FAKE]


def _refuse_traced():
    if _is_tracing() or any(torch._C._get_dispatch_mode(m) is not None for m in _MODES):
        raise GDNError("this call cannot be traced: the trace would not hold the library's kernels")


@contextlib.contextmanager
def _untraced():
    state = torch._C._get_tracing_state()
    torch._C._set_tracing_state(None)
    try:
        yield
    finally:
        torch._C._set_tracing_state(state)


def _as_one_op():
    """What the forward pass of an autograd function runs in."""
    return _untraced() if _is_tracing() else _NO_SWITCH


def _call(fn, args, dev):
    if _dispatch_modes() or _is_tracing():
        _refuse_traced()
    index = dev.index
    if torch.cuda.current_device() == index:
        status = fn(ctypes.byref(args), _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            status = fn(ctypes.byref(args), _raw_stream(index))
    if status:
        _check(status)


def _has_tangent(tensors):
    return any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def _wants_grad(*tensors):
    """Whether a call has to go through its autograd function (which has no forward mode and
    says so); one that has not calls the library directly."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    return _is_tracing() or forward_ad._current_level >= 0 and _has_tangent(tensors)


def _no_derivative(name, tensors):
    """Refuses a step whose derivative the caller expects: it advances its state in place and has none."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise GDNError(f"{name} has no gradient: call it under torch.no_grad()")
    if forward_ad._current_level >= 0 and _has_tangent(tensors):
        raise GDNError(f"{name} has no derivative")


# ------------------------------------------------------------------ short causal convolution
def _conv_args(x, weight, bias, silu, initial_state, cu_seqlens, cu_seqlens_host):
    if x.dim() != 3:
        raise GDNError("x must be [B, T, D]")
    if weight.dim() != 2:
        raise GDNError("weight must be [D, W]")
    B, T, D = x.shape
    W, dt, dev = weight.shape[1], x.dtype, x.device
    if (B | T | D | W) >> 31:
        _past_32_bits()
    a = ConvArgs()
    a.dtype = _dtype_code(x)
    a.x_stride = _rows("x", x, (B, T, D), 1, dt, dev)
    _t("weight", weight, (D, W), dt, dev)
    _t("bias", bias, (D,), dt, dev, optional=True)
    cu, host, n = _seqs(cu_seqlens, cu_seqlens_host, B, T, dev, need_host=False)
    _t("initial_state", initial_state, (n, W - 1, D), dt, dev, optional=True)
    a.B, a.T, a.D, a.W, a.num_seqs, a.silu = B, T, D, W, n, int(bool(silu))
    a.x, a.w, a.bias, a.init, a.cu_seqlens = map(_ptr, (x, weight, bias, initial_state, cu))
    _on_gpu("x", x)
    return a, host


def _rows_like(x, packed_unchecked):
    """An output of x's shape: rows behind the last sequence (possible only where
    the lengths were not checked on the host) hold zeros."""
    return x.new_zeros(x.shape) if packed_unchecked else x.new_empty(x.shape)


def gdn_conv_fwd(x, weight, bias=None, silu: bool = True, initial_state=None, cu_seqlens=None, cu_seqlens_host=None,
                 output_final_state: bool = True):
    """y, final_state (None unless output_final_state) of the short causal convolution:
    x [B, T, D], weight [D, W], bias [D], states [N, W-1, D] (the inputs before a
    sequence's start, oldest first), all of one dtype."""
    if _compiling():
        return _outside(gdn_conv_fwd, x, weight, bias, silu, initial_state, cu_seqlens, cu_seqlens_host,
                        output_final_state)
    a, host = _conv_args(x, weight, bias, silu, initial_state, cu_seqlens, cu_seqlens_host)
    y = _rows_like(x, cu_seqlens is not None and host is None)
    fin = torch.empty((a.num_seqs, a.W - 1, a.D), dtype=x.dtype, device=x.device) if output_final_state else None
    args = ConvFwdArgs()
    args.a, args.y, args.final_state = a, _ptr(y), _ptr(fin)
    _call(lib().gdn_conv_fwd, args, x.device)
    return y, fin


def gdn_conv_bwd(x, weight, dy, bias=None, silu: bool = True, initial_state=None, cu_seqlens=None,
                 cu_seqlens_host=None, dfinal=None):
    """(dx, dweight, dbias, dinitial_state), the last two None without bias / initial_state."""
    if _compiling():
        return _outside(gdn_conv_bwd, x, weight, dy, bias, silu, initial_state, cu_seqlens, cu_seqlens_host, dfinal)
    a, host = _conv_args(x, weight, bias, silu, initial_state, cu_seqlens, cu_seqlens_host)
    dev, dt = x.device, x.dtype
    _t("dy", dy, x.shape, dt, dev)
    _t("dfinal", dfinal, (a.num_seqs, a.W - 1, a.D), dt, dev, optional=True)
    dx = _rows_like(x, cu_seqlens is not None and host is None)
    dw = torch.empty_like(weight)
    db = None if bias is None else torch.empty_like(bias)
    di = None if initial_state is None else torch.empty_like(initial_state)
    args = ConvBwdArgs()
    args.a = a
    args.dy, args.dfinal, args.dx, args.dw, args.dbias, args.dinit = map(_ptr, (dy, dfinal, dx, dw, db, di))
    with _on(dev):
        ws = _workspace(lib().gdn_conv_bwd_workspace_size(ctypes.byref(args)), dev)
    args.workspace, args.workspace_bytes = ws.data_ptr(), ws.numel()
    _call(lib().gdn_conv_bwd, args, dev)
    return dx, dw, db, di


def gdn_conv_step(x, state, weight, bias=None, silu: bool = True, state_idx=None, y=None):
    """One token for each of N sequences: x [N, D], state [S, W-1, D] (advanced in place;
    sequence n uses slot n, or state_idx[n]; out-of-range indices mark padding, whose y is
    left as it was).  Two sequences of one call must not share a slot.  Returns y [N, D]."""
    if _compiling():
        return _outside(gdn_conv_step, x, state, weight, bias, silu, state_idx, y)
    if x.dim() != 2 or weight.dim() != 2:
        raise GDNError("x must be [N, D] and weight [D, W]")
    _no_derivative("gdn_conv_step", (x, state, weight, bias))
    N, D = x.shape
    W, dt, dev = weight.shape[1], x.dtype, x.device
    slots = state.shape[0]
    if (N | D | W | slots) >> 31:
        _past_32_bits()
    stride = _rows("x", x, (N, D), 1, dt, dev)
    _t("weight", weight, (D, W), dt, dev)
    _t("bias", bias, (D,), dt, dev, optional=True)
    _t("state", state, (slots, W - 1, D), dt, dev)
    _t("state_idx", state_idx, (N,), torch.int32, dev, optional=True)
    _on_gpu("x", x)
    if y is None:
        y = weight.new_empty((N, D))
    else:
        _t("y", y, (N, D), dt, dev)
    a = ConvStepArgs(_dtype_code(x), N, D, W, x.data_ptr(), stride, state.data_ptr(), _ptr(state_idx), slots,
                     weight.data_ptr(), _ptr(bias), bool(silu), y.data_ptr())
    _call(lib().gdn_conv_step, a, dev)
    return y


class _ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, silu, cu_seqlens, cu_seqlens_host, output_final_state):
        with _as_one_op():
            y, fin = gdn_conv_fwd(x, weight, bias, silu, initial_state, cu_seqlens, cu_seqlens_host,
                                  output_final_state)
        ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
        ctx.silu, ctx.cu_host = silu, _own_lengths(cu_seqlens_host)
        ctx.set_materialize_grads(False)
        return y, fin

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dfin):
        x, weight, bias, init, cu = ctx.saved_tensors
        if dy is None:
            if dfin is None:
                return (None,) * 8
            dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
        dx, dw, db, di = gdn_conv_bwd(x, weight, dy.contiguous(), bias, ctx.silu, init, cu, ctx.cu_host,
                                      None if dfin is None else dfin.contiguous())
        return dx, dw, db, di, None, None, None, None


def short_conv(x, weight, bias=None, silu: bool = True, initial_state=None, output_final_state: bool = False,
               cu_seqlens=None, cu_seqlens_host=None):
    """Short causal depthwise convolution over x [B, T, D] with weight [D, W] (W in 2..4),
    optional bias [D] and SiLU, differentiable in x, weight, bias and initial_state.
    Returns y, or (y, final_state [N, W-1, D]).  cu_seqlens (int32, B = 1) packs
    sequences; cu_seqlens_host, when given, is checked against T."""
    if _compiling():
        return _outside(short_conv, x, weight, bias, silu, initial_state, output_final_state, cu_seqlens,
                        cu_seqlens_host)
    if _wants_grad(x, weight, bias, initial_state):
        y, fin = _ShortConv.apply(x, weight, bias, initial_state, bool(silu), cu_seqlens, cu_seqlens_host,
                                  bool(output_final_state))
    else:
        y, fin = gdn_conv_fwd(x, weight, bias, silu, initial_state, cu_seqlens, cu_seqlens_host, output_final_state)
    return (y, fin) if output_final_state else y


# ------------------------------------------------------------------ selective state space scan
def _scan_args(x, dt, A, B, C, D, dt_bias, dt_softplus, h0, cu_seqlens, cu_seqlens_host, seg_mode,
               round_once=False):
    if x.dim() != 4 or B.dim() != 4:
        raise GDNError("x must be [B, T, H, Dv] and B, C [B, T, G, Dk]")
    nb, T, H, Dv = x.shape
    G, Dk = B.shape[2:]
    if (nb | T | H | Dv | G | Dk) >> 31:
        _past_32_bits()
    dev, e = x.device, x.dtype
    a = ScanArgs()
    a.dtype = _dtype_code(x)
    a.x_stride = _rows("x", x, (nb, T, H, Dv), 2, e, dev)
    a.b_stride = _rows("B", B, (nb, T, G, Dk), 2, e, dev)
    a.c_stride = _rows("C", C, (nb, T, G, Dk), 2, e, dev)
    if dt.dtype not in (e, torch.float32):
        raise GDNError(f"dt must be {e} or float32, got {dt.dtype}")
    a.dt_dtype = _dtype_code(dt)
    a.dt_stride = _rows("dt", dt, (nb, T, H), 1, dt.dtype, dev)
    _t("A", A, (H,), torch.float32, dev)
    _t("D", D, (H,), torch.float32, dev, optional=True)
    _t("dt_bias", dt_bias, (H,), torch.float32, dev, optional=True)
    cu, host, n = _seqs(cu_seqlens, cu_seqlens_host, nb, T, dev, need_host=True)
    _t("initial_state", h0, (n, H, Dk, Dv), torch.float32, dev, optional=True)
    a.B, a.T, a.H, a.G, a.Dk, a.Dv = nb, T, H, G, Dk, Dv
    a.dt_softplus, a.num_seqs, a.seg_mode = int(bool(dt_softplus)), n, int(seg_mode)
    a.round_once = int(bool(round_once))
    a.x, a.dt, a.b, a.c, a.A, a.D, a.dt_bias, a.h0, a.cu_seqlens = map(_ptr, (x, dt, B, C, A, D, dt_bias, h0, cu))
    a.cu_seqlens_host = None if host is None else host.data_ptr()
    _on_gpu("x", x)
    return a, host


def gdn_scan_fwd(x, dt, A, B, C, D=None, dt_bias=None, dt_softplus: bool = False, h0=None, cu_seqlens=None,
                 cu_seqlens_host=None, output_final_state: bool = True, save_states: bool = False, seg_mode: int = 0,
                 round_once: bool = False):
    """(y, hT) with hT None unless output_final_state, followed by the saved segment
    states if save_states (a flat fp32 tensor for gdn_scan_bwd)."""
    if _compiling():
        return _outside(gdn_scan_fwd, x, dt, A, B, C, D, dt_bias, dt_softplus, h0, cu_seqlens, cu_seqlens_host,
                        output_final_state, save_states, seg_mode, round_once)
    a, host = _scan_args(x, dt, A, B, C, D, dt_bias, dt_softplus, h0, cu_seqlens, cu_seqlens_host, seg_mode,
                         round_once)
    dev, L = x.device, lib()
    y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    hT = (torch.empty((a.num_seqs, a.H, a.Dk, a.Dv), dtype=torch.float32, device=dev) if output_final_state else None)
    args = ScanFwdArgs()
    args.a, args.y, args.hT = a, _ptr(y), _ptr(hT)
    states = None
    with _on(dev):
        if save_states:
            states = torch.empty(max(4, L.gdn_scan_states_bytes(ctypes.byref(a)) // 4), dtype=torch.float32, device=dev)
            args.h_save = _ptr(states)
        ws = _workspace(L.gdn_scan_fwd_workspace_size(ctypes.byref(args)), dev)
    args.a.workspace, args.a.workspace_bytes = ws.data_ptr(), ws.numel()
    _call(L.gdn_scan_fwd, args, dev)
    del host
    return (y, hT, states) if save_states else (y, hT)


def gdn_scan_bwd(x, dt, A, B, C, dy, D=None, dt_bias=None, dt_softplus: bool = False, h0=None, dhT=None,
                 cu_seqlens=None, cu_seqlens_host=None, states=None, seg_mode: int = 0, round_once: bool = False):
    """(dx, ddt, dA, dB, dC, dD, ddt_bias, dh0); dD, ddt_bias and dh0 are None where their
    inputs are.  states: gdn_scan_fwd(..., save_states=True) on the same inputs."""
    if _compiling():
        return _outside(gdn_scan_bwd, x, dt, A, B, C, dy, D, dt_bias, dt_softplus, h0, dhT, cu_seqlens,
                        cu_seqlens_host, states, seg_mode, round_once)
    a, host = _scan_args(x, dt, A, B, C, D, dt_bias, dt_softplus, h0, cu_seqlens, cu_seqlens_host, seg_mode,
                         round_once)
    dev, L = x.device, lib()
    _t("dy", dy, x.shape, x.dtype, dev)
    _t("dhT", dhT, (a.num_seqs, a.H, a.Dk, a.Dv), torch.float32, dev, optional=True)
    new = lambda t: None if t is None else torch.empty(t.shape, dtype=t.dtype, device=dev)
    dx, ddt, db, dc, dA, dD, dbias, dh0 = map(new, (x, dt, B, C, A, D, dt_bias, h0))
    args = ScanBwdArgs()
    args.a = a
    args.dy, args.dhT, args.dx, args.ddt, args.db, args.dc, args.dA, args.dD, args.ddt_bias, args.dh0 = map(
        _ptr, (dy, dhT, dx, ddt, db, dc, dA, dD, dbias, dh0))
    with _on(dev):
        if states is not None:
            _t("states", states, states.shape, torch.float32, dev)
            if states.numel() * 4 != max(16, L.gdn_scan_states_bytes(ctypes.byref(a))):
                raise GDNError("states are not those of a forward pass with these arguments")
            args.h_saved = _ptr(states)
        ws = _workspace(L.gdn_scan_bwd_workspace_size(ctypes.byref(args)), dev)
    args.a.workspace, args.a.workspace_bytes = ws.data_ptr(), ws.numel()
    _call(L.gdn_scan_bwd, args, dev)
    del host
    return dx, ddt, dA, db, dc, dD, dbias, dh0


def gdn_scan_step(x, dt, A, B, C, state, D=None, dt_bias=None, dt_softplus: bool = False, state_idx=None, y=None):
    """One token for each of N sequences: x [N, H, Dv], dt [N, H], B, C [N, G, Dk]; state
    [S, H, Dk, Dv] fp32 is advanced in place (slots as in gdn_decode_step).  Returns y."""
    if _compiling():
        return _outside(gdn_scan_step, x, dt, A, B, C, state, D, dt_bias, dt_softplus, state_idx, y)
    if x.dim() != 3 or B.dim() != 3:
        raise GDNError("x must be [N, H, Dv] and B, C [N, G, Dk]")
    _no_derivative("gdn_scan_step", (x, dt, A, B, C, state, D, dt_bias))
    N, H, Dv = x.shape
    G, Dk = B.shape[1:]
    slots = state.shape[0]
    if (N | H | Dv | G | Dk | slots) >> 31:
        _past_32_bits()
    dev, e = x.device, x.dtype
    code = _dtype_code(x)
    xs = _rows("x", x, (N, H, Dv), 2, e, dev)
    bs = _rows("B", B, (N, G, Dk), 2, e, dev)
    cs = _rows("C", C, (N, G, Dk), 2, e, dev)
    if dt.dtype not in (e, torch.float32):
        raise GDNError(f"dt must be {e} or float32, got {dt.dtype}")
    ds = _rows("dt", dt, (N, H), 1, dt.dtype, dev)
    _t("A", A, (H,), torch.float32, dev)
    _t("D", D, (H,), torch.float32, dev, optional=True)
    _t("dt_bias", dt_bias, (H,), torch.float32, dev, optional=True)
    _t("state", state, (slots, H, Dk, Dv), torch.float32, dev)
    _t("state_idx", state_idx, (N,), torch.int32, dev, optional=True)
    _on_gpu("x", x)
    if y is None:
        y = x.new_empty((N, H, Dv))
    else:
        _t("y", y, (N, H, Dv), e, dev)
    a = ScanStepArgs(code, _dtype_code(dt), N, H, G, Dk, Dv, x.data_ptr(), dt.data_ptr(), B.data_ptr(), C.data_ptr(),
                     xs, ds, bs, cs, A.data_ptr(), _ptr(D), _ptr(dt_bias), bool(dt_softplus), state.data_ptr(),
                     _ptr(state_idx), slots, y.data_ptr())
    _call(lib().gdn_scan_step, a, dev)
    return y


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, dt_bias, h0, dt_softplus, cu_seqlens, cu_seqlens_host, final, seg_mode,
                round_once):
        with _as_one_op():
            cu_seqlens_host = _own_lengths(cu_seqlens_host if cu_seqlens_host is not None else
                                           None if cu_seqlens is None else cu_seqlens.cpu())
            res = gdn_scan_fwd(x, dt, A, B, C, D, dt_bias, dt_softplus, h0, cu_seqlens, cu_seqlens_host, final,
                               save_states=True, seg_mode=seg_mode, round_once=round_once)
        ctx.save_for_backward(x, dt, A, B, C, D, dt_bias, h0, cu_seqlens, res[2])
        ctx.dt_softplus, ctx.cu_host, ctx.seg_mode, ctx.round_once = dt_softplus, cu_seqlens_host, seg_mode, round_once
        ctx.set_materialize_grads(False)
        return res[0], res[1]

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dhT):
        x, dt, A, B, C, D, dt_bias, h0, cu, states = ctx.saved_tensors
        if dy is None:
            if dhT is None:
                return (None,) * 14
            dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
        dx, ddt, dA, dB, dC, dD, dbias, dh0 = gdn_scan_bwd(
            x, dt, A, B, C, _gradient(dy), D, dt_bias, ctx.dt_softplus, h0,
            None if dhT is None else dhT.contiguous(), cu, ctx.cu_host, states, ctx.seg_mode,
            ctx.round_once)
        return dx, ddt, dA, dB, dC, dD, dbias, dh0, None, None, None, None, None, None


def selective_scan(x, dt, A, B, C, D=None, dt_bias=None, dt_softplus: bool = False, initial_state=None,
                   output_final_state: bool = False, cu_seqlens=None, cu_seqlens_host=None, seg_mode: int = 0,
                   round_once: bool = False):
    """Selective state space scan, differentiable in every tensor argument:

        h_t = exp(d_t A) h_{t-1} + d_t B_t x_t^T,   y_t = h_t^T C_t + D x_t,
        d_t = dt_t + dt_bias, or softplus(dt_t + dt_bias) with dt_softplus

    x [B, T, H, Dv], dt [B, T, H] (x's dtype or fp32), A, D, dt_bias [H] fp32 (A <= 0), B, C
    [B, T, G, Dk] shared by H / G heads, states [N, H, Dk, Dv] fp32.  Returns y, or
    (y, hT).  cu_seqlens (int32, B = 1) packs sequences; without its host copy
    cu_seqlens_host it is read back once (a device synchronisation).  round_once: bf16 y and
    dx are the fp32 result rounded once; without it a chunk's matrix and state are rounded
    inside as well (rms error up to a quarter above the output rounding's, 2 to 10 % less time)."""
    if _compiling():
        return _outside(selective_scan, x, dt, A, B, C, D, dt_bias, dt_softplus, initial_state, output_final_state,
                        cu_seqlens, cu_seqlens_host, seg_mode, round_once)
    if _wants_grad(x, dt, A, B, C, D, dt_bias, initial_state):
        y, hT = _SelectiveScan.apply(x, dt, A, B, C, D, dt_bias, initial_state, bool(dt_softplus), cu_seqlens,
                                     cu_seqlens_host, bool(output_final_state), int(seg_mode), bool(round_once))
    else:
        y, hT = gdn_scan_fwd(x, dt, A, B, C, D, dt_bias, dt_softplus, initial_state, cu_seqlens, cu_seqlens_host,
                             output_final_state, seg_mode=seg_mode, round_once=round_once)
    return (y, hT) if output_final_state else y


# ------------------------------------------------------------------ gated group norm
def _norm_args(x, weight, z, bias, eps, center, gate_first):
    if x.dim() < 2:
        raise GDNError("x must be [..., G, D]")
    G, D = x.shape[-2:]
    if (G | D) >> 31:
        _past_32_bits()
    dt, dev = x.dtype, x.device
    code = _dtype_code(x)
    x_stride = _rows("x", x, x.shape, 2, dt, dev)
    z_stride = 0 if z is None else _rows("z", z, x.shape, 2, dt, dev)
    shared = weight.dim() == 1
    shape = (D,) if shared else (G, D)
    _t("weight", weight, shape, dt, dev)
    _t("bias", bias, shape, dt, dev, optional=True)
    R = 1
    for n in x.shape[:-2]:
        R *= n
    if gate_first and z is None:
        raise GDNError("gate_first needs z")
    _on_gpu("x", x)
    return NormArgs(code, R, G, D, x.data_ptr(), x_stride, _ptr(z), z_stride, weight.data_ptr(), _ptr(bias), shared,
                    bool(center), bool(gate_first), eps)


def gdn_norm_fwd(x, weight, z=None, bias=None, eps: float = 1e-5, center: bool = False, gate_first: bool = False):
    """y of the gated group norm (see gated_group_norm)."""
    if _compiling():
        return _outside(gdn_norm_fwd, x, weight, z, bias, eps, center, gate_first)
    args = NormFwdArgs()
    args.a = _norm_args(x, weight, z, bias, eps, center, gate_first)
    y = x.new_empty(x.shape)
    args.y = _ptr(y)
    _call(lib().gdn_norm_fwd, args, x.device)
    return y


def gdn_norm_bwd(x, weight, dy, z=None, bias=None, eps: float = 1e-5, center: bool = False, gate_first: bool = False):
    """(dx, dweight, dz, dbias), the last two None without z / bias."""
    if _compiling():
        return _outside(gdn_norm_bwd, x, weight, dy, z, bias, eps, center, gate_first)
    args = NormBwdArgs()
    args.a = _norm_args(x, weight, z, bias, eps, center, gate_first)
    dev = x.device
    _t("dy", dy, x.shape, x.dtype, dev)
    new = lambda t: None if t is None else torch.empty(t.shape, dtype=t.dtype, device=dev)
    dx, dw, dz, db = map(new, (x, weight, z, bias))
    args.dy, args.dx, args.dw, args.dz, args.dbias = map(_ptr, (dy, dx, dw, dz, db))
    with _on(dev):
        ws = _workspace(lib().gdn_norm_bwd_workspace_size(ctypes.byref(args)), dev)
    args.workspace, args.workspace_bytes = ws.data_ptr(), ws.numel()
    _call(lib().gdn_norm_bwd, args, dev)
    return dx, dw, dz, db


class _GatedGroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, z, bias, eps, center, gate_first):
        ctx.save_for_backward(x, weight, z, bias)
        ctx.opts = (eps, center, gate_first)
        with _as_one_op():
            return gdn_norm_fwd(x, weight, z, bias, eps, center, gate_first)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, z, bias = ctx.saved_tensors
        dx, dw, dz, db = gdn_norm_bwd(x, weight, dy.contiguous(), z, bias, *ctx.opts)
        return dx, dw, dz, db, None, None, None


def gated_group_norm(x, weight, z: Optional[torch.Tensor] = None, bias=None, eps: float = 1e-5,
                     center: bool = False, gate_first: bool = False):
    """Group norm over the last dimension of x [..., G, D], channels last, with an optional
    SiLU gate z (x's shape), differentiable in x, weight, z and bias:

        v = x silu(z) with gate_first, else x
        y = (v - m) / sqrt(mean((v - m)^2) + eps) * weight + bias,   m = mean(v) with center, else 0
        y = y silu(z) with a gate and not gate_first

    weight and bias are [G, D], or [D] shared by all groups."""
    if _compiling():
        return _outside(gated_group_norm, x, weight, z, bias, eps, center, gate_first)
    if not _wants_grad(x, weight, z, bias):
        return gdn_norm_fwd(x, weight, z, bias, eps, center, gate_first)
    return _GatedGroupNorm.apply(x, weight, z, bias, float(eps), bool(center), bool(gate_first))
