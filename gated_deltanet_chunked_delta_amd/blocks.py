"""Operators of a block around its mixer: residual norm (also with an output in 8
bits), rows in 8 bits with scales, projections with their epilogue, and the gated
linear recurrence.

A block adds its input to the residual stream and normalises the sum
(``add_rms_norm``), projects it (``linear``; or, in serving, both in 8 bits:
``add_rms_norm_8bit``, ``linear_8bit``), runs a mixer -- the delta rule, the
selective scan, or ``gated_recurrence``, their channelwise sibling -- and projects
back.  As in ``layers.py`` only arguments are marshalled here, and the same rules
hold for streams, devices, strided inputs, captured graphs, derivatives and tracers;
no input needs any alignment beyond its elements'.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import layers as _layers
from .binding import GDNError, _compiling, _dtype_code, _outside, _ptr, _vp, lib as _load
from .layers import (_as_one_op, _call, _no_derivative, _on, _past_32_bits, _rows, _t, _wants_grad, _workspace)

__all__ = ["add_rms_norm", "add_rms_norm_8bit", "quantize_rows"]

_i32, _i64, _sz, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


class AddNormFwdArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("res_dtype", _i32), ("R", _i64), ("D", _i32), ("eps", _f32), ("x", _vp),
                ("x_stride", _i64), ("r", _vp), ("r_stride", _i64), ("w", _vp), ("s", _vp), ("y", _vp), ("q", _vp),
                ("q_scale", _vp)]


class AddNormBwdArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("res_dtype", _i32), ("R", _i64), ("D", _i32), ("eps", _f32), ("s", _vp),
                ("s_stride", _i64), ("w", _vp), ("dy", _vp), ("ds", _vp), ("dx", _vp), ("dr", _vp), ("dw", _vp),
                ("workspace", _vp), ("workspace_bytes", _sz)]


class QuantArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("R", _i64), ("D", _i32), ("x", _vp), ("x_stride", _i64), ("q", _vp), ("q_scale", _vp)]


_SIGNATURES = [("gdn_addnorm_fwd", AddNormFwdArgs), ("gdn_addnorm_bwd", AddNormBwdArgs), ("gdn_quant_rows", QuantArgs)]
_SIZES = [("gdn_addnorm_bwd_workspace_size", AddNormBwdArgs)]
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


def _on_gpu(name, t):
    return _layers._on_gpu(name, t)


def _flat(t, inner=1):
    """The number of rows in front of the last `inner` dimensions."""
    n = 1
    for s in t.shape[:t.dim() - inner]:
        n *= s
    return n


def _row_input(name, t):
    if t.dim() < 2:
        raise GDNError(f"{name} must be [..., D]")
    D = t.shape[-1]
    if D >> 31 or _flat(t) >> 31:
        _past_32_bits()
    return D


# ------------------------------------------------------------------ residual norm, rows in 8 bits
def _addnorm_args(x, weight, residual, eps):
    D = _row_input("x", x)
    dt, dev = x.dtype, x.device
    a = AddNormFwdArgs()
    a.dtype = a.res_dtype = _dtype_code(x)
    a.R, a.D, a.eps = _flat(x), D, eps
    a.x, a.x_stride = x.data_ptr(), _rows("x", x, x.shape, 1, dt, dev)
    _t("weight", weight, (D,), dt, dev)
    a.w = weight.data_ptr()
    s = x
    if residual is not None:
        if residual.dtype not in (dt, torch.float32):
            raise GDNError(f"residual must be {dt} or float32, got {residual.dtype}")
        a.res_dtype = _dtype_code(residual)
        a.r, a.r_stride = residual.data_ptr(), _rows("residual", residual, x.shape, 1, residual.dtype, dev)
        s = torch.empty(x.shape, dtype=residual.dtype, device=dev)
        a.s = s.data_ptr()
    _on_gpu("x", x)
    return a, s


def gdn_addnorm_fwd(x, weight, residual=None, eps: float = 1e-6):
    """(y, s) of the residual norm (see add_rms_norm); s is x itself without a residual."""
    if _compiling():
        return _outside(gdn_addnorm_fwd, x, weight, residual, eps)
    a, s = _addnorm_args(x, weight, residual, eps)
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    a.y = y.data_ptr()
    _call(lib().gdn_addnorm_fwd, a, x.device)
    return y, s


def gdn_addnorm_bwd(s, weight, dy, ds=None, eps: float = 1e-6, need=(True, True, True)):
    """(dx, dresidual, dweight) from the sum s (x itself without a residual) and the gradients
    of y and, optionally, of s; a gradient that is not in `need` is None.  dx is in dy's type,
    dresidual in s's, one tensor where the two are alike."""
    if _compiling():
        return _outside(gdn_addnorm_bwd, s, weight, dy, ds, eps, need)
    D = _row_input("s", s)
    dt, dev = dy.dtype, s.device
    if s.dtype not in (dt, torch.float32):
        raise GDNError(f"s must be {dt} or float32, got {s.dtype}")
    _t("dy", dy, s.shape, dt, dev)
    _t("ds", ds, s.shape, s.dtype, dev, optional=True)
    _t("weight", weight, (D,), dt, dev)
    a = AddNormBwdArgs()
    a.dtype, a.res_dtype = _dtype_code(dy), _dtype_code(s)
    a.R, a.D, a.eps = _flat(s), D, eps
    a.s, a.s_stride = s.data_ptr(), _rows("s", s, s.shape, 1, s.dtype, dev)
    a.w, a.dy, a.ds = weight.data_ptr(), dy.data_ptr(), _ptr(ds)
    _on_gpu("s", s)
    same = s.dtype == dt
    dx = torch.empty(s.shape, dtype=dt, device=dev) if need[0] or same and need[1] else None
    dr = torch.empty(s.shape, dtype=s.dtype, device=dev) if need[1] and not same else None
    dw = torch.empty(D, dtype=dt, device=dev) if need[2] else None
    a.dx, a.dr, a.dw = _ptr(dx), _ptr(dr), _ptr(dw)
    with _on(dev):
        ws = _workspace(lib().gdn_addnorm_bwd_workspace_size(ctypes.byref(a)), dev)
    a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel()
    _call(lib().gdn_addnorm_bwd, a, dev)
    return (dx if need[0] else None), (None if not need[1] else dx if same else dr), dw


class _AddNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        with _as_one_op():
            y, s = gdn_addnorm_fwd(x, weight, residual, eps)
        ctx.save_for_backward(s if residual is not None else x, weight)
        ctx.eps, ctx.res = eps, residual is not None
        ctx.set_materialize_grads(False)
        return (y, s) if ctx.res else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, ds=None):
        s, weight = ctx.saved_tensors
        if dy is None:
            if ds is None:
                return (None,) * 4
            dy = torch.zeros(s.shape, dtype=weight.dtype, device=s.device)
        need = ctx.needs_input_grad
        dx, dr, dw = gdn_addnorm_bwd(s, weight, dy.contiguous(), None if ds is None else ds.contiguous(), ctx.eps,
                                     (need[0], need[2], need[1]))
        return dx, dw, dr, None


def add_rms_norm(x, weight, residual=None, eps: float = 1e-6):
    """(y, s) of the residual norm over the last dimension of x [..., D], differentiable in x,
    weight and residual:

        s = x + residual   (in residual's type: x's, or fp32; x itself without a residual)
        y = s / sqrt(mean(s^2) + eps) * weight

    The norm reads s as it is stored, rounded to its type.  weight is [D]."""
    if _compiling():
        return _outside(add_rms_norm, x, weight, residual, eps)
    if not _wants_grad(x, weight, residual):
        return gdn_addnorm_fwd(x, weight, residual, float(eps))
    out = _AddNorm.apply(x, weight, residual, float(eps))
    return out if residual is not None else (out, x)


def _q8(x):
    return (torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device),
            torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device))


def add_rms_norm_8bit(x, weight, residual=None, eps: float = 1e-6):
    """(q, scale, s): the residual norm with its output in 8 bits.  q [..., D] is e4m3, scale
    [...] fp32; row y of add_rms_norm, before any rounding, is q * scale with scale =
    max(max|y|, 2^-100) / 448 and q rounded once.  No derivative."""
    if _compiling():
        return _outside(add_rms_norm_8bit, x, weight, residual, eps)
    _no_derivative("add_rms_norm_8bit", (x, weight, residual))
    a, s = _addnorm_args(x, weight, residual, eps)
    q, scale = _q8(x)
    a.q, a.q_scale = q.data_ptr(), scale.data_ptr()
    _call(lib().gdn_addnorm_fwd, a, x.device)
    return q, scale, s


def quantize_rows(x):
    """(q, scale): rows of x [..., D] in 8 bits, as add_rms_norm_8bit's output: weights laid out
    once for linear_8bit ([N, K] gives a scale for each output), or activations that come from no
    norm.  No derivative."""
    if _compiling():
        return _outside(quantize_rows, x)
    _no_derivative("quantize_rows", (x,))
    D = _row_input("x", x)
    a = QuantArgs()
    a.dtype, a.R, a.D = _dtype_code(x), _flat(x), D
    a.x, a.x_stride = x.data_ptr(), _rows("x", x, x.shape, 1, x.dtype, x.device)
    _on_gpu("x", x)
    q, scale = _q8(x)
    a.q, a.q_scale = q.data_ptr(), scale.data_ptr()
    _call(lib().gdn_quant_rows, a, x.device)
    return q, scale
