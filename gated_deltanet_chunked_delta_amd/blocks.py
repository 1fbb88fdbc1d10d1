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
from .binding import GDNError, _check, _compiling, _dtype_code, _outside, _ptr, _vp, lib as _load
from .layers import (_as_one_op, _call, _no_derivative, _on, _own_lengths, _past_32_bits, _rows, _rows_like, _seqs, _t, _wants_grad, _workspace)

__all__ = ["add_rms_norm", "add_rms_norm_8bit", "quantize_rows", "linear", "linear_8bit", "gated_recurrence", "gdn_rec_step"]

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


class RecArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("g_dtype", _i32), ("B", _i32), ("T", _i32), ("D", _i32), ("x", _vp), ("x_stride", _i64),
                ("g", _vp), ("g_stride", _i64), ("i", _vp), ("i_stride", _i64), ("scale", _vp), ("h0", _vp),
                ("cu_seqlens", _vp), ("num_seqs", _i32), ("workspace", _vp), ("workspace_bytes", _sz)]


class RecFwdArgs(ctypes.Structure):
    _fields_ = [("a", RecArgs), ("y", _vp), ("hT", _vp), ("h_save", _vp)]


class RecBwdArgs(ctypes.Structure):
    _fields_ = [("a", RecArgs), ("h_saved", _vp), ("dy", _vp), ("dhT", _vp), ("dx", _vp), ("dg", _vp), ("di", _vp),
                ("dscale", _vp), ("dh0", _vp)]


class RecStepArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("g_dtype", _i32), ("N", _i32), ("D", _i32), ("x", _vp), ("x_stride", _i64), ("g", _vp),
                ("g_stride", _i64), ("i", _vp), ("i_stride", _i64), ("scale", _vp), ("state", _vp), ("state_idx", _vp),
                ("num_slots", _i32), ("y", _vp)]


class LinearArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("out_dtype", _i32), ("M", _i64), ("N", _i32), ("K", _i32), ("x", _vp), ("x_stride", _i64),
                ("w", _vp), ("x_scale", _vp), ("w_scale", _vp), ("bias", _vp), ("r", _vp), ("r_stride", _i64), ("act", _i32),
                ("workspace", _vp), ("workspace_bytes", _sz)]


class LinearFwdArgs(ctypes.Structure):
    _fields_ = [("a", LinearArgs), ("y", _vp), ("v_save", _vp)]


class LinearBwdArgs(ctypes.Structure):
    _fields_ = [("a", LinearArgs), ("v_saved", _vp), ("dy", _vp), ("dx", _vp), ("dw", _vp), ("dbias", _vp)]


_SIGNATURES = [("gdn_addnorm_fwd", AddNormFwdArgs), ("gdn_addnorm_bwd", AddNormBwdArgs), ("gdn_quant_rows", QuantArgs),
               ("gdn_linear_fwd", LinearFwdArgs), ("gdn_linear_bwd", LinearBwdArgs),
               ("gdn_rec_fwd", RecFwdArgs), ("gdn_rec_bwd", RecBwdArgs), ("gdn_rec_step", RecStepArgs)]
_SIZES = [("gdn_addnorm_bwd_workspace_size", AddNormBwdArgs), ("gdn_rec_fwd_workspace_size", RecFwdArgs),
          ("gdn_rec_bwd_workspace_size", RecBwdArgs), ("gdn_linear_fwd_workspace_size", LinearFwdArgs),
          ("gdn_linear_bwd_workspace_size", LinearBwdArgs), ("gdn_rec_states_bytes", RecArgs)]
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


def _row_input(name, t):
    """(shape, width, number of rows)"""
    shape = t.shape
    if len(shape) < 2:
        raise GDNError(f"{name} must be [..., D]")
    D, R = shape[-1], 1
    for n in shape[:-1]:
        R *= n
    if (D | R) >> 31:
        _past_32_bits()
    return shape, D, R


def _like(t, dtype):
    """A contiguous tensor of t's shape (t's rows lie evenly apart: only a contiguous t is dense)."""
    return torch.empty_like(t) if dtype is t.dtype else torch.empty_like(t, dtype=dtype)


# ------------------------------------------------------------------ residual norm, rows in 8 bits
def _addnorm_args(x, weight, residual, eps):
    shape, D, R = _row_input("x", x)
    dt, dev = x.dtype, x.device
    code = res = _dtype_code(x)
    xs, rs, s = _rows("x", x, shape, 1, dt, dev), 0, x
    _t("weight", weight, (D,), dt, dev)
    if residual is not None:
        rdt = residual.dtype
        if rdt is not dt and rdt is not torch.float32:
            raise GDNError(f"residual must be {dt} or float32, got {rdt}")
        res, rs = _dtype_code(residual), _rows("residual", residual, shape, 1, rdt, dev)
        s = _like(x, rdt)
    _on_gpu("x", x)
    return AddNormFwdArgs(code, res, R, D, eps, x.data_ptr(), xs, _ptr(residual), rs, weight.data_ptr(),
                          None if residual is None else s.data_ptr()), s


def gdn_addnorm_fwd(x, weight, residual=None, eps: float = 1e-6):
    """(y, s) of the residual norm (see add_rms_norm); s is x itself without a residual."""
    if _compiling():
        return _outside(gdn_addnorm_fwd, x, weight, residual, eps)
    a, s = _addnorm_args(x, weight, residual, eps)
    y = torch.empty_like(x)
    a.y = y.data_ptr()
    _call(lib().gdn_addnorm_fwd, a, x.device)
    return y, s


def gdn_addnorm_bwd(s, weight, dy, ds=None, eps: float = 1e-6, need=(True, True, True)):
    """(dx, dresidual, dweight) from the sum s (x itself without a residual) and the gradients
    of y and, optionally, of s; a gradient that is not in `need` is None.  dx is in dy's type,
    dresidual in s's, one tensor where the two are alike."""
    if _compiling():
        return _outside(gdn_addnorm_bwd, s, weight, dy, ds, eps, need)
    _, D, R = _row_input("s", s)
    dt, dev = dy.dtype, s.device
    if s.dtype not in (dt, torch.float32):
        raise GDNError(f"s must be {dt} or float32, got {s.dtype}")
    _t("dy", dy, s.shape, dt, dev)
    _t("ds", ds, s.shape, s.dtype, dev, optional=True)
    _t("weight", weight, (D,), dt, dev)
    a = AddNormBwdArgs()
    a.dtype, a.res_dtype = _dtype_code(dy), _dtype_code(s)
    a.R, a.D, a.eps = R, D, eps
    a.s, a.s_stride = s.data_ptr(), _rows("s", s, s.shape, 1, s.dtype, dev)
    a.w, a.dy, a.ds = weight.data_ptr(), dy.data_ptr(), _ptr(ds)
    _on_gpu("s", s)
    same = s.dtype == dt
    dx = torch.empty_like(dy) if need[0] or same and need[1] else None
    dr = torch.empty_like(s) if need[1] and not same else None
    dw = torch.empty_like(weight) if need[2] else None
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
    return torch.empty_like(x, dtype=torch.float8_e4m3fn), x.new_empty(x.shape[:-1], dtype=torch.float32)


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
    shape, D, R = _row_input("x", x)
    code, stride = _dtype_code(x), _rows("x", x, shape, 1, x.dtype, x.device)
    _on_gpu("x", x)
    q, scale = _q8(x)
    a = QuantArgs(code, R, D, x.data_ptr(), stride, q.data_ptr(), scale.data_ptr())
    _call(lib().gdn_quant_rows, a, x.device)
    return q, scale


# ------------------------------------------------------------------ projections
GDN_E4M3 = 2
_ACTS = {None: 0, "silu": 1, "gelu": 2}


def _linear_args(x, weight, bias, activation, residual, out_dtype):
    if weight.dim() != 2:
        raise GDNError("weight must be [N, K]")
    xshape, K, M = _row_input("x", x)
    N, dev, dt = weight.shape[0], x.device, x.dtype
    if N >> 31:
        _past_32_bits()
    if activation not in _ACTS:
        raise GDNError(f"unknown activation {activation!r} (None, 'silu' or 'gelu')")
    xs, rs = _rows("x", x, xshape, 1, dt, dev), 0
    _t("weight", weight, (N, K), dt, dev)
    _t("bias", bias, (N,), out_dtype, dev, optional=True)
    shape = (*xshape[:-1], N)
    if residual is not None:
        rs = _rows("residual", residual, shape, 1, out_dtype, dev)
    _on_gpu("x", x)
    return LinearArgs(0, 0, M, N, K, x.data_ptr(), xs, weight.data_ptr(), None, None, _ptr(bias), _ptr(residual), rs,
                      _ACTS[activation]), shape


def _linear_run(a, shape, out_dtype, dev, save):
    y = torch.empty(shape, dtype=out_dtype, device=dev)
    v = torch.empty(shape, dtype=torch.float32, device=dev) if save else None
    args = LinearFwdArgs(a, y.data_ptr(), _ptr(v))
    L = lib()
    if a.M > 64:  # (up to that many rows a product takes no workspace)
        with _on(dev):
            ws = _workspace(L.gdn_linear_fwd_workspace_size(ctypes.byref(args)), dev)
        args.a.workspace, args.a.workspace_bytes = ws.data_ptr(), ws.numel()
    _call(L.gdn_linear_fwd, args, dev)
    return y, v


def gdn_linear_fwd(x, weight, bias=None, activation=None, residual=None, save: bool = False):
    """(y, v) of the projection (see linear): v [..., N] fp32 is the value before the activation,
    for gdn_linear_bwd, with an activation and save; else None."""
    if _compiling():
        return _outside(gdn_linear_fwd, x, weight, bias, activation, residual, save)
    return _linear_fwd(x, weight, bias, activation, residual, save, False)


def _linear_fwd(x, weight, bias, activation, residual, save, train):
    """gdn_linear_fwd; with train, sizes of which a gradient is too large are refused."""
    code = _dtype_code(x)
    a, shape = _linear_args(x, weight, bias, activation, residual, x.dtype)
    a.dtype = a.out_dtype = code
    if train and (a.M | a.N | a.K) >> 16:  # (below: no gradient is too large)
        b = LinearBwdArgs(a, dx=1, dw=1)  # (its size alone is asked for; without rows x is null)
        with _on(x.device):
            if lib().gdn_linear_bwd_workspace_size(ctypes.byref(b)) == 0:
                _check(1)
    return _linear_run(a, shape, x.dtype, x.device, save and activation is not None)


def gdn_linear_bwd(x, weight, dy, activation=None, v=None, need=(True, True, True)):
    """(dx, dweight, dbias) of the projection; a gradient that is not in `need` is None.  v:
    gdn_linear_fwd(..., save=True) on the same inputs, with an activation."""
    if _compiling():
        return _outside(gdn_linear_bwd, x, weight, dy, activation, v, need)
    code = _dtype_code(x)
    a, shape = _linear_args(x, weight, None, activation, None, x.dtype)
    dt, dev = x.dtype, x.device
    a.dtype = a.out_dtype = code
    _t("dy", dy, shape, dt, dev)
    _t("v", v, shape, torch.float32, dev, optional=activation is None)
    if not any(need):
        return None, None, None
    args = LinearBwdArgs()
    dx = torch.empty(x.shape, dtype=dt, device=dev) if need[0] else None
    dw = torch.empty_like(weight) if need[1] else None
    db = torch.empty(a.N, dtype=dt, device=dev) if need[2] else None
    args.a, args.v_saved, args.dy, args.dx, args.dw, args.dbias = a, _ptr(v), dy.data_ptr(), *map(_ptr, (dx, dw, db))
    with _on(dev):
        ws = _workspace(lib().gdn_linear_bwd_workspace_size(ctypes.byref(args)), dev)
    args.a.workspace, args.a.workspace_bytes = ws.data_ptr(), ws.numel()
    _call(lib().gdn_linear_bwd, args, dev)
    return dx, dw, db


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, activation):
        need = ctx.needs_input_grad
        with _as_one_op():
            y, v = _linear_fwd(x, weight, bias, activation, residual, any(need[:3]), any(need[:3]))
        ctx.save_for_backward(x, weight, v)
        ctx.act = activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, v = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = gdn_linear_bwd(x, weight, dy.contiguous(), ctx.act, v, need[:3]) if any(need[:3]) else (None,) * 3
        return dx, dw, db, dy if need[3] else None, None


def linear(x, weight, bias=None, activation=None, residual=None):
    """Projection with its epilogue, differentiable in x, weight, bias and residual:

        y = act(x weight^T + bias) + residual

    x [..., K], weight [N, K], bias [N], residual [..., N], all of one dtype (bf16 or fp32);
    activation None, "silu" or "gelu" (its tanh form).  Sums are fp32 and y is rounded once.  With
    an activation a training pass keeps the value before it in fp32 (4 bytes an output).  A
    training pass takes fewer than 2^22 rows in bf16, 2^21 in fp32, along which the weight's
    gradient sums (gdn_linear_bwd takes more for the other gradients)."""
    if _compiling():
        return _outside(linear, x, weight, bias, activation, residual)
    if not _wants_grad(x, weight, bias, residual):
        return gdn_linear_fwd(x, weight, bias, activation, residual)[0]
    return _Linear.apply(x, weight, bias, residual, activation)


def linear_8bit(x, x_scale, weight, weight_scale, bias=None, activation=None, residual=None, out_dtype=torch.bfloat16):
    """linear of 8-bit rows: x [..., K] e4m3 with x_scale [...] (add_rms_norm_8bit, quantize_rows),
    weight [N, K] e4m3 with weight_scale [N] (quantize_rows); bias, residual and y in out_dtype (bf16
    or fp32).  No derivative."""
    if _compiling():
        return _outside(linear_8bit, x, x_scale, weight, weight_scale, bias, activation, residual, out_dtype)
    _no_derivative("linear_8bit", (x, x_scale, weight, weight_scale, bias, residual))
    if x.dtype is not torch.float8_e4m3fn:
        raise GDNError(f"x must be {torch.float8_e4m3fn}, got {x.dtype}")
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise GDNError(f"unsupported out_dtype {out_dtype}")
    a, shape = _linear_args(x, weight, bias, activation, residual, out_dtype)
    _t("x_scale", x_scale, x.shape[:-1], torch.float32, x.device)
    _t("weight_scale", weight_scale, (a.N,), torch.float32, x.device)
    a.dtype, a.out_dtype = GDN_E4M3, 1 if out_dtype is torch.bfloat16 else 0
    a.x_scale, a.w_scale = x_scale.data_ptr(), weight_scale.data_ptr()
    return _linear_run(a, shape, out_dtype, x.device, False)[0]


# ------------------------------------------------------------------ gated linear recurrence
def _gate_dtype(x, g):
    if g.dtype not in (x.dtype, torch.float32):
        raise GDNError(f"g must be {x.dtype} or float32, got {g.dtype}")
    return g.dtype


def _rec_args(x, g, i, scale, h0, cu_seqlens, cu_seqlens_host):
    if x.dim() != 3:
        raise GDNError("x must be [B, T, D]")
    B, T, D = x.shape
    if (B | T | D) >> 31:
        _past_32_bits()
    dt, dev = x.dtype, x.device
    a = RecArgs()
    a.dtype, a.x_stride = _dtype_code(x), _rows("x", x, (B, T, D), 1, dt, dev)
    gdt = _gate_dtype(x, g)
    a.g_dtype, a.g_stride = _dtype_code(g), _rows("g", g, (B, T, D), 1, gdt, dev)
    a.i_stride = 0 if i is None else _rows("i", i, (B, T, D), 1, dt, dev)
    _t("scale", scale, (D,), torch.float32, dev, optional=True)
    cu, host, n = _seqs(cu_seqlens, cu_seqlens_host, B, T, dev, need_host=False)
    _t("initial_state", h0, (n, D), torch.float32, dev, optional=True)
    a.B, a.T, a.D, a.num_seqs = B, T, D, n
    a.x, a.g, a.i, a.scale, a.h0, a.cu_seqlens = map(_ptr, (x, g, i, scale, h0, cu))
    _on_gpu("x", x)
    return a, cu is not None and host is None


def gdn_rec_fwd(x, g, i=None, scale=None, h0=None, cu_seqlens=None, cu_seqlens_host=None,
                output_final_state: bool = True, save_states: bool = False):
    """(y, hT) with hT None unless output_final_state, followed by the chunks' states if
    save_states (a flat fp32 tensor for gdn_rec_bwd)."""
    if _compiling():
        return _outside(gdn_rec_fwd, x, g, i, scale, h0, cu_seqlens, cu_seqlens_host, output_final_state, save_states)
    a, unchecked = _rec_args(x, g, i, scale, h0, cu_seqlens, cu_seqlens_host)
    dev, L = x.device, lib()
    args = RecFwdArgs()
    y = _rows_like(x, True) if unchecked else torch.empty_like(x)
    hT = torch.empty((a.num_seqs, a.D), dtype=torch.float32, device=dev) if output_final_state else None
    args.a, args.y, args.hT = a, y.data_ptr(), _ptr(hT)
    states = None
    with _on(dev):
        if save_states:
            states = torch.empty(L.gdn_rec_states_bytes(ctypes.byref(a)) // 4, dtype=torch.float32, device=dev)
            args.h_save = states.data_ptr()
        ws = _workspace(L.gdn_rec_fwd_workspace_size(ctypes.byref(args)), dev)
    args.a.workspace, args.a.workspace_bytes = ws.data_ptr(), ws.numel()
    _call(L.gdn_rec_fwd, args, dev)
    return (y, hT, states) if save_states else (y, hT)


def gdn_rec_bwd(x, g, dy, i=None, scale=None, h0=None, dhT=None, cu_seqlens=None, cu_seqlens_host=None, states=None):
    """(dx, dg, di, dscale, dh0); the last three are None where their inputs are.  states:
    gdn_rec_fwd(..., save_states=True) on the same inputs."""
    if _compiling():
        return _outside(gdn_rec_bwd, x, g, dy, i, scale, h0, dhT, cu_seqlens, cu_seqlens_host, states)
    a, unchecked = _rec_args(x, g, i, scale, h0, cu_seqlens, cu_seqlens_host)
    dev, L = x.device, lib()
    _t("dy", dy, x.shape, x.dtype, dev)
    _t("dhT", dhT, (a.num_seqs, a.D), torch.float32, dev, optional=True)
    args = RecBwdArgs()
    dx, dg = _rows_like(x, unchecked), _rows_like(g, unchecked)
    di = None if i is None else _rows_like(i, unchecked)
    ds, dh0 = (None if t is None else torch.empty_like(t) for t in (scale, h0))
    args.a = a
    args.dy, args.dhT, args.dx, args.dg, args.di, args.dscale, args.dh0 = map(_ptr, (dy, dhT, dx, dg, di, ds, dh0))
    with _on(dev):
        if states is not None:
            _t("states", states, states.shape, torch.float32, dev)
            if states.numel() * 4 != L.gdn_rec_states_bytes(ctypes.byref(a)):
                raise GDNError("states are not those of a forward pass with these arguments")
            args.h_saved = states.data_ptr()
        ws = _workspace(L.gdn_rec_bwd_workspace_size(ctypes.byref(args)), dev)
    args.a.workspace, args.a.workspace_bytes = ws.data_ptr(), ws.numel()
    _call(L.gdn_rec_bwd, args, dev)
    return dx, dg, di, ds, dh0


class _GatedRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, g, i, scale, h0, cu_seqlens, cu_seqlens_host, final):
        with _as_one_op():
            y, hT, states = gdn_rec_fwd(x, g, i, scale, h0, cu_seqlens, cu_seqlens_host, final, save_states=True)
        ctx.save_for_backward(x, g, i, scale, h0, cu_seqlens, states)
        ctx.cu_host = _own_lengths(cu_seqlens_host)
        ctx.set_materialize_grads(False)
        return y, hT

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dhT):
        x, g, i, scale, h0, cu, states = ctx.saved_tensors
        if dy is None:
            if dhT is None:
                return (None,) * 8
            dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
        dx, dg, di, ds, dh0 = gdn_rec_bwd(x, g, dy.contiguous(), i, scale, h0,
                                          None if dhT is None else dhT.contiguous(), cu, ctx.cu_host, states)
        return dx, dg, di, ds, dh0, None, None, None


def gated_recurrence(x, g, i=None, scale=None, initial_state=None, output_final_state: bool = False, cu_seqlens=None,
                     cu_seqlens_host=None):
    """Gated linear recurrence over x [B, T, D], channel by channel, differentiable in every
    tensor argument:

        h_t = exp(L_t) h_{t-1} + m_t sigmoid(i_t) x_t,   y_t = h_t
        L_t = g_t, m_t = 1;   with scale:  L_t = -scale sigmoid(g_t), m_t = sqrt(1 - exp(2 L_t))

    g [B, T, D] is in x's dtype or fp32: log decays (<= 0), or logits with scale [D] (fp32, >= 0);
    i [B, T, D], when given, are logits of the input's gate.  States [N, D] are fp32.  Returns y, or
    (y, hT).  cu_seqlens (int32, B = 1) packs sequences; cu_seqlens_host, when given, is checked
    against T."""
    if _compiling():
        return _outside(gated_recurrence, x, g, i, scale, initial_state, output_final_state, cu_seqlens, cu_seqlens_host)
    if _wants_grad(x, g, i, scale, initial_state):
        y, hT = _GatedRecurrence.apply(x, g, i, scale, initial_state, cu_seqlens, cu_seqlens_host,
                                       bool(output_final_state))
    else:
        y, hT = gdn_rec_fwd(x, g, i, scale, initial_state, cu_seqlens, cu_seqlens_host, output_final_state)
    return (y, hT) if output_final_state else y


def gdn_rec_step(x, g, state, i=None, scale=None, state_idx=None, y=None):
    """One token for each of N sequences: x, g, i [N, D] (as gated_recurrence); state [S, D] fp32 is
    advanced in place (slots as in gdn_decode_step: sequence n uses slot n, or state_idx[n];
    out-of-range indices mark padding, whose y is left as it was; no two sequences of a call
    share a slot).  Returns y [N, D]."""
    if _compiling():
        return _outside(gdn_rec_step, x, g, state, i, scale, state_idx, y)
    if x.dim() != 2:
        raise GDNError("x must be [N, D]")
    _no_derivative("gdn_rec_step", (x, g, state, i, scale))
    N, D = x.shape
    slots = state.shape[0]
    if (N | D | slots) >> 31:
        _past_32_bits()
    dt, dev = x.dtype, x.device
    code = _dtype_code(x)
    xs = _rows("x", x, (N, D), 1, dt, dev)
    gs = _rows("g", g, (N, D), 1, _gate_dtype(x, g), dev)
    ist = 0 if i is None else _rows("i", i, (N, D), 1, dt, dev)
    _t("scale", scale, (D,), torch.float32, dev, optional=True)
    _t("state", state, (slots, D), torch.float32, dev)
    _t("state_idx", state_idx, (N,), torch.int32, dev, optional=True)
    _on_gpu("x", x)
    if y is None:
        y = torch.empty_like(x)
    else:
        _t("y", y, (N, D), dt, dev)
    a = RecStepArgs(code, _dtype_code(g), N, D, x.data_ptr(), xs, g.data_ptr(), gs, _ptr(i), ist, _ptr(scale),
                    state.data_ptr(), _ptr(state_idx), slots, y.data_ptr())
    _call(lib().gdn_rec_step, a, dev)
    return y
