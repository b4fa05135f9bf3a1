"""Matrices in 8 bits with a scale per block of 128, the norm that writes them and
the products that read them.

Low-level calls (names of the C entry points in include/flce.h, caller-owned
buffers optional):
    rms_norm_add_fwd, rms_norm_add_bwd, quantize8 (quantize8_pair with the
    transpose), gemm8
Autograd front ends:
    rms_norm_add(x, residual, weight=None, *, eps=1e-5) -> y, summed
    linear8(x, W)

A step that calls ``backward()`` is captured as ``ops`` says: run before on the
capture stream, with no eager graph of the same leaves alive.
"""
from __future__ import annotations

import dataclasses
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _abi
from .api import _cuda, _dtype_code
from .ops import (_addr, _call, _matrix, _norm_params, _on, _output, _row_stride, _rows_of,
                  _status, _stream, _vector, _workspace, NormGrads, norm_bwd_workspace_bytes)

_F32, _E4M3 = torch.float32, torch.float8_e4m3fn


@dataclasses.dataclass
class Quant8:
    """A matrix [R, K] in 8 bits (include/flce.h): data[r, k] * scales[r / rows, k / 128]."""
    data: torch.Tensor    # [R, K] float8_e4m3fn, rows of a multiple of 16 bytes
    scales: torch.Tensor  # [ceil(R / rows), ceil(K / 128)] f32
    rows: int = 1         # rows to a scale: 1 or 128


def _new8(R, K, rows, device):
    ld = -(-K // 16) * 16
    return Quant8(torch.empty_strided((R, K), (ld, 1), dtype=_E4M3, device=device),
                  torch.empty(R if rows == 1 else -(-R // 128), -(-K // 128), dtype=_F32,
                              device=device), rows)


def _matrix8(q, name, device):
    """A matrix in 8 bits: rows, columns, row stride."""
    if not isinstance(q, Quant8):
        raise ValueError(f"{name} must be a Quant8")
    data, scales, rows = q.data, q.scales, q.rows
    if rows != 1 and rows != 128:
        raise ValueError(f"{name}.rows must be 1 or 128")
    R, K, ld = _matrix(data, "data", device)
    if data.dtype is not _E4M3:
        raise TypeError(f"{name}.data must be float8_e4m3fn")
    if not isinstance(scales, torch.Tensor) or scales.get_device() != device.index:
        _on(scales, f"{name}.scales", device)
    G = -(-K // 128)
    if scales.dtype is not _F32 or scales.shape != (R if rows == 1 else -(-R // 128), G) or \
            not scales.is_contiguous():
        raise ValueError(f"{name}.scales must be a contiguous float32 tensor: {rows} rows and "
                         "128 columns to a scale")
    return R, K, ld if R > 1 else -(-K // 16) * 16


def _output8(q, name, R, K, rows, device):
    """An optional caller-owned matrix in 8 bits, or a new one; its row stride."""
    if q is None:
        q = _new8(R, K, rows, device)
        return q, -(-K // 16) * 16
    has_R, has_K, ld = _matrix8(q, name, device)
    if has_R != R or has_K != K or q.rows != rows:
        raise ValueError(f"{name} must be [{R}, {K}] with {rows} rows to a scale")
    return q, ld


# ------------------------------------------------- the norm of a residual stream

@dataclasses.dataclass
class NormAddOut:
    """Outputs of rms_norm_add_fwd (None where not asked for)."""
    y: Optional[torch.Tensor]
    summed: Optional[torch.Tensor]
    rstd: torch.Tensor  # [N] f32
    quant: Optional[Quant8]


def rms_norm_add_fwd(x, residual=None, weight=None, eps=1e-5, *, want_y=True, want_quant=False,
                     y=None, summed=None, rstd=None, quant=None) -> NormAddOut:
    """The residual stream summed = x + residual (dtype of x; ``summed`` may be x or
    residual itself) and its RMS norm, rows [N, D] of bf16 or fp32, row strides
    free: y in x's dtype, and with ``want_quant`` (or a ``quant`` to write) in 8
    bits with a scale per 128 columns.  residual None: the norm of x, which is not
    copied unless ``summed`` is given."""
    N, D, ldx = _matrix(x, "x")
    dev, dt = x.device, x.dtype
    if weight is None:
        wdt, w = _abi.FLCE_F32, 0
    else:
        wdt, w = _dtype_code(_vector(weight, "weight", D, dev)), weight.data_ptr()
    ldr = lds = ldy = ldq = r = sum_ = y_ = q_ = scales = 0
    if residual is not None:
        has_N, has_D, ldr = _matrix(residual, "residual", dev)
        if has_N != N or has_D != D or residual.dtype is not dt:
            raise ValueError("residual must have the shape and dtype of x")
        r = residual.data_ptr()
    if residual is not None or summed is not None:
        summed = _output(summed, "summed", (N, D), dt, dev)
        lds, sum_ = _row_stride(summed, "summed", N, D), summed.data_ptr()
    if want_y or y is not None:
        y = _output(y, "y", (N, D), dt, dev)
        ldy, y_ = _row_stride(y, "y", N, D), y.data_ptr()
    if want_quant or quant is not None:
        quant, ldq = _output8(quant, "quant", N, D, 1, dev)
        q_, scales = quant.data.data_ptr(), quant.scales.data_ptr()
    elif y is None:
        raise ValueError("one of y and quant must be asked for")
    rstd = _output(rstd, "rstd", (N,), _F32, dev)
    rc = _call.rms_norm_add_fwd(x.data_ptr(), _dtype_code(x), N, D, ldx, r, ldr, w, wdt,
                                float(eps), sum_, lds, y_, ldy, q_, ldq, scales, rstd.data_ptr(),
                                _stream(dev))
    _abi.check(rc, "rms_norm_add_fwd")
    return NormAddOut(y, summed, rstd, quant)


def rms_norm_add_bwd(summed, grad_y, grad_summed, rstd, weight=None, *, want_grad_x=True,
                     want_grad_weight=None, grad_x=None, grad_weight=None, accumulate=False,
                     ws=None) -> NormGrads:
    """Gradients of rms_norm_add_fwd: grad_x, that of x and of the residual alike, is
    the norm's plus grad_summed, what comes back along the stream (None: nothing;
    ``grad_x`` may be grad_y or grad_summed itself); grad_weight as in rms_norm_bwd."""
    N, D, lds = _matrix(summed, "summed")
    dev = summed.device
    ldgy = _matrix(grad_y, "grad_y", dev)[2]
    ldgs = 0
    if grad_summed is not None:
        ldgs = _matrix(grad_summed, "grad_summed", dev)[2]
    for g, name in ((grad_y, "grad_y"), (grad_summed, "grad_summed")):
        if g is not None and (g.shape != (N, D) or g.dtype is not summed.dtype):
            raise ValueError(f"{name} must have the shape and dtype of summed")
    wdt = _norm_params(D, weight, None, dev)
    if rstd is None:
        raise ValueError("rstd must be given")
    _vector(rstd, "rstd", N, dev, _F32)
    want_w = weight is not None if want_grad_weight is None else want_grad_weight
    if accumulate and want_w and grad_weight is None:
        raise ValueError("accumulate needs the gradient to add to")
    gx = _output(grad_x, "grad_x", (N, D), summed.dtype, dev) if want_grad_x else None
    gw = _output(grad_weight, "grad_weight", (D,), _F32, dev) if want_w else None
    ws, ws_bytes = _workspace(ws, dev, norm_bwd_workspace_bytes, N, D) if want_w else (None, 0)
    rc = _call.rms_norm_add_bwd(_addr(summed), _dtype_code(summed), N, D, lds, _addr(grad_y), ldgy,
                                _addr(grad_summed), ldgs, _addr(weight), wdt, _addr(rstd),
                                _addr(gx), 0 if gx is None else _row_stride(gx, "grad_x", N, D),
                                _addr(gw), 1 if accumulate else 0, _addr(ws), ws_bytes,
                                _stream(dev))
    _abi.check(rc, "rms_norm_add_bwd")
    return NormGrads(gx, gw, None)


class _RMSNormAdd(torch.autograd.Function):
    """Takes tensors of any shape, so that x and residual get one tensor as gradient:
    autograd then gives each leaf memory of its own, which it does not for two views."""
    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        D = x.shape[-1]
        y, summed = (torch.empty(x.shape, dtype=x.dtype, device=x.device) for _ in range(2))
        o = rms_norm_add_fwd(_rows_of(x.reshape(-1, D)), _rows_of(residual.reshape(-1, D)), weight,
                             eps, y=y.view(-1, D), summed=summed.view(-1, D))
        ctx.save_for_backward(summed, weight, o.rstd)
        ctx.set_materialize_grads(False)
        return y, summed

    @staticmethod
    @once_differentiable
    def backward(ctx, gy, gs):
        summed, weight, rstd = ctx.saved_tensors
        need_x, need_r, need_w, _ = ctx.needs_input_grad
        if gy is None:  # only the stream goes on
            return gs if need_x else None, gs if need_r else None, None, None
        D = summed.shape[-1]
        o = rms_norm_add_bwd(summed.view(-1, D), _rows_of(gy.reshape(-1, D)),
                             None if gs is None else _rows_of(gs.reshape(-1, D)), rstd, weight,
                             want_grad_x=need_x or need_r, want_grad_weight=need_w)
        g = None if o.grad_x is None else o.grad_x.view(summed.shape)
        return g if need_x else None, g if need_r else None, o.grad_weight, None


def rms_norm_add(x, residual, weight=None, *, eps=1e-5):
    """The residual stream x + residual [..., D] and its RMS norm over the last
    dimension: returns (y, summed)."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must have a last dimension to normalise")
    if not isinstance(residual, torch.Tensor) or residual.shape != x.shape:
        raise ValueError("residual must have the shape of x")
    return _RMSNormAdd.apply(x, residual, weight, float(eps))


# --------------------------------------------------------------- to 8 bits, products

def _quantize8(x, rows, plain, transposed, q, qt):
    R, C, ldx = _matrix(x, "x")
    dev = x.device
    if rows not in (1, 128):
        raise ValueError("rows must be 1 or 128")
    ldq = ldqt = 0
    if plain:
        q, ldq = _output8(q, "out", R, C, rows, dev)
    if transposed:
        qt, ldqt = _output8(qt, "out_t", C, R, rows, dev)
    rc = _call.quantize8(x.data_ptr(), _dtype_code(x), R, C, ldx, rows,
                         q.data.data_ptr() if plain else 0, ldq,
                         q.scales.data_ptr() if plain else 0,
                         qt.data.data_ptr() if transposed else 0, ldqt,
                         qt.scales.data_ptr() if transposed else 0, _stream(dev))
    _abi.check(rc, "quantize8")
    return q, qt


def quantize8(x, rows=1, *, transpose=False, out=None) -> Quant8:
    """x [R, C] (bf16 or fp32, row stride free) in 8 bits, one scale for 128 columns of
    ``rows`` rows (1 or 128); with ``transpose`` that of x^T [C, R]."""
    if transpose:
        return _quantize8(x, rows, False, True, None, out)[1]
    return _quantize8(x, rows, True, False, out, None)[0]


def quantize8_pair(x, rows=1, *, out=None, out_t=None):
    """(x, x^T) in 8 bits, each with ``rows`` of its rows to a scale, x read once."""
    return _quantize8(x, rows, True, True, out, out_t)


def gemm8(a: Quant8, b: Quant8, bias=None, *, out=None, out_dtype=torch.float32,
          accumulate=False, status=None) -> torch.Tensor:
    """a b^T (+ bias [N], bf16 or fp32) of a [M, K] (rows 1) and b [N, K] (rows 1 or
    128): [M, N] in ``out`` or a new tensor of ``out_dtype`` (bf16 or fp32).  From one
    token's head or layer to a long batch's (whose results are stored fastest in rows
    of a multiple of 16 bytes: an ``out`` with padding where N is odd).  ``accumulate``
    adds to the fp32 ``out``.  A wait inside the kernel that gives up leaves NaN, and FLCE_ETIMEOUT
    in ``status`` (new_status), if given."""
    if not isinstance(a, Quant8) or a.rows != 1:
        raise ValueError("a must be a Quant8 with one row to a scale")
    dev = _cuda(a.data, "a.data").device
    M, K, lda = _matrix8(a, "a", dev)
    N, Kb, ldb = _matrix8(b, "b", dev)
    if K != Kb:
        raise ValueError(f"b must be [N, {K}]")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    _vector(bias, "bias", N, dev)
    if status is not None:
        _status(status, dev)
    out = _output(out, "out", (M, N), out_dtype if out is None else out.dtype, dev)
    ldo = _row_stride(out, "out", M, N)
    rc = _call.gemm8(a.data.data_ptr(), lda, a.scales.data_ptr(), M, b.data.data_ptr(), ldb,
                     b.scales.data_ptr(), b.rows, N, K, _addr(bias),
                     _abi.FLCE_F32 if bias is None else _dtype_code(bias), out.data_ptr(),
                     _dtype_code(out), ldo, 1 if accumulate else 0, _addr(status), _stream(dev))
    _abi.check(rc, "gemm8")
    return out


class _Linear8(torch.autograd.Function):
    """recorded: whether a backward pass can follow (needs_input_grad does not say so: it
    stays true for a leaf where gradients are switched off)."""
    @staticmethod
    def forward(ctx, x, W, recorded):
        need_x, need_w = (need and recorded for need in ctx.needs_input_grad[:2])
        x8, x8t = _quantize8(_rows_of(x), 1, True, need_w, None, None)
        w8, w8t = _quantize8(_rows_of(W), 128, True, need_x, None, None)
        ctx.dtypes = x.dtype, W.dtype
        saved = []
        for q in (x8t, w8t):
            saved += [None, None] if q is None else [q.data, q.scales]
        ctx.save_for_backward(*saved)
        return gemm8(x8, w8, out_dtype=x.dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        xt, xt_scales, wt, wt_scales = ctx.saved_tensors
        need_x, need_w, _ = ctx.needs_input_grad
        dx, dw = ctx.dtypes
        if not (need_x or need_w):
            return None, None, None
        g8, g8t = _quantize8(_rows_of(g), 1, need_x, need_w, None, None)
        gx = gemm8(g8, Quant8(wt, wt_scales, 128), out_dtype=dx) if need_x else None
        gW = None
        if need_w and g.shape[0] == 0:  # no token
            gW = torch.zeros(g.shape[1], xt.shape[0], dtype=dw, device=g.device)
        elif need_w:
            gW = gemm8(g8t, Quant8(xt, xt_scales), out_dtype=dw)
        return gx, gW, None


def linear8(x, W):
    """x W^T with x [..., K] and W [N, K] (bf16 or fp32), rounded to 8 bits for the
    product (x by rows, W by squares of 128), and both gradients the same way from
    the incoming one; results in x's dtype, the gradient of W in W's."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must have a last dimension")
    if not isinstance(W, torch.Tensor) or W.dim() != 2 or W.shape[1] != x.shape[-1]:
        raise ValueError(f"W must be [N, {x.shape[-1]}]")
    y = _Linear8.apply(x.reshape(-1, x.shape[-1]), W, torch.is_grad_enabled())
    return y.view(*x.shape[:-1], W.shape[0])
