"""The operators around the loss head: embedding lookup, norms, 4-bit head.

Low-level calls (names of the C entry points in include/flce.h, caller-owned
buffers optional):
    embedding_fwd, embedding_bwd, layer_norm_fwd, layer_norm_bwd,
    rms_norm_fwd, rms_norm_bwd, head4_quantize, head4_logits
Autograd front ends:
    embedding(ids, W, *, scale=1.0, padding_idx=None, status=None)
    layer_norm(x, weight=None, bias=None, *, eps=1e-5)
    rms_norm(x, weight=None, *, eps=1e-5)

As in ``api``, PyTorch only allocates and supplies the current stream.  A
training step with a tied table keeps one fp32 gradient for both of its uses:
``flce_bwd(..., grad_W=gW)`` writes it and ``embedding_bwd(..., grad_W=gW,
accumulate_grad_W=True)`` adds the input side's rows.

To capture a step that calls ``backward()`` into a CUDA graph, run it before on
the capture stream and drop every eager graph of the same leaves (the loss
tensors that hold them): a leaf's gradient accumulation belongs to the stream
it was first used on, and one that an eager graph keeps alive pulls that
stream into the capture.
"""
from __future__ import annotations

import dataclasses
import functools
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _abi
from .api import _cuda, _dtype_code, new_status
from .api import _stream as _stream_of

_call = _abi.packed
_Tensor, _INT32, _INT64 = torch.Tensor, torch.int32, torch.int64

# A call on a few tokens costs less on the device than its checks here, so these
# ask a tensor for each property once.  The stream's handle comes from the same
# place that torch.cuda.current_stream takes it from.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device):
    if _raw_stream is None or device.index is None:
        return _stream_of(device)
    return _raw_stream(device.index)


def _addr(t):
    return 0 if t is None else t.data_ptr()


def _on(t, name, device):
    """t lies on `device` (a tensor elsewhere has another index, on the host -1)."""
    if not isinstance(t, _Tensor) or t.get_device() != device.index:
        _cuda(t, name)
        raise ValueError(f"{name} must be on {device}")


def _matrix(t, name, device=None):
    """A CUDA [rows, cols] argument with unit column stride: rows, cols, row stride."""
    if device is None:
        _cuda(t, name)
    else:
        _on(t, name, device)
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be 2-D with unit stride along its rows")
    rows, cols = shape
    return rows, cols, stride[0] if rows > 1 else cols


def _row_stride(t, name, rows, cols):
    """The row stride of a [rows, cols] output on the right device."""
    stride = t.stride()
    if stride[1] != 1 and cols > 1:
        raise ValueError(f"{name} must be 2-D with unit stride along its rows")
    return stride[0] if rows > 1 else cols


def _rows_of(t):
    """t as the calls take it: unit column stride, rows that do not overlap."""
    ok = (t.shape[1] <= 1 or t.stride(1) == 1) and (t.shape[0] <= 1 or t.stride(0) >= t.shape[1])
    return t if ok else t.contiguous()


def _output(t, name, shape, dtype, device):
    """An optional caller-owned output, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device.index:
        raise ValueError(f"{name} must be {dtype} of shape {list(shape)} on {device}")
    if len(shape) == 1 and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _vector(t, name, n, device, dtype=None):
    """An optional contiguous [n] argument."""
    if t is None:
        return None
    _on(t, name, device)
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{n}] tensor")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    return t


def _ids(ids, device):
    if not isinstance(ids, _Tensor) or ids.get_device() != device.index:
        _on(ids, "ids", device)
    shape = ids.shape
    if ids.dtype is not _INT64 or len(shape) != 1:
        raise ValueError("ids must be int64 of shape [N]")
    return ids.contiguous(), shape[0]


def _padding(padding_idx, V):
    if padding_idx is None:
        return -1
    p = int(padding_idx)
    if not 0 <= p < V:
        raise ValueError(f"padding_idx must lie in [0, {V})")
    return p


@functools.lru_cache(maxsize=512)
def _workspace_bytes(query, device_index, *sizes):
    """A workspace query's answer for a device: the plans go by its SMs."""
    with torch.cuda.device(device_index):
        return query(*sizes)


def _workspace(ws, device, query, *sizes):
    """The caller's workspace or a new one, and its bytes."""
    if ws is None:
        nbytes = _workspace_bytes(query, device.index, *sizes)
        return (torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes) if nbytes > 0 \
            else (None, 0)
    if not isinstance(ws, _Tensor) or ws.get_device() != device.index or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on {device}")
    return ws, ws.nbytes


def _status(status, device):
    """The caller's status word or a new one."""
    if status is None:
        return new_status(device)
    if not isinstance(status, _Tensor) or status.get_device() != device.index or \
            status.dtype is not _INT32 or status.numel() < 1:
        raise ValueError(f"status must be an int32 word on {device} (new_status)")
    return status


# ------------------------------------------------------------------ embedding

def embedding_fwd(ids, W, scale=1.0, *, out=None, status=None) -> torch.Tensor:
    """out[i] = scale * W[ids[i]] for ids [N] int64 and W [V, D] (bf16 or fp32,
    row stride free).  An id outside [0, V) gives a row of zeros and sets
    ``status`` (FLCE_ELABEL; a word of the caller's, else nobody can read it).
    ``out``/``status`` let a caller reuse buffers."""
    V, D, ldw = _matrix(W, "W")
    dev = W.device
    ids, N = _ids(ids, dev)
    out = _output(out, "out", (N, D), W.dtype, dev)
    ldo = _row_stride(out, "out", N, D)
    status = _status(status, dev)
    rc = _call.embedding_fwd(ids.data_ptr(), W.data_ptr(), _dtype_code(W), N, D, V, ldw,
                             float(scale), out.data_ptr(), ldo, status.data_ptr(), _stream(dev))
    _abi.check(rc, "embedding_fwd")
    return out


def embedding_bwd_workspace_bytes(N: int, D: int, V: int) -> int:
    """Bytes of device workspace embedding_bwd needs on the current device."""
    return int(_abi.embedding_bwd_workspace_bytes(N, D, V))


def embedding_bwd(ids, grad_out, V, scale=1.0, padding_idx=None, *, grad_W=None,
                  accumulate_grad_W=False, grad_dtype=torch.float32, ws=None,
                  status=None) -> torch.Tensor:
    """Gradient [V, D] of the table: scale times the sum of the rows of
    ``grad_out`` [N, D] by id, in fp32 and in a fixed order.  Written whole
    (``grad_W``, or a new tensor of ``grad_dtype``), or with
    ``accumulate_grad_W`` added to the fp32 ``grad_W``, whose other rows are
    not touched.  Tokens with id ``padding_idx`` are left out."""
    N, D, ldg = _matrix(grad_out, "grad_out")
    dev = grad_out.device
    ids, n = _ids(ids, dev)
    if n != N:
        raise ValueError(f"ids must be int64 of shape [{N}]")
    V = int(V)
    if accumulate_grad_W and grad_W is None:
        raise ValueError("accumulate_grad_W needs grad_W")
    grad_W = _output(grad_W, "grad_W", (V, D), grad_dtype if grad_W is None else grad_W.dtype, dev)
    ldw = _row_stride(grad_W, "grad_W", V, D)
    ws, ws_bytes = _workspace(ws, dev, embedding_bwd_workspace_bytes, N, D, V)
    status = _status(status, dev)
    rc = _call.embedding_bwd(_addr(ids), _addr(grad_out), _dtype_code(grad_out), N, D, V, ldg,
                             float(scale), _padding(padding_idx, V), _addr(grad_W),
                             _dtype_code(grad_W), ldw, 1 if accumulate_grad_W else 0, _addr(ws),
                             ws_bytes, _addr(status), _stream(dev))
    _abi.check(rc, "embedding_bwd")
    return grad_W


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, W, scale, padding_idx, status):
        if status is None and W.is_cuda:
            status = new_status(W.device)
        out = embedding_fwd(ids, W, scale, status=status)
        ctx.save_for_backward(ids)
        ctx.args = (W.shape[0], W.dtype, scale, padding_idx)
        ctx.status = status
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        (ids,) = ctx.saved_tensors
        V, dtype, scale, padding_idx = ctx.args
        gW = embedding_bwd(ids, _rows_of(g), V, scale, padding_idx, grad_dtype=dtype,
                           status=ctx.status)
        return None, gW, None, None, None


def embedding(ids, W, *, scale=1.0, padding_idx=None, status=None):
    """Embedding lookup scale * W[ids] with ids [...] int64, W [V, D]; returns
    [..., D].  The backward forms the dense gradient of W in W's dtype (one
    rounding of the fp32 sums); ids equal to ``padding_idx`` leave their row's
    gradient 0.  An id outside [0, V) gives a row of zeros and no gradient; both
    passes say so in ``status`` (new_status, read by check_status), if given:
    without it such ids go unseen."""
    if not isinstance(W, torch.Tensor) or W.dim() != 2:
        raise ValueError("W must be 2-D")
    if not isinstance(ids, torch.Tensor):
        raise ValueError("ids must be an int64 tensor")
    _padding(padding_idx, W.shape[0])
    out = _Embedding.apply(ids.reshape(-1), W, float(scale), padding_idx, status)
    return out.view(*ids.shape, W.shape[1])


# ---------------------------------------------------------------------- norms

@dataclasses.dataclass
class NormOut:
    """Outputs of a norm's forward (mean is None for rms_norm)."""
    y: torch.Tensor
    mean: Optional[torch.Tensor]   # [N] f32
    rstd: torch.Tensor             # [N] f32


@dataclasses.dataclass
class NormGrads:
    """Gradients of a norm's backward (None where not requested)."""
    grad_x: Optional[torch.Tensor]
    grad_weight: Optional[torch.Tensor]  # fp32
    grad_bias: Optional[torch.Tensor]    # fp32


def _norm_params(D, weight, bias, device):
    _vector(weight, "weight", D, device)
    _vector(bias, "bias", D, device)
    if weight is not None and bias is not None and weight.dtype is not bias.dtype:
        raise TypeError("weight and bias must share one dtype")
    p = weight if weight is not None else bias
    return _abi.FLCE_F32 if p is None else _dtype_code(p)


def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, *, y=None, mean=None,
                   rstd=None) -> NormOut:
    """Layer norm of the rows of x [N, D] (bf16 or fp32, row stride free) with
    weight and bias [D] (each optional, bf16 or fp32).  Returns y (dtype of x;
    ``y`` may be x itself) and the fp32 mean and rstd the backward needs."""
    N, D, ldx = _matrix(x, "x")
    dev = x.device
    wdt = _norm_params(D, weight, bias, dev)
    y = _output(y, "y", (N, D), x.dtype, dev)
    ldy = _row_stride(y, "y", N, D)
    mean = _output(mean, "mean", (N,), torch.float32, dev)
    rstd = _output(rstd, "rstd", (N,), torch.float32, dev)
    rc = _call.layer_norm_fwd(x.data_ptr(), _dtype_code(x), N, D, ldx, _addr(weight), _addr(bias),
                              wdt, float(eps), y.data_ptr(), ldy, mean.data_ptr(), rstd.data_ptr(),
                              _stream(dev))
    _abi.check(rc, "layer_norm_fwd")
    return NormOut(y, mean, rstd)


def rms_norm_fwd(x, weight=None, eps=1e-5, *, y=None, rstd=None) -> NormOut:
    """RMS norm of the rows of x [N, D]: layer norm without the mean and bias."""
    N, D, ldx = _matrix(x, "x")
    dev = x.device
    wdt = _norm_params(D, weight, None, dev)
    y = _output(y, "y", (N, D), x.dtype, dev)
    ldy = _row_stride(y, "y", N, D)
    rstd = _output(rstd, "rstd", (N,), torch.float32, dev)
    rc = _call.rms_norm_fwd(x.data_ptr(), _dtype_code(x), N, D, ldx, _addr(weight), wdt,
                            float(eps), y.data_ptr(), ldy, rstd.data_ptr(), _stream(dev))
    _abi.check(rc, "rms_norm_fwd")
    return NormOut(y, None, rstd)


def norm_bwd_workspace_bytes(N: int, D: int) -> int:
    """Bytes of device workspace layer_norm_bwd and rms_norm_bwd need on the current
    device."""
    return int(_abi.norm_bwd_workspace_bytes(N, D))


def _norm_bwd_args(x, N, D, grad_y, rstd, want_x, want_w, want_b, grad_x, grad_weight,
                   grad_bias, accumulate, ws):
    dev = x.device
    if grad_y.shape != (N, D) or grad_y.dtype is not x.dtype:
        raise ValueError("grad_y must have the shape and dtype of x")
    _vector(rstd, "rstd", N, dev, torch.float32)
    if rstd is None:
        raise ValueError("rstd must be given")
    if accumulate and ((want_w and grad_weight is None) or (want_b and grad_bias is None)):
        raise ValueError("accumulate needs the gradients to add to")
    gx = _output(grad_x, "grad_x", (N, D), x.dtype, dev) if want_x else None
    gw = _output(grad_weight, "grad_weight", (D,), torch.float32, dev) if want_w else None
    gb = _output(grad_bias, "grad_bias", (D,), torch.float32, dev) if want_b else None
    ws, ws_bytes = _workspace(ws, dev, norm_bwd_workspace_bytes, N, D) if want_w or want_b \
        else (None, 0)
    return gx, 0 if gx is None else _row_stride(gx, "grad_x", N, D), gw, gb, ws, ws_bytes


def layer_norm_bwd(x, grad_y, mean, rstd, weight=None, *, want_grad_x=True,
                   want_grad_weight=None, want_grad_bias=False, grad_x=None, grad_weight=None,
                   grad_bias=None, accumulate=False, ws=None) -> NormGrads:
    """Gradients of layer_norm_fwd from its x, mean, rstd and the incoming
    grad_y: grad_x (dtype of x; ``grad_x`` may be grad_y itself), grad_weight
    and grad_bias (fp32; added to the given ones when ``accumulate``)."""
    N, D, ldx = _matrix(x, "x")
    ldg = _matrix(grad_y, "grad_y", x.device)[2]
    wdt = _norm_params(D, weight, None, x.device)
    if mean is None:
        raise ValueError("mean must be given")
    _vector(mean, "mean", N, x.device, torch.float32)
    want_w = weight is not None if want_grad_weight is None else want_grad_weight
    gx, ldgx, gw, gb, ws, ws_bytes = _norm_bwd_args(x, N, D, grad_y, rstd, want_grad_x, want_w,
                                                    want_grad_bias, grad_x, grad_weight, grad_bias,
                                                    accumulate, ws)
    rc = _call.layer_norm_bwd(_addr(x), _dtype_code(x), N, D, ldx, _addr(grad_y), ldg,
                              _addr(weight), wdt, _addr(mean), _addr(rstd), _addr(gx), ldgx,
                              _addr(gw), _addr(gb),
                              1 if accumulate else 0, _addr(ws), ws_bytes, _stream(x.device))
    _abi.check(rc, "layer_norm_bwd")
    return NormGrads(gx, gw, gb)


def rms_norm_bwd(x, grad_y, rstd, weight=None, *, want_grad_x=True, want_grad_weight=None,
                 grad_x=None, grad_weight=None, accumulate=False, ws=None) -> NormGrads:
    """Gradients of rms_norm_fwd (see layer_norm_bwd)."""
    N, D, ldx = _matrix(x, "x")
    ldg = _matrix(grad_y, "grad_y", x.device)[2]
    wdt = _norm_params(D, weight, None, x.device)
    want_w = weight is not None if want_grad_weight is None else want_grad_weight
    gx, ldgx, gw, _, ws, ws_bytes = _norm_bwd_args(x, N, D, grad_y, rstd, want_grad_x, want_w,
                                                   False, grad_x, grad_weight, None, accumulate, ws)
    rc = _call.rms_norm_bwd(_addr(x), _dtype_code(x), N, D, ldx, _addr(grad_y), ldg, _addr(weight),
                            wdt, _addr(rstd), _addr(gx), ldgx, _addr(gw), 1 if accumulate else 0,
                            _addr(ws), ws_bytes, _stream(x.device))
    _abi.check(rc, "rms_norm_bwd")
    return NormGrads(gx, gw, None)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        x = _rows_of(x)
        out = layer_norm_fwd(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, out.mean, out.rstd)
        return out.y

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        x, weight, mean, rstd = ctx.saved_tensors
        need_x, need_w, need_b, _ = ctx.needs_input_grad
        # grad_weight / grad_bias are fp32; autograd casts them to the parameter
        # dtype when that differs
        o = layer_norm_bwd(x, _rows_of(g), mean, rstd, weight, want_grad_x=need_x,
                           want_grad_weight=need_w, want_grad_bias=need_b)
        return o.grad_x, o.grad_weight, o.grad_bias, None


class _RMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, eps):
        x = _rows_of(x)
        out = rms_norm_fwd(x, weight, eps)
        ctx.save_for_backward(x, weight, out.rstd)
        return out.y

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        x, weight, rstd = ctx.saved_tensors
        need_x, need_w, _ = ctx.needs_input_grad
        o = rms_norm_bwd(x, _rows_of(g), rstd, weight, want_grad_x=need_x,
                         want_grad_weight=need_w)
        return o.grad_x, o.grad_weight, None


def _norm_rows(x):
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must have a last dimension to normalise")
    return x.reshape(-1, x.shape[-1])


def layer_norm(x, weight=None, bias=None, *, eps=1e-5):
    """Layer norm over the last dimension of x [..., D]; weight and bias [D]
    are optional and may be fp32 beside a bf16 x."""
    return _LayerNorm.apply(_norm_rows(x), weight, bias, float(eps)).view(x.shape)


def rms_norm(x, weight=None, *, eps=1e-5):
    """RMS norm over the last dimension of x [..., D]."""
    return _RMSNorm.apply(_norm_rows(x), weight, float(eps)).view(x.shape)


# ------------------------------------------------------------------- 4-bit head

@dataclasses.dataclass
class Head4:
    """A head's weights in 4 bits (layout: include/flce.h, head4 section)."""
    packed: torch.Tensor            # [V, >= ceil(D / 128) * 64] uint8
    scales: torch.Tensor            # [V, ceil(D / group)] bf16 or f32
    zeros: Optional[torch.Tensor]   # [V, ceil(D / group)] uint8, or None (all 8)
    D: int
    group: int = 128

    @property
    def V(self):
        return self.packed.shape[0]


def _head4_args(head, device):
    V, width, ldp = _matrix(head.packed, "packed", device)
    if head.group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    if width < (head.D + 127) // 128 * 64:
        raise ValueError("packed must hold ceil(D / 128) * 64 bytes per row")
    shape = (V, -(-head.D // head.group))
    _on(head.scales, "scales", device)
    if head.scales.shape != shape or not head.scales.is_contiguous():
        raise ValueError(f"scales must be a contiguous {list(shape)} tensor")
    if head.zeros is not None:
        _on(head.zeros, "zeros", device)
        if head.zeros.shape != shape or not head.zeros.is_contiguous():
            raise ValueError(f"zeros must be a contiguous {list(shape)} tensor")
    if head.packed.dtype is not torch.uint8 or \
            (head.zeros is not None and head.zeros.dtype is not torch.uint8):
        raise TypeError("packed and zeros must be uint8")
    return V, ldp


def head4_quantize(W, group=128, *, zero_point=False, scale_dtype=None) -> Head4:
    """Rounds a head W [V, D] (bf16 or fp32, finite, row stride free) to 4 bits
    with a scale, and with ``zero_point`` a zero point, per ``group`` columns
    (32, 64 or 128) of a row.  ``scale_dtype`` defaults to W's."""
    V, D, ldw = _matrix(W, "W")
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    G = -(-D // group)
    head = Head4(torch.empty(V, -(-D // 128) * 64, dtype=torch.uint8, device=W.device),
                 torch.empty(V, G, dtype=scale_dtype or W.dtype, device=W.device),
                 torch.empty(V, G, dtype=torch.uint8, device=W.device) if zero_point else None,
                 D, group)
    ldp = head.packed.shape[1]
    rc = _abi.head4_quantize(_addr(W), _dtype_code(W), V, D, ldw, group, _addr(head.packed), ldp,
                             _addr(head.scales), _dtype_code(head.scales), _addr(head.zeros),
                             _stream(W.device))
    _abi.check(rc, "head4_quantize")
    return head


def head4_logits(x, head: Head4, bias=None, *, out=None,
                 out_dtype=torch.float32, status=None) -> torch.Tensor:
    """Logits [M, V] of the hidden states x [M, D] (bf16 or fp32): x times the
    head's 4-bit weights transposed (+ bias [V], dtype of x).  Made for M up to
    a few tens (decoding); ``out`` (bf16 or fp32) or ``out_dtype`` sets the
    logits' dtype.  A wait inside the kernel that gives up leaves NaN in its
    logits, and FLCE_ETIMEOUT in ``status`` (new_status), if given."""
    M, D, ldx = _matrix(x, "x")
    if D != head.D:
        raise ValueError(f"x must be [M, {head.D}]")
    dev = x.device
    V, ldp = _head4_args(head, dev)
    _vector(bias, "bias", V, dev, x.dtype)
    if status is not None:
        _status(status, dev)
    out = _output(out, "out", (M, V), out_dtype if out is None else out.dtype, dev)
    ldo = _row_stride(out, "out", M, V)
    dt = _dtype_code(x)
    rc = _call.head4_logits(x.data_ptr(), dt, M, D, ldx, head.packed.data_ptr(), ldp,
                            head.scales.data_ptr(), _dtype_code(head.scales), _addr(head.zeros),
                            head.group, V, _addr(bias), out.data_ptr(), _dtype_code(out), ldo,
                            _addr(status), _stream(dev))
    _abi.check(rc, "head4_logits")
    return out
