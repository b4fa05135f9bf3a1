"""Beam search on the head's logits.

Low-level calls (names of the C entry points in include/flce.h, caller-owned
buffers optional):
    beam_select   the best continuations of each request's beams
    beam_reorder_ caches and histories put in the order of the beams selected
"""
from __future__ import annotations

import dataclasses
import functools
import struct

import torch

from . import _abi
from .api import _dtype_code
from .ops import _addr, _call, _matrix, _on, _output, _status, _stream, _vector, _workspace


@dataclasses.dataclass
class BeamOut:
    """What beam_select selects, best first (reusable through ``out=``)."""
    scores: torch.Tensor   # [B, num] f32
    tokens: torch.Tensor   # [B, num] i64
    parents: torch.Tensor  # [B, num] i64, a beam of the request: 0 .. K - 1


def beam_select_workspace_bytes(B: int, K: int, V: int, num: int) -> int:
    """Bytes of device workspace beam_select needs."""
    return int(_abi.beam_select_workspace_bytes(B, K, V, num))


def beam_select(logits, scores, beams, num=None, *, finished=None, pad_id=0, out=None,
                ws=None) -> BeamOut:
    """Of each request's ``beams`` rows of logits [B * beams, V] (bf16 or fp32, row
    stride free) the ``num`` (default: beams) best continuations by score plus log
    probability; scores [B * beams] f32.  Beams marked in ``finished`` ([B * beams]
    bool) go on with ``pad_id`` at their own score.  Ties, -infinity and NaN:
    include/flce.h."""
    R, V, ld = _matrix(logits, "logits")
    dev = logits.device
    K = int(beams)
    num = K if num is None else int(num)
    if K < 1 or R % K != 0:
        raise ValueError("logits must have a multiple of `beams` rows")
    B = R // K
    if scores is None:
        raise ValueError("scores must be given")
    _vector(scores, "scores", R, dev, torch.float32)
    if finished is not None:
        _vector(finished, "finished", R, dev)
        if finished.dtype not in (torch.bool, torch.uint8):
            raise TypeError("finished must be bool or uint8")
    if out is None:
        tokens = torch.empty(B, num, dtype=torch.int64, device=dev)
        out = BeamOut(torch.empty(B, num, dtype=torch.float32, device=dev), tokens,
                      torch.empty_like(tokens))
    else:
        for t, name, dt in ((out.scores, "scores", torch.float32),
                            (out.tokens, "tokens", torch.int64),
                            (out.parents, "parents", torch.int64)):
            _output(t, "out." + name, (B, num), dt, dev)
            if not t.is_contiguous():
                raise ValueError(f"out.{name} must be contiguous")
    ws, ws_bytes = _workspace(ws, dev, beam_select_workspace_bytes, B, K, V, num)
    rc = _call.beam_select(logits.data_ptr(), _dtype_code(logits), B, K, V, ld, scores.data_ptr(),
                           _addr(finished), int(pad_id), num, out.scores.data_ptr(),
                           out.tokens.data_ptr(), out.parents.data_ptr(), _addr(ws), ws_bytes,
                           _stream(dev))
    _abi.check(rc, "beam_select")
    return out


@functools.lru_cache(maxsize=512)
def _runs(shape, stride, size):
    """A state's row stride, and its rows as runs: how many, how far apart, how long, in
    bytes; None where that takes more than one outer stride."""
    dims = sorted((st, n) for n, st in zip(shape[1:], stride[1:]) if n != 1)
    run = 1
    while dims and dims[0][0] == run:
        run *= dims.pop(0)[1]
    outer, step = 1, 0
    if dims:
        step = dims[0][0]
        while dims and dims[0][0] == step * outer:
            outer *= dims.pop(0)[1]
    if dims:
        return None
    return stride[0] * size, outer, step * size, run * size


def beam_reorder_(states, parents, *, status=None) -> None:
    """Puts the beams' states in the order of ``parents`` [B, K] (beam_select's), in
    place: of each tensor [B * K, ...] row b * K + k becomes what row
    b * K + parents[b, k] was.  A state may be a slice (the filled part of a cache)
    whose rows have at most one gap in their order in memory.  A parent outside
    [0, K) leaves its row as it was and sets FLCE_ELABEL in ``status``
    (new_status), if given."""
    if not isinstance(parents, torch.Tensor) or not parents.is_cuda or \
            parents.dtype is not torch.int64 or parents.dim() != 2 or \
            not parents.is_contiguous():
        raise ValueError("parents must be a contiguous int64 CUDA tensor [B, K]")
    dev = parents.device
    index = dev.index
    B, K = parents.shape
    R = B * K
    rows, shape, stride, dtype, runs = [], None, None, None, ()
    for i, t in enumerate(states):
        if not isinstance(t, torch.Tensor) or t.get_device() != index:
            _on(t, f"states[{i}]", dev)
        # caches mostly come in one layout
        if t.shape != shape or t.stride() != stride or t.dtype is not dtype:
            shape, stride, dtype = t.shape, t.stride(), t.dtype
            if len(shape) < 1 or shape[0] != R:
                raise ValueError(f"states[{i}] must have {R} rows")
            runs = _runs(shape, stride, t.element_size()) if t.numel() > 0 else ()
            if runs is None:
                raise ValueError(f"states[{i}]: more than one gap in a row's order in memory")
        if runs:
            rows.append(t.data_ptr())
            rows += runs
    if not rows:
        return
    if status is not None:
        _status(status, dev)
    rc = _abi.beam_reorder(struct.pack("=" + "Qqqqq" * (len(rows) // 5), *rows), len(rows) // 5, B,
                           K, parents.data_ptr(), None if status is None else status.data_ptr(),
                           _stream(dev))
    _abi.check(rc, "beam_reorder")
