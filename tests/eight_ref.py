"""Plain forms of the operators in 8 bits and of beam search, with bounds (the
notation of ops_ref.py).

Rounding to e4m3 is off by at most half a step, 2^-4 of a normal number (from 2^-6
on) and 2^-10 below.  A block's 128 products are exact in fp32; the tensor cores'
sum of them, in an order and with roundings of their own, is taken as off by at
most one step (2 u) of the magnitudes' sum for each term.
"""
import torch

from ops_ref import U, d, half

MOST, LEAST = 448.0, 2.0 ** -100
E4M3 = torch.float8_e4m3fn


def ceil(n, k):
    return -(-n // k)


def blocks(t, rows):
    """t [R, K] as [R / rows, rows, K / 128, 128], filled up with zeros."""
    R, K = t.shape
    full = torch.zeros(ceil(R, rows) * rows, ceil(K, 128) * 128, dtype=t.dtype)
    full[:R, :K] = t
    return full.view(-1, rows, full.shape[1] // 128, 128)


def quantize(t, rows):
    """(data, scales) by the definition, in fp32 on the host: bits are compared."""
    R, K = t.shape
    b = blocks(t.detach().cpu().float(), rows)
    a = b.abs().amax((1, 3)).clamp_min(LEAST)
    top = torch.full_like(a, MOST)
    q = (b * (top / a)[:, None, :, None]).reshape(-1, b.shape[2] * 128)[:R, :K]
    return q.to(E4M3), a / top


def spread(scales, rows, R, K):
    return scales.repeat_interleave(rows, 0)[:R].repeat_interleave(128, 1)[:, :K]


def value(q):
    """What a Quant8 stands for, in 64 bits."""
    R, K = q.data.shape
    return q.data.cpu().double() * spread(d(q.scales), q.rows, R, K)


def rounded8(y, bound, q, what=""):
    """q is y [N, D] (64 bits, a kernel's fp32 value within `bound`) in 8 bits by rows."""
    N, D = y.shape
    a = blocks(y.abs(), 1).amax((1, 3)).clamp_min(LEAST)
    off = blocks(bound.expand(N, D), 1).amax((1, 3))
    scales = d(q.scales)
    assert ((scales - a / MOST).abs() <= (off + 2 * U * a) / MOST).all(), (what, "scales")
    s = spread(scales, 1, N, D)
    v = y / s
    step = (v.abs() * 2.0 ** -4).clamp_min(2.0 ** -10)
    # the number rounded is within the bound and three fp32 roundings of v
    slack = (bound / s + 4 * U * v.abs()) * 1.25
    err = (q.data.cpu().double() - v).abs()
    assert (err <= step + slack).all(), (what, "numbers", float((err - step - slack).max()))


def gemm(a, b, bias, base, dtype):
    """(y, bound) of gemm8."""
    x, w = value(a), value(b)
    y, mag = x @ w.t(), x.abs() @ w.t().abs()
    K = x.shape[1]
    bound = (min(K, 128) * 2 + ceil(K, 128) + 4) * U * mag
    if bias is not None:
        y = y + d(bias)
        bound = bound + U * y.abs()
    if base is not None:
        y = y + d(base)
        bound = bound + U * y.abs()
    return y, bound + (half(dtype) * (y.abs() + bound) if dtype != torch.float32 else 0)


def beam(logits, scores, K, num, finished, pad):
    """Scores [B, num] in 64 bits, tokens, parents: the definition, candidate by candidate."""
    z, s = d(logits), d(scores)
    R, V = z.shape
    out = []
    for b in range(R // K):
        total = torch.full((K, V), float("-inf"), dtype=torch.float64)
        for k in range(K):
            r = b * K + k
            if not torch.isfinite(s[r]):
                continue
            if finished is not None and bool(finished[r]):
                total[k, pad] = s[r]
                continue
            lse = torch.logsumexp(z[r], 0)
            if torch.isfinite(lse):
                total[k] = s[r] + (z[r] - lse)
        order = torch.sort(total.flatten(), descending=True, stable=True)
        out.append((order.values[:num], order.indices[:num] % V, order.indices[:num] // V))
    return [torch.stack(x) for x in zip(*out)]
