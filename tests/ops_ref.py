"""Plain 64-bit forms of the operators around the loss head, each with a bound
on how far a kernel that sums in fp32 may be from it.

``u`` = 2^-24 is half a step of fp32 and ``half(t)`` half a step of the stored
type relative to the value (``torch.finfo(t).eps / 2``).  A sum of n terms in
fp32, in chains of at most ``c`` additions, is off by at most c u times the sum
of the magnitudes.  The kernels keep at least 32 partial sums per row, so a row
of D terms has chains of at most D / 32 + 16 (the partial sums' own additions,
a few per level, are the 16); sums over rows may be one chain.
"""
import torch

U = 2.0 ** -24


def half(t):
    return torch.finfo(t).eps / 2


def d(t):
    return None if t is None else t.detach().cpu().double()


def chain(D):
    return -(-D // 32) + 16


def close(got, ref, bound, what=""):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= bound + 1e-38)
    # equal infinities and NaN in the same places are equal
    bad &= ~((got == ref) | (got.isnan() & ref.isnan()))
    if bad.any():
        i = tuple(int(k) for k in bad.nonzero()[0])
        raise AssertionError((what, "at", i, "got", float(got[i]), "want", float(ref[i]), "bound",
                              float(bound[i]) if isinstance(bound, torch.Tensor) else bound,
                              "bad", int(bad.sum()), "of", bad.numel()))


# ------------------------------------------------------------------ embedding

def embedding(ids, W, scale, dtype):
    """W rounded product: scale to fp32, the product in fp32, the store."""
    V = W.shape[0]
    ids, W = ids.cpu(), d(W)
    ok = (ids >= 0) & (ids < V)
    y = W[ids.clamp(0, V - 1)] * scale * ok[:, None]
    return y, y.abs() * (half(dtype) + 2 * U)


def embedding_grad(ids, dy, V, scale, padding_idx, base, dtype):
    ids, dy = ids.cpu(), d(dy)
    keep = (ids >= 0) & (ids < V)
    if padding_idx is not None:
        keep &= ids != padding_idx
    ids, dy = ids[keep], dy[keep]
    D = dy.shape[1]
    g = torch.zeros(V, D, dtype=torch.float64).index_add_(0, ids, dy * scale)
    mag = torch.zeros(V, D, dtype=torch.float64).index_add_(0, ids, (dy * scale).abs())
    n = torch.bincount(ids, minlength=V)[:, None].double()
    bound = (n + 3) * U * mag
    if base is not None:
        g = g + d(base)
        bound = bound + U * (d(base).abs() + mag)
    return g, bound + half(dtype) * g.abs() * (dtype != torch.float32)


# ---------------------------------------------------------------------- norms

def norm(x, w, b, eps, center, dtype):
    """(y, bound), (mean, bound), (rstd, bound)."""
    x, w, b = d(x), d(w), d(b)
    N, D = x.shape
    c = chain(D)
    zero = torch.zeros(N, 1, dtype=torch.float64)
    mean = x.mean(1, keepdim=True) if center else zero
    dm = (c + 2) * U * x.abs().mean(1, keepdim=True) if center else zero
    r = x - mean
    var = r.square().mean(1, keepdim=True)
    # around mean + dm the mean square grows by dm^2; each square and sum rounds;
    # a difference x - mean is rounded by u |x - mean| (2 u in its square)
    rel = (c + 6) * U + dm.square() / (var + eps)
    rstd = (var + eps).rsqrt()
    h = r * rstd
    y = h if w is None else h * w
    wa = 1.0 if w is None else w.abs()
    err = wa * (rstd * dm + h.abs() * (rel + 6 * U))
    out = y if b is None else y + b
    err = err + U * (y.abs() + (0 if b is None else b.abs()))
    err = err * (1 + half(dtype)) + half(dtype) * out.abs()
    return ((out, err), (mean[:, 0], dm[:, 0] + U * mean[:, 0].abs()),
            (rstd[:, 0], rstd[:, 0] * (rel[:, 0] + 4 * U)))


def norm_grad(x, dy, mean, rstd, w, center, dtype):
    """(dx, bound), (dw, bound), (db, bound) from the saved statistics."""
    x, dy, w = d(x), d(dy), d(w)
    N, D = x.shape
    c = chain(D)
    m = d(mean)[:, None] if center else torch.zeros(N, 1, dtype=torch.float64)
    r = d(rstd)[:, None]
    h = (x - m) * r
    dh = 3 * U * h.abs() + 2 * U * (x.abs() + m.abs()) * r
    g = dy if w is None else dy * w
    c1 = g.mean(1, keepdim=True) if center else torch.zeros(N, 1, dtype=torch.float64)
    c2 = (g * h).mean(1, keepdim=True)
    dc1 = (c + 4) * U * g.abs().mean(1, keepdim=True) if center else 0.0
    dc2 = (c + 4) * U * (g * h).abs().mean(1, keepdim=True) + (g.abs() * dh).mean(1, keepdim=True)
    dx = r * (g - c1 - h * c2)
    mag = r * (g.abs() + c1.abs() + (h * c2).abs())
    err = r * (dc1 + h.abs() * dc2 + c2.abs() * dh) + 6 * U * mag
    err = err * (1 + half(dtype)) + half(dtype) * dx.abs()
    dw, dwe = (dy * h).sum(0), (N + 4) * U * (dy * h).abs().sum(0) + (dy.abs() * dh).sum(0)
    db, dbe = dy.sum(0), (N + 4) * U * dy.abs().sum(0)
    return (dx, err), (dw, dwe), (db, dbe)


# ----------------------------------------------------------------- 4-bit head

def unpack4(packed, D):
    """q [V, D] from the layout of include/flce.h, word by word."""
    p = packed.cpu().contiguous().to(torch.int64)
    q = torch.empty(p.shape[0], D, dtype=torch.float64)
    for k in range(D):
        w, t, j = k % 128 // 32, k % 32 // 8, k % 8
        bit = 4 * (j // 2 + 4 * (j % 2))
        byte = k // 128 * 64 + 4 * (4 * t + w) + bit // 8
        q[:, k] = (p[:, byte] >> (bit % 8)) & 15
    return q


def head4_weights(packed, scales, zeros, D, group):
    q = unpack4(packed, D)
    of = torch.arange(D) // group
    z = 8.0 if zeros is None else zeros.cpu().double()[:, of]
    return (q - z) * d(scales)[:, of]


def head4(x, Wq, bias, group, dtype):
    """Tensor-core sums may cut instead of round: a step of fp32 each (2 u)."""
    x = d(x)
    D = x.shape[1]
    y = x @ Wq.t()
    mag = x.abs() @ Wq.abs().t()
    if bias is not None:
        y = y + d(bias)
        mag = mag + d(bias).abs()
    err = (chain(D) + 16) * 2 * U * mag
    return y, err * (1 + half(dtype)) + half(dtype) * y.abs() * (dtype != torch.float32)
