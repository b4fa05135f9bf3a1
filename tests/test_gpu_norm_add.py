"""The residual norm, forward (y, 8 bits, both) and backward, against 64-bit forms
(bounds: ops_ref.py, eight_ref.py)."""
import pytest
import torch

import eight_ref as E
import ops_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


@pytest.fixture(scope="module")
def lh():
    import lm_head_linear_fwd_gb300 as m
    return m


def _randn(shape, dtype, seed, std=1.0, mean=0.0, pad=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    N, D = shape
    flat = torch.randn(N * (D + pad) + shift, generator=g).mul_(std).add_(mean).to(dtype).cuda()
    return flat[shift:].view(N, D + pad)[:, :D]


def _vec(D, dtype, seed):
    return _randn((1, D), dtype, seed, 0.3, 1.0)[0].contiguous()


def _check(x, res, w, o, quant):
    dt = x.dtype
    full = R.d(x) + (0 if res is None else R.d(res))
    r = o.summed if o.summed is not None else x
    # fp32 sum, then the type: the sum of two numbers may take two roundings
    R.close(r, full, full.abs() * (R.half(dt) + 2 * R.U), "summed")
    y, _, rstd = R.norm(r, w, None, EPS, False, F32)
    R.close(o.rstd, *rstd, "rstd")
    if o.y is not None:
        R.close(o.y, y[0], y[1] + (R.half(dt) * y[0].abs() * 1.01 if dt == BF else 0), "y")
    if quant:
        E.rounded8(*y, o.quant)


SHAPES = [(1, 1), (1, 2), (3, 7), (5, 64), (3, 129), (40, 768), (7, 1601), (3, 4096), (2, 5120),
          (3, 8191), (2, 16384), (2, 20001), (1, 70000), (700, 200), (1000, 33)]
LAYOUT = [(BF, BF, 0, 0), (BF, F32, 3, 1), (F32, F32, 0, 0), (F32, BF, 2, 3), (BF, BF, 8, 8)]


@pytest.mark.parametrize("N,D", SHAPES)
@pytest.mark.parametrize("dtype,wdtype,pad,shift", LAYOUT)
def test_forward(lh, N, D, dtype, wdtype, pad, shift):
    x = _randn((N, D), dtype, 1, 0.5, 0.0, pad, shift)
    res = _randn((N, D), dtype, 2, 2.0, 0.5, pad, shift)
    w = _vec(D, wdtype, 3)
    o = lh.rms_norm_add_fwd(x, res, w, EPS, want_quant=True)
    _check(x, res, w, o, True)
    for kw in (dict(), dict(want_y=False, want_quant=True)):  # each output alone
        p = lh.rms_norm_add_fwd(x, res, w, EPS, **kw)
        assert torch.equal(p.summed, o.summed) and torch.equal(p.rstd, o.rstd)
        if p.y is not None:
            assert torch.equal(p.y, o.y) and p.quant is None
        else:
            assert torch.equal(p.quant.data.view(torch.uint8), o.quant.data.view(torch.uint8))
            assert torch.equal(p.quant.scales, o.quant.scales)
    # the stream in place, other strides, y in x's place
    res2 = torch.empty(N, D + pad, dtype=dtype, device="cuda")[:, :D].copy_(res)
    x2 = torch.empty(N, D + 5, dtype=dtype, device="cuda")[:, :D].copy_(x)
    # (rows that begin elsewhere are added up in another order)
    p = lh.rms_norm_add_fwd(x2, res2, w, EPS, summed=res2, y=x2)
    assert torch.equal(res2, o.summed) and p.y is x2
    _check(x, res, w, p, False)
    # neighbours of the outputs
    wide = torch.full((N, D + 5), 7.0, dtype=dtype, device="cuda")
    also = torch.full((N, D + 5), 7.0, dtype=dtype, device="cuda")
    ldq = E.ceil(D, 16) * 16 + 32
    q8 = torch.full((N, ldq), 0x55, dtype=torch.uint8, device="cuda")
    q = lh.Quant8(q8.view(E.E4M3)[:, 16:16 + D], torch.empty(N, E.ceil(D, 128), device="cuda"))
    p = lh.rms_norm_add_fwd(x, res, w, EPS, y=wide[:, 2:2 + D], summed=also[:, 3:3 + D], quant=q)
    assert torch.equal(also[:, 3:3 + D], o.summed)
    _check(x, res, w, p, True)
    assert (wide[:, :2] == 7).all() and (wide[:, 2 + D:] == 7).all()
    assert (also[:, :3] == 7).all() and (also[:, 3 + D:] == 7).all()
    assert (q8[:, :16] == 0x55).all() and (q8[:, 16 + D:] == 0x55).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [96, 1601, 21000])
def test_without_residual(lh, dtype, D):
    x, w = _randn((9, D), dtype, 1), _vec(D, F32, 2)
    o = lh.rms_norm_add_fwd(x, None, w, EPS, want_quant=True)
    assert o.summed is None
    _check(x, None, w, o, True)
    kept = torch.empty_like(x)
    p = lh.rms_norm_add_fwd(x, None, w, EPS, summed=kept, want_quant=True)
    assert torch.equal(kept, x) and torch.equal(p.y, o.y)
    o = lh.rms_norm_add_fwd(x, x, None, EPS)  # the same rows twice, no weight
    _check(x, x, None, o, False)


@pytest.mark.parametrize("D", [256, 21000])
def test_forward_values(lh, D):
    """Rows of zeros, tiny, huge, with an infinity, with a NaN; many rows."""
    N = 2500 if D < 1000 else 12
    x, res = _randn((N, D), F32, 1), _randn((N, D), F32, 2)
    x[0], res[0] = 0.0, 0.0
    x[1] *= 1e-25
    res[1] = 0.0
    x[2, 5], res[3, 9] = float("inf"), float("nan")
    o = lh.rms_norm_add_fwd(x, res, None, EPS, want_quant=True)
    keep = torch.ones(N, dtype=torch.bool)
    keep[2:4] = False
    k = keep.cuda()
    part = lh.NormAddOut(o.y[k], o.summed[k], o.rstd[k],
                         lh.Quant8(o.quant.data.view(torch.uint8)[k].view(E.E4M3),
                                   o.quant.scales[k]))
    _check(x[k], res[k], None, part, True)
    assert (o.y[0] == 0).all() and (o.quant.scales[0] == E.LEAST / 448).all()
    assert o.y[2, 5].isnan() and o.quant.data.float()[2, 5].isnan()
    assert o.y[3].isnan().all() and o.quant.scales[3].isnan().all()
    assert o.quant.data.float()[3].isnan().all()


@pytest.mark.parametrize("N,D", SHAPES + [(333, 4096)])
@pytest.mark.parametrize("dtype,wdtype,pad,shift", LAYOUT)
def test_backward(lh, N, D, dtype, wdtype, pad, shift):
    r = _randn((N, D), dtype, 1, 2.0, 0.5, pad, shift)
    gy = _randn((N, D), dtype, 4, 0.1, 0.02, pad, shift)
    gs = _randn((N, D), dtype, 5, 0.2, 0.0, pad, shift)
    w = _vec(D, wdtype, 2)
    rstd = lh.rms_norm_fwd(r, w, EPS).rstd
    o = lh.rms_norm_add_bwd(r, gy, gs, rstd, w)
    (dx, bx), dw, _ = R.norm_grad(r, gy, None, rstd, w, False, F32)
    want = dx + R.d(gs)
    # one fp32 addition more, one rounding to the type
    R.close(o.grad_x, want, bx + 2 * R.U * (dx.abs() + R.d(gs).abs()) +
            (R.half(dtype) * (want.abs() + bx) * 1.01 if dtype == BF else 0), "grad_x")
    R.close(o.grad_weight, *dw, "grad_weight")
    again = lh.rms_norm_add_bwd(r, gy, gs, rstd, w)
    assert torch.equal(again.grad_x, o.grad_x) and torch.equal(again.grad_weight, o.grad_weight)
    # in place of either gradient, beside neighbours, without the stream, without grad_x
    for which in (0, 1):
        g2 = [torch.empty(N, D + pad, dtype=dtype, device="cuda")[:, :D].copy_(t) for t in (gy, gs)]
        lh.rms_norm_add_bwd(r, g2[0], g2[1], rstd, w, grad_x=g2[which])
        assert torch.equal(g2[which], o.grad_x)
    wide = torch.full((N, D + 5), 7.0, dtype=dtype, device="cuda")
    gw = torch.full((D,), 0.25, device="cuda")
    lh.rms_norm_add_bwd(r, gy, gs, rstd, w, grad_x=wide[:, 2:2 + D], grad_weight=gw,
                        accumulate=True)
    # (rows that begin elsewhere are added up in another order)
    R.close(wide[:, 2:2 + D], want, bx + 2 * R.U * (dx.abs() + R.d(gs).abs()) +
            (R.half(dtype) * (want.abs() + bx) * 1.01 if dtype == BF else 0), "grad_x, wide")
    R.close(gw, dw[0] + 0.25, dw[1] + R.U * (dw[0].abs() + 0.5), "grad_weight, added")
    assert (wide[:, :2] == 7).all() and (wide[:, 2 + D:] == 7).all()
    plain = lh.rms_norm_bwd(r, gy, rstd, w)
    p = lh.rms_norm_add_bwd(r, gy, None, rstd, w)
    assert torch.equal(p.grad_x, plain.grad_x) and torch.equal(p.grad_weight, plain.grad_weight)
    p = lh.rms_norm_add_bwd(r, gy, gs, rstd, w, want_grad_x=False)
    assert p.grad_x is None and torch.equal(p.grad_weight, plain.grad_weight)


def test_empty(lh):
    x = torch.empty(0, 64, device="cuda")
    o = lh.rms_norm_add_fwd(x, x, None, EPS, want_quant=True)
    assert o.y.shape == (0, 64) and o.quant.scales.shape == (0, 1)
    w = torch.ones(64, device="cuda")
    g = lh.rms_norm_add_bwd(x, x, x, o.rstd, w)
    assert (g.grad_weight == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_autograd(lh, dtype):
    """Both outputs used, one of them, the residual twice; against 64-bit autograd and,
    in fp32, against differences."""
    N, D = 6, 160
    x, res, w = _randn((N, D), dtype, 1), _randn((N, D), dtype, 2), _vec(D, dtype, 3)
    cy, cs = _randn((N, D), F32, 4), _randn((N, D), F32, 5)

    def loss(x, res, w, use, f):
        y, s = f(x, res, w)
        return sum((t * c.to(t.dtype)).sum() for t, c, u in ((y, cy, "y"), (s, cs, "s")) if u in use)

    def plain(x, res, w):
        r = x + res
        return r * (r.square().mean(1, keepdim=True) + EPS).rsqrt() * w, r
    for use in ("ys", "y", "s"):
        t = [v.clone().requires_grad_() for v in (x, res, w)]
        loss(*t, use, lambda *a: lh.rms_norm_add(*a, eps=EPS)).backward()
        t64 = [v.double().requires_grad_() for v in (x, res, w)]
        loss(*t64, use, plain).backward()
        for a, b in zip(t, t64):
            if b.grad is None:
                assert a.grad is None
                continue
            # bf16: r, y's and the stream's gradient are rounded before they are used
            tol = 1e-5 if dtype == F32 else 8 * 2.0 ** -8
            assert (a.grad.double() - b.grad).abs().max() <= tol * max(1.0, b.grad.abs().max()), use
    if dtype == F32:
        v = _randn((N, D), F32, 6)
        g = torch.autograd.grad(loss(*(t0 := [q.clone().requires_grad_() for q in (x, res, w)]), "ys",
                                     lambda *a: lh.rms_norm_add(*a, eps=EPS)), t0[0])[0]
        h = 2.0 ** -8
        f = [loss(x + e * v, res, w, "ys", lambda *a: lh.rms_norm_add(*a, eps=EPS)).double()
             for e in (h, -h)]
        # central differences: h^2 of the third derivative, and the loss's rounding over 2 h
        assert abs((f[0] - f[1]) / (2 * h) - (g.double() * v.double()).sum()) < 0.05
    y, s = lh.rms_norm_add(x.view(2, 3, D), res.view(2, 3, D), w)
    assert y.shape == s.shape == (2, 3, D)


@pytest.mark.parametrize("use", ["both", "y", "summed"])
@pytest.mark.parametrize("shape", [(6, 40), (2, 3, 40), (40,)])
def test_gradients_of_leaves_accumulate(lh, shape, use):
    """x and residual get equal gradients, each in memory of its own: a second backward
    pass adds to each once (g + g = 2 g exactly)."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x, r = (torch.randn(shape, device="cuda", generator=g).requires_grad_() for _ in range(2))
    w = torch.randn(40, device="cuda", generator=g).requires_grad_()
    gy, gs = (torch.randn(shape, device="cuda", generator=g) for _ in range(2))
    kept = gs.clone()
    for passes in (1, 2, 3):
        y, s = lh.rms_norm_add(x, r, w)
        outs, grads = {"both": ((y, s), (gy, gs)), "y": ((y,), (gy,)),
                       "summed": ((s,), (gs,))}[use]
        torch.autograd.backward(outs, grads)
        if passes == 1:
            first = x.grad.clone()
            assert torch.equal(r.grad, first)
        assert x.grad.data_ptr() != r.grad.data_ptr()
        if passes == 2:
            assert torch.equal(x.grad, 2 * first) and torch.equal(r.grad, 2 * first)
    assert torch.equal(gs, kept)
