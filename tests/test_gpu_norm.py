"""Layer norm and RMS norm, forward and backward, against 64-bit forms
(bounds: tests/ops_ref.py)."""
import pytest
import torch

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


def _vec(D, dtype, seed, mean):
    return _randn((1, D), dtype, seed, 0.3, mean)[0].contiguous()


def _fwd(lh, x, w, b, center, **kw):
    return lh.layer_norm_fwd(x, w, b, EPS, **kw) if center else lh.rms_norm_fwd(x, w, EPS, **kw)


def _check_fwd(lh, x, w, b, center, o):
    y, mean, rstd = R.norm(x, w, b, EPS, center, x.dtype)
    R.close(o.rstd, *rstd, "rstd")
    if center:
        R.close(o.mean, *mean, "mean")
    R.close(o.y, *y, "y")


SHAPES = [(1, 1), (1, 2), (2, 7), (5, 64), (3, 129), (40, 768), (7, 1601), (3, 4096), (2, 5120),
          (3, 8191), (2, 16384), (2, 20001), (1, 70000)]
LAYOUT = [(BF, BF, 0, 0), (BF, F32, 0, 0), (BF, F32, 3, 1), (F32, F32, 0, 0), (F32, BF, 2, 3),
          (BF, BF, 8, 8), (F32, F32, 1, 0)]


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("N,D", SHAPES)
@pytest.mark.parametrize("dtype,wdtype,pad,shift", LAYOUT)
def test_forward(lh, center, N, D, dtype, wdtype, pad, shift):
    x = _randn((N, D), dtype, 1, 2.0, 0.5, pad, shift)
    w, b = _vec(D, wdtype, 2, 1.0), _vec(D, wdtype, 3, 0.0) if center else None
    o = _fwd(lh, x, w, b, center)
    _check_fwd(lh, x, w, b, center, o)
    wide = torch.full((N, D + 5), 7.0, dtype=dtype, device="cuda")
    _fwd(lh, x, w, b, center, y=wide[:, 2:2 + D])
    assert torch.equal(wide[:, 2:2 + D], o.y)
    assert (wide[:, :2] == 7).all() and (wide[:, 2 + D:] == 7).all()
    x2 = x.clone() if pad == 0 else torch.empty(N, D + pad, dtype=dtype,
                                                device="cuda")[:, :D].copy_(x)
    _fwd(lh, x2, w, b, center, y=x2)  # in place
    assert torch.equal(x2, o.y)


@pytest.mark.parametrize("center", [True, False])
def test_forward_values(lh, center):
    """No weights; a far mean; a constant row; an infinity, a NaN; many rows."""
    D = 1000
    x = _randn((2500, D), F32, 1)
    x[0] += 3e4
    x[1] = 5.0
    x[2] = 0.0
    x[3, 17], x[4, 18] = float("inf"), float("nan")
    x[5] *= 1e-20
    o = _fwd(lh, x, None, None, center)
    keep = torch.arange(2500) > 4
    keep[:3] = True
    _check_fwd(lh, x[keep.cuda()], None, None, center,
               lh.NormOut(o.y[keep.cuda()], o.mean[keep.cuda()] if center else None,
                          o.rstd[keep.cuda()]))
    assert o.y[4].isnan().all() and o.rstd[4].isnan()
    assert o.y[3, 17].isnan()
    assert o.y[5:].isfinite().all() and o.y[:3].isfinite().all()
    if center:  # each of weight and bias alone
        w, b = _vec(D, F32, 2, 1.0), _vec(D, F32, 3, 0.0)
        _check_fwd(lh, x[5:9], w, None, True, lh.layer_norm_fwd(x[5:9], w, None, EPS))
        _check_fwd(lh, x[5:9], None, b, True, lh.layer_norm_fwd(x[5:9], None, b, EPS))


def _bwd(lh, x, dy, mean, rstd, w, center, **kw):
    if center:
        return lh.layer_norm_bwd(x, dy, mean, rstd, w, **kw)
    kw.pop("want_grad_bias", None)
    return lh.rms_norm_bwd(x, dy, rstd, w, **kw)


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("N,D", SHAPES + [(1000, 96), (700, 1601), (333, 4096)])
@pytest.mark.parametrize("dtype,wdtype,pad,shift", LAYOUT)
def test_backward(lh, center, N, D, dtype, wdtype, pad, shift):
    x = _randn((N, D), dtype, 1, 2.0, 0.5, pad, shift)
    dy = _randn((N, D), dtype, 4, 0.1, 0.02, pad, shift)
    w = _vec(D, wdtype, 2, 1.0)
    f = _fwd(lh, x, w, None, center)
    o = _bwd(lh, x, dy, f.mean, f.rstd, w, center, want_grad_bias=True)
    dx, dw, db = R.norm_grad(x, dy, f.mean, f.rstd, w, center, dtype)
    R.close(o.grad_x, *dx, "grad_x")
    R.close(o.grad_weight, *dw, "grad_weight")
    if center:
        R.close(o.grad_bias, *db, "grad_bias")
    again = _bwd(lh, x, dy, f.mean, f.rstd, w, center, want_grad_bias=True)
    assert torch.equal(again.grad_x, o.grad_x) and torch.equal(again.grad_weight, o.grad_weight)
    # other layouts of the output, the incoming gradient overwritten, sums added to
    wide = torch.full((N, D + 5), 7.0, dtype=dtype, device="cuda")
    _bwd(lh, x, dy, f.mean, f.rstd, w, center, grad_x=wide[:, 2:2 + D])
    assert torch.equal(wide[:, 2:2 + D], o.grad_x)
    assert (wide[:, :2] == 7).all() and (wide[:, 2 + D:] == 7).all()
    dy2 = torch.empty(N, D + pad, dtype=dtype, device="cuda")[:, :D].copy_(dy)
    gw = torch.full((D,), 0.25, device="cuda")
    _bwd(lh, x, dy2, f.mean, f.rstd, w, center, grad_x=dy2, grad_weight=gw,
         grad_bias=torch.zeros(D, device="cuda"), accumulate=True) if center else \
        _bwd(lh, x, dy2, f.mean, f.rstd, w, center, grad_x=dy2, grad_weight=gw, accumulate=True)
    assert torch.equal(dy2, o.grad_x)
    R.close(gw, dw[0] + 0.25, dw[1] + R.U * (dw[0].abs() + 0.5), "accumulated grad_weight")


def test_backward_subsets(lh):
    x, dy = _randn((50, 300), BF, 1), _randn((50, 300), BF, 2)
    w = _vec(300, F32, 3, 1.0)
    f = lh.layer_norm_fwd(x, w, None, EPS)
    full = lh.layer_norm_bwd(x, dy, f.mean, f.rstd, w, want_grad_bias=True)
    for wx in (True, False):
        for ww in (True, False):
            for wb in (True, False):
                o = lh.layer_norm_bwd(x, dy, f.mean, f.rstd, w, want_grad_x=wx,
                                      want_grad_weight=ww, want_grad_bias=wb)
                for want, a, b in ((wx, o.grad_x, full.grad_x), (ww, o.grad_weight,
                                                                 full.grad_weight),
                                   (wb, o.grad_bias, full.grad_bias)):
                    assert torch.equal(a, b) if want else a is None
    # no weight: its gradient can still be asked for
    o = lh.layer_norm_bwd(x, dy, f.mean, f.rstd, None, want_grad_weight=True)
    dx, dw, _ = R.norm_grad(x, dy, f.mean, f.rstd, None, True, BF)
    R.close(o.grad_x, *dx)
    R.close(o.grad_weight, *dw)


def test_empty(lh):
    x = torch.empty(0, 40, device="cuda")
    o = lh.layer_norm_fwd(x)
    assert o.y.shape == (0, 40) and o.mean.shape == (0,)
    z = torch.ones(40, device="cuda")
    g = lh.layer_norm_bwd(x, x, o.mean, o.rstd, z, want_grad_bias=True)
    assert (g.grad_weight == 0).all() and (g.grad_bias == 0).all()
    g = lh.rms_norm_bwd(x, x, o.rstd, z, grad_weight=z, accumulate=True)
    assert (z == 1).all()


def test_far_rows(lh):
    """Offsets beyond 2^31 elements."""
    N, ld, D = 70000, 32768, 64
    x = torch.zeros(N, ld, dtype=BF, device="cuda")[:, 100:100 + D]
    at = torch.tensor([0, 65535, 65536, N - 1], device="cuda")
    rows = _randn((4, D), BF, 1)
    x[at] = rows
    o = lh.layer_norm_fwd(x, y=x)
    y, mean, rstd = R.norm(rows, None, None, EPS, True, BF)
    R.close(o.y[at], *y)
    x[at] = rows
    dy = torch.zeros(N, D, dtype=BF, device="cuda")
    dy[at] = _randn((4, D), BF, 2)
    g = lh.layer_norm_bwd(x, dy, o.mean, o.rstd, None, want_grad_weight=True)
    dx, dw, _ = R.norm_grad(rows, dy[at], o.mean[at], o.rstd[at], None, True, BF)
    R.close(g.grad_x[at], *dx)
    R.close(g.grad_weight, *dw)


@pytest.mark.parametrize("center", [True, False])
def test_autograd_against_differences(lh, center):
    D = 37
    x = _randn((4, 5 * D), F32, 1).view(4, 5, D).requires_grad_(True)
    w, b = _vec(D, F32, 2, 1.0).requires_grad_(True), _vec(D, F32, 3, 0.0).requires_grad_(True)
    v = _randn((20, D), F32, 4)
    y = lh.layer_norm(x, w, b) if center else lh.rms_norm(x, w)
    assert y.shape == x.shape
    (y.view(20, D) * v).sum().backward()

    def f(x, w, b):
        r = x - x.mean(-1, keepdim=True) if center else x
        h = r * (r.square().mean(-1, keepdim=True) + EPS).rsqrt() * w
        return ((h + b if center else h).view(20, D) * R.d(v)).sum()

    g = torch.Generator().manual_seed(5)
    args = [R.d(x), R.d(w), R.d(b)]
    grads = [x.grad, w.grad, b.grad]
    for k in range(3 if center else 2):
        t = torch.randn(args[k].shape, dtype=torch.float64, generator=g)
        up, dn = list(args), list(args)
        up[k], dn[k] = args[k] + 1e-5 * t, args[k] - 1e-5 * t
        diff = (f(*up) - f(*dn)) / 2e-5
        got = (R.d(grads[k]) * t).sum()
        # fp32 sums of 740 terms at most (~50 u) and the differences' own 1e-8
        assert abs(got - diff) <= 1e-5 * (R.d(grads[k]) * t).abs().sum(), k
    # a broadcast incoming gradient (stride 0), a transposed input
    xt = _randn((D, 20), F32, 6).t().requires_grad_(True)
    (lh.layer_norm(xt, w, b) if center else lh.rms_norm(xt, w)).sum().backward()
    assert xt.grad.shape == (20, D)


def test_stream_and_graph(lh):
    x, dy = _randn((200, 520), BF, 1), _randn((200, 520), BF, 2)
    w, b = _vec(520, F32, 3, 1.0), _vec(520, F32, 4, 0.0)
    f = lh.layer_norm_fwd(x, w, b)
    dx, gw, gb = torch.empty_like(dy), torch.empty(520, device="cuda"), torch.empty(520,
                                                                                  device="cuda")
    ws = torch.empty(lh.norm_bwd_workspace_bytes(200, 520), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        lh.layer_norm_fwd(x, w, b, y=f.y, mean=f.mean, rstd=f.rstd)
        lh.layer_norm_bwd(x, dy, f.mean, f.rstd, w, want_grad_bias=True, grad_x=dx,
                          grad_weight=gw, grad_bias=gb, ws=ws)

    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(_randn((200, 520), BF, 7))
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        e = lh.layer_norm_fwd(x, w, b)
        o = lh.layer_norm_bwd(x, dy, e.mean, e.rstd, w, want_grad_bias=True)
        assert torch.equal(f.y, e.y) and torch.equal(dx, o.grad_x)
        assert torch.equal(gw, o.grad_weight) and torch.equal(gb, o.grad_bias)
