"""Rounding to 8 bits (bit for bit) and the products in 8 bits, against 64-bit forms
(bounds: eight_ref.py)."""
import pytest
import torch

import eight_ref as E
import ops_ref as R

pytestmark = pytest.mark.gpu
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.fixture(scope="module")
def lh():
    import lm_head_linear_fwd_gb300 as m
    return m


def _randn(shape, dtype, seed, std=1.0, pad=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    N, D = shape
    flat = torch.randn(N * (D + pad) + shift, generator=g).mul_(std).to(dtype).cuda()
    return flat[shift:].view(N, D + pad)[:, :D]


def _same(q, want, rows, what):
    data, scales = want
    assert q.rows == rows
    assert torch.equal(q.scales.cpu(), scales), (what, "scales")
    assert torch.equal(q.data.cpu().view(U8), data.view(U8)), (what, "numbers")


@pytest.mark.parametrize("N,D", [(1, 1), (1, 128), (2, 130), (17, 96), (128, 128), (129, 257),
                                 (300, 1601), (64, 4096), (1000, 40)])
@pytest.mark.parametrize("dtype,pad,shift", [(BF, 0, 0), (BF, 3, 1), (F32, 0, 0), (F32, 1, 2),
                                             (BF, 8, 8)])
def test_quantize(lh, N, D, dtype, pad, shift):
    x = _randn((N, D), dtype, 1, 0.7, pad, shift)
    x *= torch.rand(N, 1, generator=torch.Generator().manual_seed(2)).mul(-12).exp2().cuda()
    x[0, 0] = 0.0
    if N > 20:
        x[5] = 0.0
        x[6] *= 1e-30
    xt = x.t().contiguous()
    for rows in (1, 128):
        want, want_t = E.quantize(x, rows), E.quantize(xt, rows)
        q = lh.quantize8(x, rows)
        _same(q, want, rows, "alone")
        _same(lh.quantize8(x, rows, transpose=True), want_t, rows, "transposed")
        a, b = lh.quantize8_pair(x, rows)
        _same(a, want, rows, "pair")
        _same(b, want_t, rows, "pair transposed")
        # outputs inside larger ones
        big = torch.full((N, E.ceil(D, 16) * 16 + 32), 0x55, dtype=U8, device="cuda")
        big_t = torch.full((D, E.ceil(N, 16) * 16 + 32), 0x55, dtype=U8, device="cuda")
        o = lh.Quant8(big.view(E.E4M3)[:, 16:16 + D], torch.empty_like(a.scales), rows)
        t = lh.Quant8(big_t.view(E.E4M3)[:, 16:16 + N], torch.empty_like(b.scales), rows)
        lh.quantize8_pair(x, rows, out=o, out_t=t)
        _same(o, want, rows, "inside")
        _same(t, want_t, rows, "inside transposed")
        for m, n in ((big, D), (big_t, N)):
            assert (m[:, :16] == 0x55).all() and (m[:, 16 + n:] == 0x55).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_values(lh, dtype):
    """Blocks with an infinity or NaN, the largest and the smallest numbers."""
    x = _randn((300, 384), dtype, 1)
    x[3, 5], x[150, 200], x[280, 380] = float("inf"), float("nan"), float("-inf")
    x[10], x[11] = torch.finfo(dtype).max, torch.finfo(dtype).tiny
    x[12] = 2.0 ** -133
    for rows in (1, 128):
        q, t = lh.quantize8_pair(x, rows)
        v = q.data.float()
        R0, C0 = (slice(3, 4), slice(0, 128)) if rows == 1 else (slice(0, 128), slice(0, 128))
        assert q.scales[0 if rows == 128 else 3, 0] == float("inf") and v[3, 5].isnan()
        block = v[R0, C0].clone()
        block[3 - R0.start, 5] = 0
        assert (block == 0).all()
        R1 = slice(150, 151) if rows == 1 else slice(128, 256)
        assert v[R1, 128:256].isnan().all() and q.scales[1 if rows == 128 else 150, 1].isnan()
        assert v[280, 380].isnan()
        assert t.data.float()[5, 3].isnan() and t.data.float()[200, 150].isnan()
        keep = torch.isfinite(q.scales)
        want = E.quantize(x.cpu(), rows)
        assert torch.equal(q.scales.cpu()[keep.cpu()], want[1][keep.cpu()])
        if rows == 1:
            assert torch.equal(q.data.cpu()[10:13].view(U8), want[0][10:13].view(U8))


def _operand(lh, R0, K, rows, seed, wild=False):
    g = torch.Generator().manual_seed(seed)
    ld = E.ceil(K, 16) * 16 + 16 * (seed % 3)
    data = (torch.randn(R0, ld, generator=g) * 100).clamp(-448, 448).to(E.E4M3).cuda()
    scales = torch.rand(R0 if rows == 1 else E.ceil(R0, 128), E.ceil(K, 128), generator=g) + 0.5
    if wild:
        scales *= (torch.rand(scales.shape, generator=g) * 40 - 20).exp2()
    return lh.Quant8(data[:, :K], scales.cuda(), rows)


SIZES = [(1, 1, 1), (1, 128, 128), (1, 300, 257), (2, 129, 1000), (5, 1000, 96), (16, 768, 768),
         (17, 513, 300), (33, 200, 2048), (64, 130, 129), (77, 768, 1601), (100, 2000, 640),
         (128, 128, 4096), (129, 257, 128), (250, 300, 384), (300, 1000, 1601), (513, 640, 100),
         (1000, 1024, 512), (1, 8000, 64), (3, 64, 9000), (700, 130, 3000),
         # more tiles than SMs, clusters of each size and tile, both kernels above 64 tokens
         (3, 30000, 300), (40, 20500, 130), (50, 8192, 512), (20, 4096, 2048), (100, 10000, 200),
         (70, 10240, 384), (2000, 2600, 400)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("rows", [1, 128])
def test_gemm(lh, M, N, K, rows):
    a, b = _operand(lh, M, K, 1, 1), _operand(lh, N, K, rows, 2)
    g = torch.Generator().manual_seed(3)
    for dtype, bdtype in ((F32, None), (BF, BF), (F32, F32)):
        bias = None if bdtype is None else torch.randn(N, generator=g).mul_(1e3).to(bdtype).cuda()
        st = lh.new_status("cuda")
        y = lh.gemm8(a, b, bias, out_dtype=dtype, status=st)
        R.close(y, *E.gemm(a, b, bias, None, dtype), ("y", dtype))
        assert torch.equal(lh.gemm8(a, b, bias, out_dtype=dtype), y)
        wide = torch.full((M, N + 5), 7.0, dtype=dtype, device="cuda")
        lh.gemm8(a, b, bias, out=wide[:, 2:2 + N])
        assert torch.equal(wide[:, 2:2 + N], y)
        assert (wide[:, :2] == 7).all() and (wide[:, 2 + N:] == 7).all()
        lh.check_status(st)
        # rows of whole 16-byte blocks, which the last columns do not fill
        wide = torch.full((M, E.ceil(N, 8) * 8 + 8), 7.0, dtype=dtype, device="cuda")
        lh.gemm8(a, b, bias, out=wide[:, :N])
        assert torch.equal(wide[:, :N], y) and (wide[:, N:] == 7).all()
    base = torch.randn(M, N, generator=g).mul_(1e4).cuda()
    out = base.clone()
    lh.gemm8(a, b, bias, out=out, accumulate=True)
    R.close(out, *E.gemm(a, b, bias, base, F32), "accumulate")
    wide = torch.full((M, E.ceil(N, 8) * 8 + 8), 7.0, device="cuda")
    wide[:, :N] = base
    lh.gemm8(a, b, bias, out=wide[:, :N], accumulate=True)
    assert torch.equal(wide[:, :N], out) and (wide[:, N:] == 7).all()


def test_gemm_scales(lh):
    """Scales over 80 powers of two, blocks of zeros, an infinite scale, a NaN."""
    M, N, K = 40, 200, 900
    for rows in (1, 128):
        a, b = _operand(lh, M, K, 1, 4, True), _operand(lh, N, K, rows, 5, True)
        a.data.view(U8)[3] = 0
        R.close(lh.gemm8(a, b), *E.gemm(a, b, None, None, F32))
        a.scales[7, 2], b.scales[1 if rows == 128 else 130, 3] = float("nan"), float("inf")
        y = lh.gemm8(a, b)
        assert y[7].isnan().all()
        bad = y[:, 128:] if rows == 128 else y[:, 130]
        assert not bad.isfinite().any()
        rest = y[:, :128] if rows == 128 else y[:, :130]
        assert rest[:7].isfinite().all() and rest[8:].isfinite().all()


def test_gemm_far(lh):
    """Outputs past 2^31 elements."""
    M, N, K = 16500, 131072, 64
    a, b = _operand(lh, M, K, 1, 1), _operand(lh, N, K, 128, 2)
    y = lh.gemm8(a, b, out_dtype=BF)
    for rows in (slice(0, 3), slice(M - 3, M)):
        part = lh.Quant8(a.data[rows], a.scales[rows].contiguous())
        R.close(y[rows], *E.gemm(part, b, None, None, BF))
    # every row is one of few: rows repeat
    a.data.view(U8)[:] = a.data.view(U8)[:1].clone()
    a.scales[:] = a.scales[:1].clone()
    lh.gemm8(a, b, out=y)
    assert (y == y[:1]).all()


def test_empty(lh):
    x = torch.empty(0, 64, device="cuda")
    q = lh.quantize8(x)
    w = lh.quantize8(torch.ones(8, 64, device="cuda"), 128)
    assert lh.gemm8(q, w).shape == (0, 8)
    x, W = torch.empty(0, 64, device="cuda", requires_grad=True), \
        torch.ones(8, 64, device="cuda", requires_grad=True)
    lh.linear8(x, W).sum().backward()
    assert x.grad.shape == (0, 64) and (W.grad == 0).all()


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32)])
def test_linear(lh, dtype, wdtype):
    """The three products of what the roundings stand for, in 64 bits."""
    M, K, N = 200, 300, 260
    x = _randn((M, K), dtype, 1).requires_grad_()
    W = _randn((N, K), wdtype, 2, K ** -0.5).requires_grad_()
    gy = _randn((M, N), dtype, 3, 1e-3)
    y = lh.linear8(x.view(2, 100, K), W)
    assert y.shape == (2, 100, N) and y.dtype is dtype
    y.backward(gy.view(2, 100, N))
    xd, wd = x.detach(), W.detach()
    x8, x8t = lh.quantize8_pair(xd)
    w8, w8t = lh.quantize8_pair(wd, 128)
    g8, g8t = lh.quantize8_pair(gy)
    R.close(y.view(M, N), *E.gemm(x8, w8, None, None, dtype), "y")
    R.close(x.grad, *E.gemm(g8, w8t, None, None, dtype), "grad_x")
    R.close(W.grad, *E.gemm(g8t, x8t, None, None, wdtype), "grad_W")
    # e4m3 is off by 2^-4 at most, about 2^-5.3 on average, per factor, with random
    # signs: near the gradient of the unrounded product
    for got, want in ((y.view(M, N), xd.double() @ wd.double().t()),
                      (x.grad, gy.double() @ wd.double()),
                      (W.grad, gy.double().t() @ xd.double())):
        assert (got.double() - want).norm() <= 2 * 2.0 ** -4 * want.norm()
    for need in ((True, False), (False, True)):
        t = [v.detach().clone().requires_grad_(r) for v, r in zip((x, W), need)]
        lh.linear8(*t).backward(gy)
        for v, full in zip(t, (x, W)):
            assert (v.grad is None) if not v.requires_grad else torch.equal(v.grad, full.grad)


def test_side_stream_and_graph(lh):
    """A captured norm, product and quantisation, replayed on new inputs, on a stream
    of its own."""
    M, K, N = 24, 640, 300
    x, res, w = _randn((M, K), BF, 1), _randn((M, K), BF, 2), torch.ones(K, device="cuda")
    W8 = lh.quantize8(_randn((N, K), BF, 3), 128)

    def step():
        o = lh.rms_norm_add_fwd(x, res, w, want_y=False, want_quant=True)
        return lh.gemm8(o.quant, W8), o.summed
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, summed = step()
    for seed in (5, 6):
        x.copy_(_randn((M, K), BF, seed))
        graph.replay()
        want = step()
        assert torch.equal(y, want[0]) and torch.equal(summed, want[1])


def test_captured_training_step(lh):
    """Norm, product and both backward passes captured on one stream, replayed on new
    inputs: the eager step's gradients."""
    N, K, M = 300, 640, 200
    W, w = _randn((M, K), BF, 3), torch.ones(K, device="cuda")
    gy = _randn((N, M), BF, 4).reshape(2, N // 2, M)
    leaves = [_randn((N, K), BF, seed).reshape(2, N // 2, K).clone() for seed in (1, 2)]
    leaves = [t.requires_grad_() for t in (*leaves, w.clone(), W.clone())]

    def step(x, res, w, W):
        y, summed = lh.rms_norm_add(x, res, w)
        torch.autograd.backward((lh.linear8(y, W), summed), (gy, summed.detach()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(*leaves)
    torch.cuda.current_stream().wait_stream(s)
    for t in leaves:
        t.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(*leaves)
    for seed in (5, 6):
        with torch.no_grad():
            leaves[0].copy_(_randn((N, K), BF, seed).view_as(leaves[0]))
        graph.replay()
        eager = [t.detach().clone().requires_grad_() for t in leaves]
        step(*eager)
        for a, b in zip(leaves, eager):
            assert torch.equal(a.grad, b.grad)
