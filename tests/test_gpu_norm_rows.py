"""The norms where a team of threads works on many rows in turn (rows copied ahead into
places that were used before), on every shape of team, dense rows throughout
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


def _rows(N, D, dtype, seed, std=1.0, mean=0.0, pad=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    flat = torch.randn(N * (D + pad) + shift, generator=g).mul_(std).add_(mean).to(dtype).cuda()
    return flat[shift:].view(N, D + pad)[:, :D]


def _vec(D, dtype, seed, mean):
    return _rows(1, D, dtype, seed, 0.3, mean)[0].contiguous()


# (N, D): five rows or more for each team of 152 SMs.  1281..1536, 2049..2560 and
# 2561..3071 columns give teams of 96, 160 and 192 threads, several to a block.
SHAPES = {BF: [(50000, 64), (7000, 769), (4600, 1500), (4600, 1501), (3100, 1600), (3100, 1601),
               (2500, 2400), (2500, 2401), (2500, 2600), (2500, 2601), (800, 5120), (800, 5119),
               (800, 8190)],
          F32: [(50000, 36), (4600, 1500), (4600, 1501), (1700, 1600), (2500, 2401), (1700, 2600),
                (800, 5120), (800, 6001), (800, 8192)]}
CASES = [(dtype, N, D) for dtype, shapes in SHAPES.items() for N, D in shapes]


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("dtype,N,D", CASES + [(BF, 500, 12000), (BF, 500, 12001), (BF, 800, 20480),
                                               (F32, 500, 9000), (F32, 500, 9001)])
def test_forward(lh, center, dtype, N, D):
    x = _rows(N, D, dtype, 1, 2.0, 0.5)
    w, b = _vec(D, F32, 2, 1.0), _vec(D, F32, 3, 0.0) if center else None

    def run(x):
        return lh.layer_norm_fwd(x, w, b, EPS) if center else lh.rms_norm_fwd(x, w, EPS)

    o = run(x)
    y, mean, rstd = R.norm(x, w, b, EPS, center, dtype)
    R.close(o.y, *y, "y")
    R.close(o.rstd, *rstd, "rstd")
    if center:
        R.close(o.mean, *mean, "mean")
    # rows that start inside 16-byte blocks: the same bits
    other = torch.empty(N * (D + 3) + 1, dtype=dtype, device="cuda")[1:].view(N, D + 3)[:, :D]
    p = run(other.copy_(x))
    assert torch.equal(p.y, o.y) and torch.equal(p.rstd, o.rstd)


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("dtype,N,D", CASES)
def test_backward(lh, center, dtype, N, D):
    x, dy = _rows(N, D, dtype, 1, 2.0, 0.5), _rows(N, D, dtype, 4, 0.1, 0.02)
    w = _vec(D, F32, 2, 1.0)
    f = lh.layer_norm_fwd(x, w, None, EPS) if center else lh.rms_norm_fwd(x, w, EPS)

    def run(x, dy):
        if center:
            return lh.layer_norm_bwd(x, dy, f.mean, f.rstd, w, want_grad_bias=True)
        return lh.rms_norm_bwd(x, dy, f.rstd, w)

    o = run(x, dy)
    dx, dw, db = R.norm_grad(x, dy, f.mean, f.rstd, w, center, dtype)
    R.close(o.grad_x, *dx, "grad_x")
    R.close(o.grad_weight, *dw, "grad_weight")
    if center:
        R.close(o.grad_bias, *db, "grad_bias")
    shifted = [torch.empty(N * (D + 3) + 1, dtype=dtype, device="cuda")[1:].view(N, D + 3)[:, :D]
               for _ in range(2)]
    p = run(shifted[0].copy_(x), shifted[1].copy_(dy))
    for a, b in ((p.grad_x, o.grad_x), (p.grad_weight, o.grad_weight), (p.grad_bias, o.grad_bias)):
        assert a is b is None or torch.equal(a, b)
