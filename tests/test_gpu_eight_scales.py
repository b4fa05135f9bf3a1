"""Scales of opposite sizes in gemm8: what counts is their product, in the kernel for few
tokens, in that on CTA pairs and for either kind of the weights' scales alike."""
import pytest
import torch

import eight_ref as E
import ops_ref as R
import test_gpu_eight as T
from test_gpu_eight import lh  # noqa: F401  (the fixture)
from test_gpu_eight_pairs import _on_pairs

pytestmark = pytest.mark.gpu
F32, U8 = torch.float32, torch.uint8
# one tile per CTA, clusters that share a tile's blocks, CTA pairs
SIZES = [(40, 20500, 900), (20, 300, 1500), (300, 5000, 1300)]


def _operands(lh, M, N, K, rows):
    a, b = T._operand(lh, M, K, 1, 4), T._operand(lh, N, K, rows, 5)
    if M > 64:
        assert _on_pairs(M, N)
    return a, b


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("large", ["a", "b"])
def test_opposite(lh, M, N, K, rows, large):  # noqa: F811
    """2^e and 2^-e with e up to 120: the products are near 1, a block's sum (up to 2^25)
    times either scale would leave fp32's range."""
    a, b = _operands(lh, M, N, K, rows)
    e = torch.linspace(0, 120, a.scales.shape[1]).round().cuda()
    e = e if large == "a" else -e
    a.scales *= e.exp2()
    b.scales *= (-e).exp2()
    for out_dtype in (F32, torch.bfloat16):
        R.close(lh.gemm8(a, b, out_dtype=out_dtype), *E.gemm(a, b, None, None, out_dtype))


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("rows", [1, 128])
def test_products_out_of_range(lh, M, N, K, rows):  # noqa: F811
    """A product above fp32's range counts as infinite, NaN where the sum is 0, and one
    below as 0, by the row and the columns that have it."""
    a, b = _operands(lh, M, N, K, rows)
    c0 = N // 2 // 128 * 128
    at = slice(c0, c0 + 128)  # the columns of one scale for 128, or each with its own
    group = slice(c0 // 128, c0 // 128 + 1) if rows == 128 else at
    a.scales[1, 2], a.scales[2, 2] = 2.0 ** 100, 2.0 ** 100
    a.scales[M - 1, 3] = 2.0 ** -100
    b.scales[group, 2], b.scales[group, 3] = 2.0 ** 100, 2.0 ** -100
    a.data.view(U8)[2, 256:384] = 0  # a block whose sums are 0
    y = lh.gemm8(a, b)
    want = E.value(a) @ E.value(b).t()
    assert (y[1, at].abs() == float("inf")).all()
    assert torch.equal(y[1, at].sign().cpu(), want[1, at].sign().float())
    assert y[2, at].isnan().all()
    y[1:3, at] = want[1:3, at] = 0  # the rest by its values, the smallest among them
    mag = E.value(a).abs() @ E.value(b).abs().t()
    mag[1:3, at] = 0
    bound = (256 + E.ceil(K, 128) + 4) * R.U * mag + 1e-30
    R.close(y, want, bound)
