"""gemm8's kernel for many tokens (256 x 256 tiles on CTA pairs) over more blocks of 128
columns than its scales are handed over for at a time, with several tiles to a pair, and
a layer's training pass whose products all go to it (bounds: eight_ref.py)."""
import os
import re

import pytest
import torch

import eight_ref as E
import ops_ref as R
import test_gpu_eight as T
from test_gpu_eight import lh  # noqa: F401  (the fixture)

BF, F32 = torch.bfloat16, torch.float32
gpu = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _on_pairs(M, N):
    """Whether a product goes to the pairs on this GPU: more tiles of 64 x 128 than SMs
    (tile_tokens in gemm8.cu, whose rule test_the_rule reads)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return M > 64 and -(-M // 64) * -(-N // 128) > sms


def test_the_rule():
    """The sizes below are chosen by this rule and these numbers of blocks."""
    src = open(os.path.join(ROOT, "lm_head_linear_fwd_gb300", "csrc", "gemm8.cu")).read()
    assert "if (M > 64 && (M + 63) / 64 * tiles_n > sms) return 0;" in src
    src = open(os.path.join(ROOT, "lm_head_linear_fwd_gb300", "csrc", "gemm8_pair.cuh")).read()
    ahead, ring = (int(re.search(rf"constexpr int {n} = (\d+);", src).group(1))
                   for n in ("kAhead", "kRing"))
    assert ahead * ring <= 16


# 9, 16, 18, 20 and 25 blocks: within and past the ring of scales, by fours and not; from
# 40 tiles to 88, of which some pairs have two
SIZES = [(300, 5000, 1100), (300, 5000, 2048), (1100, 4100, 2177), (2000, 2600, 2560),
         (2000, 2600, 3200)]


@gpu
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("rows", [1, 128])
def test_gemm_on_pairs(lh, M, N, K, rows):  # noqa: F811
    """Types, bias, outputs with and without whole 16-byte rows, sums added to."""
    assert _on_pairs(M, N)
    T.test_gemm(lh, M, N, K, rows)


@gpu
@pytest.mark.parametrize("M,N", [(300, 5000), (1100, 4100)])
@pytest.mark.parametrize("rows", [1, 128])
def test_scales_on_pairs(lh, M, N, rows):  # noqa: F811
    """Scales over 80 powers of two, blocks of zeros; a NaN and an infinity in the last
    row's and the last columns' scales stay in them."""
    K = 1500
    assert _on_pairs(M, N) and M % 256 and N % 256
    a, b = T._operand(lh, M, K, 1, 4, True), T._operand(lh, N, K, rows, 5, True)
    a.data.view(torch.uint8)[3] = 0
    y = lh.gemm8(a, b)
    R.close(y, *E.gemm(a, b, None, None, F32))
    a.scales[M - 1, 2], b.scales[-1, 9] = float("nan"), float("inf")
    z = lh.gemm8(a, b)
    last = N - 1 if rows == 1 else (N - 1) // 128 * 128
    assert z[M - 1].isnan().all() and not z[:, last:].isfinite().any()
    assert torch.equal(z[:M - 1, :last], y[:M - 1, :last])


@gpu
@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32)])
def test_linear_on_pairs(lh, dtype, wdtype):  # noqa: F811
    """y, grad_x and grad_W of 18, 12 and 11 blocks, all of them on the pairs."""
    M, K, N = 1300, 2200, 1500
    assert _on_pairs(M, N) and _on_pairs(M, K) and _on_pairs(N, K)
    x = T._randn((M, K), dtype, 1).requires_grad_()
    W = T._randn((N, K), wdtype, 2, K ** -0.5).requires_grad_()
    gy = T._randn((M, N), dtype, 3, 1e-3)
    y = lh.linear8(x, W)
    y.backward(gy)
    x8, x8t = lh.quantize8_pair(x.detach())
    w8, w8t = lh.quantize8_pair(W.detach(), 128)
    g8, g8t = lh.quantize8_pair(gy)
    R.close(y, *E.gemm(x8, w8, None, None, dtype), "y")
    R.close(x.grad, *E.gemm(g8, w8t, None, None, dtype), "grad_x")
    R.close(W.grad, *E.gemm(g8t, x8t, None, None, wdtype), "grad_W")
