"""linear8 rounds to 8 bits, transposed, what its backward pass will read and nothing
else: with gradients switched off only its own product's operands."""
import contextlib

import pytest
import torch

from test_eight_refusals import abi, mods  # noqa: F401  (fixtures)

no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="fake tensors on a stand-in for the library; CPU only")


@no_gpu
@pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")
@pytest.mark.parametrize("mode,x_grad,w_grad,xt,wt", [
    ("grad", True, True, True, True), ("grad", False, True, True, False),
    ("grad", True, False, False, True), ("grad", False, False, False, False),
    ("no_grad", True, True, False, False), ("no_grad", False, True, False, False),
    ("inference", True, True, False, False)])
def test_what_is_rounded(mods, mode, x_grad, w_grad, xt, wt):  # noqa: F811
    eight, _, reached = mods
    x = torch.zeros(2, 3, 64, device="cuda:0", requires_grad=x_grad)
    W = torch.zeros(40, 64, device="cuda:0", requires_grad=w_grad)
    with {"grad": contextlib.nullcontext, "no_grad": torch.no_grad,
          "inference": torch.inference_mode}[mode]():
        y = eight.linear8(x, W)
    assert y.shape == (2, 3, 40) and y.requires_grad == (mode == "grad" and (x_grad or w_grad))
    # (x, dt, R, C, ldx, rows, q, ldq, scales, qt, ldqt, scales_t, stream)
    calls = [a for n, a in reached if n == "quantize8"]
    assert [n for n, _ in reached] == ["quantize8", "quantize8", "gemm8"]
    assert [(a[5], a[7] > 0, a[10] > 0) for a in calls] == [(1, True, xt), (128, True, wt)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(50, 300, 260), (1300, 2200, 1500)])
def test_the_same_product(M, K, N):
    import lm_head_linear_fwd_gb300 as lh
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16).requires_grad_()
    W = torch.randn(N, K, device="cuda", generator=g).mul_(K ** -0.5).requires_grad_()
    y = lh.linear8(x, W)
    with torch.no_grad():
        assert torch.equal(lh.linear8(x, W), y)
    with torch.inference_mode():
        assert torch.equal(lh.linear8(x, W), y)
    y.sum().backward()
    assert x.grad is not None and W.grad is not None
