"""The 4-bit head near the ends of fp32 (bounds: tests/ops_ref.py)."""
import pytest
import torch

import ops_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("M", [2, 12, 20])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype,sdt", [(BF, BF), (BF, F32), (F32, F32)])
def test_scales_of_any_magnitude(M, group, dtype, sdt):
    """Scales up to 2^127, with tokens that leave the logits within range, and tokens of
    zeros; scales down to 2^-120, with large tokens."""
    import lm_head_linear_fwd_gb300 as lh
    V, D = 300, 384
    g = torch.Generator().manual_seed(M)
    packed = torch.randint(0, 256, (V, D // 2), generator=g, dtype=torch.uint8).cuda()
    zeros = torch.randint(0, 16, (V, D // group), generator=g, dtype=torch.uint8).cuda()
    for lo, hi, std in ((110, 127.9, 2.0 ** -30), (-120, -100, 2.0 ** 90), (-8, 0, 1.0)):
        e = torch.rand(V, D // group, generator=g) * (hi - lo) + lo
        scales = torch.exp2(e.double()).to(sdt).cuda()
        x = torch.randn(M, D, generator=g).mul_(std).to(dtype).cuda()
        x[0] = 0
        y = lh.head4_logits(x, lh.Head4(packed, scales, zeros, D, group))
        assert (y[0] == 0).all() and y.isfinite().all()
        Wq = R.head4_weights(packed, scales, zeros, D, group)
        R.close(y, *R.head4(x, Wq, None, group, F32), (lo, hi))
