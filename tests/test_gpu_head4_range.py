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


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype,sdt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_rounding_a_table_up_to_the_largest_values(group, dtype, sdt):
    """With zero points, a group whose range passes fp32's: scale, zero point and nibbles
    of the definition, and weights that come back within half a step."""
    import lm_head_linear_fwd_gb300 as lh
    V, D = 200, 256
    g = torch.Generator().manual_seed(group)
    most = torch.finfo(dtype).max
    W = ((torch.rand(V, D, generator=g, dtype=torch.float64) * 2 - 1) * most).to(dtype)
    W[0, 0::group], W[0, 1::group] = most, -most   # the widest range
    W[1] = W[1].abs()                              # one sign: within range
    h = lh.head4_quantize(W.cuda(), group, zero_point=True, scale_dtype=sdt)
    Wg = W.double().view(V, D // group, group)
    lo, hi = Wg.amin(2).clamp(max=0), Wg.amax(2).clamp(min=0)
    # the range and the quotient round in turn, as in fp32 without its upper end
    s = (((hi - lo) / 2).float().double() / 7.5).float().to(sdt)
    assert torch.equal(h.scales.cpu(), s) and s.isfinite().all()
    s = s.double()
    z = (-lo / s).float().round().clamp(0, 15)
    assert torch.equal(h.zeros.cpu().float(), z)
    q = ((Wg / s[:, :, None]).float().round() + z[:, :, None]).clamp(0, 15).view(V, D)
    assert torch.equal(R.unpack4(h.packed, D).float(), q)
    # a scale of fp32 covers the range; one of bf16 is off by 2^-8 of up to 15 steps
    Wq = R.head4_weights(h.packed, h.scales, h.zeros, D, group)
    step = s.repeat_interleave(group, 1)
    assert ((Wq - W.double()).abs() <= step * (1.0 + (0 if sdt == F32 else 15 * 2.0 ** -8))).all()
