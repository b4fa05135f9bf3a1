"""The residual norm to 8 bits with weights that are not finite: an infinite one makes its
block's scale infinite and the block's finite numbers 0, a NaN its block NaN, wherever the
block lies; blocks beside it stay as they are."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lh():
    import lm_head_linear_fwd_gb300 as m
    return m


# rows on 16-byte boundaries whose last block is short, full ones, one block, rows off
# them, rows too wide to hold
@pytest.mark.parametrize("N,D,pad", [(5, 200, 0), (3, 132, 0), (40, 1032, 0), (7, 256, 0),
                                     (2, 8, 0), (3, 5128, 0), (5, 201, 0), (4, 1601, 3),
                                     (2, 21000, 0)])
@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32)])
def test_weights(lh, N, D, pad, dtype, wdtype):
    g = torch.Generator(device="cuda").manual_seed(D)
    x, r = (torch.randn(N, D + pad, device="cuda", generator=g).abs().add(0.1).to(dtype)[:, :D]
            for _ in range(2))
    w = torch.rand(D, device="cuda", generator=g).add(0.5).to(wdtype)
    want = lh.rms_norm_add_fwd(x, r, w, want_quant=True)
    G = -(-D // 128)
    for at in {0, D // 2, (D - 1) // 128 * 128, D - 2, D - 1}:
        block, cols = at // 128, slice(at // 128 * 128, min(D, at // 128 * 128 + 128))
        rest = torch.ones(D, dtype=torch.bool, device="cuda")
        rest[cols] = False
        for value in (float("inf"), float("-inf"), float("nan")):
            v = w.clone()
            v[at] = value
            o = lh.rms_norm_add_fwd(x, r, v, want_quant=True)
            q, first = o.quant.data.float(), want.quant.data.float()
            others = torch.arange(G, device="cuda") != block
            assert torch.equal(o.quant.scales[:, others], want.quant.scales[:, others])
            assert torch.equal(q[:, rest], first[:, rest])
            keep = torch.arange(D, device="cuda") != at
            assert torch.equal(o.y[:, keep], want.y[:, keep])
            scale = o.quant.scales[:, block]
            if value == value:
                assert (o.y[:, at] == value).all()
                assert (scale == float("inf")).all(), at
                inside = q[:, cols].clone()
                assert inside[:, at - cols.start].isnan().all()
                inside[:, at - cols.start] = 0
                assert (inside == 0).all(), at
            else:
                assert scale.isnan().all() and q[:, cols].isnan().all()
