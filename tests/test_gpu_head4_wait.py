"""What a wait of the 4-bit head that gives up leaves behind, without a GPU fault: a
barrier that nothing completes, with a short limit."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_wait_that_gave_up_is_reported_and_its_sums_are_nan():
    import lm_head_linear_fwd_gb300 as lh
    from lm_head_linear_fwd_gb300 import _abi
    for _ in range(3):
        st = lh.new_status("cuda")
        y = torch.zeros(4, device="cuda")
        rc = _abi.head4_wait_selftest(y.data_ptr(), st.data_ptr(), 20_000_000,
                                      torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        assert int(st.item()) == -9  # FLCE_ETIMEOUT
        assert y[:3].tolist() == [1.0, 1.0, 1.0] and y[3].isnan()
    assert _abi.head4_wait_selftest(y.data_ptr(), st.data_ptr(), 3_000_000_000, None) == -2
    # the context is intact, and an ordinary call says nothing
    W = torch.randn(500, 256, device="cuda", dtype=torch.bfloat16)
    x = torch.randn(20, 256, device="cuda", dtype=torch.bfloat16)
    st = lh.new_status("cuda")
    z = lh.head4_logits(x, lh.head4_quantize(W), status=st)
    lh.check_status(st)
    assert z.isfinite().all()
