"""Ids out of range through the autograd front end of the lookup."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_caller_sees_bad_ids():
    import lm_head_linear_fwd_gb300 as lh
    V, D = 10, 24
    W = torch.randn(V, D, device="cuda", requires_grad=True)
    good = torch.tensor([[1, 2, 9], [0, 1, 1]], device="cuda")
    st = lh.new_status("cuda")
    lh.embedding(good, W, scale=2.0, status=st).sum().backward()
    lh.check_status(st)
    want = W.grad.clone()
    for bad in (-1, V, 2 ** 40):
        for use in (True, False):  # with and without a graph of autograd
            st = lh.new_status("cuda")
            W.grad = None
            with torch.set_grad_enabled(use):
                y = lh.embedding(torch.cat([good, torch.full((2, 1), bad, device="cuda")], 1), W,
                                 scale=2.0, status=st)
            assert (y[:, 3] == 0).all() and torch.equal(y[:, :3], W.detach()[good] * 2)
            with pytest.raises(lh.FlceError):
                lh.check_status(st)
            if use:
                st.zero_()
                y.sum().backward()
                assert torch.equal(W.grad, want)
                assert int(st.item()) == -5  # the backward pass says so too
    with pytest.raises(ValueError):
        lh.embedding(good, W, status=torch.zeros(1, dtype=torch.int32))
