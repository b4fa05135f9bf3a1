"""beam_select's limits are those of its header (no GPU needed): sizes whose blocks pass a
launch's count are refused before anything is enqueued."""
import pytest
import torch

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="host-validation tests use stand-in pointers; CPU only")
ESHAPE, ECUDA = -2, -7
LEAST = 2 ** 31


@pytest.fixture(scope="module")
def abi():
    import __graft_entry__
    __graft_entry__.build()
    from lm_head_linear_fwd_gb300 import _abi
    return _abi


@pytest.mark.parametrize("V", [1, 2040, 2041, 2042, 2047, 2048, 4088, 4089, 4096, 1 << 20])
def test_blocks(abi, V):
    """64 B and B K ceil((V + 7) / 2048) below 2^31."""
    K, per = 64, -(-(V + 7) // 2048)
    most = min((LEAST - 1) // (K * per), (LEAST - 1) // 64)  # requests
    for B, fits in ((most, True), (most + 1, False)):
        assert (B * K * per < LEAST) == fits
        need = abi.beam_select_workspace_bytes(B, K, V, 1)
        rc = abi.beam_select(1 << 20, 0, B, K, V, V, 1 << 50, None, 0, 1, 1 << 51, 1 << 52, 1 << 53,
                             1 << 54, 1 << 49, None)
        assert (need > 0) == fits and rc == (ECUDA if fits else ESHAPE), (B, need, rc)
