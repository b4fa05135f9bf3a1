"""beam_reorder writes its states in place while other blocks still read the parents, so a
state that covers them, or the status word, is refused (no GPU needed: a call that passes
every check ends at the missing device)."""
import random
import struct

import pytest
import torch

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="host-validation tests use stand-in pointers; CPU only")
A, FAR = 0x100000, 0x10000000  # never dereferenced
EINVAL, ECUDA = -1, -7


@pytest.fixture(scope="module")
def abi():
    import __graft_entry__
    __graft_entry__.build()
    from lm_head_linear_fwd_gb300 import _abi
    return _abi


def _call(abi, state, parents=FAR, status=None, B=2, K=3):
    return abi.beam_reorder(struct.pack("=Qqqqq", *state), 1, B, K, parents, status, None)


@pytest.mark.parametrize("state,apart,meet", [
    # one run of 64 bytes to each of six rows; the parents are 48 bytes, the status four
    ((A, 64, 1, 0, 64), (-48, 6 * 64), (-40, 0, 8, 6 * 64 - 8)),
    # rows of 8 bytes 64 apart, and runs of 8 in steps of 64
    ((A, 64, 1, 0, 8), (-48, 8, 16, 72, 5 * 64 + 8), (0, 24, 64, 5 * 64)),
    ((A, 128, 2, 64, 8), (-48, 8, 16, 72, 80, 5 * 128 + 72), (0, 24, 64, 5 * 128 + 64)),
    # the rows within a step of the runs
    ((A, 8, 2, 128, 8), (-48, 48, 80, 128 + 48), (0, 40, 88, 128 + 40))])
def test_parents(abi, state, apart, meet):
    for at in apart:
        assert _call(abi, state, A + at) == ECUDA, at
    for at in meet:
        assert _call(abi, state, A + at) == EINVAL, at


def test_status(abi):
    assert _call(abi, (A, 64, 1, 0, 64), FAR, FAR + 44) == EINVAL  # inside the parents
    for at, rc in ((-4, ECUDA), (0, EINVAL), (4, EINVAL), (8, ECUDA), (60, ECUDA), (64, EINVAL),
                   (5 * 64 + 8, ECUDA)):
        assert _call(abi, (A, 64, 1, 0, 8), status=A + at) == rc, at


def test_against_bytes_marked_one_by_one(abi):
    rng, met = random.Random(7), 0
    for _ in range(2000):
        B, K = rng.randint(1, 2), rng.randint(1, 3)
        R, outer, inner = B * K, rng.randint(1, 3), rng.randint(1, 12)
        step = inner + rng.randint(0, 60)
        row = (outer - 1) * step + inner + rng.randint(0, 60)
        if rng.random() < 0.3:  # rows inside a step
            row = inner + rng.randint(0, 20)
            step = (R - 1) * row + inner + rng.randint(0, 60)
        data, parents, status = A + rng.randint(0, 99), A + 8 * rng.randint(0, 40), \
            A + 4 * rng.randint(0, 80)
        bytes_ = {data + r * row + o * step + i for r in range(R) for o in range(outer)
                  for i in range(inner)}
        shared = bool(bytes_ & (set(range(parents, parents + 8 * R)) |
                                set(range(status, status + 4))))
        rc = _call(abi, (data, row, outer, step, inner), parents, status, B, K)
        if set(range(parents, parents + 8 * R)) & set(range(status, status + 4)):
            shared = True
        assert rc == (EINVAL if shared else ECUDA)
        met += shared
    assert 300 < met < 1700  # of 2000


def test_nothing_of_a_state(abi):
    assert _call(abi, (A, 64, 0, 0, 64), A) == _call(abi, (A, 64, 1, 0, 0), A, A + 64) == 0
