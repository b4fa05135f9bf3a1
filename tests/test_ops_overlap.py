"""Matrices that lie in one buffer: calls whose rows share no byte are taken, calls
whose rows do are refused.  The refusals are told apart without a GPU: a call that
passes every check ends at the missing device."""
import itertools
import random

import pytest
import torch

import ops_ref as R

no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="host-validation tests use stand-in pointers; CPU only")
A, FAR = 0x10000000, 0x7000000000  # never dereferenced
EINVAL, ECUDA = -1, -7
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def abi():
    import __graft_entry__
    __graft_entry__.build()
    from lm_head_linear_fwd_gb300 import _abi
    return _abi


def _fwd(abi, x, y, N, D, ldx, ldy, dt=0):
    return abi.layer_norm_fwd(x, dt, N, D, ldx, None, None, 1, 1e-5, y, ldy, None, None, None)


def _calls(abi, x, y, N, D, ldx, ldy):
    """Every call that reads [N, D] at x and writes [N, D] at y (bf16)."""
    return {
        "layer_norm_fwd": _fwd(abi, x, y, N, D, ldx, ldy),
        "rms_norm_fwd": abi.rms_norm_fwd(x, 0, N, D, ldx, None, 1, 1e-5, y, ldy, None, None),
        "layer_norm_bwd x": abi.layer_norm_bwd(x, 0, N, D, ldx, FAR, D, None, 1, FAR, FAR, y, ldy,
                                               None, None, 0, None, 0, None),
        "rms_norm_bwd dy": abi.rms_norm_bwd(FAR, 0, N, D, D, x, ldx, None, 1, FAR, y, ldy, None, 0,
                                            None, 0, None),
        "embedding_fwd": abi.embedding_fwd(FAR, x, 0, N, D, N, ldx, 1.0, y, ldy, FAR, None),
        "embedding_bwd": abi.embedding_bwd(FAR, x, 0, N, D, N, ldx, 1.0, -1, y, 0, ldy, 0, FAR,
                                           1 << 40, FAR, None)}


@no_gpu
def test_slices_of_one_buffer(abi):
    N, D = 5, 24
    apart = [("left and right halves", 0, D, 2 * D, 2 * D), ("right and left", D, 0, 2 * D, 2 * D),
             ("thirds", 2 * D, 0, 3 * D, 3 * D), ("even and odd rows", 0, D, 2 * D, 2 * D),
             ("a gap between", 0, D + 8, 2 * D + 16, 2 * D + 16),
             ("far rows", 0, N * D, D, D), ("strides with a common gap", 0, D, 2 * D, 4 * D),
             ("the last columns of rows before", 3 * 2 * D + D, 0, 2 * D, 2 * D)]
    for name, x, y, ldx, ldy in apart:
        for call, rc in _calls(abi, A + 2 * x, A + 2 * y, N, D, ldx, ldy).items():
            assert rc == ECUDA, (name, call, rc)
    meet = [("one column shared", 0, D - 1, 2 * D, 2 * D), ("from the right", D + 1, 0, 2 * D, 2 * D),
            ("next row reached", D + 1, 2 * D, 2 * D, 2 * D), ("shifted rows", 0, 2 * D, D, D),
            ("other strides", 0, 8, 2 * D, 3 * D), ("inside", 8, 0, 2 * D, D),
            ("the last row alone", 0, (N - 1) * 2 * D + D - 1, 2 * D, 2 * D)]
    for name, x, y, ldx, ldy in meet:
        for call, rc in _calls(abi, A + 2 * x, A + 2 * y, N, D, ldx, ldy).items():
            assert rc == EINVAL, (name, call, rc)


@no_gpu
def test_against_bytes_marked_one_by_one(abi):
    """Random places and strides: never taken where a byte is shared, and refused only
    there when the strides are equal (or a side has one row)."""
    rng = random.Random(5)
    seen = {True: 0, False: 0}
    for _ in range(6000):
        N, D = rng.randint(1, 6), rng.randint(1, 9)
        ldx = D + rng.randint(0, 14)
        ldy = ldx if rng.random() < 0.6 else D + rng.randint(0, 14)
        x, y = 200, 200 + rng.randint(-140, 140)
        if x == y:
            continue
        if N == 1:
            ldx = ldy = D
        rows = [{p + i * ld + j for i in range(N) for j in range(D)} for p, ld in ((x, ldx), (y, ldy))]
        shared = bool(rows[0] & rows[1])
        rc = _fwd(abi, A + 4 * x, A + 4 * y, N, D, ldx, ldy, dt=1)
        assert rc in (EINVAL, ECUDA)
        if shared or ldx == ldy:
            assert (rc == EINVAL) == shared, (N, D, ldx, ldy, y - x)
        seen[shared] += 1
    assert min(seen.values()) > 500


@no_gpu
def test_head4_outputs_lie_apart_from_inputs(abi):
    V, D, M, group = 40, 200, 3, 64
    G, ldp = 4, 128
    P = [A + (k << 24) for k in range(6)]

    def logits(**kw):
        a = dict(x=P[0], dt=0, M=M, D=D, ldx=D, packed=P[1], ldp=ldp, scales=P[2], dts=1,
                 zeros=P[3], group=group, V=V, bias=P[4], y=P[5], dty=1, ldy=V, status=None,
                 stream=None)
        assert set(kw) <= set(a)
        return abi.head4_logits(*dict(a, **kw).values())

    assert logits() == ECUDA
    n = 4 * M * V
    ends = {"x": 2 * M * D, "packed": V * ldp, "scales": 4 * V * G, "zeros": V * G, "bias": 2 * V}
    for k, (name, size) in enumerate(ends.items()):
        step = 16 if name == "packed" else 4
        for at in (P[5] - size + step, P[5], P[5] + n - step):
            assert logits(**{name: at}) == EINVAL, (name, at)
        for at in (P[5] - (size + step - 1) // step * step, P[5] + n):
            assert logits(**{name: at}) == ECUDA, (name, at)
    # x and y as slices of the columns of one buffer
    assert logits(x=P[5] + 2 * 80, ldx=300, ldy=300, dty=0) == ECUDA
    assert logits(x=P[5] + 2 * 39, ldx=300, ldy=300, dty=0) == EINVAL
    assert logits(M=0, x=P[5]) == 0

    def quantize(**kw):
        a = dict(W=P[0], dt=0, V=V, D=D, ldw=D, group=group, packed=P[1], ldp=ldp, scales=P[2],
                 dts=1, zeros=P[3], stream=None)
        assert set(kw) <= set(a)
        return abi.head4_quantize(*dict(a, **kw).values())

    assert quantize() == quantize(zeros=None) == ECUDA
    for kw in (dict(packed=P[0]), dict(scales=P[0] + 2 * V * D - 4), dict(zeros=P[0] + 1),
               dict(scales=P[1]), dict(zeros=P[1] + V * ldp - 1), dict(zeros=P[2])):
        assert quantize(**kw) == EINVAL, kw
    assert quantize(scales=P[0] + 2 * V * D) == quantize(zeros=P[1] + V * ldp) == ECUDA


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,gap", [(64, 0), (37, 0), (201, 3), (1600, 1)])
def test_column_slices_and_rows_in_turn(dtype, D, gap):
    """The same bits as apart, and what lies between stays."""
    import lm_head_linear_fwd_gb300 as lh
    N, V = 700, 90
    g = torch.Generator().manual_seed(D)

    def rnd(*shape, std=1.0, dt=dtype):
        return torch.randn(*shape, generator=g).mul_(std).to(dt).cuda()

    x, dy, w = rnd(N, D), rnd(N, D, std=0.1), rnd(D, dt=F32)
    W, ids = rnd(V, D), torch.randint(0, V, (N,), generator=g).cuda()
    f = lh.layer_norm_fwd(x, w)
    b = lh.layer_norm_bwd(x, dy, f.mean, f.rstd, w)
    y = lh.embedding_fwd(ids, W, 2.0)
    gW = lh.embedding_bwd(ids, dy, V, 2.0, grad_dtype=dtype)

    def columns(rows):
        buf = torch.full((rows, 2 * D + 2 * gap), 7.0, dtype=dtype, device="cuda")
        return buf, buf[:, :D], buf[:, D + gap:2 * D + gap]

    def rows_in_turn(rows):
        buf = torch.full((2 * rows, D + gap), 7.0, dtype=dtype, device="cuda")
        return buf, buf[0::2, :D], buf[1::2, :D]

    for make, flip in itertools.product((columns, rows_in_turn), (False, True)):
        buf, p, q = make(N)
        if flip:
            p, q = q, p
        p.copy_(x)
        lh.layer_norm_fwd(p, w, y=q)
        assert torch.equal(q, f.y) and torch.equal(p, x)
        lh.layer_norm_bwd(p, dy, f.mean, f.rstd, w, grad_x=q)
        assert torch.equal(q, b.grad_x) and torch.equal(p, x)
        p.copy_(dy)
        lh.layer_norm_bwd(x, p, f.mean, f.rstd, w, grad_x=q)
        assert torch.equal(q, b.grad_x) and torch.equal(p, dy)
        p[:V].copy_(W)
        lh.embedding_fwd(ids, p[:V], 2.0, out=q)
        assert torch.equal(q, y) and torch.equal(p[:V], W)
        p.copy_(dy)
        lh.embedding_bwd(ids, p, V, 2.0, grad_W=q[:V])
        assert torch.equal(q[:V], gW) and torch.equal(p, dy)
        if gap:
            assert (buf[:, -gap:] == 7).all()
    R.close(y, *R.embedding(ids, W, 2.0, dtype))
