"""What the operators around the loss head refuse (no GPU needed): the C entry
points return a status before they touch the device, the Python calls raise.
Stand-in pointers are used only where no GPU could be reached with them."""
import pytest
import torch

no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="host-validation tests use stand-in pointers; CPU only")
A, B, C = 0x100000, 0x10000000, 0x20000000  # never dereferenced
EINVAL, ESHAPE, EDTYPE, EALIGN, EWORKSPACE, ENOSUP = -1, -2, -3, -4, -6, -8


@pytest.fixture(scope="module")
def abi():
    import __graft_entry__
    __graft_entry__.build()
    from lm_head_linear_fwd_gb300 import _abi
    return _abi


def _caller(fn, base):
    def call(**kw):
        assert set(kw) <= set(base)
        return fn(*dict(base, **kw).values())
    return call


@no_gpu
def test_embedding_fwd(abi):
    call = _caller(abi.embedding_fwd, dict(ids=A, W=B, dt=0, N=4, D=8, V=10, ldw=8, scale=1.0,
                                           out=C, ldo=8, status=A, stream=None))
    assert call(dt=2) == EDTYPE
    assert call(N=-1) == call(D=0) == call(V=0) == call(V=1 << 31) == ESHAPE
    assert call(ldw=7) == call(ldo=7) == call(ldo=1 << 60) == ESHAPE
    assert call(ids=None) == call(W=None) == call(out=None) == call(status=None) == EINVAL
    assert call(ids=A + 4) == call(W=B + 1) == call(out=C + 1) == call(status=A + 2) == EALIGN
    assert call(out=B + 64) == EINVAL  # overlaps the table


@no_gpu
def test_embedding_bwd(abi):
    call = _caller(abi.embedding_bwd, dict(ids=A, dy=B, dt=0, N=4, D=8, V=10, ldg=8, scale=1.0,
                                           pad=-1, gW=C, dtg=1, ldw=8, acc=0, ws=A, wsb=1 << 30,
                                           status=A, stream=None))
    assert call(dt=2) == call(dtg=5) == EDTYPE
    assert call(N=-1) == call(N=1 << 31) == call(D=0) == call(V=0) == call(ldg=7) == ESHAPE
    assert call(ldw=7) == ESHAPE
    assert call(acc=2) == call(ids=None) == call(dy=None) == call(gW=None) == EINVAL
    assert call(status=None) == call(gW=B) == EINVAL
    assert call(acc=1, dtg=0) == ENOSUP
    assert call(dy=B + 1) == call(gW=C + 2) == EALIGN
    need = abi.embedding_bwd_workspace_bytes(4, 8, 10)
    if need:
        assert call(ws=None) == call(wsb=need - 1) == EWORKSPACE
        assert call(ws=A + 8) == EALIGN


@no_gpu
def test_norm_fwd(abi):
    ln = _caller(abi.layer_norm_fwd, dict(x=A, dt=0, N=4, D=8, ldx=8, w=B, b=B, wdt=1, eps=1e-5,
                                          y=C, ldy=8, mean=B, rstd=B, stream=None))
    rms = _caller(abi.rms_norm_fwd, dict(x=A, dt=0, N=4, D=8, ldx=8, w=B, wdt=1, eps=1e-5, y=C,
                                         ldy=8, rstd=B, stream=None))
    for call in (ln, rms):
        assert call(dt=9) == call(wdt=-1) == EDTYPE
        assert call(N=-1) == call(D=0) == call(ldx=7) == call(ldy=7) == ESHAPE
        assert call(x=None) == call(y=None) == EINVAL
        assert call(x=A + 1) == call(y=C + 1) == call(w=B + 2) == call(rstd=B + 2) == EALIGN
        assert call(y=A + 16) == EINVAL          # overlaps x
        assert call(y=A, ldy=16) == EINVAL       # in place with another stride
    assert ln(b=B + 2) == ln(mean=B + 1) == EALIGN


@no_gpu
def test_norm_bwd(abi):
    ln = _caller(abi.layer_norm_bwd, dict(x=A, dt=0, N=4, D=8, ldx=8, dy=B, ldg=8, w=C, wdt=1,
                                          mean=C, rstd=C, dx=0x30000000, lddx=8, gw=C, gb=C, acc=0,
                                          ws=C, wsb=1 << 30, stream=None))
    rms = _caller(abi.rms_norm_bwd, dict(x=A, dt=0, N=4, D=8, ldx=8, dy=B, ldg=8, w=C, wdt=1,
                                         rstd=C, dx=0x30000000, lddx=8, gw=C, acc=0, ws=C,
                                         wsb=1 << 30, stream=None))
    for call in (ln, rms):
        assert call(dt=9) == call(wdt=4) == EDTYPE
        assert call(N=-1) == call(D=0) == call(ldx=7) == call(ldg=7) == call(lddx=7) == ESHAPE
        assert call(x=None) == call(dy=None) == call(rstd=None) == call(acc=2) == EINVAL
        assert call(dx=A) == call(dx=B + 16) == call(dx=B, lddx=9) == EINVAL
        assert call(x=A + 1) == call(gw=C + 2) == call(rstd=C + 1) == EALIGN
        assert call(ws=None) == call(wsb=0) == EWORKSPACE
        assert call(ws=C + 8) == EALIGN
    assert ln(mean=None) == EINVAL
    assert ln(gb=C + 2) == EALIGN
    assert abi.norm_bwd_workspace_bytes(0, 8) == abi.norm_bwd_workspace_bytes(4, 0) == 0


@no_gpu
def test_head4(abi):
    call = _caller(abi.head4_logits, dict(x=A, dt=0, M=2, D=200, ldx=200, packed=B, ldp=128,
                                          scales=C, dts=0, zeros=None, group=64, V=10, bias=None,
                                          y=0x30000000, dty=1, ldy=10, status=None,
                                          stream=None))
    assert call(dt=2) == call(dts=2) == call(dty=2) == EDTYPE
    assert call(M=-1) == call(D=0) == call(V=0) == call(group=48) == call(ldp=112) == ESHAPE
    assert call(ldx=199) == call(ldy=9) == ESHAPE
    assert call(x=None) == call(packed=None) == call(scales=None) == call(y=None) == EINVAL
    assert call(packed=B + 8) == call(ldp=136) == call(scales=C + 1) == call(bias=C + 1) == EALIGN
    q = _caller(abi.head4_quantize, dict(W=A, dt=0, V=10, D=200, ldw=200, group=64, packed=B,
                                         ldp=128, scales=C, dts=0, zeros=None, stream=None))
    assert q(dt=2) == q(dts=3) == EDTYPE
    assert q(V=0) == q(ldw=199) == q(group=256) == q(ldp=64) == ESHAPE
    assert q(W=None) == q(packed=None) == q(scales=None) == EINVAL
    assert q(W=A + 1) == q(packed=B + 4) == EALIGN


def test_python_calls_refuse(abi):
    import lm_head_linear_fwd_gb300 as lh
    x, w = torch.zeros(4, 8), torch.zeros(8)
    ids = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: lh.embedding_fwd(ids, x), lambda: lh.embedding(ids, x),
                 lambda: lh.embedding_bwd(ids, x, 10), lambda: lh.layer_norm_fwd(x, w),
                 lambda: lh.layer_norm(x), lambda: lh.rms_norm(x, w),
                 lambda: lh.rms_norm_bwd(x, x, torch.ones(4)), lambda: lh.head4_quantize(x),
                 lambda: lh.head4_logits(x, lh.Head4(x, x, None, 8, 32)),
                 lambda: lh.embedding(ids, x, padding_idx=4),
                 lambda: lh.embedding(ids, x, padding_idx=-1),
                 lambda: lh.layer_norm(torch.tensor(1.0)), lambda: lh.embedding([1], x)):
        with pytest.raises(ValueError):  # no CPU path, bad padding, bad shapes
            call()


@pytest.mark.gpu
def test_python_calls_refuse_on_the_device(abi):
    import lm_head_linear_fwd_gb300 as lh
    x, w = torch.zeros(4, 8, device="cuda"), torch.zeros(8, device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    st = torch.ones(4, device="cuda")
    for call in (lambda: lh.embedding_fwd(ids, x.t()), lambda: lh.embedding_fwd(ids.int(), x),
                 lambda: lh.embedding_fwd(ids, x, out=x[:3]),
                 lambda: lh.embedding_fwd(ids, x, out=x.bfloat16()),
                 lambda: lh.embedding_bwd(ids[:3], x, 10),
                 lambda: lh.embedding_bwd(ids, x, 10, 1.0, 10),
                 lambda: lh.embedding_bwd(ids, x, 10, accumulate_grad_W=True),
                 lambda: lh.layer_norm_fwd(x, w[:7]), lambda: lh.layer_norm_fwd(x.t()),
                 lambda: lh.layer_norm_bwd(x, x, None, st, w),
                 lambda: lh.layer_norm_bwd(x, x.bfloat16(), st, st, w),
                 lambda: lh.rms_norm_bwd(x, x, st[:3], w),
                 lambda: lh.rms_norm_bwd(x, x, st, w, accumulate=True),
                 lambda: lh.head4_quantize(x, 16),
                 lambda: lh.head4_logits(x[:, :7], lh.head4_quantize(x, 32)),
                 lambda: lh.head4_logits(x, lh.Head4(x.byte(), st, None, 8, 32))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: lh.embedding_fwd(ids, x.half()), lambda: lh.layer_norm_fwd(x.half()),
                 lambda: lh.layer_norm_fwd(x, w, w.bfloat16()), lambda: lh.layer_norm_fwd(x, w.half()),
                 lambda: lh.rms_norm_bwd(x, x, st.bfloat16(), w),
                 lambda: lh.head4_logits(x, lh.head4_quantize(x, 32), st.bfloat16())):
        with pytest.raises((TypeError, ValueError)):
            call()
    with pytest.raises(lh.FlceError):  # adding to a bf16 gradient
        lh.embedding_bwd(ids, x, 10, grad_W=torch.zeros(10, 8, dtype=torch.bfloat16, device="cuda"),
                         accumulate_grad_W=True)
    with pytest.raises(lh.FlceError):  # rows that overlap
        lh.layer_norm_fwd(w.expand(4, 8))


@no_gpu
def test_arguments_from_memory_reach_their_places(abi):
    """flce_call answers as the entry point does, with every argument wrong in turn."""
    P = [A + (k << 28) for k in range(9)]
    calls = {
        "embedding_fwd": [P[0], P[1], 0, 4, 8, 10, 8, 1.0, P[2], 8, P[3], 0],
        "embedding_bwd": [P[0], P[1], 0, 4, 8, 10, 8, 1.0, -1, P[2], 1, 8, 0, P[3], 1 << 20, P[4],
                          0],
        "layer_norm_fwd": [P[0], 0, 4, 8, 8, P[1], P[2], 0, 1e-5, P[3], 8, P[4], P[5], 0],
        "rms_norm_fwd": [P[0], 0, 4, 8, 8, P[1], 0, 1e-5, P[2], 8, P[3], 0],
        "layer_norm_bwd": [P[0], 0, 4, 8, 8, P[1], 8, P[2], 0, P[3], P[4], P[5], 8, P[6], P[7], 0,
                           P[8], 1 << 20, 0],
        "rms_norm_bwd": [P[0], 0, 4, 8, 8, P[1], 8, P[2], 0, P[3], P[4], 8, P[5], 0, P[6], 1 << 20,
                         0],
        "head4_logits": [P[0], 0, 2, 100, 100, P[1], 64, P[2], 0, P[3], 64, 10, P[4], P[5], 0, 10,
                         P[6], 0]}
    for name, good in calls.items():
        types = abi._SIGNATURES[name][1]
        assert len(types) == len(good), name
        refused = 0
        for k, t in enumerate(types[:-1]):  # (any stream is taken)
            for bad in {abi._f: (2.0,), abi._p: (0, good[k] + 1)}.get(t, (-7, 1 << 40)):
                if t is abi._i and bad > 9:
                    bad = 9
                args = good[:k] + [bad] + good[k + 1:]
                want = getattr(abi, name)(*args)
                assert getattr(abi.packed, name)(*args) == want < 0, (name, k, bad, want)
                refused += want != -7  # not only the missing device
        assert refused >= len(types)
    call = abi.load().flce_call
    assert call(99, bytes(96), 96) == ENOSUP
    assert call(0, bytes(88), 88) == call(0, None, 96) == EINVAL
