"""What the 8-bit operators and beam search refuse (no GPU needed): the C entry points
return a status before they touch the device, the Python calls raise.  Stand-in
pointers are used only where no GPU could be reached with them; a call that passes
every check ends at the missing device."""
import contextlib
import random
import struct
import types

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="host-validation tests use stand-in pointers; CPU only")
pytestmark = [no_gpu, pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")]
A, B, C, D_ = 0x100000, 0x10000000, 0x20000000, 0x30000000  # never dereferenced
E, F, G = 0x40000000, 0x50000000, 0x60000000
EINVAL, ESHAPE, EDTYPE, EALIGN, EWORKSPACE, ECUDA, ENOSUP = -1, -2, -3, -4, -6, -7, -8


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


def test_rms_norm_add_fwd(abi):
    call = _caller(abi.rms_norm_add_fwd, dict(
        x=A, dt=0, N=4, D=40, ldx=40, res=B, ldr=40, w=C, wdt=1, eps=1e-5, sum=D_, lds=40, y=E,
        ldy=40, q=F, ldq=48, scales=G, rstd=G + 4096, stream=None))
    assert call(dt=2) == call(wdt=7) == EDTYPE
    assert call(N=-1) == call(D=0) == call(ldx=39) == call(ldr=39) == call(lds=39) == ESHAPE
    assert call(ldy=39) == call(ldq=32) == ESHAPE
    assert call(x=None) == call(y=None, q=None, scales=None) == EINVAL
    assert call(q=None) == call(scales=None) == EINVAL
    for bad in (dict(x=A + 1), dict(res=B + 1), dict(sum=D_ + 1), dict(y=E + 1), dict(w=C + 2),
                dict(q=F + 8), dict(ldq=40), dict(ldq=56), dict(scales=G + 2), dict(rstd=G + 1)):
        assert call(**bad) == EALIGN, bad
    for bad in (dict(sum=A + 16), dict(y=B + 16), dict(sum=A, lds=48), dict(y=B, ldy=48),
                dict(q=A), dict(q=B + 32), dict(q=D_), dict(q=E), dict(y=D_), dict(sum=E + 2),
                dict(scales=F), dict(scales=E), dict(scales=A)):
        assert call(**bad) == EINVAL, bad
    for good in (dict(), dict(res=None), dict(sum=None), dict(sum=A), dict(sum=B), dict(y=A),
                 dict(y=B), dict(sum=B, y=A), dict(q=None, scales=None), dict(y=None),
                 dict(w=None, rstd=None)):
        assert call(**good) == ECUDA, good
    assert call(N=0) == 0


def test_rms_norm_add_bwd(abi):
    call = _caller(abi.rms_norm_add_bwd, dict(
        sum=A, dt=0, N=4, D=8, lds=8, gy=B, ldgy=8, gs=C, ldgs=8, w=D_, wdt=1, rstd=D_ + 4096,
        gx=E, ldgx=8, gw=F, acc=0, ws=G, wsb=1 << 30, stream=None))
    assert call(dt=9) == call(wdt=4) == EDTYPE
    assert call(N=-1) == call(D=0) == call(lds=7) == call(ldgy=7) == call(ldgs=7) == ESHAPE
    assert call(ldgx=7) == ESHAPE
    assert call(sum=None) == call(gy=None) == call(rstd=None) == call(acc=2) == EINVAL
    assert call(gx=A) == call(gx=B + 16) == call(gx=C + 16) == call(gx=C, ldgx=9) == EINVAL
    assert call(gs=C + 1) == call(gy=B + 1) == call(gw=F + 2) == call(rstd=D_ + 1) == EALIGN
    assert call(ws=None) == call(wsb=0) == EWORKSPACE
    assert call(gx=C) == call(gx=B) == call(gs=None) == ECUDA


def test_quantize8(abi):
    call = _caller(abi.quantize8, dict(x=A, dt=0, R=200, C=40, ldx=40, rows=1, q=B, ldq=48,
                                       scales=C, qt=D_, ldqt=208, scales_t=E, stream=None))
    assert call(dt=2) == EDTYPE
    assert call(rows=2) == call(rows=0) == call(rows=64) == EINVAL
    assert call(R=-1) == call(C=0) == call(ldx=39) == call(ldq=32) == call(ldqt=192) == ESHAPE
    assert call(R=1 << 37, C=1 << 20, ldx=1 << 20, ldq=1 << 20, ldqt=1 << 38) == ESHAPE
    assert call(x=None) == call(q=None) == call(scales_t=None) == EINVAL
    assert call(q=None, scales=None, qt=None, scales_t=None) == EINVAL
    assert call(x=A + 1) == call(q=B + 8) == call(ldq=40) == call(qt=D_ + 4) == EALIGN
    assert call(ldqt=201) == call(scales=C + 1) == call(scales_t=E + 2) == EALIGN
    assert call(q=A) == call(qt=A + 160) == call(qt=B) == call(scales=B) == call(scales_t=C) == EINVAL
    assert call() == call(rows=128) == call(q=None, scales=None) == ECUDA
    assert call(R=0) == 0


def test_gemm8(abi):
    call = _caller(abi.gemm8, dict(a=A, lda=48, sa=B, M=5, b=C, ldb=48, sb=D_, rows=128, N=70, K=40,
                                   bias=E, dtb=1, y=F, dty=0, ldy=70, acc=0, status=G, stream=None))
    assert call(dty=2) == call(dtb=-1) == EDTYPE
    assert call(rows=2) == call(acc=2) == call(a=None) == call(b=None) == call(y=None) == EINVAL
    assert call(sa=None) == call(sb=None) == EINVAL
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(M=1 << 31), dict(N=1 << 31), dict(K=1 << 31),
                dict(lda=32), dict(ldb=32), dict(ldy=69)):
        assert call(**bad) == ESHAPE, bad
    for bad in (dict(a=A + 8), dict(b=C + 4), dict(lda=40), dict(ldb=56), dict(y=F + 1),
                dict(sa=B + 2), dict(sb=D_ + 1), dict(bias=E + 2), dict(status=G + 2)):
        assert call(**bad) == EALIGN, bad
    assert call(acc=1) == ENOSUP
    for bad in (dict(y=A), dict(y=C), dict(y=B), dict(y=D_), dict(y=E)):
        assert call(**bad) == EINVAL, bad
    assert call() == call(bias=None, status=None) == call(acc=1, dty=1) == call(rows=1) == ECUDA
    assert call(M=0, a=None, sa=None, y=None) == 0


def test_beam_select(abi):
    need = abi.beam_select_workspace_bytes(3, 4, 1000, 4)
    assert need >= 3 * 4 * (4 * 8 + 8)
    call = _caller(abi.beam_select, dict(z=A, dt=0, B=3, K=4, V=1000, ld=1000, s=B, fin=B + 4096,
                                         pad=0, num=4, os=C, ot=D_, op=E, ws=F, wsb=need,
                                         stream=None))
    assert call(dt=3) == EDTYPE
    for bad in (dict(B=-1), dict(K=0), dict(K=65), dict(V=0), dict(V=(1 << 20) + 1), dict(num=0),
                dict(num=65), dict(ld=999), dict(V=1, K=2, num=3), dict(B=1 << 26)):
        assert call(**bad) == ESHAPE, bad
    for bad in (dict(z=None), dict(s=None), dict(os=None), dict(ot=None), dict(op=None),
                dict(pad=-1), dict(pad=1000), dict(os=A), dict(ot=C), dict(op=D_), dict(ws=C),
                dict(os=B), dict(ot=B + 4096), dict(ws=A)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(z=A + 1), dict(s=B + 2), dict(os=C + 2), dict(ot=D_ + 4), dict(op=E + 4),
                dict(ws=F + 8)):
        assert call(**bad) == EALIGN, bad
    assert call(ws=None) == call(wsb=need - 1) == EWORKSPACE
    assert call() == call(fin=None, pad=-1) == ECUDA
    assert call(B=0) == 0
    for sizes in ((0, 4, 10, 4), (-1, 4, 10, 4), (1, 0, 10, 4), (1, 4, 10, 65)):
        assert abi.beam_select_workspace_bytes(*sizes) == 0


def _states(*rows):
    return b"".join(struct.pack("=Qqqqq", *r) for r in rows)


def test_beam_reorder(abi):
    def call(*rows, n=None, B_=2, K=3, parents=B, status=C):
        return abi.beam_reorder(_states(*rows), len(rows) if n is None else n, B_, K, parents,
                                status, None)
    good = (A, 64, 1, 0, 64)
    assert call(good) == call((A, 64, 2, 32, 20)) == call((A, 8, 2, 64, 8)) == ECUDA
    assert call(good, parents=None) == call((0, 64, 1, 0, 64)) == EINVAL
    assert call(good, status=None) == ECUDA
    assert call(good, parents=B + 4) == call(good, status=C + 2) == EALIGN
    assert call(good, K=0) == call(good, K=65) == call(good, B_=-1) == call(good, n=-1) == ESHAPE
    for bad in ((A, 63, 1, 0, 64), (A, 64, 2, 10, 20), (A, 64, 2, 32, -1), (A, -64, 1, 0, 64),
                (A, 40, 2, 32, 20), (A, 8, 2, 32, 8), (A, 1 << 61, 1, 0, 8),
                (A, 64, 1 << 40, 1 << 30, 8), (A, 0, 1, 0, 8)):
        assert call(bad) == ESHAPE, bad
    assert abi.beam_reorder(None, 1, 2, 3, B, C, None) == EINVAL
    assert call() == call((0, 0, 0, 0, 0)) == call(good, B_=0) == 0


def test_states_that_meet(abi):
    """Random places and strides against bytes marked one by one: states that share a
    byte are never taken; the layouts that caches come in are."""
    def run(x, y, Bn, K):
        return abi.beam_reorder(_states(x, y), 2, Bn, K, B, C, None)

    def marked(t, R):
        p, rs, outer, os_, inner = t
        return {p + r * rs + o * os_ + i for r in range(R) for o in range(outer)
                for i in range(inner)}
    rng, met = random.Random(3), 0
    for _ in range(3000):
        Bn, K = rng.randint(1, 2), rng.randint(1, 3)
        pair = []
        for _ in range(2):
            outer, inner = rng.randint(1, 3), rng.randint(1, 6)
            os_ = inner + rng.randint(0, 12)
            rs = (outer - 1) * os_ + inner + rng.randint(0, 12)
            if rng.random() < 0.3:  # rows inside a step
                rs = inner + rng.randint(0, 3)
                os_ = (Bn * K - 1) * rs + inner + rng.randint(0, 9)
            pair.append((A + rng.randint(0, 60), rs, outer, os_, inner))
        shared = bool(marked(pair[0], Bn * K) & marked(pair[1], Bn * K))
        rc = run(*pair, Bn, K)
        assert rc in (EINVAL, ECUDA)
        assert not shared or rc == EINVAL, pair
        met += shared
    assert met > 300
    # K and V of [R, 2, H, L, D], of [R, H, 2, L, D], of [2, L, R, H D], filled parts
    H, L, D, R = 3, 40, 16, 6
    full = H * L * D
    for x, y in (((A, 2 * full, H, L * D, 10 * D), (A + full, 2 * full, H, L * D, 10 * D)),
                 ((A, 2 * full, H, 2 * L * D, 10 * D), (A + L * D, 2 * full, H, 2 * L * D, 10 * D)),
                 ((A, H * D, 10, R * H * D, H * D), (A + L * R * H * D, H * D, 10, R * H * D, H * D)),
                 ((A, full, 1, 0, full), (A + R * full, full, 1, 0, full))):
        assert run(x, y, 2, 3) == ECUDA
    assert run((A, full, 1, 0, full), (A, full, 1, 0, full), 2, 3) == EINVAL


# ------------------------------------------------------------------ Python calls

@pytest.fixture
def mods(monkeypatch, abi):
    from lm_head_linear_fwd_gb300 import beam, eight, ops
    reached = []
    names = [n for n in vars(ops._call) if not n.startswith("_")]
    stand_in = types.SimpleNamespace(reached=reached, **{
        n: (lambda n: lambda *args: reached.append((n, args)) or 0)(n) for n in names})
    for m in (eight, beam):
        monkeypatch.setattr(m, "_call", stand_in)
        monkeypatch.setattr(m, "_stream", lambda device: 0)
    monkeypatch.setattr(beam._abi, "beam_reorder",
                        lambda *args: reached.append(("beam_reorder", args)) or 0)
    monkeypatch.setattr(eight, "norm_bwd_workspace_bytes", lambda *a: 4096)
    monkeypatch.setattr(torch.cuda, "device", lambda index: contextlib.nullcontext())
    with FakeTensorMode():
        yield eight, beam, reached


N, D, V = 4, 160, 30


def _args(op, dev="cuda:0"):
    def z(*shape, dt=torch.float32):
        return torch.zeros(*shape, dtype=dt, device=dev)
    f8, i64 = torch.float8_e4m3fn, torch.int64
    st = z(1, dt=torch.int32)
    return {
        "rms_norm_add_fwd": dict(x=z(N, D), residual=z(N, D), weight=z(D), y=z(N, D),
                                 summed=z(N, D), rstd=z(N), q=z(N, D, dt=f8), scales=z(N, 2)),
        "rms_norm_add_bwd": dict(summed=z(N, D), grad_y=z(N, D), grad_summed=z(N, D), rstd=z(N),
                                 weight=z(D), grad_x=z(N, D), grad_weight=z(D),
                                 ws=z(4096, dt=torch.uint8)),
        "quantize8": dict(x=z(N, D), q=z(N, D, dt=f8), scales=z(N, 2), qt=z(D, 16, dt=f8),
                          scales_t=z(D, 1)),
        "gemm8": dict(a=z(N, D, dt=f8), sa=z(N, 2), b=z(V, D, dt=f8), sb=z(1, 2), bias=z(V),
                      out=z(N, V), status=st),
        "beam_select": dict(logits=z(N, V), scores=z(N), finished=z(N, dt=torch.bool),
                            os=z(2, 2), ot=z(2, 2, dt=i64), op=z(2, 2, dt=i64),
                            ws=z(4096, dt=torch.uint8)),
        "beam_reorder": dict(state=z(N, 7), other=z(N, 2, 3), parents=z(2, 2, dt=i64), status=st),
    }[op]


def _make(mods, op, a):
    eight, beam, _ = mods
    a = dict(a)
    if op == "rms_norm_add_fwd":
        a["quant"] = eight.Quant8(a.pop("q"), a.pop("scales"))
        return eight.rms_norm_add_fwd(**a)
    if op == "quantize8":
        return eight.quantize8_pair(a["x"], out=eight.Quant8(a["q"], a["scales"]),
                                    out_t=eight.Quant8(a["qt"][:, :N], a["scales_t"]))
    if op == "gemm8":
        return eight.gemm8(eight.Quant8(a["a"], a["sa"]), eight.Quant8(a["b"], a["sb"], 128),
                           a["bias"], out=a["out"], status=a["status"])
    if op == "beam_select":
        return beam.beam_select(a["logits"], a["scores"], 2, finished=a["finished"],
                                out=beam.BeamOut(a["os"], a["ot"], a["op"]), ws=a["ws"])
    if op == "beam_reorder":
        return beam.beam_reorder_([a["state"], a["other"]], a["parents"], status=a["status"])
    return getattr(eight, op)(**a)


OPS = ["rms_norm_add_fwd", "rms_norm_add_bwd", "quantize8", "gemm8", "beam_select", "beam_reorder"]


@pytest.mark.parametrize("op", OPS)
def test_every_tensor_lies_on_the_same_gpu(mods, op):
    good = _args(op)
    _make(mods, op, good)
    assert [n for n, _ in mods[2]] == [op]
    for dev in ("cuda:1", "cpu"):
        other = _args(op, dev)
        for name in good:
            with pytest.raises(ValueError):
                _make(mods, op, dict(good, **{name: other[name]}))
    assert len(mods[2]) == 1


def _refused(mods, which, **kw):
    with pytest.raises((ValueError, TypeError)):
        _make(mods, which, dict(_args(which), **kw))


def test_shapes_and_types(mods):
    def z(*shape, dt=torch.float32):
        return torch.zeros(shape, dtype=dt, device="cuda:0")
    f8, bf, i64 = torch.float8_e4m3fn, torch.bfloat16, torch.int64
    for kw in (dict(residual=z(N, D + 1)), dict(residual=z(N, D, dt=bf)), dict(weight=z(D + 1)),
               dict(summed=z(N, D, dt=bf)), dict(y=z(N + 1, D)), dict(q=z(N, D, dt=torch.uint8)),
               dict(q=z(N, D + 16, dt=f8)), dict(scales=z(N, 3)), dict(scales=z(N, 2, dt=bf)),
               dict(rstd=z(N + 1)), dict(x=z(N, D, 1)), dict(x=z(D, N).t())):
        _refused(mods, "rms_norm_add_fwd", **kw)
    for kw in (dict(grad_y=z(N, D, dt=bf)), dict(grad_summed=z(N, D + 1)), dict(rstd=None),
               dict(grad_x=z(N, D, dt=bf)), dict(grad_weight=z(D, dt=bf)), dict(weight=z(D - 1))):
        _refused(mods, "rms_norm_add_bwd", **kw)
    for kw in (dict(q=z(N, D)), dict(scales=z(N, 1)), dict(qt=z(D, 32, dt=bf)),
               dict(scales_t=z(D, 2)), dict(x=z(N, D + 1))):
        _refused(mods, "quantize8", **kw)
    for kw in (dict(a=z(N, D + 16, dt=f8)), dict(sa=z(N, 1)), dict(b=z(V, D)), dict(sb=z(V, 2)),
               dict(bias=z(V + 1)), dict(out=z(N, V + 1)), dict(out=z(V, N).t()),
               dict(status=z(1))):
        _refused(mods, "gemm8", **kw)
    for kw in (dict(logits=z(N + 1, V)), dict(logits=z(V, N).t()), dict(scores=z(N, dt=bf)),
               dict(scores=None), dict(finished=z(N)), dict(finished=z(N - 1, dt=torch.bool)),
               dict(os=z(2, 3)), dict(ot=z(2, 2)), dict(op=z(2, 2, dt=torch.int32)),
               dict(ot=z(2, 4, dt=i64)[:, ::2])):
        _refused(mods, "beam_select", **kw)
    for kw in (dict(state=z(N + 1, 7)), dict(state=z()), dict(parents=z(2, 2)),
               dict(parents=z(4, dt=i64)), dict(parents=z(2, 4, dt=i64)[:, ::2]),
               dict(other=z(N, 2, 3, 4, 5)[:, :, :2, :3]), dict(status=z(1))):
        _refused(mods, "beam_reorder", **kw)
    eight, beam, reached = mods
    f = eight.Quant8(z(N, D, dt=f8), z(1, 2), 128)
    with pytest.raises(ValueError):
        eight.gemm8(f, f)  # a by rows only
    with pytest.raises(ValueError):
        eight.gemm8(eight.Quant8(z(N, D, dt=f8), z(N, 2)), f, accumulate=True)
    with pytest.raises(ValueError):
        eight.quantize8(z(N, D), 64)
    with pytest.raises(ValueError):
        eight.rms_norm_add_fwd(z(N, D), want_y=False)
    with pytest.raises(ValueError):
        eight.rms_norm_add(z(N, D), z(N, D + 1))
    with pytest.raises(ValueError):
        eight.linear8(z(N, D), z(V, D + 1))
    with pytest.raises(ValueError):
        beam.beam_select(z(N, V), z(N), 3)
    assert not reached


def test_runs_of_a_state():
    from lm_head_linear_fwd_gb300.beam import _runs

    def runs(t):
        return _runs(t.shape, t.stride(), t.element_size())
    t = torch.empty(6, 4, 10, 8, dtype=torch.bfloat16)
    assert runs(t) == (640, 1, 0, 640)
    assert runs(t[:, :, :7]) == (640, 4, 160, 112)
    assert runs(t[:, 1]) == (640, 1, 0, 160)
    assert runs(t.transpose(1, 2)) == (640, 1, 0, 640)
    assert runs(t[:, :, :, 2]) == (640, 40, 16, 2)
    assert runs(t[:, :2, :7, :3]) is None
    assert runs(t[:, 1:2, :7, :3]) == (640, 7, 16, 6)
    assert runs(t.transpose(0, 1)) == (160, 6, 640, 160)
    assert runs(torch.empty(6)) == (4, 1, 0, 4)
