"""Arguments of another device, type or layout than a call needs are refused before
their address is taken.  Fake tensors stand in for those of two GPUs; a call whose
checks all pass ends at a stand-in for the library."""
import contextlib
import types

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="fake tensors of two GPUs; on a machine without one only")
pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")


@pytest.fixture
def ops(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    from lm_head_linear_fwd_gb300 import ops as m
    names = [n for n in vars(m._call) if not n.startswith("_")]
    stand_in = types.SimpleNamespace(**{n: (lambda n: lambda *args: reached.append((n, args)) or 0)(n)
                                        for n in names})
    reached = stand_in.reached = []
    monkeypatch.setattr(m, "_call", stand_in)
    monkeypatch.setattr(m, "_stream", lambda device: 0)
    monkeypatch.setattr(m, "embedding_bwd_workspace_bytes", lambda *a: 4096)
    monkeypatch.setattr(m, "norm_bwd_workspace_bytes", lambda *a: 4096)
    monkeypatch.setattr(torch.cuda, "device", lambda index: contextlib.nullcontext())
    with FakeTensorMode():
        yield m


N, D, V = 4, 128, 10


def _args(op, dev="cuda:0"):
    """The tensors of a call by name, all in order."""
    def z(*shape, dt=torch.float32):
        return torch.zeros(*shape, dtype=dt, device=dev)
    ids, st, ws = z(N, dt=torch.int64), z(1, dt=torch.int32), z(4096, dt=torch.uint8)
    row, vec, stat = z(N, D), z(D), z(N)
    return {
        "embedding_fwd": dict(ids=ids, W=z(V, D), out=row, status=st),
        "embedding_bwd": dict(ids=ids, grad_out=row, grad_W=z(V, D), ws=ws, status=st),
        "layer_norm_fwd": dict(x=row, weight=vec, bias=z(D), y=z(N, D), mean=stat, rstd=z(N)),
        "rms_norm_fwd": dict(x=row, weight=vec, y=z(N, D), rstd=stat),
        "layer_norm_bwd": dict(x=row, grad_y=z(N, D), mean=stat, rstd=z(N), weight=vec,
                               grad_x=z(N, D), grad_weight=z(D), grad_bias=z(D), ws=ws),
        "rms_norm_bwd": dict(x=row, grad_y=z(N, D), rstd=stat, weight=vec, grad_x=z(N, D),
                             grad_weight=z(D), ws=ws),
        "head4_logits": dict(x=row, packed=z(V, 64, dt=torch.uint8), scales=z(V, 1),
                             zeros=z(V, 1, dt=torch.uint8), bias=z(V), out=z(N, V), status=st),
    }[op]


def _call(ops, op, a, group=128):
    a = dict(a)
    if op == "embedding_bwd":
        a["V"] = V
    if op == "layer_norm_bwd":
        a["want_grad_bias"] = True
    if op == "head4_logits":
        a["head"] = ops.Head4(a.pop("packed"), a.pop("scales"), a.pop("zeros"), D, group)
    return getattr(ops, op)(**a)


OPS = ["embedding_fwd", "embedding_bwd", "layer_norm_fwd", "rms_norm_fwd", "layer_norm_bwd",
       "rms_norm_bwd", "head4_logits"]


@no_gpu
@pytest.mark.parametrize("op", OPS)
def test_every_tensor_lies_on_the_same_gpu(ops, op):
    good = _args(op)
    _call(ops, op, good)
    assert [n for n, _ in ops._call.reached] == [op]
    elsewhere = _args(op, "cuda:1"), _args(op, "cpu")
    for name in good:
        for other in elsewhere:
            with pytest.raises(ValueError):
                _call(ops, op, dict(good, **{name: other[name]}))
    assert len(ops._call.reached) == 1


@no_gpu
@pytest.mark.parametrize("op", ["embedding_fwd", "embedding_bwd", "head4_logits"])
def test_status_is_a_word(ops, op):
    good = _args(op)
    for bad in (torch.zeros(1, dtype=torch.int64, device="cuda:0"),
                torch.zeros(1, device="cuda:0"), torch.zeros(0, dtype=torch.int32, device="cuda:0"),
                0):
        with pytest.raises(ValueError):
            _call(ops, op, dict(good, status=bad))
    assert not ops._call.reached
    _call(ops, op, dict(good, status=None))
    assert ops._call.reached


@no_gpu
@pytest.mark.parametrize("op", ["embedding_bwd", "layer_norm_bwd", "rms_norm_bwd"])
def test_workspace_counts_in_bytes(ops, op):
    good = _args(op)
    with pytest.raises(ValueError):
        _call(ops, op, dict(good, ws=torch.zeros(4096, 2, dtype=torch.uint8, device="cuda:0")[:, 0]))
    for ws, nbytes in ((torch.zeros(1024, device="cuda:0"), 4096), (good["ws"], 4096), (None, 4096)):
        _call(ops, op, dict(good, ws=ws))
        assert nbytes in ops._call.reached.pop()[1]


@no_gpu
def test_group_of_a_head(ops):
    for group in (0, -64, 48, 256):
        with pytest.raises(ValueError):
            _call(ops, "head4_logits", _args("head4_logits"), group=group)
    assert not ops._call.reached


@no_gpu
@pytest.mark.parametrize("op", ["embedding_bwd", "layer_norm_bwd", "rms_norm_bwd"])
def test_workspace_is_asked_for_on_the_tensors_device(ops, op, monkeypatch):
    """A device's answer is not another's: they differ in SMs."""
    current, asked = [0], []

    @contextlib.contextmanager
    def device(index):
        old, current[0] = current[0], index
        yield
        current[0] = old

    def query(*sizes):
        asked.append(current[0])
        return 1000 + current[0]

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(ops, "embedding_bwd_workspace_bytes", query)
    monkeypatch.setattr(ops, "norm_bwd_workspace_bytes", query)
    for index in (1, 0, 1, 0):
        _call(ops, op, dict(_args(op, f"cuda:{index}"), ws=None))
        assert 1000 + index in ops._call.reached[-1][1], index
    assert sorted(asked) == [0, 1]  # once for each


@pytest.mark.gpu
@pytest.mark.parametrize("op", OPS)
def test_host_tensors_beside_device_ones(op):
    from lm_head_linear_fwd_gb300 import ops
    good, host = _args(op, "cuda"), _args(op, "cpu")
    if "ids" in good:
        good["ids"].fill_(V - 1)
    if "ws" in good:  # what these sizes need
        need = ops.embedding_bwd_workspace_bytes(N, D, V) if op == "embedding_bwd" \
            else ops.norm_bwd_workspace_bytes(N, D)
        good["ws"] = torch.zeros(-(-need // 4), device="cuda")
    _call(ops, op, good)
    for name in good:
        with pytest.raises(ValueError):
            _call(ops, op, dict(good, **{name: host[name]}))
    if "status" in good:
        with pytest.raises(ValueError):
            _call(ops, op, dict(good, status=torch.zeros(1, dtype=torch.int64, device="cuda")))
    _call(ops, op, good)
    torch.cuda.synchronize()
