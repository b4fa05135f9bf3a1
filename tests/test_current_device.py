"""The library launches on the current device: calls on tensors of another one are refused
before they reach it (the default stream's handle is the same on every device, so that a
kernel would run on one GPU with addresses of another).  Fake tensors stand in for those
of two GPUs."""
import contextlib
import types

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

pytestmark = [pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="fake tensors of two GPUs; on a machine without one only"),
              pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")]


@pytest.fixture
def lib(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import lm_head_linear_fwd_gb300 as lh
    from lm_head_linear_fwd_gb300 import api, beam, eight, ops
    reached, current = [], [0]

    def stand_in(name):
        return lambda *args: reached.append(name) or 0
    names = [n for n in vars(ops._call) if not n.startswith("_")]
    call = types.SimpleNamespace(**{n: stand_in(n) for n in names})
    for m in (ops, eight, beam):
        monkeypatch.setattr(m, "_call", call)
    for m, n in ((ops, "head4_quantize"), (beam, "beam_reorder"), (api, "ce_logits_bwd"),
                 (api, "flce_grad_scale")):
        monkeypatch.setattr(m._abi, n, stand_in(n))
    for m in (eight, ops):
        monkeypatch.setattr(m, "norm_bwd_workspace_bytes", lambda *a: 4096)
    monkeypatch.setattr(api, "_current_device", lambda: current[0], raising=False)
    monkeypatch.setattr(ops, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device: types.SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(torch.cuda, "device", lambda index: contextlib.nullcontext())
    with FakeTensorMode():
        yield lh, reached, current


def _calls(lh, dev):
    def z(*shape, dt=torch.float32):
        return torch.zeros(*shape, dtype=dt, device=dev)
    x, i64 = z(4, 160), torch.int64
    q = lh.Quant8(z(4, 160, dt=torch.float8_e4m3fn), z(4, 2))
    w = lh.Quant8(z(30, 160, dt=torch.float8_e4m3fn), z(1, 2), 128)
    return {
        "embedding_fwd": lambda: lh.embedding_fwd(z(4, dt=i64), z(30, 160)),
        "rms_norm_fwd": lambda: lh.rms_norm_fwd(x),
        "layer_norm_fwd": lambda: lh.layer_norm_fwd(x),
        "head4_quantize": lambda: lh.head4_quantize(z(30, 128)),
        "rms_norm_add_fwd": lambda: lh.rms_norm_add_fwd(x, x),
        "rms_norm_add_bwd": lambda: lh.rms_norm_add_bwd(x, x, x, z(4), z(160)),
        "quantize8": lambda: lh.quantize8(x),
        "gemm8": lambda: lh.gemm8(q, w),
        "beam_select": lambda: lh.beam_select(x, z(4), 2, ws=z(4096, dt=torch.uint8)),
        "beam_reorder": lambda: lh.beam_reorder_([x], z(2, 2, dt=i64)),
        "ce_logits_bwd": lambda: lh.ce_logits_bwd(x, z(4, dt=i64), z(4), z(1, dt=i64), z(1))}


def test_on_the_current_device_only(lib):
    lh, reached, current = lib
    for device, here in ((0, 0), (1, 1), (1, 0), (0, 1)):
        current[0] = here
        for name, call in _calls(lh, f"cuda:{device}").items():
            del reached[:]
            if device == here:
                call()
                assert reached == [name]
            else:
                with pytest.raises(ValueError, match="current device"):
                    call()
                assert not reached, name
