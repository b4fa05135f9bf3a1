"""The example that runs the operators together: it learns, its hand-written
backward agrees with the one autograd composes, and it decodes from 4 bits."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "tied_lm", os.path.join(ROOT, "examples", "tied_lm.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("vocab,width", [(1000, 256), (777, 200)])
def test_learns_and_decodes(example, vocab, width):
    losses, right = example.main(["--steps", "60", "--vocab", str(vocab), "--width", str(width)])
    assert losses[-1] < 0.05 * losses[0], losses[::10]
    assert right >= 0.9


def test_gradients_agree_with_autograd(example):
    lh = example.lh
    V, D, N = 500, 256, 700
    model = example.TiedLM(V, D, torch.device("cuda"), seed=3)
    g = torch.Generator().manual_seed(4)
    ids = torch.randint(V, (N,), generator=g).cuda()
    labels = torch.randint(V, (N,), generator=g).cuda()
    loss, grads = model.loss_and_grads(ids, labels)
    p = {k: v.clone().requires_grad_() for k, v in model.p.items()}

    def run(table, head):
        e = lh.embedding(ids, table, scale=model.scale)
        u = lh.layer_norm(e, p["w1"], p["b1"])
        h = lh.layer_norm(torch.addmm(e, u, p["A"]), p["w2"], p["b2"])
        return lh.flce(h, head, labels, reduction="mean")
    # the table's two uses as two leaves: each gradient is rounded to bf16 once
    table, head = (p["W"].detach().clone().requires_grad_() for _ in range(2))
    want = run(table, head)
    want.backward()
    assert abs(want.item() - loss.item()) <= 1e-5 * loss.item()
    half = 2.0 ** -8
    for got, refs in ((grads["W"], (table.grad, head.grad)), (grads["w1"], (p["w1"].grad,)),
                      (grads["b1"], (p["b1"].grad,)), (grads["w2"], (p["w2"].grad,)),
                      (grads["b2"], (p["b2"].grad,))):
        ref = sum(r.double() for r in refs)
        bound = half * sum(r.double().abs() for r in refs)
        # fp32 sums of up to N terms in another order
        slack = N * 2.0 ** -24 * sum(r.double().abs().max() for r in refs)
        assert ((got.double() - ref).abs() <= bound * 1.01 + slack).all()
    assert grads["W"].dtype == torch.float32
    lh.check_status(model.status)
