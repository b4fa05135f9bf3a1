"""The example's beam decoder against a search written out on the host, step by step on
the same logits."""
import importlib.util
import os

import pytest
import torch

import eight_ref as E

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "tied_lm", os.path.join(ROOT, "examples", "tied_lm.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("vocab,width,K", [(300, 128, 3), (777, 200, 1), (500, 96, 8)])
def test_beams(example, vocab, width, K):
    lh, B, length = example.lh, 2, 5
    model = example.TiedLM(vocab, width, torch.device("cuda"), seed=5)
    first = torch.tensor([7, 11], device="cuda")
    history, score = example.BeamDecoder(model, B, K, length).run(first)
    head = lh.quantize8(model.p["W"], 128)
    ids, scores = first.repeat_interleave(K), torch.tensor(([0.0] + [float("-inf")] * (K - 1)) * B)
    kept = torch.zeros(B * K, 0, dtype=torch.int64)
    for _ in range(length):
        z = lh.gemm8(lh.quantize8(model.hidden(ids)[-1].y), head)
        best, token, parent = E.beam(z, scores, K, K, None, 0)
        rows = (parent + K * torch.arange(B)[:, None]).flatten()
        kept = torch.cat([kept[rows], token.flatten()[:, None]], 1)
        ids, scores = token.flatten().cuda(), best.flatten().float()
    assert torch.equal(history.cpu(), kept.view(B, K, length)[:, 0])
    # fp32 scores of five steps, each off by one fp32 rounding and the sum's
    assert (score.cpu().double() - best[:, 0]).abs().max() <= 5 * 2e-5
    lh.check_status(model.status)
