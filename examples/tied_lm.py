"""A small language model with a tied table, trained and decoded with this
package's operators: ``python examples/tied_lm.py [--steps N] [--vocab V] [--width D]``.

    e = embedding(ids, W, sqrt(D));  u = layer_norm(e);  h = layer_norm(e + u A);
    loss = flce(h, W, next ids)

Training writes its own backward: the head's gradient of the table (flce_bwd) and
the lookup's (embedding_bwd) are summed in one fp32 buffer.  Decoding reads the table
in 4 bits (head4_quantize, head4_logits), one captured graph per token, or, with several
beams to a sequence, in 8 (quantize8, gemm8, beam_select, beam_reorder_).  The tokens
follow a random permutation, so what there is to learn is the permutation.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lm_head_linear_fwd_gb300 as lh  # noqa: E402

BF = torch.bfloat16


class TiedLM:
    """fp32 parameters, bf16 copies to compute with."""

    def __init__(self, V, D, device, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.V, self.D, self.scale = V, D, math.sqrt(D)
        self.master = {
            "W": torch.randn(V, D, generator=g).mul_(D ** -0.5),
            "A": torch.randn(D, D, generator=g).mul_(D ** -0.5),
            "w1": torch.ones(D), "b1": torch.zeros(D), "w2": torch.ones(D), "b2": torch.zeros(D)}
        self.master = {k: v.to(device) for k, v in self.master.items()}
        self.p = {k: v.to(BF) for k, v in self.master.items()}
        self.grad_W = torch.empty(V, D, device=device)  # fp32, of both uses of the table
        self.m = {k: torch.zeros_like(v) for k, v in self.master.items()}
        self.v = {k: torch.zeros_like(v) for k, v in self.master.items()}
        self.t = 0
        self.status = lh.new_status(device)

    def hidden(self, ids):
        p = self.p
        e = lh.embedding_fwd(ids, p["W"], self.scale, status=self.status)
        n1 = lh.layer_norm_fwd(e, p["w1"], p["b1"])
        r = torch.addmm(e, n1.y, p["A"])
        return e, n1, r, lh.layer_norm_fwd(r, p["w2"], p["b2"])

    def loss_and_grads(self, ids, labels):
        p = self.p
        e, n1, r, n2 = self.hidden(ids)
        out = lh.flce_fwd(n2.y, p["W"], labels, reduction="mean", status=self.status)
        one = torch.ones(1, device=ids.device)
        back = lh.flce_bwd(n2.y, p["W"], labels, out.lse, out.n_valid, one, reduction="mean",
                           grad_W=self.grad_W, status=self.status)
        g2 = lh.layer_norm_bwd(r, back.grad_H, n2.mean, n2.rstd, p["w2"], want_grad_bias=True)
        g1 = lh.layer_norm_bwd(e, g2.grad_x @ p["A"].t(), n1.mean, n1.rstd, p["w1"],
                               want_grad_bias=True)
        lh.embedding_bwd(ids, g2.grad_x + g1.grad_x, self.V, self.scale, grad_W=self.grad_W,
                         accumulate_grad_W=True, status=self.status)
        return out.loss, {"W": self.grad_W, "A": (n1.y.t() @ g2.grad_x).float(),
                          "w1": g1.grad_weight, "b1": g1.grad_bias,
                          "w2": g2.grad_weight, "b2": g2.grad_bias}

    def step(self, ids, labels, lr):
        loss, grads = self.loss_and_grads(ids, labels)
        self.t += 1
        for k, g in grads.items():  # Adam
            self.m[k].lerp_(g, 0.1)
            self.v[k].lerp_(g * g, 0.02)
            m = self.m[k] / (1 - 0.9 ** self.t)
            v = self.v[k] / (1 - 0.98 ** self.t)
            self.master[k].sub_(lr * m / (v.sqrt() + 1e-8))
            self.p[k].copy_(self.master[k])
        return loss


class Decoder:
    """One token of each of M sequences per replay, from the table in 4 bits."""

    def __init__(self, model, M, group=64):
        self.head = lh.head4_quantize(model.p["W"], group, zero_point=True)
        device = model.p["W"].device
        self.ids = torch.zeros(M, dtype=torch.int64, device=device)
        self.logits = torch.empty(M, model.V, device=device)

        def token():
            h = model.hidden(self.ids)[-1].y
            lh.head4_logits(h, self.head, out=self.logits, status=model.status)
            self.ids.copy_(self.logits.argmax(1))

        side = torch.cuda.Stream(device)
        side.wait_stream(torch.cuda.current_stream(device))
        with torch.cuda.stream(side):
            token()  # warm-up: libraries allocate on their first call
        torch.cuda.current_stream(device).wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            token()

    def run(self, first, length):
        """[length, M]: the tokens that follow `first`."""
        self.ids.copy_(first)
        out = []
        for _ in range(length):
            self.graph.replay()
            out.append(self.ids.clone())
        return torch.stack(out)


class BeamDecoder:
    """B sequences of K beams each, from the table in 8 bits; the beams' histories are
    what moves with them."""

    def __init__(self, model, B, K, length):
        self.model, self.B, self.K = model, B, K
        device = model.p["W"].device
        self.head = lh.quantize8(model.p["W"], 128)
        self.history = torch.zeros(B * K, length, dtype=torch.int64, device=device)
        # the first step has one beam to go on from
        self.start = torch.full((B, K), float("-inf"), device=device)
        self.start[:, 0] = 0.0

    def run(self, first):
        """The best history of each sequence after `first` [B], and its score."""
        model, K = self.model, self.K
        ids, scores = first.repeat_interleave(K), self.start.flatten()
        for t in range(self.history.shape[1]):
            h = lh.quantize8(model.hidden(ids)[-1].y)
            best = lh.beam_select(lh.gemm8(h, self.head, status=model.status), scores, K)
            lh.beam_reorder_([self.history[:, :t]] if t else [], best.parents,
                             status=model.status)
            ids, scores = best.tokens.flatten(), best.scores.flatten()
            self.history[:, t] = ids
        return self.history.view(self.B, K, -1)[:, 0].clone(), best.scores[:, 0]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--vocab", type=int, default=1000)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--lr", type=float, default=3e-3)
    a = ap.parse_args(argv)
    device = torch.device("cuda")
    gen = torch.Generator().manual_seed(1)
    follows = torch.randperm(a.vocab, generator=gen).to(device)
    model = TiedLM(a.vocab, a.width, device)
    losses = []
    for i in range(a.steps):
        ids = torch.randint(a.vocab, (a.tokens,), generator=gen).to(device)
        losses.append(model.step(ids, follows[ids], a.lr))
        if i % 20 == 0 or i + 1 == a.steps:
            print(f"step {i:4d}  loss {losses[-1].item():.4f}")
    first = torch.arange(4, device=device)
    got = Decoder(model, 4).run(first, 16)
    want = []
    for _ in range(16):
        first = follows[first]
        want.append(first)
    right = (got == torch.stack(want)).float().mean().item()
    beams = BeamDecoder(model, 4, 3, 16).run(torch.arange(4, device=device))[0]
    lh.check_status(model.status)
    print(f"decoded from 4 bits: {100 * right:.0f}% of 64 tokens right")
    same = (beams.t() == torch.stack(want)).float().mean().item()
    print(f"with 3 beams from 8 bits: {100 * same:.0f}%")
    return [x.item() for x in losses], right


if __name__ == "__main__":
    main()
