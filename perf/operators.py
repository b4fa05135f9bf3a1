"""Timed cases of the operators around the loss head.

The loss head reads the hidden states H and the (tied) embedding table W.  The
operators here are what a program runs next to it:

* ``embedding``       the lookup H0 = scale * W[ids] at the model's input
* ``embedding_grad``  its gradient, dense [V, D], fresh or added to the head's
* ``layer_norm``      the norm before the head (forward), and ``layer_norm_grad``
* ``rms_norm``        the same without the mean (forward), and ``rms_norm_grad``
* ``head4``           the head when it answers: logits of a few tokens from
                      4-bit weights with a scale (and zero point) per group

A case is a plain dict; ``prepare`` makes its inputs on the GPU from a seed,
``run`` makes one pass (the plain torch form, or the library's calls where
``own`` is set), ``work`` counts what a pass cannot do without and ``exact``
is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


# --------------------------------------------------------------------- cases

def listed():
    return [
        # the token embeddings of a decoding batch of 16 requests, GPT-2 sized table
        {"name": "embedding_decode", "op": "embedding", "N": 16, "D": 768, "V": 50257,
         "dt": "bf16", "scale": 1.0, "pad": 0},
        # a long packed training batch, inputs scaled by sqrt(D)
        {"name": "embedding_long", "op": "embedding", "N": 65536, "D": 5120, "V": 151936,
         "dt": "bf16", "scale": 71.5541752799933, "pad": 0},
        # the table's own gradient in a small model, in the table's type, one id for padding
        {"name": "embedding_grad_small", "op": "embedding_grad", "N": 2048, "D": 768, "V": 32777,
         "dt": "bf16", "gdt": "bf16", "scale": 1.0, "pad": 0, "padding_idx": 0,
         "accumulate": False},
        # tied weights: the input side's gradient added to the fp32 gradient of the head
        {"name": "embedding_grad_tied", "op": "embedding_grad", "N": 8192, "D": 4096, "V": 128256,
         "dt": "bf16", "gdt": "f32", "scale": 64.0, "pad": 0, "padding_idx": -1,
         "accumulate": True},
        # one decoding step of four requests
        {"name": "layer_norm_decode", "op": "layer_norm", "N": 4, "D": 768, "dt": "bf16",
         "wdt": "f32", "bias": True, "pad": 0},
        # the norm before the head on a long packed batch
        {"name": "layer_norm_long", "op": "layer_norm", "N": 65536, "D": 5120, "dt": "bf16",
         "wdt": "bf16", "bias": True, "pad": 0},
        # an odd width in an odd stride: rows that start inside 16-byte blocks
        {"name": "layer_norm_grad_odd", "op": "layer_norm_grad", "N": 8191, "D": 1601,
         "dt": "bf16", "wdt": "f32", "bias": True, "pad": 6},
        # an fp32 model's norm
        {"name": "rms_norm_f32", "op": "rms_norm", "N": 8192, "D": 4096, "dt": "f32",
         "wdt": "f32", "bias": False, "pad": 0},
        # the norm's backward pass at the Llama-3 8B head's batch
        {"name": "rms_norm_grad", "op": "rms_norm_grad", "N": 8192, "D": 4096, "dt": "bf16",
         "wdt": "bf16", "bias": False, "pad": 0},
        # next-token logits of one request, Llama-3 8B's head
        {"name": "head4_single", "op": "head4", "M": 1, "D": 4096, "V": 128256, "dt": "bf16",
         "group": 128, "zero": False, "sdt": "bf16", "bias": False, "out": "f32"},
        # a few fp32 tokens, small groups with zero points, odd vocabulary and a bias
        {"name": "head4_few", "op": "head4", "M": 5, "D": 768, "V": 50257, "dt": "f32",
         "group": 32, "zero": True, "sdt": "f32", "bias": True, "out": "f32"},
        # a decoding batch of 32 requests on the largest head
        {"name": "head4_batch", "op": "head4", "M": 32, "D": 5120, "V": 151936, "dt": "bf16",
         "group": 64, "zero": False, "sdt": "bf16", "bias": False, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: a multiple of 64, a multiple of 8, or any."""
    d = _log(rng, lo, hi)
    kind = rng.random()
    if kind < 0.4:
        return max(64, d // 64 * 64)
    return max(8, d // 8 * 8) if kind < 0.7 else d


def draw(rng):
    c = _draw(rng)
    return c if 3072 not in c.values() else draw(rng)


def _draw(rng):
    op = rng.choice(["embedding", "embedding_grad", "layer_norm", "layer_norm_grad", "rms_norm",
                     "rms_norm_grad", "head4"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    if op == "head4":
        D = _width(rng, 64, 5120)
        return {"op": op, "M": _log(rng, 1, 32 if dt == "bf16" else 10), "D": D,
                "V": _log(rng, 256, 151936), "dt": dt, "group": rng.choice([32, 64, 128]),
                "zero": rng.random() < 0.5, "sdt": rng.choice(["bf16", "f32"]),
                "bias": rng.random() < 0.5, "out": rng.choice(["bf16", "f32"])}
    D = _width(rng, 64, 5120)
    N = _log(rng, 1, 65536 if dt == "bf16" else 32768)
    pad = rng.choice([0, 0, 8, rng.randrange(1, 16)])
    if op in ("embedding", "embedding_grad"):
        V = _log(rng, 256, 151936)
        c = {"op": op, "N": N, "D": D, "V": V, "dt": dt,
             "scale": rng.choice([1.0, math.sqrt(D)]), "pad": pad}
        if op == "embedding_grad":
            acc = rng.random() < 0.4
            c.update(gdt="f32" if acc else rng.choice(["f32", dt]),
                     padding_idx=rng.choice([-1, 0]), accumulate=acc)
        return c
    return {"op": op, "N": N, "D": D, "dt": dt, "wdt": rng.choice([dt, "f32"]),
            "bias": op.startswith("layer") and rng.random() < 0.8, "pad": pad}


# -------------------------------------------------------------------- inputs

_EPS = 1e-5


def _zipf(V):
    p = np.arange(1, V + 1, dtype=np.float64) ** -1.1
    return p / p.sum()


def _ids(g, N, V):
    cdf = torch.from_numpy(np.cumsum(_zipf(V))).cuda()
    u = torch.rand(N, dtype=torch.float64, device="cuda", generator=g)
    return torch.searchsorted(cdf, u, right=True).clamp_(max=V - 1)


def _rows(g, N, D, dt, pad, std=1.0, shift=0.0):
    """[N, D] normal values in rows of D + pad elements."""
    t = torch.empty(N, D + pad, dtype=_DT[dt], device="cuda")
    t.normal_(shift, std, generator=g)
    return t[:, :D]


def _groups(c):
    return -(-c["D"] // c["group"])


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": c}
    op, D = c["op"], c["D"]
    if op in ("embedding", "embedding_grad"):
        s["ids"] = _ids(g, c["N"], c["V"])
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if op == "embedding":
            s["W"] = _rows(g, c["V"], D, c["dt"], c["pad"], 0.02)
            s["y"] = torch.empty(c["N"], D, dtype=_DT[c["dt"]], device="cuda")
        else:
            s["dy"] = _rows(g, c["N"], D, c["dt"], c["pad"], 1e-3)
            if c["accumulate"]:  # the gradient that the head left there
                s["gW"] = _rows(g, c["V"], D, c["gdt"], 0, 1e-3)
            else:
                s["gW"] = torch.empty(c["V"], D, dtype=_DT[c["gdt"]], device="cuda")
    elif op == "head4":
        V, M, G = c["V"], c["M"], _groups(c)
        s["x"] = _rows(g, M, D, c["dt"], 0)
        s["packed"] = torch.randint(0, 256, (V, -(-D // 128) * 64), dtype=torch.uint8,
                                    device="cuda", generator=g)
        scale = torch.rand(V, G, device="cuda", generator=g) * 0.004 + 0.004
        s["scales"] = scale.to(_DT[c["sdt"]])
        s["zeros"] = torch.randint(0, 16, (V, G), dtype=torch.uint8, device="cuda",
                                   generator=g) if c["zero"] else None
        s["bias"] = _rows(g, 1, V, c["dt"], 0, 0.1)[0] if c["bias"] else None
        s["y"] = torch.empty(M, V, dtype=_DT[c["out"]], device="cuda")
    else:
        N = c["N"]
        s["x"] = _rows(g, N, D, c["dt"], c["pad"], 1.5, 0.25)
        s["w"] = (1 + 0.1 * torch.randn(D, device="cuda", generator=g)).to(_DT[c["wdt"]])
        s["b"] = (0.1 * torch.randn(D, device="cuda", generator=g)).to(_DT[c["wdt"]]) \
            if c["bias"] else None
        layer = op.startswith("layer")
        if op.endswith("grad"):
            # the statistics that the forward saved
            xd = s["x"].double()
            mean = xd.mean(1) if layer else torch.zeros(N, dtype=torch.float64, device="cuda")
            var = (xd - mean[:, None]).square_().mean(1)
            s["mean"] = mean.float() if layer else None
            s["rstd"] = (var + _EPS).rsqrt().float()
            s["dy"] = _rows(g, N, D, c["dt"], c["pad"], 1e-2)
            s["dx"] = torch.empty(N, D, dtype=_DT[c["dt"]], device="cuda")
            s["dw"] = torch.empty(D, dtype=torch.float32, device="cuda")
            s["db"] = torch.empty(D, dtype=torch.float32, device="cuda") if c["bias"] else None
        else:
            s["y"] = torch.empty(N, D, dtype=_DT[c["dt"]], device="cuda")
            s["mean"] = torch.empty(N, dtype=torch.float32, device="cuda") if layer else None
            s["rstd"] = torch.empty(N, dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------- plain form

def _plain_embedding(s, c):
    return (s["W"][s["ids"]].float() * c["scale"]).to(_DT[c["dt"]])


def _plain_embedding_grad(s, c):
    rows = s["dy"].float() * c["scale"]
    if c["padding_idx"] >= 0:
        rows = torch.where((s["ids"] != c["padding_idx"])[:, None], rows, 0.0)
    if c["accumulate"]:
        return s["gW"].index_add_(0, s["ids"], rows)
    total = torch.zeros(c["V"], c["D"], dtype=torch.float32, device="cuda")
    return total.index_add_(0, s["ids"], rows).to(_DT[c["gdt"]])


def _plain_norm(s, c):
    x = s["x"].float()
    mean = None
    if c["op"].startswith("layer"):
        mean = x.mean(1)
        x = x - mean[:, None]
    rstd = (x.square().mean(1) + _EPS).rsqrt()
    y = x * rstd[:, None] * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    return y.to(_DT[c["dt"]]), mean, rstd


def _plain_norm_grad(s, c):
    x, dy = s["x"].float(), s["dy"].float()
    if s["mean"] is not None:
        x = x - s["mean"][:, None]
    xhat = x * s["rstd"][:, None]
    gw = dy * s["w"].float()
    dx = gw - xhat * (gw * xhat).mean(1, keepdim=True)
    if s["mean"] is not None:
        dx = dx - gw.mean(1, keepdim=True)
    dx = (dx * s["rstd"][:, None]).to(_DT[c["dt"]])
    return dx, (dy * xhat).sum(0), dy.sum(0) if s["b"] is not None else None


def _plain_head4(s, c):
    V, D = c["V"], c["D"]
    p = s["packed"]
    # [V, blocks, t, w, bytes 0..3] -> nibbles n = 0..7 of each 32-bit word
    q = torch.stack((p & 15, p >> 4), -1).view(V, -1, 4, 4, 2, 4)
    # nibble n = 4 * hi + lo holds column 2 * lo + hi of the word's eight
    q = q.permute(0, 1, 3, 2, 5, 4).reshape(V, -1)[:, :D].float()
    group = c["group"]
    z = s["zeros"].float().repeat_interleave(group, 1)[:, :D] if c["zero"] else 8.0
    w = (q - z) * s["scales"].float().repeat_interleave(group, 1)[:, :D]
    y = s["x"].float() @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(_DT[c["out"]])


# ---------------------------------------------------------- the library's form

def _own(s, c):
    import lm_head_linear_fwd_gb300 as lh
    op = c["op"]
    if op == "embedding":
        return lh.embedding_fwd(s["ids"], s["W"], c["scale"], out=s["y"], status=s["status"])
    if op == "embedding_grad":
        return lh.embedding_bwd(s["ids"], s["dy"], c["V"], c["scale"],
                                c["padding_idx"] if c["padding_idx"] >= 0 else None,
                                grad_W=s["gW"], accumulate_grad_W=c["accumulate"],
                                status=s["status"])
    if op == "layer_norm":
        o = lh.layer_norm_fwd(s["x"], s["w"], s["b"], _EPS, y=s["y"], mean=s["mean"],
                              rstd=s["rstd"])
        return o.y, o.mean, o.rstd
    if op == "rms_norm":
        o = lh.rms_norm_fwd(s["x"], s["w"], _EPS, y=s["y"], rstd=s["rstd"])
        return o.y, None, o.rstd
    if op == "layer_norm_grad":
        o = lh.layer_norm_bwd(s["x"], s["dy"], s["mean"], s["rstd"], s["w"],
                              want_grad_bias=s["b"] is not None, grad_x=s["dx"],
                              grad_weight=s["dw"], grad_bias=s["db"])
        return o.grad_x, o.grad_weight, o.grad_bias
    if op == "rms_norm_grad":
        o = lh.rms_norm_bwd(s["x"], s["dy"], s["rstd"], s["w"], grad_x=s["dx"],
                            grad_weight=s["dw"])
        return o.grad_x, o.grad_weight, None
    head = lh.Head4(s["packed"], s["scales"], s["zeros"], c["D"], c["group"])
    return lh.head4_logits(s["x"], head, s["bias"], out=s["y"])


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    op = c["op"]
    if op == "embedding":
        return _plain_embedding(state, c)
    if op == "embedding_grad":
        return _plain_embedding_grad(state, c)
    if op == "head4":
        return _plain_head4(state, c)
    return _plain_norm_grad(state, c) if op.endswith("grad") else _plain_norm(state, c)


# ----------------------------------------------------------------------- work

def _distinct(N, V):
    """Expected number of distinct ids among N."""
    return float(-np.expm1(N * np.log1p(-_zipf(V))).sum())


def work(case):
    c, op, D = case, case["op"], case["D"]
    e = _SIZE[c["dt"]]
    if op == "embedding":
        return {"bytes": 8 * c["N"] + (_distinct(c["N"], c["V"]) + c["N"]) * D * e,
                "flops": c["N"] * D}
    if op == "embedding_grad":
        out = 8 * _distinct(c["N"], c["V"]) * D if c["accumulate"] \
            else c["V"] * D * _SIZE[c["gdt"]]
        return {"bytes": 8 * c["N"] + c["N"] * D * e + out, "flops": 2 * c["N"] * D}
    if op == "head4":
        V, M, G = c["V"], c["M"], _groups(c)
        return {"bytes": V * D / 2 + V * G * (_SIZE[c["sdt"]] + (1 if c["zero"] else 0))
                + M * D * e + M * V * _SIZE[c["out"]] + (V * e if c["bias"] else 0),
                "flops": 2 * M * V * D}
    N, vectors = c["N"], 1 + (1 if c["bias"] else 0)
    stats = (2 if op.startswith("layer") else 1) * 4 * N
    if op.endswith("grad"):
        return {"bytes": 3 * N * D * e + stats + D * _SIZE[c["wdt"]] + 4 * D * vectors,
                "flops": 12 * N * D}
    return {"bytes": 2 * N * D * e + stats + D * _SIZE[c["wdt"]] * vectors, "flops": 7 * N * D}


# ------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c, op, D = s["case"], case["op"], case["D"]
    if op == "embedding":
        return torch.index_select(s["W"], 0, s["ids"]).double().mul_(c["scale"])
    if op == "embedding_grad":
        # tokens sorted by id: each id's rows lie together, summed by a running sum per id
        ids, dy = s["ids"], s["dy"]
        if c["padding_idx"] >= 0:
            keep = ids != c["padding_idx"]
            ids, dy = ids[keep], dy[keep]
        total = s["gW"].double() if c["accumulate"] \
            else torch.zeros(c["V"], D, dtype=torch.float64, device="cuda")
        at, order = torch.sort(ids, stable=True)
        v, n = torch.unique_consecutive(at, return_counts=True)
        for a in range(0, D, 512):
            rows = dy[order, a:a + 512].double().mul_(c["scale"])
            total[v, a:a + 512] += torch.segment_reduce(rows, "sum", lengths=n, axis=0) \
                if len(v) else 0.0
        return total
    if op == "head4":
        V, group = c["V"], c["group"]
        col = np.arange(D)
        block, r = col // 128, col % 128
        w, t, j = r // 32, r % 32 // 8, r % 8
        nibble = j // 2 + 4 * (j % 2)
        at = torch.from_numpy(block * 64 + (4 * t + w) * 4 + nibble // 2).cuda()
        shift = torch.from_numpy((nibble % 2 * 4).astype(np.uint8)).cuda()
        of = torch.from_numpy(col // group).cuda()
        x = s["x"].double()
        y = torch.empty(c["M"], V, dtype=torch.float64, device="cuda")
        for a in range(0, V, 16384):
            q = ((s["packed"][a:a + 16384, at] >> shift) & 15).double()
            q -= s["zeros"][a:a + 16384, of].double() if c["zero"] else 8
            q *= s["scales"][a:a + 16384, of].double()
            y[:, a:a + 16384] = torch.einsum("md,vd->mv", x, q)
        return y + s["bias"].double() if s["bias"] is not None else y
    layer = op.startswith("layer")
    x, w = s["x"].double(), s["w"].double()
    if not op.endswith("grad"):
        mean = x.sum(1) / D if layer else None
        if layer:
            x -= mean[:, None]
        rstd = 1 / torch.sqrt((x * x).sum(1) / D + _EPS)
        y = torch.einsum("nd,n,d->nd", x, rstd, w)
        return y + s["b"].double() if s["b"] is not None else y, mean, rstd
    if layer:
        x -= s["mean"].double()[:, None]
    x *= s["rstd"].double()[:, None]
    dy = s["dy"].double()
    c1 = torch.einsum("nd,nd,d->n", dy, x, w) / D
    dw, db = torch.einsum("nd,nd->d", dy, x), dy.sum(0) if s["b"] is not None else None
    x *= -c1[:, None]
    x += dy * w
    if layer:
        x -= (dy @ w / D)[:, None]
    return x * s["rstd"].double()[:, None], dw, db
