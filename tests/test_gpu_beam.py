"""Beam search against the definition in 64 bits (eight_ref.beam): tokens and parents
exactly, scores to fp32.  Random logits are apart by far more than the sum's rounding."""
import pytest
import torch

import eight_ref as E

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NINF, NAN, INF = float("-inf"), float("nan"), float("inf")


@pytest.fixture(scope="module")
def lh():
    import lm_head_linear_fwd_gb300 as m
    return m


def _logits(R, V, dtype, seed, pad=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    flat = torch.randn(R * (V + pad) + shift, generator=g).mul_(3).to(dtype).cuda()
    return flat[shift:].view(R, V + pad)[:, :V]


def _scores(R, seed):
    return torch.rand(R, generator=torch.Generator().manual_seed(seed)).mul_(-5).cuda()


def _check(o, want, exact=True):
    scores, tokens, parents = want
    assert torch.equal(o.parents.cpu(), parents)
    assert torch.equal(o.tokens.cpu(), tokens)
    got = o.scores.cpu().double()
    fine = scores.isfinite()
    assert torch.equal(got[~fine], scores[~fine])
    # lse: terms of 2^-22 relative, a chain of some hundred fp32 additions; one rounding
    assert ((got - scores).abs()[fine] <= 1e-5 + 2.0 ** -23 * scores.abs()[fine]).all()


@pytest.mark.parametrize("B,K,V,num", [(1, 1, 1, 1), (1, 1, 5, 5), (2, 3, 7, 4), (1, 4, 50257, 4),
                                       (3, 5, 8192, 10), (2, 4, 8193, 64), (5, 64, 300, 64),
                                       (2, 2, 40, 64), (1, 7, 16384, 1), (70, 2, 1000, 4),
                                       (2, 8, 128256, 16), (1, 2, 1 << 20, 33)])
@pytest.mark.parametrize("dtype,pad,shift", [(BF, 0, 0), (F32, 0, 0), (BF, 3, 1), (F32, 2, 3)])
def test_select(lh, B, K, V, num, dtype, pad, shift):
    z, s = _logits(B * K, V, dtype, 1, pad, shift), _scores(B * K, 2)
    o = lh.beam_select(z, s, K, num)
    _check(o, E.beam(z, s, K, num, None, 0))
    done = torch.rand(B * K, generator=torch.Generator().manual_seed(3)) < 0.3
    o = lh.beam_select(z, s, K, num, finished=done.cuda(), pad_id=V // 2)
    _check(o, E.beam(z, s, K, num, done, V // 2))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_ties_and_masks(lh, dtype):
    """Equal logits, few allowed tokens, beams that do not count, the first step's
    scores, ascending and descending rows."""
    K, V = 4, 20000
    z, s = _logits(2 * K, V, dtype, 1), _scores(2 * K, 2)
    z[0] = 1.0                        # every token the same
    z[1] = z[1].round()               # many ties
    z[2] = NINF
    z[2, [19999, 8191, 8192]] = 0.5   # three tokens allowed, equal
    z[4] = torch.arange(V) / 256.0
    z[5] = -torch.arange(V) / 256.0
    z[6, ::2] = 0.0
    z[6, 1::2] = -0.0                 # equal zeros
    s[:K] = s[0]
    for num in (1, 4, 40, 64):
        _check(lh.beam_select(z, s, K, num), E.beam(z, s, K, num, None, 0))
    first = torch.tensor([0.0, NINF, NINF, NINF] * 2, device="cuda")
    _check(lh.beam_select(z, first, K), E.beam(z, first, K, K, None, 0))
    # nothing of a beam: a NaN, an infinity, nothing allowed, no score; all of these
    z[3, 7], z[5, 9] = NAN, INF
    z[6], s[7] = NINF, NAN
    o = lh.beam_select(z, s, K, 50)
    _check(o, E.beam(z, s, K, 50, None, 0))
    z[:] = NINF
    done = torch.zeros(2 * K, dtype=torch.uint8, device="cuda")
    done[2] = done[5] = 1
    for num in (2, 50):
        _check(lh.beam_select(z, s, K, num, finished=done, pad_id=11),
               E.beam(z, s, K, num, done.cpu(), 11))
        _check(lh.beam_select(z, s, K, num), E.beam(z, s, K, num, None, 0))


@pytest.mark.parametrize("R,V,dtype,shift", [(320, 70001, F32, 1), (600, 70000, BF, 0),
                                             (1280, 131072, BF, 0)])
def test_many_long_rows(lh, R, V, dtype, shift):
    """Enough rows for several tiles to a block: rows that rise, fall and stay, whose
    candidates overflow the first tile's bound, masked parts, ties."""
    K = 4
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.empty(R * V + shift, dtype=dtype, device="cuda")[shift:].view(R, V)
    z.normal_(0.0, 3.0, generator=g)
    z[0] = torch.arange(V, device="cuda") / 4096.0
    z[1] = -torch.arange(V, device="cuda") / 4096.0
    z[5] = 0.25
    z[9, :40000] = NINF
    z[10] = NINF
    z[10, V - 1] = 1.0
    z[17] = z[17].round()
    z[18, 20000:60000] += 30.0
    z[R - 1] = torch.arange(V, device="cuda") // 8192
    s = _scores(R, 2)
    for num in (1, 4, 16, 40):
        o = lh.beam_select(z, s, K, num)
        for b in (0, 1, 2, 4, 33, R // K - 1):
            rows = slice(b * K, b * K + K)
            part = lh.BeamOut(o.scores[b:b + 1], o.tokens[b:b + 1], o.parents[b:b + 1])
            _check(part, E.beam(z[rows], s[rows], K, num, None, 0))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("num", [5, 64])
def test_masked_long_rows(lh, dtype, num):
    """Several tiles to a block over a vocabulary that is masked in part: tiles without a
    logit before, between and behind others, fewer logits than are asked for, equal ones
    around a tile's end."""
    R, V, K = 320, 70000, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.empty(R, V, dtype=dtype, device="cuda").normal_(0.0, 3.0, generator=g)
    z[0:4, :V // 2] = NINF
    z[4:8, V // 2:] = NINF
    z[8:12, :8192 + 17] = NINF
    z[12:16, 100:V - 100] = torch.finfo(dtype).min
    z[16:20] = NINF
    z[16:20, 8191:8195] = 2.0
    z[20:24] = 0.0
    z[24:28, 8192:] = z[24:28, :8192].max()
    s = _scores(R, 4)
    o = lh.beam_select(z, s, K, num)
    for b in range(8):
        rows = slice(b * K, b * K + K)
        part = lh.BeamOut(o.scores[b:b + 1], o.tokens[b:b + 1], o.parents[b:b + 1])
        _check(part, E.beam(z[rows], s[rows], K, num, None, 0))


def test_buffers_and_graph(lh):
    """Caller-owned outputs and workspace; captured with the reordering and replayed."""
    B, K, V = 3, 4, 3000
    z, s = _logits(B * K, V, F32, 1), _scores(B * K, 2)
    ws = torch.empty(lh.beam_select_workspace_bytes(B, K, V, K), dtype=torch.uint8, device="cuda")
    hist = torch.randint(0, V, (B * K, 9), device="cuda")
    cache = torch.randn(B * K, 2, 5, 8, device="cuda")
    out = lh.beam_select(z, s, K, ws=ws)
    lh.beam_reorder_([hist, cache], out.parents)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lh.beam_select(z, s, K, out=out, ws=ws)
        lh.beam_reorder_([hist, cache], out.parents)
    for seed in (4, 5):
        z.copy_(_logits(B * K, V, F32, seed))
        before = hist.clone(), cache.clone()
        graph.replay()
        _check(out, E.beam(z, s, K, K, None, 0))
        rows = (out.parents + K * torch.arange(B, device="cuda")[:, None]).flatten()
        assert torch.equal(hist, before[0][rows]) and torch.equal(cache, before[1][rows])


def _rows(parents):
    B, K = parents.shape
    return (parents + K * torch.arange(B, device=parents.device)[:, None]).flatten()


@pytest.mark.parametrize("B,K", [(1, 1), (1, 4), (3, 5), (40, 2), (2, 64)])
def test_reorder(lh, B, K):
    """Types, slices and orders of dimensions; rows outside a slice stay as they are."""
    R = B * K
    g = torch.Generator().manual_seed(B * 100 + K)
    parents = torch.randint(0, K, (B, K), generator=g).cuda()
    whole = [torch.randint(0, 100, shape, generator=g).to(dt).cuda() for shape, dt in (
        ((R,), torch.int64), ((R, 7), torch.int64), ((R, 3), torch.uint8), ((R, 5), BF),
        ((R, 2, 40, 16), BF), ((R, 2, 40, 16), F32), ((3, R, 10, 8), BF), ((R, 2, 3, 40, 16), BF),
        ((R, 130, 64), torch.uint8), ((R, 0, 4), BF), ((R, 1001), torch.bool))]
    views = [whole[0], whole[1][:, 1:6], whole[2], whole[3][:, 1:4], whole[4][:, :, :33],
             whole[5][:, :, 3:7, :].transpose(1, 2)[:, :, :, :], whole[6].transpose(0, 1)[:, :, :7],
             whole[7][:, 0, :, :10], whole[7][:, 1, :, 2:9], whole[8], whole[9], whole[10][:, 1:]]
    want = [w.clone() for w in whole]
    of = [0, 1, 2, 3, 4, 5, 6, 7, 7, 8, 9, 10]
    cut = [lambda w: w, lambda w: w[:, 1:6], lambda w: w, lambda w: w[:, 1:4],
           lambda w: w[:, :, :33], lambda w: w[:, :, 3:7, :].transpose(1, 2),
           lambda w: w.transpose(0, 1)[:, :, :7], lambda w: w[:, 0, :, :10],
           lambda w: w[:, 1, :, 2:9], lambda w: w, lambda w: w, lambda w: w[:, 1:]]
    rows = _rows(parents)
    for i, c in zip(of, cut):
        v = c(want[i])
        v.copy_(v[rows].clone())
    st = lh.new_status("cuda")
    lh.beam_reorder_(views, parents, status=st)
    for w, e in zip(whole, want):
        assert torch.equal(w, e), w.shape
    lh.check_status(st)


def test_reorder_many_and_far(lh):
    """More states than a launch takes; rows past 4 GB."""
    parents = torch.tensor([[1, 0, 0, 2]], device="cuda")
    states = [torch.randn(4, 3 + i % 5, device="cuda") for i in range(150)]
    want = [t[_rows(parents)] for t in states]
    lh.beam_reorder_(states, parents)
    assert all(torch.equal(a, b) for a, b in zip(states, want))
    big = torch.empty(4, 3 * 2 ** 29 + 16, dtype=torch.uint8, device="cuda")
    for k in range(4):
        big[k] = k + 1
        big[k, -1] = 10 + k
    lh.beam_reorder_([big], parents)
    for k, p in enumerate(parents[0].tolist()):
        assert (big[k, :-1] == p + 1).all() and big[k, -1] == 10 + p


def test_reorder_bad_parent(lh):
    """A parent that is no beam leaves its row and is reported."""
    t = torch.arange(8, device="cuda")
    st = lh.new_status("cuda")
    lh.beam_reorder_([t], torch.tensor([[1, 4, -1, 0], [3, 3, 3, 3]], device="cuda"), status=st)
    assert t.tolist() == [1, 1, 2, 0, 7, 7, 7, 7]
    with pytest.raises(lh.FlceError):
        lh.check_status(st)


def test_decoding_chain(lh):
    """As a program uses them: residual norm to 8 bits, the head's product, selection,
    reordering; each step's result from the one before it."""
    B, K, D, V = 2, 3, 256, 1000
    g = torch.Generator().manual_seed(1)
    table = torch.randn(V, D, generator=g).mul_(0.2).to(BF).cuda()
    head = lh.quantize8(table, 128)
    w = torch.ones(D, dtype=BF, device="cuda")
    stream = torch.randn(B * K, D, generator=g).to(BF).cuda()
    tokens = torch.zeros(B * K, 6, dtype=torch.int64, device="cuda")
    scores = torch.tensor([0.0, NINF, NINF] * B, device="cuda")
    done = torch.zeros(B * K, dtype=torch.bool, device="cuda")
    st = lh.new_status("cuda")
    for t in range(6):
        x = lh.embedding_fwd(tokens[:, t - 1].contiguous(), table, status=st) if t else stream * 0.5
        o = lh.rms_norm_add_fwd(x, stream, w, want_y=False, want_quant=True, summed=stream)
        logits = lh.gemm8(o.quant, head, status=st)
        want = E.value(o.quant) @ E.value(head).t()
        assert (logits.cpu().double() - want).abs().max() <= 1e-4 * want.abs().max()
        best = lh.beam_select(logits, scores, K, finished=done, pad_id=0)
        _check(best, E.beam(logits, scores, K, K, done.cpu(), 0))
        kept = stream.clone(), tokens.clone()
        lh.beam_reorder_([stream, tokens], best.parents, status=st)
        rows = _rows(best.parents)
        assert torch.equal(stream, kept[0][rows]) and torch.equal(tokens, kept[1][rows])
        tokens[:, t] = best.tokens.flatten()
        scores = best.scores.flatten()
        done = done[rows] | (best.tokens.flatten() % 7 == 0)
    lh.check_status(st)
