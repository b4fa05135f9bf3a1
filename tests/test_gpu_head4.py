"""The 4-bit head: rounding, layout and logits against 64-bit forms
(bounds: tests/ops_ref.py)."""
import pytest
import torch

import ops_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lh():
    import lm_head_linear_fwd_gb300 as m
    return m


def _randn(shape, dtype, seed, std=1.0, pad=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    N, D = shape
    flat = torch.randn(N * (D + pad) + shift, generator=g).mul_(std).to(dtype).cuda()
    return flat[shift:].view(N, D + pad)[:, :D]


def _head(lh, V, D, group, zero, sdt, seed, extra=0):
    """Random bits in every place, those past column D too."""
    g = torch.Generator().manual_seed(seed)
    G = -(-D // group)
    wide = torch.randint(0, 256, (V, -(-D // 128) * 64 + extra), generator=g, dtype=torch.uint8)
    scales = (torch.rand(V, G, generator=g) * 0.02 + 0.001).to(sdt)
    zeros = torch.randint(0, 16, (V, G), generator=g, dtype=torch.uint8).cuda() if zero else None
    packed = wide.cuda()[:, :-(-D // 128) * 64]
    return lh.Head4(packed, scales.cuda(), zeros, D, group)


def _check(lh, x, head, bias, dtype, **kw):
    y = lh.head4_logits(x, head, bias, out_dtype=dtype, **kw)
    Wq = R.head4_weights(head.packed, head.scales, head.zeros, head.D, head.group)
    ref, bound = R.head4(x, Wq, bias, head.group, dtype)
    R.close(y, ref, bound, (tuple(x.shape), head.V, head.group))
    return y


@pytest.mark.parametrize("M,D,V", [(1, 1, 1), (1, 32, 5), (1, 128, 16), (2, 130, 17),
                                   (1, 768, 1003), (3, 257, 40), (8, 1000, 33), (9, 640, 100),
                                   (17, 384, 65), (32, 512, 300), (33, 96, 31), (70, 200, 50),
                                   (1, 4096, 130), (4, 5120, 20), (0, 64, 8)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype,sdt,out,zero", [(BF, BF, F32, False), (BF, F32, BF, True),
                                                (F32, F32, F32, True), (F32, BF, BF, False)])
def test_logits(lh, M, D, V, group, dtype, sdt, out, zero):
    pad, shift = (0, 0) if group == 64 else (3, 1)
    x = _randn((M, D), dtype, 1, 1.0, pad, shift)
    head = _head(lh, V, D, group, zero, sdt, 2, extra=16 if group == 32 else 0)
    bias = _randn((1, V), dtype, 3)[0] if group != 128 else None
    y = _check(lh, x, head, bias, out)
    assert torch.equal(lh.head4_logits(x, head, bias, out_dtype=out), y)
    if M:  # an output inside a wider buffer
        wide = torch.full((M, V + 3), 7.0, dtype=out, device="cuda")
        lh.head4_logits(x, head, bias, out=wide[:, 1:1 + V])
        assert torch.equal(wide[:, 1:1 + V], y)
        assert (wide[:, 0] == 7).all() and (wide[:, 1 + V:] == 7).all()


@pytest.mark.parametrize("M,group,dtype", [(1, 32, BF), (12, 64, BF), (20, 64, BF), (32, 32, BF),
                                           (7, 128, F32), (3, 64, F32)])
def test_logits_of_many_rows_and_columns(lh, M, group, dtype):
    """More tiles than a launch holds at once, more columns than stay on chip."""
    V, D = 90001, 2600
    x = _randn((M, D), dtype, 11)
    head = _head(lh, V, D, group, True, BF, 12)
    y = lh.head4_logits(x, head)
    for rows in (slice(0, 300), slice(38800, 39300), slice(77700, 78100), slice(89700, 90001)):
        part = lh.Head4(head.packed[rows], head.scales[rows], head.zeros[rows], D, group)
        Wq = R.head4_weights(part.packed, part.scales, part.zeros, D, group)
        ref, bound = R.head4(x, Wq, None, group, F32)
        R.close(y[:, rows], ref, bound, (M, group, rows))
    # every row, up to the order of the sums of rows that split a tile's columns
    again = torch.cat([lh.head4_logits(x, lh.Head4(head.packed[i:i + 45000],
                                                   head.scales[i:i + 45000],
                                                   head.zeros[i:i + 45000], D, group))
                       for i in range(0, V, 45000)], 1)
    scale = (x.float().abs().sum(1, keepdim=True) * 15 * 0.021)
    assert ((y - again).abs() <= scale * (D + 8) * 2.0 ** -24).all()


@pytest.mark.parametrize("M", [3, 12, 32])
def test_specials_stay_in_their_token(lh, M):
    head = _head(lh, 300, 600, 64, True, BF, 13)
    x = _randn((M, 600), BF, 14)
    want = lh.head4_logits(x, head)
    x[1, 5], x[2, 599] = float("inf"), float("nan")
    y = lh.head4_logits(x, head)
    keep = [m for m in range(M) if m not in (1, 2)]
    assert torch.equal(y[keep], want[keep])
    assert not y[1].isfinite().any() and y[2].isnan().all()


def test_one_hot_reads_every_weight(lh):
    """x = e_k gives column k of the weights exactly (bf16 scales, fp32 logits)."""
    D, V = 300, 70
    for zero, group in ((False, 128), (True, 32)):
        head = _head(lh, V, D, group, zero, BF, 5)
        Wq = R.head4_weights(head.packed, head.scales, head.zeros, D, group)
        y = lh.head4_logits(torch.eye(D, dtype=BF, device="cuda"), head)
        assert torch.equal(y.cpu().double(), Wq.t())


def test_fp32_tokens_keep_their_bits(lh):
    """fp32 x enters in parts that add up to it: full precision, extremes, specials."""
    D, V = 256, 40
    head = _head(lh, V, D, 64, True, F32, 6)
    x = _randn((6, D), F32, 7)
    x[1] *= 1e30
    x[2] *= 1e-30
    x[3] = 3e38 * x[3].sign()
    x[3, 1:] = 0
    _check(lh, x, head, None, F32)
    x = _randn((3, D), F32, 8)
    x[0, 5], x[1, 9] = float("inf"), float("nan")
    y = lh.head4_logits(x, head)
    assert not y[0].isfinite().any() and y[1].isnan().all() and y[2].isfinite().all()


@pytest.mark.parametrize("V,D,group,zero,dtype,sdt", [
    (5, 128, 128, False, F32, F32), (33, 200, 32, True, F32, F32), (40, 129, 64, False, BF, BF),
    (7, 1000, 128, True, BF, F32), (1, 1, 32, False, F32, BF), (64, 768, 64, True, BF, BF)])
def test_quantize(lh, V, D, group, zero, dtype, sdt):
    W = _randn((V, D), dtype, 9, 0.05, 5, 1)
    W[0, :min(D, group)] = 0  # a group of zeros
    if V > 2:
        W[2] = W[2].abs() + 0.01  # one sign only
    h = lh.head4_quantize(W, group, zero_point=zero, scale_dtype=sdt)
    G = -(-D // group)
    assert h.scales.shape == (V, G) and h.scales.dtype == sdt and h.packed.shape[0] == V
    # the same steps in fp32, element by element
    Wf = torch.zeros(V, G * group).copy_(torch.nn.functional.pad(W.float().cpu(),
                                                                 (0, G * group - D)))
    Wg = Wf.view(V, G, group)
    lo, hi = Wg.amin(2).clamp(max=0), Wg.amax(2).clamp(min=0)
    s = (hi - lo) / 15 if zero else torch.maximum(hi, -lo) / 7
    s = s.to(sdt).float()
    s[s == 0] = 1
    z = (-lo / s).round().clamp(0, 15) if zero else torch.full_like(s, 8)
    q = ((Wg / s[:, :, None]).round() + z[:, :, None]).clamp(0, 15).view(V, -1)[:, :D]
    assert torch.equal(h.scales.float().cpu(), s)
    if zero:
        assert torch.equal(h.zeros.cpu().float(), z)
    assert torch.equal(R.unpack4(h.packed, D).float(), q)
    # and through the product: within half a step of the scale of each weight
    y = lh.head4_logits(torch.eye(D, device="cuda"), h).cpu().t()
    step = s.repeat_interleave(group, 1)[:, :D]
    if sdt == F32 and not zero:
        assert ((y - W.float().cpu()).abs() <= step * 0.5 * (1 + 1e-6)).all()


@pytest.mark.parametrize("D", [1, 7, 65, 127, 129, 250])
def test_quantize_leaves_zeros_past_the_last_column(lh, D):
    W = _randn((50, D), BF, 22)
    for zero in (False, True):
        h = lh.head4_quantize(W, 32, zero_point=zero)
        every = R.unpack4(h.packed, h.packed.shape[1] * 2)
        assert (every[:, D:] == 0).all() and (every[:, :D] != 0).any()


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("dtype,group", [(F32, 32), (BF, 64), (F32, 128), (BF, 128)])
def test_quantize_halves_and_extremes(lh, dtype, group, zero):
    """Quotients that end in one half, scales near the ends of fp32, many rows: the
    nibbles of an exact division, rounded to even."""
    V, D = 9001, 640
    g = torch.Generator().manual_seed(21)
    W = torch.randint(-14, 15, (V, D), generator=g).float() / 2 + 0.0
    W[:, ::group] = 7.0 if not zero else 7.5   # the group's largest: scales of 1 (and 2^k)
    if zero:
        W[:, 1::group] = -7.5
        W.clamp_(-7.5, 7.5)
    W *= 2.0 ** torch.randint(-90, 91, (V, 1), generator=g).float()
    W[:40] *= 0
    W[40:80] = torch.randn(40, D, generator=g) * 2e-38
    W[80:120] = torch.randn(40, D, generator=g) * 1e37
    W[120:4000] = torch.randn(3880, D, generator=g)
    W = W.to(dtype)
    h = lh.head4_quantize(W.cuda(), group, zero_point=zero, scale_dtype=dtype)
    Wg = W.float().view(V, D // group, group)
    lo, hi = Wg.amin(2).clamp(max=0), Wg.amax(2).clamp(min=0)
    s = ((hi - lo) / 15 if zero else torch.maximum(hi, -lo) / 7).to(dtype).float()
    s[s == 0] = 1
    z = (-lo / s).round().clamp(0, 15) if zero else torch.full_like(s, 8)
    q = ((Wg / s[:, :, None]).round() + z[:, :, None]).clamp(0, 15).view(V, D)
    assert torch.equal(h.scales.float().cpu(), s)
    if zero:
        assert torch.equal(h.zeros.cpu().float(), z)
    assert torch.equal(R.unpack4(h.packed, D).float(), q)


def test_stream_graph_and_far_rows(lh):
    D, V = 512, 1000
    head = _head(lh, V, D, 128, False, BF, 1)
    x = _randn((4, D), BF, 2)
    want = lh.head4_logits(x, head)
    out = torch.empty_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lh.head4_logits(x, head, out=out)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lh.head4_logits(x, head, out=out)
    x.copy_(_randn((4, D), BF, 3))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, lh.head4_logits(x, head))
    # packed rows beyond 2^31 bytes
    V, ld = 70000, 32768
    wide = torch.zeros(V, ld, dtype=torch.uint8, device="cuda")
    wide[:, :64] = torch.randint(0, 256, (V, 64), dtype=torch.uint8, device="cuda")
    far = lh.Head4(wide[:, :64], torch.rand(V, 1, device="cuda"), None, 128, 128)
    x = _randn((2, 128), BF, 4)
    y = lh.head4_logits(x, far)
    near = lh.Head4(wide[:, :64].contiguous(), far.scales, None, 128, 128)
    assert torch.equal(y, lh.head4_logits(x, near))
    rows = torch.tensor([0, 65535, 65536, V - 1])
    Wq = R.head4_weights(wide[rows.cuda(), :64], far.scales[rows.cuda()], None, 128, 128)
    ref, bound = R.head4(x, Wq, None, 128, F32)
    R.close(y[:, rows.cuda()], ref, bound)
