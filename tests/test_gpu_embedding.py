"""Embedding lookup and the gradient of the table against 64-bit forms
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
    """Normal values [N, D] in rows of D + pad elements from element `shift`."""
    g = torch.Generator().manual_seed(seed)
    N, D = shape
    flat = torch.randn(N * (D + pad) + shift, generator=g).mul_(std).to(dtype).cuda()
    return flat[shift:].view(N, D + pad)[:, :D]


def _ids(N, V, seed, kind="uniform"):
    g = torch.Generator().manual_seed(seed)
    if kind == "same":
        return torch.full((N,), V // 2, dtype=torch.int64).cuda()
    if kind == "heavy":  # most tokens on a few ids, the rest spread
        a = torch.randint(0, V, (N,), generator=g)
        few = torch.randint(0, min(V, 3), (N,), generator=g)
        return torch.where(torch.rand(N, generator=g) < 0.8, few, a).cuda()
    return torch.randint(0, V, (N,), generator=g).cuda()


SHAPES = [(1, 1, 1), (1, 8, 5), (3, 7, 11), (17, 64, 100), (256, 129, 50), (1000, 768, 977),
          (33, 1600, 3), (5, 4097, 64)]


@pytest.mark.parametrize("N,D,V", SHAPES)
@pytest.mark.parametrize("dtype,pad,shift", [(BF, 0, 0), (BF, 3, 1), (F32, 0, 0), (F32, 5, 3),
                                             (BF, 8, 0), (BF, 0, 4)])
def test_lookup(lh, N, D, V, dtype, pad, shift):
    W = _randn((V, D), dtype, 1, 0.5, pad, shift)
    ids = _ids(N, V, 2)
    for scale in (1.0, 45.2548339959):
        st = lh.new_status("cuda")
        y = lh.embedding_fwd(ids, W, scale, status=st)
        lh.check_status(st)
        ref, bound = R.embedding(ids, W, scale, dtype)
        R.close(y, ref, bound, "y")
        if scale == 1.0:
            assert torch.equal(y, W[ids])
    # a caller's output inside a wider buffer; what lies around it stays
    wide = torch.full((N, D + 6), 7.0, dtype=dtype, device="cuda")
    lh.embedding_fwd(ids, W, 1.0, out=wide[:, 3:3 + D])
    assert torch.equal(wide[:, 3:3 + D], W[ids])
    assert (wide[:, :3] == 7).all() and (wide[:, 3 + D:] == 7).all()


def test_lookup_bad_ids_and_special_values(lh):
    V, D = 10, 40
    W = _randn((V, D), BF, 3)
    W[4, 5], W[4, 6], W[7] = float("inf"), float("nan"), 0.0
    ids = torch.tensor([4, -1, 7, 10, 2 ** 40, -2 ** 62, 9], device="cuda")
    st = lh.new_status("cuda")
    y = lh.embedding_fwd(ids, W, 2.0, status=st)
    with pytest.raises(lh.FlceError):
        lh.check_status(st)
    assert int(st.item()) == -5
    assert (y[[1, 3, 4, 5]] == 0).all()
    assert torch.equal(torch.nan_to_num(y[0], nan=1.5), torch.nan_to_num(W[4] * 2, nan=1.5))
    assert torch.equal(y[6], W[9] * 2)


@pytest.mark.parametrize("N,D,V", SHAPES + [(2000, 48, 37), (777, 520, 5000), (4100, 24, 300)])
@pytest.mark.parametrize("kind", ["uniform", "heavy", "same"])
@pytest.mark.parametrize("dtype,gdtype,pad,shift", [(BF, F32, 0, 0), (BF, BF, 0, 0),
                                                    (F32, F32, 3, 1), (BF, F32, 5, 1),
                                                    (F32, BF, 0, 0)])
def test_gradient(lh, N, D, V, kind, dtype, gdtype, pad, shift):
    dy = _randn((N, D), dtype, 5, 0.1, pad, shift)
    ids = _ids(N, V, 6, kind)
    for scale, padding in ((1.0, None), (27.7, V // 2)):
        st = lh.new_status("cuda")
        gW = torch.full((V, D), float("nan"), dtype=gdtype, device="cuda")
        lh.embedding_bwd(ids, dy, V, scale, padding, grad_W=gW, status=st)
        lh.check_status(st)
        ref, bound = R.embedding_grad(ids, dy, V, scale, padding, None, gdtype)
        R.close(gW, ref, bound, "grad_W")
    again = lh.embedding_bwd(ids, dy, V, scale, padding, grad_dtype=gdtype)
    assert torch.equal(again, gW)  # the same bits


@pytest.mark.parametrize("N,D,V,kind", [(1, 8, 4, "same"), (300, 130, 1000, "uniform"),
                                        (2000, 96, 50, "heavy"), (1500, 257, 9, "same"),
                                        (64, 768, 20000, "uniform")])
@pytest.mark.parametrize("dtype,pad", [(BF, 0), (F32, 0), (BF, 7)])
def test_gradient_added(lh, N, D, V, kind, dtype, pad):
    dy = _randn((N, D), dtype, 7, 0.1)
    ids = _ids(N, V, 8, kind)
    base = _randn((V, D), F32, 9, 1.0, pad)
    gW = torch.empty(V, D + pad, device="cuda")[:, :D].copy_(base)
    touched = torch.zeros(V, dtype=torch.bool, device="cuda")
    touched[ids] = True
    gW[~touched] = float("nan")  # rows no id names are not touched
    lh.embedding_bwd(ids, dy, V, 3.3, None, grad_W=gW, accumulate_grad_W=True)
    ref, bound = R.embedding_grad(ids, dy, V, 3.3, None, base, F32)
    t = touched.cpu()
    R.close(gW[touched], ref[t], bound[t], "grad_W")
    assert gW[~touched].isnan().all()


def test_gradient_empty_bad_and_masked(lh):
    V, D = 20, 24
    for acc in (False, True):
        gW = torch.ones(V, D, device="cuda")
        lh.embedding_bwd(torch.empty(0, dtype=torch.int64, device="cuda"),
                         torch.empty(0, D, device="cuda"), V, grad_W=gW, accumulate_grad_W=acc)
        assert (gW == (1 if acc else 0)).all()
    ids = torch.tensor([3, 5, 3, 99, -1, 5, 2 ** 33 + 3], device="cuda")
    dy = _randn((7, D), F32, 1)
    dy[3:5], dy[6] = float("nan"), float("inf")  # bad ids: not used
    dy[[1, 5]] = float("nan")                    # padding: not used
    st = lh.new_status("cuda")
    g = lh.embedding_bwd(ids, dy, V, 1.0, 5, status=st)
    assert int(st.item()) == -5
    ref, bound = R.embedding_grad(ids[[0, 2]], dy[[0, 2]], V, 1.0, None, None, F32)
    R.close(g, ref, bound)
    # every token masked
    st = lh.new_status("cuda")
    g = lh.embedding_bwd(torch.full((50,), 5, device="cuda"),
                         torch.full((50, D), float("nan"), device="cuda"), V, 1.0, 5, status=st)
    lh.check_status(st)
    assert (g == 0).all()
    # an inf and a NaN reach their own row only
    dy = _randn((40, D), BF, 2)
    ids = _ids(40, V, 3)
    ids[7], ids[9] = 11, 12
    dy[7, 3], dy[9, 4] = float("inf"), float("nan")
    g = lh.embedding_bwd(ids, dy, V)
    bad = (~g.isfinite()).nonzero().tolist()
    assert bad == [[11, 3], [12, 4]]


def test_long_token_lists(lh):
    """More tokens than one block's share of the sort, on few columns."""
    D = 4
    for N, V, kind in ((70001, 151936, "uniform"), (70001, 151936, "heavy"), (40000, 2, "uniform"),
                       (150000, 300, "same")):
        ids = _ids(N, V, 4, kind)
        dy = _randn((N, D), F32, 5)
        g = lh.embedding_bwd(ids, dy, V, 1.0)
        ref, bound = R.embedding_grad(ids, dy, V, 1.0, None, None, F32)
        R.close(g, ref, bound, (N, V, kind))


def test_far_rows(lh):
    """Offsets beyond 2^31 elements in the table and in its gradient."""
    V, ld, D = 70000, 32768, 64
    W = torch.zeros(V, ld, dtype=BF, device="cuda")[:, 100:100 + D]
    ids = torch.tensor([V - 1, 0, V - 2, 65536, 65535, V - 1], device="cuda")
    rows = _randn((6, D), BF, 1)
    W[ids] = rows
    y = lh.embedding_fwd(ids, W, 1.0)
    assert torch.equal(y, W[ids])
    dy = _randn((6, D), BF, 2)
    lh.embedding_bwd(ids, dy, V, 1.0, grad_W=W)
    ref, bound = R.embedding_grad(ids, dy, V, 1.0, None, None, BF)
    R.close(W, ref, bound)


def test_autograd_streams_and_graph(lh):
    V, D = 500, 96
    W = _randn((V, D), F32, 1).requires_grad_(True)
    ids = _ids(60, V, 2).view(3, 20)
    ids[0, 0] = 4
    y = lh.embedding(ids, W, scale=2.5, padding_idx=4)
    assert y.shape == (3, 20, D)
    v = _randn((60, D), F32, 3).view(3, 20, D)
    (y * v).sum().backward()
    ref, bound = R.embedding_grad(ids.view(-1), v.view(-1, D), V, 2.5, 4, None, F32)
    R.close(W.grad, ref, bound)
    # directional difference of the lookup (linear, so exact up to fp64 rounding)
    t = torch.randn(V, D, dtype=torch.float64, generator=torch.Generator().manual_seed(4))
    t[4] = 0  # the padding row's gradient is left out by definition
    diff = 0.0
    for s in (1, -1):
        Wd = R.d(W) + s * 1e-3 * t
        diff += s * (Wd[ids.cpu()] * 2.5 * R.d(v)).sum() / 2e-3
    assert abs((R.d(W.grad) * t).sum() - diff) <= 1e-5 * (ref.abs() * t.abs()).sum()
    # broadcast gradient (stride 0) and a bf16 table
    Wb = W.detach().to(BF).requires_grad_(True)
    lh.embedding(ids, Wb).sum().backward()
    ref, bound = R.embedding_grad(ids.view(-1), torch.ones(60, D), V, 1.0, None, None, BF)
    R.close(Wb.grad, ref, bound)
    # another stream than the tensors' own, then a graph
    dy = v.reshape(60, D)
    flat = ids.reshape(-1)
    want = lh.embedding_bwd(flat, dy, V, 1.5)
    s = torch.cuda.Stream()
    st = lh.new_status("cuda")
    ws = torch.empty(max(1, lh.embedding_bwd_workspace_bytes(60, D, V)), dtype=torch.uint8,
                     device="cuda")
    out = torch.empty(60, D, device="cuda")
    g = torch.empty(V, D, device="cuda")
    s.wait_stream(torch.cuda.current_stream())

    def step():
        lh.embedding_fwd(flat, W.detach(), 1.5, out=out, status=st)
        lh.embedding_bwd(flat, dy, V, 1.5, grad_W=g, ws=ws, status=st)

    with torch.cuda.stream(s):
        step()
    s.synchronize()
    assert torch.equal(g, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    flat.copy_(_ids(60, V, 9))
    for _ in range(2):
        g.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(g, lh.embedding_bwd(flat, dy, V, 1.5))
        assert torch.equal(out, lh.embedding_fwd(flat, W.detach(), 1.5))
    lh.check_status(st)
