"""The table's gradient for long token lists (above 128 tokens per SM the tokens are
sorted by one cluster), against 64-bit sums (bounds: tests/ops_ref.py)."""
import pytest
import torch

import ops_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lh():
    import lm_head_linear_fwd_gb300 as m
    return m


def _sorted_by_the_cluster(N):
    return N > 128 * torch.cuda.get_device_properties(0).multi_processor_count


def _ids(N, V, seed, kind):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, V, (N,), generator=g)
    if kind == "heavy":
        few = torch.randint(0, min(V, 3), (N,), generator=g)
        ids = torch.where(torch.rand(N, generator=g) < 0.8, few, ids)
    if kind == "bad":  # some out of range, on either side
        at = torch.randperm(N, generator=g)[:N // 50]
        ids[at] = torch.where(at % 2 == 0, -1 - at, V + at * 2 ** 20)
    return ids.cuda()


def _rows(N, D, dtype, seed, pad=0, std=0.1):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(N, D + pad, generator=g).mul_(std).to(dtype).cuda()[:, :D]


@pytest.mark.parametrize("N,D,V", [(20001, 24, 977), (40000, 9, 151936), (66000, 40, 5)])
@pytest.mark.parametrize("kind", ["uniform", "heavy", "bad"])
@pytest.mark.parametrize("dtype,gdtype,pad", [(BF, F32, 0), (BF, BF, 3), (F32, F32, 0),
                                              (F32, BF, 1)])
def test_fresh(lh, N, D, V, kind, dtype, gdtype, pad):
    assert _sorted_by_the_cluster(N)
    ids, dy = _ids(N, V, 1, kind), _rows(N, D, dtype, 2, pad)
    for padding in (None, V // 2):
        st = lh.new_status("cuda")
        gW = torch.full((V, D), float("nan"), dtype=gdtype, device="cuda")
        lh.embedding_bwd(ids, dy, V, 2.5, padding, grad_W=gW, status=st)
        assert int(st.item()) == (-5 if kind == "bad" else 0)
        ref, bound = R.embedding_grad(ids, dy, V, 2.5, padding, None, gdtype)
        R.close(gW, ref, bound, (kind, padding))
        again = lh.embedding_bwd(ids, dy, V, 2.5, padding, grad_dtype=gdtype)
        assert torch.equal(again, gW)  # the same bits


@pytest.mark.parametrize("N,D,V,kind", [(20001, 24, 977, "uniform"), (40000, 9, 151936, "heavy"),
                                        (20001, 130, 6, "heavy"), (40000, 8, 3000, "bad")])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_added(lh, N, D, V, kind, dtype):
    assert _sorted_by_the_cluster(N)
    ids, dy = _ids(N, V, 3, kind), _rows(N, D, dtype, 4)
    base = _rows(V, D, F32, 5, std=1.0)
    for padding in (None, 1):
        touched = torch.zeros(V, dtype=torch.bool, device="cuda")
        touched[ids[(ids >= 0) & (ids < V)]] = True
        if padding is not None:
            touched[padding] = False
        gW = base.clone()
        gW[~touched] = float("nan")  # rows that get nothing are not touched
        lh.embedding_bwd(ids, dy, V, 3.3, padding, grad_W=gW, accumulate_grad_W=True)
        ref, bound = R.embedding_grad(ids, dy, V, 3.3, padding, base, F32)
        t = touched.cpu()
        R.close(gW[touched], ref[t], bound[t], (kind, padding))
        assert gW[~touched].isnan().all()
        again = base.clone()
        lh.embedding_bwd(ids, dy, V, 3.3, padding, grad_W=again, accumulate_grad_W=True)
        assert torch.equal(again[touched], gW[touched])


def test_in_a_graph_and_on_another_stream(lh):
    N, D, V = 20001, 16, 700
    assert _sorted_by_the_cluster(N)
    ids, dy = _ids(N, V, 6, "uniform"), _rows(N, D, BF, 7)
    ws = torch.empty(lh.embedding_bwd_workspace_bytes(N, D, V), dtype=torch.uint8, device="cuda")
    st = lh.new_status("cuda")
    g, add = torch.empty(V, D, device="cuda"), torch.zeros(V, D, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        lh.embedding_bwd(ids, dy, V, 1.5, 3, grad_W=g, ws=ws, status=st)
        lh.embedding_bwd(ids, dy, V, 1.5, 3, grad_W=add, accumulate_grad_W=True, ws=ws, status=st)

    with torch.cuda.stream(side):
        step()
    side.synchronize()
    want = lh.embedding_bwd(ids, dy, V, 1.5, 3)
    assert torch.equal(g, want) and torch.equal(add, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    ids.copy_(_ids(N, V, 8, "heavy"))
    want = lh.embedding_bwd(ids, dy, V, 1.5, 3)
    for _ in range(3):
        g.fill_(float("nan"))
        add.zero_()
        ws.fill_(255)  # nothing is kept in the workspace between calls
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(g, want) and torch.equal(add, want)
    lh.check_status(st)


@pytest.mark.parametrize("N", [300, 20001])
def test_more_rows_than_a_block_marks_at_once(lh, N):
    """Each block fills more rows than its bitmap holds (65536), for both ways to order
    the tokens."""
    V = 11_000_003
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert V > 65536 * sms
    ids, dy = _ids(N, V, 9, "uniform"), _rows(N, 1, F32, 10)
    ids[:4] = torch.tensor([0, V - 1, 65535, 65536], device="cuda")
    gW = torch.full((V, 1), float("nan"), device="cuda")
    lh.embedding_bwd(ids, dy, V, 1.0, grad_W=gW)
    ref, bound = R.embedding_grad(ids, dy, V, 1.0, None, None, F32)
    R.close(gW, ref, bound)


def test_places_lie_within_the_list(lh, monkeypatch):
    """The checked build looks at every place that a token is put at: none leaves the
    list, and the bits are those of the ordinary build, for both ways to order tokens."""
    from lm_head_linear_fwd_gb300 import _abi, build
    ordinary, checked = _abi.load(), _abi.open_library(build.build(checked=True))
    for N, kind in ((300, "uniform"), (5000, "heavy"), (20001, "bad"), (40000, "heavy")):
        V, D = 1500, 8
        ids, dy = _ids(N, V, 11, kind), _rows(N, D, BF, 12)
        got = []
        for lib in (ordinary, checked):
            monkeypatch.setattr(_abi, "_lib", lib)
            st = lh.new_status("cuda")
            got.append(lh.embedding_bwd(ids, dy, V, 1.0, 3, status=st))
            assert int(st.item()) == (-5 if kind == "bad" else 0)
        assert torch.equal(*got)
