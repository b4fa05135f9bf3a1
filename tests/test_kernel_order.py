"""Orders within kernels that no run can be relied on to show, read from the
source (no GPU needed)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "lm_head_linear_fwd_gb300", "csrc")


def kernels():
    """(name, body without comments) of every __global__ function."""
    out = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        src = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__ void\s+(?:__launch_bounds__\([^{;]*?\)\s+)?(\w+)\(", src):
            start = src.index("{", m.end())
            depth, end = 1, start + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(src[end], 0)
                end += 1
            out.append((m.group(1), src[start:end]))
    return out


KERNELS = kernels()
REMOTE = [k for k in KERNELS if "mapa_shared(" in k[1]]


def test_every_kernel_is_seen():
    names = {n for n, _ in KERNELS}
    assert {"embedding_sort_kernel", "ce_bwd_resident_kernel", "norm_bwd_kernel",
            "head4_many_kernel", "tc_gemm_pair_kernel"} <= names
    assert {"embedding_sort_kernel", "ce_bwd_resident_kernel"} <= {n for n, _ in REMOTE}


@pytest.mark.parametrize("name,body", REMOTE, ids=[n for n, _ in REMOTE])
def test_cluster_has_started_before_its_shared_memory_is_used(name, body):
    """Another CTA's shared memory may be accessed once that CTA has started, which a
    cluster barrier shows; the last such access comes before the last barrier, so that
    no CTA has ended."""
    uses = [m.start() for m in re.finditer(r"mapa_shared\(", body)]
    syncs = [m.start() for m in re.finditer(r"cluster_sync\(\)", body)]
    assert syncs and syncs[0] < uses[0], name
    assert syncs[-1] > uses[-1], name


def test_a_wait_that_gave_up_is_reported_after_the_last_one():
    """head4_many_kernel: the flag is read for the report behind a barrier of the block
    that all warps pass after their waits, and the tensor memory is freed after that."""
    body = dict(KERNELS)["head4_many_kernel"]
    reads = [m.start() for m in re.finditer(r"some_wait_failed\(failed\)", body)]
    assert len(reads) == 1 and not re.search(r"[^a-z]\*failed\b", body.replace("int* failed", ""))
    assert body.rindex("add_sums()") < reads[0]
    assert reads[0] < body.index("set_status(a.status, FLCE_ETIMEOUT)") < body.index("tmem_dealloc(")
    src = open(os.path.join(CSRC, "head4_many.cuh")).read()
    helper = src[src.index("bool some_wait_failed"):]
    assert helper.index("__syncthreads()") < helper.index("*failed != 0")
