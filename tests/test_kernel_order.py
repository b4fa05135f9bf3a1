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
