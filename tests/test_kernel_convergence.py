"""Cluster barriers are aligned instructions: all lanes of a warp have to come to them
together.  Where one lane has worked alone before, the warp is joined first (read from
the source, no GPU needed)."""
import re

from test_kernel_order import KERNELS

BODIES = dict(KERNELS)


def _branches(body, *heads):
    """The parts of a kernel that begin with each of `heads`."""
    at = [body.index(h) for h in heads] + [body.rindex("tc_fence_before();")]
    assert at == sorted(at)
    return [body[a:b] for a, b in zip(at, at[1:])]


def test_pairs():
    """Each role's last statement joins its warps; then comes the last barrier."""
    body = BODIES["gemm8_pair_kernel"]
    copies, products, scales, sums = _branches(body, "if (warp == 0) {\n", "} else if (warp <= 2) {",
                                               "} else if (warp < 4) {", "setmaxnreg.inc")
    assert re.search(r"__syncwarp\(\);\s*$", copies)
    assert re.search(r"__syncwarp\(\);\s*}\s*$", products)  # the leader's; the other's do nothing
    assert re.search(r"__syncwarp\(\);\s*} else {\s*asm volatile\(\"$", scales)
    assert re.search(r"__syncwarp\(\);\s*}\s*$", sums)
    assert re.search(r"tc_fence_before\(\);\s*cluster_sync\(\);", body[body.rindex("__syncwarp()"):])


def test_clusters_that_share_a_tile():
    body = BODIES["gemm8_kernel"]
    # the warps that copy and issue come to both barriers joined, and so do the others
    assert re.search(r"if \(g\.split > 1 && warp < 2\) \{\s*__syncwarp\(\);\s*cluster_sync\(\);"
                     r"\s*cluster_sync\(\);", body)
    assert re.search(r"__syncwarp\(\);\s*cluster_sync\(\);\s*const uint32_t mine", body)
    assert body.count("cluster_sync();") == 4
