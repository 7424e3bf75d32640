"""Kernels that reach into another CTA's shared memory do so only after a barrier of
the cluster: until then that CTA may not have started, and its memory is not there.
Checked on the sources, since a run that goes wrong depends on when CTAs start."""
import os
import re

import pytest

from ffn_gated_activation_b200 import _build

CSRC = os.path.join(_build.PKG_DIR, "csrc")
FILES = [os.path.join(CSRC, n) for n in sorted(os.listdir(CSRC)) if n.endswith((".cu", ".cuh"))]
BARRIER = re.compile(r"\b(cluster_sync|cluster_wait_started)\(\)")


def kernels(text):
    """(name, body) of each __global__ function."""
    for m in re.finditer(r"__global__", text):
        opening = re.compile(r"\b(situ_\w+)\([^;{]*\)\s*\{").search(text, m.end())
        if opening is None:
            continue
        depth, at = 1, opening.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield opening.group(1), re.sub(r"//[^\n]*", "", text[opening.end():at])


@pytest.mark.parametrize("path", FILES, ids=[os.path.basename(p) for p in FILES])
def test_a_cluster_barrier_comes_before_the_first_remote_access(path):
    for name, body in kernels(open(path).read()):
        first = body.find("peer_addr(")
        if first >= 0:
            barrier = BARRIER.search(body)
            assert barrier is not None and barrier.start() < first, name


def test_the_kernels_are_found():
    names = {n for p in FILES for n, body in kernels(open(p).read()) if "peer_addr(" in body}
    assert {"situ_nvfp4_small_kernel", "situ_nvfp4_gemm_kernel", "situ_fused_gemm_2sm_kernel"} <= names
