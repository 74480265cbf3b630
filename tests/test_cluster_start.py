"""A CTA may touch another CTA's shared memory only once that CTA is known to have started, which a cluster barrier
shows and being scheduled together does not.  So in the text of every kernel the first remote access comes after a
cluster barrier (read from the sources; no GPU)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mbarrier_gemm_pipelines_gb300", "csrc")
REMOTE = re.compile(r"\b(mapa_shared|ld_shared_cluster\w*|st_shared_cluster\w*|mbar_arrive_cluster)\s*\(")
BARRIER = re.compile(r"\b(cluster_sync_all|cluster_wait)\s*\(")


def kernels():
    """(file, name, body) of every __global__ function with a body, and of every device function that is a kernel's
    whole body (their names end in _cta)."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
        for m in re.finditer(r"__global__|__device__ __forceinline__ void (?=\w+_cta\()", text):
            name = re.compile(r"(\w+_(?:kernel|cta))\s*\(").search(text, m.end())
            start = text.index("{", name.end())
            depth, at = 0, start
            while True:
                depth += {"{": 1, "}": -1}.get(text[at], 0)
                at += 1
                if depth == 0:
                    break
            yield os.path.basename(path), name.group(1), text[start:at]


FOUND = [(f, n, b) for f, n, b in kernels() if REMOTE.search(b)]


def test_kernels_are_found():
    names = {n for _, n, _ in FOUND}
    assert {"moe_router_kernel", "dz_kernel", "tile_cta", "linear_pair_kernel"} <= names


@pytest.mark.parametrize("file,name,body", FOUND, ids=[n for _, n, _ in FOUND])
def test_barrier_before_the_first_remote_access(file, name, body):
    barrier = BARRIER.search(body)
    assert barrier is not None and barrier.start() < REMOTE.search(body).start()
