"""A kernel that may be launched before the grid in front of it has ended sees that grid's writes only after a
griddepcontrol.wait of its own.  So in the text of every kernel that waits, the wait depends on nothing and comes before
the first load, store or TMA copy of global memory that the text shows (read from the sources; no GPU)."""
import re

import pytest

from test_cluster_start import kernels

WAIT = re.compile(r"ptx::griddep_wait\(\)")
GLOBAL = re.compile(r"\b(tma_load_\w+|tma_store_\w+|load_slice|__ldg|__ldcg|atomicAdd|load_raw|load8_raw)\b\s*[(<]")
FOUND = [(n, b) for _, n, b in kernels() if WAIT.search(b)]


def test_kernels_are_found():
    assert {"moe_router_kernel", "moe_expert_kernel", "moe_combine_kernel", "dz_kernel", "dbias_kernel", "tile_cta",
            "linear_pair_kernel", "repitch_kernel", "dropout_add_vec_kernel"} <= {n for n, _ in FOUND}


@pytest.mark.parametrize("name,body", FOUND, ids=[n for n, _ in FOUND])
def test_the_wait_is_unconditional_and_first(name, body):
    waits = list(WAIT.finditer(body))
    assert len(waits) == 1
    before = body[:waits[0].start()].rstrip()
    assert before.endswith((";", "{", "}")), "a wait under a condition"
    assert not GLOBAL.search(before)
