"""Kernels launched programmatically are resident while the kernel before them still
writes their inputs, so none may read through the non-coherent path, which is for
memory that nobody writes during the kernel's life."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "allreduce_residual_rmsnorm_gb300", "csrc")
FILES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


def code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def reached(name, seen=None):
    """A source and the headers of the package that it includes, over all levels."""
    seen = set() if seen is None else seen
    if name not in seen and name in FILES:
        seen.add(name)
        for inc in re.findall(r'#\s*include\s+"([^"]+)"', code(name)):
            reached(inc, seen)
    return seen


@pytest.mark.parametrize("source", [f for f in FILES if f.endswith(".cu")])
def test_sources_with_a_grid_wait_hold_no_non_coherent_load(source):
    files = reached(source)
    if not any("pdl_wait()" in code(f).replace("void pdl_wait()", "") for f in files):
        return
    for f in files:
        assert not re.search(r"\.global\.nc\b|__ldg\s*\(", code(f)), f


def test_the_check_sees_the_kernels_that_wait():
    waiting = {f for f in FILES if "pdl_wait()" in code(f).replace("void pdl_wait()", "")}
    assert {"block_quant.cu", "expert_combine.cu", "fused_rows.cuh", "matmul_wide.cu"} <= waiting
