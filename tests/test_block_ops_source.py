"""Rules of the operators' sources that no run on a GPU is sure to show broken."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "expert_slot_cache_lru_gb300", "csrc")


def code(name):
    """A source file without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


EARLY = sorted(f for f in os.listdir(CSRC) if re.search(r"\bpdl_wait\(\)", code(f)))


def test_the_files_with_early_launched_kernels():
    assert {"block_norm.cu", "fp4.cu", "route.cu", "tile_gemm.cuh"} <= set(EARLY)


@pytest.mark.parametrize("name", EARLY)
def test_early_launched_kernels_load_coherently(name):
    """A kernel that is resident while the one before it still writes may not read
    through the non-coherent path, nor let the compiler choose it."""
    assert not re.findall(r"__ldg\w*\(|ld\.global(?:\.\w+)*\.nc|__restrict__", code(name))


@pytest.mark.parametrize("name", EARLY)
def test_loops_over_rows_do_not_pass_the_type(name):
    """rows + gridDim passes 2^31 where rows nears it."""
    assert not re.findall(r"for \(int \w+ = blockIdx[^;]*;[^;]*;[^;)]*\+= gridDim", code(name))


@pytest.mark.parametrize("name", EARLY + ["fp4_linear.cu", "tc_host.cu"])
def test_sizes_come_from_the_device(name):
    """The number of SMs is asked for, not written down."""
    assert not re.findall(r"\b152\b", code(name))
