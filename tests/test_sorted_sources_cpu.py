"""Rules of the sorted rows' and the 8-bit integer products' kernels that their sources show."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_shared_expert_gb300", "csrc")


@pytest.mark.parametrize("name", ["sorted.cu", "int8.cu", "int8.cuh", "int8_tc.cuh", "int8_few.cu", "int8_cols.cu", "int8_pair.cu"])
def test_nothing_is_read_by_the_read_only_path(name):
    # its contract is memory that nobody writes while the grid lives, and these grids begin while the kernel before them
    # still writes their inputs
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"__ldg\b|ld\.global\.nc", text)


@pytest.mark.parametrize("name", ["sorted.cu", "int8.cu", "int8_few.cu", "int8_cols.cu", "int8_pair.cu"])
def test_every_kernel_waits_for_the_one_before_it(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    kernels = re.split(r"__global__ void", text)[1:]
    assert kernels and all("pdl_wait()" in k for k in kernels)
