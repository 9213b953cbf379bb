"""Rules of the routed experts' kernels that their sources show."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_shared_expert_gb300", "csrc")


@pytest.mark.parametrize("name", ["route.cu", "fp8.cu", "fp8_cols.cu", "fp8_pair.cu", "fp8.cuh", "fp8_tc.cuh"])
def test_nothing_is_read_by_the_read_only_path(name):
    # Its contract is memory that nobody writes while the grid lives, and these grids begin while the kernel before
    # them still writes their inputs.
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"__ldg\b|ld\.global\.nc", text)
