"""What the 8-bit integer products' sources have to say for themselves, since no run can show that it holds by chance."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_shared_expert_gb300", "csrc")


def test_shared_arrays_of_bytes_say_how_they_are_aligned():
    # they are read as words; an array's own type promises the alignment of one value only
    found = 0
    for path in glob.glob(os.path.join(CSRC, "int8*.cu")):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for line in re.findall(r"(?<!extern )__shared__[^;]*;", text):
            if re.search(r"\bu?int(8|16)_t\b", line):
                found += 1
                assert re.search(r"__align__\((4|8|16)\)|alignas\((4|8|16)\)", line), (os.path.basename(path), line)
    assert found
