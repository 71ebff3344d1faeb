"""The operators' kernels start while the launch before them still runs, and
some of their inputs are also their outputs, so none of their loads may be
marked read-only: such a load is free to move ahead of the wait for that launch
and past a store to the same place, and no run on a GPU shows that it did not."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparsity_gemm_b200", "csrc")


@pytest.mark.parametrize("name", ["norm.cu", "route.cu", "lora.cu", "vec.cuh"])
def test_no_load_is_marked_read_only(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"__ldg|ld\.global\.nc|__restrict__|__ldcs|__ldlu", text)
