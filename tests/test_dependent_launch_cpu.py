"""Kernels that may start before the kernel ahead of them has ended read what that kernel
writes.  A load that promises the compiler memory that never changes while the kernel runs
(__ldg, a const pointer with __restrict__), or one that it may move like arithmetic (__ldcs),
could be placed ahead of the wait."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_08_b200", "csrc")
SOURCES = [p for p in sorted(glob.glob(os.path.join(CSRC, "*.cu"))) if "launch_dependent(" in open(p).read()]


def test_the_sources_are_found():
    assert len(SOURCES) == 5


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_inputs_are_read_by_ordinary_loads(path):
    text = re.sub(r"//[^\n]*", "", open(path).read())
    assert not re.findall(r"\b(__ldg|__ldcs|__ldca|__ldcg|ldg_stream)\s*\(", text)
    kernels = re.findall(r"__global__[^{]*\{", text)
    assert len(kernels) == text.count("wait_for_inputs();")
    for k in kernels:
        assert not re.findall(r"\bconst\s+[\w:]+\s*\*\s*__restrict__\s*\w+", k), k
