"""The operators' kernels start while the kernel ahead of them may still be
writing what they read, and wait on the device (griddepcontrol.wait).  Read-only
loads are for memory that nobody writes while a kernel runs, and may be moved
ahead of that wait: the sources hold none, and nothing that lets the compiler
make one."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp4_mixture_experts_gb300", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "mxfp4_*.cu*")) + [os.path.join(CSRC, "block_norm.cu")])


def code(path):
    text = open(path).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_the_operators_sources_are_there():
    assert len(FILES) == 7


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
@pytest.mark.parametrize("what", [r"__ldg\b", r"ld\.global(\.\w+)*\.nc\b", r"__restrict__"])
def test_no_read_only_loads(path, what):
    assert not re.search(what, code(path))
