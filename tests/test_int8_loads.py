"""Loads of the 8-bit kernels that start while the kernel in front of them still
runs.  What that kernel writes may change during theirs, so it must not be
read as read-only data: such a load may be served, or moved by the compiler, as
if nothing wrote there, past the wait for the kernel in front.  CPU only: the
sources are read."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "expanded_rank_matrix_b200", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "int8*.cu")) + glob.glob(os.path.join(CSRC, "int8*.cuh")))
# launched in the ordinary way: the kernel in front has ended when they start
PLAIN = ("pack_b_kernel", "pack_c_kernel")


def _code(path):
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    text = re.sub(r"//[^\n]*", "", text)
    for name in PLAIN:
        text = re.sub(r"__global__[^{;]*\b%s\(.*?\n\}\n" % name, "", text, flags=re.S)
    return text


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_read_only_loads(path):
    code = _code(path)
    for word in ("__ldg", "global.nc", "__restrict__", "__ldcs", "__ldlu"):
        assert word not in code, word


def test_kernels_left_out_are_launched_plainly():
    code = "".join(re.sub(r"//[^\n]*", "", open(p).read()) for p in SOURCES)
    for name in PLAIN:
        body = re.search(r"__global__[^{;]*\b%s\(.*?\n\}\n" % name, code, flags=re.S).group(0)
        assert "pdl_wait" not in body
        assert f"launch_chained({name}" not in code and f"{name}<<<" in code


def test_every_chained_kernel_waits():
    for path in SOURCES:
        for body in re.findall(r"__global__[^{;]*\(.*?\n\}\n", _code(path), flags=re.S):
            assert "pdl_wait()" in body, body[:200]
