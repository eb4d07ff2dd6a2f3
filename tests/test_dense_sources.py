"""What the dense operators' kernels must hold to because they are launched while the kernel before them
still runs (programmatic dependent launches): read from their sources, no GPU."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rvq_compressed_expert_gb300", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "dense*.cu*")) + glob.glob(os.path.join(CSRC, "mx4*.cu")) +
               [os.path.join(CSRC, "tc_dev.cuh")])


def code(path):
    """The source without its comments."""
    text = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_no_read_only_loads(path):
    """A kernel's lifetime includes the end of the one before it, which may write what this one reads behind its
    wait; read-only loads (ld.global.nc, __ldg, and what the compiler makes of const __restrict__) are for memory
    that nobody writes in that time."""
    found = re.findall(r"ld\.global[.\w:]*\.nc|__ldg\b|__restrict__|ldg_nc", code(path))
    assert not found, found
