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


def test_kernels_release_behind_their_own_wait():
    """A kernel lets the one behind it begin only after its own wait, in one place, whatever its arguments: what a
    kernel may rely on before its wait is that all but the kernel before it are complete."""
    release = r"launch_dependents"
    (helper,) = [p for p in FILES if re.search(release, code(p))]
    body = re.search(r"void (\w+)\(\) \{\s*grid_wait\(\);\s*asm volatile\(\"griddepcontrol\.launch_dependents;\" ::: \"memory\"\);\s*\}",
                     code(helper))
    assert body and len(re.findall(release, code(helper))) == 1
    name = body.group(1)
    launched = 0
    for p in FILES:
        text = code(p)
        for part in re.split(r"__global__ void", text)[1:]:
            kernel = part[:part.index("\n}\n") if "\n}\n" in part else len(part)]
            if not re.search(r"tc::grid_wait", kernel):
                assert re.search(r"debug_wait_kernel|cluster_probe_kernel", kernel), kernel[:200]
                continue
            launched += 1
            # one call, at the kernel's own level or in its loading warp's branch, under no condition of its own, and no CTA
            # leaves before it
            lines = [l for l in kernel.split("\n") if f"tc::{name}()" in l]
            assert len(lines) == 1 and lines[0].strip() == f"tc::{name}();", (p, lines)
            assert "return;" not in kernel[:kernel.index(lines[0])], p
    assert launched == 8
