"""What the training operators' kernels must hold to because they are launched while the kernel before them still runs
(programmatic dependent launches): read from their sources, no GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rvq_compressed_expert_gb300", "csrc")
FILES = [os.path.join(CSRC, n) for n in ("norm.cu", "group_mm.cu", "ortho.cu", "tile_mma.cuh", "train.cuh")]


def code(path):
    """The source without its comments."""
    text = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_no_read_only_loads(path):
    """The kernel before may write what this one reads behind its wait: no loads by the read-only path."""
    found = re.findall(r"ld\.global[.\w:]*\.nc|__ldg\b|__restrict__|ldg_nc", code(path))
    assert not found, found


def test_kernels_wait_and_release_once():
    """Every kernel waits for the one before it and lets the next begin in one place, by all threads, before it reads or
    writes anything but its own shared and tensor memory, and leaves nowhere before."""
    kernels = 0
    for path in FILES:
        for part in re.split(r"__global__ void", code(path))[1:]:
            kernel = part[:part.index("\n}\n")]
            kernels += 1
            assert kernel.count("tc::grid_wait_release();") == 1, (path, kernel[:120])
            before = kernel[:kernel.index("tc::grid_wait_release();")]
            assert "return" not in before.split("{", 1)[1] and "tma_load" not in before and "P.x" not in before
            line = [l for l in kernel.split("\n") if "grid_wait_release" in l][0]
            assert line == "    tc::grid_wait_release();", (path, line)  # the kernel's own level: under no condition
    assert kernels == 12
    launches = sum(len(re.findall(r"<<<", code(p))) for p in FILES)
    assert launches == 0  # all by launches that may overlap


def test_waits_are_bounded():
    """No wait on a barrier but the bounded ones."""
    for path in FILES:
        text = code(path)
        for m in re.finditer(r"mbarrier\.try_wait", text):
            around = text[max(0, m.start() - 400):m.start()]
            assert "kWaitPolls" in around, path
        assert not re.search(r"while\s*\(\s*(?:!|true|1)", text), path


def test_waits_for_many_pieces_scale_with_them():
    """A tile's sum may be over 2^24 pieces of k, seconds of work: who waits from its start for its last piece, or for its
    sums, waits as much longer (wait_tile); the plain wait is for what one piece takes."""
    text = code(os.path.join(CSRC, "tile_mma.cuh"))
    waits = re.findall(r"(mbar_wait|wait_tile|wait_cluster)\((bar_\w+)([^;{]*)", text)
    long = {b for f, b, _ in waits if f == "wait_tile"}
    assert long == {"bar_accf", "bar_land"}
    for f, b, rest in waits:  # the loader's last waits, once it gave up, are for copies on their way
        assert f == "wait_tile" or b not in long or "land >> i" in rest, (f, b)
    (clearing,) = re.findall(r"pieces \+= T\.pieces;\s*if \(T\.left == 64\) continue;\s*if \(!all\(dense::wait_tile\(bar_land[^;]*, pieces\)\)\)", text)
