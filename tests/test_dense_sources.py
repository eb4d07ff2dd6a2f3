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


def test_loads_ahead_of_the_wait_see_what_is_complete():
    """Weights that a kernel asks for before its own wait: copies stand behind the fence that makes complete kernels'
    writes visible to them, loads are answered by L2 (relaxed at the GPU's scope), not by an SM's cache."""
    copies = loads = 0
    for p in FILES:
        text = code(p)
        for part in re.split(r"__global__ void", text)[1:]:
            if "tc::grid_wait_release()" not in part:
                continue
            before = part[:part.index("tc::grid_wait_release()")]
            fetch = re.search(r"const auto fetch = \[&\]\(.*?\n    \};", before, flags=re.S)
            run = re.sub(r"const auto \w+ = \[&?\]\(.*?\n\s*\};", "", before, flags=re.S)  # not what is only defined there
            at = [m.start() for m in re.finditer(r"\b(?:load_\w+|tc::tma_load\w*)\(", run)]
            if at:
                copies += 1
                assert "tc::see_complete();" in run and run.index("tc::see_complete();") < min(at), p
            if re.search(r"\bfetch\(", run):
                loads += 1
                assert "load_stream(" in fetch.group(0), p
                bare = re.sub(r"load_stream8?\([^:]*", "", fetch.group(0))
                assert not re.search(r"\.(?:codes|scales)\b|\bwd\b", bare), (p, bare)
    assert (copies, loads) == (2, 2)
    text = code(os.path.join(CSRC, "dense_gemv.cu"))
    for name in ("load_stream", "load_stream8"):
        body = re.search(name + r"\(const \w+ \*p\) \{.*?\n\}", text, flags=re.S).group(0)
        assert "ld.relaxed.gpu.global" in body


def test_a_wait_for_a_tile_goes_by_the_clock():
    """Polls return early beside other waits of the CTA: a product over many pieces of k is waited for by time."""
    body = re.search(r"bool wait_tile\(.*?\n\}", code(os.path.join(CSRC, "dense_gemm.cuh")), flags=re.S).group(0)
    assert re.search(r"end = tc::clock_ns\(\) \+ \d+ull \+ 2000ull \* \(uint32_t\)pieces;", body)
    assert re.search(r"do \{\s*if \(tc::mbar_wait\([^;]*\)\) return true;\s*\} while \(tc::clock_ns\(\) < end\);\s*return false;", body)
