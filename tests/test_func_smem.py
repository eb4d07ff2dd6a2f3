"""The size a kernel's dynamic shared memory is allowed (csrc/func_smem.h) under two host threads, against
fakes of the two CUDA calls: whatever the order, the attribute ends at least as large as every size that
was granted, and as the cache believes.  Compiled for the host; no GPU."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rvq_compressed_expert_gb300", "csrc")
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")

PROGRAM = r"""
#include "func_smem.h"
#include <chrono>
#include <cstdio>
#include <thread>

// The driver's side: one attribute.  The larger request takes effect at once and is slow to return; the smaller
// one is made meanwhile, unless something holds it back.
static std::atomic<int> attribute{0}, calls{0};
static std::atomic<bool> large_set{false};
extern "C" cudaError_t cudaGetDevice(int *d) { *d = 0; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int bytes) {
    ++calls;
    attribute = bytes;
    if (bytes == 200000) {
        large_set = true;
        std::this_thread::sleep_for(std::chrono::milliseconds(300));
    }
    return cudaSuccess;
}
int main() {
    static wm::SmemAttr a;
    int bad = 0;
    std::thread large([&] {
        wm::ensure_smem(a, &a, 200000);
        if (attribute < 200000) { std::puts("the larger size was granted, then lowered"); ++bad; }
    });
    std::thread small([&] {
        while (!large_set) std::this_thread::yield();
        wm::ensure_smem(a, &a, 100000);
    });
    large.join();
    small.join();
    wm::ensure_smem(a, &a, 200000);  // a later call of the larger size
    if (attribute < 200000) { std::puts("the cache believes in a size that is not set"); ++bad; }
    if (a.bytes[0] != attribute) { std::puts("cache and attribute differ"); ++bad; }
    const int before = calls;
    wm::ensure_smem(a, &a, 150000);
    if (calls != before) { std::puts("a granted size was asked for again"); ++bad; }
    return bad;
}
"""


def test_two_threads_raise_one_kernels_shared_memory(tmp_path):
    if not os.path.exists(os.path.join(CUDA, "include", "cuda_runtime_api.h")):
        pytest.skip("no CUDA headers")
    src, exe = tmp_path / "smem.cpp", tmp_path / "smem"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, "-I", os.path.join(CUDA, "include"), str(src),
                    "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
