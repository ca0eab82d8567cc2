"""Host-side state shared by the entry points, compiled alone against a stand-in for the CUDA runtime (no GPU)."""
import os
import shutil
import subprocess

import pytest

from paged_kv_chunk_gb300 import build

# Two threads want different limits of one kernel.  The stand-in's call for the larger takes effect at once and
# returns late, so a caller that does not wait for it sets the smaller one in between.
PROGRAM = r"""
#include <chrono>
#include <cstdio>
#include <thread>

#include "host_common.h"

static int limit = 0;

extern "C" cudaError_t cudaGetDevice(int* dev)
{
    *dev = 3;
    return cudaSuccess;
}

extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int value)
{
    limit = value;
    if (value == 2000) std::this_thread::sleep_for(std::chrono::milliseconds(400));
    return cudaSuccess;
}

static void kernel() {}
static int done[64];

int main()
{
    bool ok[2] = {false, false};
    std::thread wide([&] { ok[0] = oasr::ensure_smem(kernel, 2000, done); });
    std::this_thread::sleep_for(std::chrono::milliseconds(100));
    std::thread narrow([&] { ok[1] = oasr::ensure_smem(kernel, 1000, done); });
    wide.join();
    narrow.join();
    std::printf("%d %d %d %d\n", ok[0], ok[1], limit, done[3]);
    return 0;
}
"""


def test_a_shared_memory_limit_is_never_lowered(tmp_path):
    cxx = shutil.which("g++")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    if not cxx or not os.path.exists(os.path.join(include, "cuda_runtime.h")):
        pytest.skip("needs a host compiler and the CUDA headers")
    src = tmp_path / "limit.cpp"
    src.write_text(PROGRAM)
    exe = str(tmp_path / "limit")
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", str(src), "-o", exe, "-I", include, "-I", build.INCLUDE,
                    "-I", build.CSRC], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True, timeout=60).stdout.split()
    assert out == ["1", "1", "2000", "2000"]
