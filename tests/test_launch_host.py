"""The largest shared memory that a kernel may ask for (csrc/sv_launch.cuh), set by host threads at the same time: the
order in which they come must not leave less than one of them asked for.  The runtime's calls are stand-ins that hold the
thread with the larger size between its call and its note of it."""
import os
import shutil
import subprocess

import pytest

from speculative_decoding_verify_spec_gb300 import _build

RUNTIME = r"""
#pragma once
enum cudaError_t { cudaSuccess = 0, cudaErrorInvalidValue = 1, cudaErrorInvalidDevice = 101 };
enum cudaFuncAttribute { cudaFuncAttributeMaxDynamicSharedMemorySize, cudaFuncAttributePreferredSharedMemoryCarveout };
cudaError_t cudaGetDevice(int *dev);
cudaError_t set_attribute(cudaFuncAttribute what, int value);
template <typename K>
cudaError_t cudaFuncSetAttribute(K *, cudaFuncAttribute what, int value) { return set_attribute(what, value); }
"""

PROGRAM = r"""
#include <chrono>
#include <cstdio>
#include <thread>

#include "sv_launch.cuh"

static std::atomic<int> attribute{0}, calls{0}, inside{0}, small_done{0};
static int refuse = 0;
static const int kSmall = 60000, kLarge = 90000;

cudaError_t cudaGetDevice(int *dev) { return *dev = 0, cudaSuccess; }
cudaError_t set_attribute(cudaFuncAttribute what, int value) {
    if (what != cudaFuncAttributeMaxDynamicSharedMemorySize) return cudaSuccess;
    if (refuse) return cudaErrorInvalidValue;
    ++calls;
    attribute = value;
    if (value == kLarge) {  // long enough for the other thread to come through, if nothing holds it
        inside = 1;
        for (int i = 0; i < 300 && !small_done; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
    }
    return cudaSuccess;
}
static void kernel() {}
static std::atomic<int> allowed[64];

int main() {
    refuse = 1;
    if (sv::allow_shared(kernel, 1000, allowed) == cudaSuccess) return 1;  // an error is passed on ..
    refuse = 0;
    if (sv::allow_shared(kernel, 1000, allowed) != cudaSuccess || attribute != 1000) return 2;  // .. and not remembered
    std::thread large([] { sv::allow_shared(kernel, kLarge, allowed); });
    std::thread small([] {
        while (!inside) std::this_thread::yield();
        sv::allow_shared(kernel, kSmall, allowed);
        small_done = 1;
    });
    large.join(), small.join();
    if (attribute != kLarge) return 3;
    const int before = calls;
    if (sv::allow_shared(kernel, kSmall, allowed) != cudaSuccess || sv::allow_shared(kernel, kLarge, allowed) != cudaSuccess) return 4;
    if (calls != before || attribute != kLarge) return 5;  // known: no further calls
    if (sv::allow_shared(kernel, kLarge + 16, allowed) != cudaSuccess || attribute != kLarge + 16) return 6;
    return 0;
}
"""


def test_the_largest_size_stays_whatever_the_threads_order(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "cuda_runtime.h").write_text(RUNTIME)
    (tmp_path / "main.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "main")
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", str(tmp_path), "-I", os.path.join(_build.PKG, "csrc"),
                    str(tmp_path / "main.cpp"), "-o", exe], check=True)
    assert subprocess.run([exe], timeout=60).returncode == 0
