"""The once-per-device set-up on the CPU: csrc/api.cpp against a stand-in for the HIP runtime that counts which kernels are
touched. A family of kernels is set up by its own first call, once, and no other family with it."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_delta_memory_amd", "csrc")

STAND_IN = r"""
#include <hip/hip_runtime_api.h>
#include <cstdio>
#include "sdm_launch.hpp"
static char kernels[4][3];   // Phase 1, read side, slot selection, recurrence
static int touched[4], device;
static int list(int f, const void** fns, int cap) {
    int n = 0;
    for (; n < 3 && n < cap; ++n) fns[n] = &kernels[f][n];
    return n;
}
namespace sdm {
int p1_lds_kernels(const void** fns, int cap) { return list(0, fns, cap); }
int read_lds_kernels(const void** fns, int cap) { return list(1, fns, cap); }
int slot_lds_kernels(const void** fns, int cap) { return list(2, fns, cap); }
int glr_lds_kernels(const void** fns, int cap) { return list(3, fns, cap); }
}
hipError_t hipGetDevice(int* d) { *d = device; return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) { *v = 163840; return hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipFuncGetAttributes(hipFuncAttributes* a, const void* f) {
    a->sharedSizeBytes = 0;
    for (int i = 0; i < 4; ++i) touched[i] += f >= kernels[i] && f < kernels[i] + 3;
    return hipSuccess;
}
hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int) { return hipSuccess; }
int main() {
    int lds = 0;
    auto say = [&]() { std::printf("%d%d%d%d ", touched[0], touched[1], touched[2], touched[3]); };
    for (int twice = 0; twice < 2; ++twice) { sdm::device_setup(&lds); say(); }
    for (int twice = 0; twice < 2; ++twice) { sdm::device_setup(nullptr, sdm::KernelFamily::slots); say(); }
    for (int twice = 0; twice < 2; ++twice) { sdm::device_setup(nullptr, sdm::KernelFamily::recurrence); say(); }
    device = 1;
    sdm::device_setup(nullptr, sdm::KernelFamily::recurrence);
    say();
    std::printf("%d\n", lds);
}
"""


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h"),
                    reason="g++ or the HIP headers are missing")
def test_each_family_is_set_up_by_its_own_first_call(tmp_path):
    src, exe = tmp_path / "stand_in.cpp", tmp_path / "stand_in"
    src.write_text(STAND_IN)
    # Everything else that api.cpp calls stays undefined: nothing here reaches it.
    subprocess.run(["g++", "-std=c++17", "-w", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", "/opt/rocm/include",
                    str(src), os.path.join(CSRC, "api.cpp"), "-Wl,--unresolved-symbols=ignore-all", "-pthread", "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert out == ["3300", "3300", "3330", "3330", "3333", "3333", "3336", "163840"]
