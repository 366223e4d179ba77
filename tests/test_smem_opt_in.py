"""CPU check of the opt-in to large dynamic shared memory, against a fake of the two runtime calls that it makes: it is
made on every device that a kernel is launched on, once, and again after a failure."""
import os
import re
import subprocess

from paged_kv_cache_25_gb300 import build

PROGRAM = r"""
#include "smem_opt_in.h"
#include <cstdio>

static int device = 0, sets[70] = {}, last = 0;
static cudaError_t answer = cudaSuccess;
extern "C" cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute a, int v)
{
    if (a == cudaFuncAttributeMaxDynamicSharedMemorySize && answer == cudaSuccess) { ++sets[device]; last = v; }
    return answer;
}

int main()
{
    static pa::SmemOptIn one, other;
    const int kernel = 0;
    int bad = 0;
    for (int round = 0; round < 3; ++round)
        for (device = 0; device < 64; device += 9) bad += one(&kernel, 100000 + device) != cudaSuccess;
    for (int d = 0; d < 64; ++d) bad += sets[d] != (d % 9 == 0 ? 1 : 0);
    bad += last != 100063;
    device = 9;
    bad += other(&kernel, 5) != cudaSuccess || sets[9] != 2;          // another kernel's object knows nothing yet
    device = 1;
    answer = cudaErrorInvalidValue;
    bad += one(&kernel, 7) != cudaErrorInvalidValue;                  // what failed is tried again
    answer = cudaSuccess;
    bad += one(&kernel, 7) != cudaSuccess || sets[1] != 1;
    device = 66;                                                      // more devices than it remembers
    for (int i = 0; i < 2; ++i) bad += one(&kernel, 8) != cudaSuccess;
    bad += sets[66] != 2;
    std::printf("%d\n", bad);
    return bad;
}
"""


def test_every_device_is_opted_in(tmp_path):
    src, exe = tmp_path / "opt_in.cpp", tmp_path / "opt_in"
    src.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-I", build.SRC, "-isystem", cuda, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_no_kernel_opts_in_another_way():
    for name in os.listdir(build.SRC):
        with open(os.path.join(build.SRC, name)) as f:
            uses = len(re.findall(r"cudaFuncSetAttribute", f.read()))
        assert uses == (1 if name == "smem_opt_in.h" else 0), name
