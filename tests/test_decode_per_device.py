"""What the decoding operators' launchers keep is kept for each device: on the host, with a stand-in for the current device."""
import os
import shutil
import subprocess

import pytest

import implicit_gemm_convolution_gb300._build as build

PROGRAM = r"""
#include "decode.h"
#include <cstdio>
static int device = 0;
extern "C" cudaError_t cudaGetDevice(int *d) { *d = device; return device < -1 ? cudaErrorNoDevice : cudaSuccess; }
int main() {
    static om::PerDevice kept;
    if (!kept.here() || kept.here()->load() != 0) return 1;
    kept.here()->store(7);
    if (kept.here()->load() != 7) return 2;
    device = 1;                               // another device: nothing is known of it
    if (!kept.here() || kept.here()->load() != 0) return 3;
    kept.here()->store(9);
    device = 0;
    if (kept.here()->load() != 7) return 4;
    device = 63;
    if (!kept.here() || kept.here()->load() != 0) return 5;
    for (int d : {64, 1000, -1, -2}) {        // behind the last place, or no device: asked for each time
        device = d;
        if (kept.here()) return 6;
    }
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_values_are_kept_for_each_device(tmp_path):
    src, exe = tmp_path / "kept.cpp", tmp_path / "kept"
    src.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, "-I", cuda, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0
