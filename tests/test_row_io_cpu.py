"""What the row operators read of gamma, compiled for the host with the address sanitizer: the C values that it has, and
nothing beside them, at every remainder of C by 8, type and alignment."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "implicit_gemm_conv_amd", "csrc")
CLANG = "/opt/rocm/llvm/bin/clang++"

PROGRAM = r"""
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#define __device__
#define __forceinline__ inline
static inline float __builtin_amdgcn_exp2f(float x) { return exp2f(x); }
static inline float __builtin_amdgcn_rcpf(float x) { return 1.0f / x; }
#include "row_io.hpp"

int main() {
    long bad = 0;
    for (int kind = 0; kind < 3; ++kind)
        for (int C = 1; C <= 40; ++C)
            for (int odd = 0; odd < 8; ++odd) {  // gamma at a 16-byte multiple, and some values past it
                const int size = kind == igc::KIND_F32 ? 4 : 2;
                char* own = (char*)malloc((C + odd) * size);
                char* gamma = own + odd * size;
                for (int c = 0; c < C; ++c) {  // 1, 2, 3, ... in every type
                    const float v = (float)(c + 1);
                    uint32_t w;
                    memcpy(&w, &v, 4);
                    const uint16_t h = kind == igc::KIND_BF16 ? (uint16_t)(w >> 16) : __builtin_bit_cast(uint16_t, (_Float16)v);
                    size == 4 ? memcpy(gamma + 4 * c, &w, 4) : memcpy(gamma + 2 * c, &h, 2);
                }
                for (int c = 0; c < C + 8; c += 8) {
                    float g[8];
                    igc::load_gamma<true>(gamma, kind, c, C, g);
                    for (int i = 0; i < 8; ++i) bad += g[i] != (c + i < C ? (float)(c + i + 1) : 0.0f);
                    if (C >= 8) {
                        igc::load_gamma<false>(gamma, kind, c, C, g);
                        for (int i = 0; i < 8; ++i) bad += g[i] != (c + i < C ? (float)(c + i + 1) : 0.0f);
                    }
                    igc::load_gamma<true>(nullptr, kind, c, C, g);
                    for (int i = 0; i < 8; ++i) bad += g[i] != 1.0f;
                }
                free(own);
            }
    printf("%ld\n", bad);
    return 0;
}
"""


@pytest.mark.skipif(not os.path.exists(CLANG), reason="needs ROCm's clang")
def test_gamma_is_read_inside_its_values(tmp_path):
    src, exe, inc = tmp_path / "gamma.cpp", tmp_path / "gamma", tmp_path / "hip"
    inc.mkdir()
    (inc / "hip_runtime.h").write_text("")  # (what it would define is above)
    src.write_text(PROGRAM)
    subprocess.run([CLANG, "-O1", "-g", "-std=c++20", "-mf16c", "-Xarch_host", "-fsanitize=address", "-I", str(tmp_path), "-I",
                    CSRC, str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stderr[:2000]
    assert int(run.stdout) == 0
