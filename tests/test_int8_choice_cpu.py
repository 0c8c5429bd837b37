"""The built-in choice of the 8-bit product says the K parts that run: as many partial outputs as the workspace holds, and
the same schedule when it is handed back as a tune."""
import os

import pytest

import implicit_gemm_conv_amd as igc

pytestmark = pytest.mark.skipif(not os.path.exists(igc.LIB_PATH), reason="libigc.so not built")


@pytest.mark.parametrize("M", [1, 8, 16, 20, 33, 64, 100, 256, 300, 777, 1024])
def test_choice_says_the_parts_that_run(M):
    splits = 0
    for N in (64, 256, 321, 1000, 2048, 3760, 4096, 8192):
        for K in (512, 1001, 2048, 4097, 6882, 8192, 12345, 16384, 32768, 65536, 131071):
            t = igc.igc_gemm_int8_default_tune(M, N, K)
            need = igc.igc_gemm_int8_workspace_bytes(M, N, K)
            parts = max(1, t.k_splits)
            splits += parts > 1
            partials = parts * M * ((N + 3) // 4 * 4) * 4 if parts > 1 else 0
            assert need == (partials + 255) // 256 * 256, (M, N, K, t.astuple(), t.k_splits, need)
            if t.bm:
                assert igc.igc_gemm_int8_workspace_bytes(M, N, K, t) == need
    assert splits > 0
