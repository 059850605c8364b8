"""A workspace for a number of tokens serves every smaller number: the sizes
never fall as tokens rise (no GPU)."""
import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def rf():
    import routed_expert_fp4_amd as rf
    if not os.path.exists(rf.LIB_PATH):
        from routed_expert_fp4_amd import build
        build.build_library()
    rf.lib()
    return rf


@pytest.mark.parametrize("N,K,G", [(7168, 3584, 32), (3584, 7168, 128), (1001, 4099, 64), (64, 256, 128),
                                   (65536, 7168, 128), (300, 10001, 64), (1, 1, 32), (40, 131072, 256),
                                   (4096, 3136, 64), (1 << 22, 40, 32)])
def test_dense_product(rf, N, K, G):
    pitch = (-(-K // 2) + 15) // 16 * 16
    m = rf.moe_quant_matrix(N, K, G, rf.MOE_DT_BF16, 0x100000, pitch, 0x200000, -(-K // G), None, 0)
    for dtype in (rf.MOE_DT_F32, rf.MOE_DT_BF16, rf.MOE_DT_F16):
        last = 256
        for C in range(1, rf.MOE_MAX_TOKENS + 1):
            n = rf.lib().moe_quant_workspace_size(ctypes.byref(m), dtype, C)
            assert n >= last, f"{C} tokens need {n} bytes, {C - 1} {last} (type {dtype})"
            last = n
