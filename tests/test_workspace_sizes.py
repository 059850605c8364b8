"""A workspace for a number of tokens serves every smaller number: the sizes
never fall as tokens, sequences or experts rise (no GPU)."""
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


@pytest.mark.parametrize("E", [1, 64, 896, 1024])
@pytest.mark.parametrize("S", [1, 2, 61, 5000, 65535])
def test_balance_by_tokens(rf, E, S):
    sizes = list(range(1, 5000)) + list(range(5000, 70000, 7)) + [1 << 17, (1 << 20) - 1, 1 << 20]
    sizes += [(limit << s) + d for s in range(3, 11) for limit in (256, 1024) for d in (-1, 0, (1 << s) - 1, 1 << s)]
    last, before = 1, 0
    for C in sorted(c for c in set(sizes) if c <= rf.MOE_MAX_BATCH_TOKENS):
        n = rf.lib().moe_balance_workspace_size(C, E, S)
        assert n >= last, f"{C} tokens need {n} bytes, {before} {last}"
        last, before = n, C


@pytest.mark.parametrize("C", [1, 32, 33, 2056, 40000, 1 << 20])
def test_balance_by_sequences_and_experts(rf, C):
    size = rf.lib().moe_balance_workspace_size
    for E in (1, 64, 65, 1024):
        at = [size(C, E, S) for S in (1, 2, 3, 128, 65535)]
        assert at == sorted(at)
    at = [size(C, E, 9) for E in range(1, 1025)]
    assert at == sorted(at)
