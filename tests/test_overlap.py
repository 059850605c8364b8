"""Outputs that overlap inputs are refused, slices of one buffer between each
other's rows are not (no GPU: every call ends at a check, with a workspace or
without)."""
import ctypes
import os

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def rf():
    import routed_expert_fp4_amd as rf
    if not os.path.exists(rf.LIB_PATH):
        from routed_expert_fp4_amd import build
        build.build_library()
    rf.lib()
    return rf


def test_dense_product(rf):
    N, K, X = 64, 256, 0x40000000
    m = rf.moe_quant_matrix(N, K, 128, rf.MOE_DT_BF16, 0x100000, 128, 0x200000, 2, None, 0)

    def call(dtype, C, xp, y, yp):
        return rf.lib().moe_quant_linear(ctypes.byref(m), dtype, P(X), xp, C, P(y), yp, 0, None, 0, None)

    inv, free = rf.MOE_ERR_INVALID_ARG, rf.MOE_ERR_WORKSPACE      # no overlap: the next check, the workspace
    for dtype, b in ((rf.MOE_DT_F32, 4), (rf.MOE_DT_BF16, 2), (rf.MOE_DT_F16, 2)):
        for C in (1, 5, 40):
            end = X + ((C - 1) * 256 + 256) * b
            assert call(dtype, C, 256, X, 64) == inv
            assert call(dtype, C, 256, end, 64) == free           # right behind x
            assert call(dtype, C, 256, end - b, 64) == inv
            assert call(dtype, C, 256, X + 4 * b, 64) == inv
            assert call(dtype, C, 256, X - ((C - 1) * 64 + 64) * b, 64) == free
            assert call(dtype, C, 256, X - ((C - 1) * 64 + 63) * b, 64) == inv
            # x and y as columns of one buffer of 320 and more
            assert call(dtype, C, 320, X + 256 * b, 320) == free
            assert call(dtype, C, 400, X - 64 * b, 400) == free
            assert call(dtype, C, 320, X + 255 * b, 320) == inv
            assert call(dtype, C, 320, X - 63 * b, 320) == inv
            if C > 1:
                assert call(dtype, C, 300, X + 256 * b, 300) == inv   # row t of y over row t + 1 of x
                # pitches that differ: some rows of y meet x, or none does
                assert call(dtype, C, 400, X + 300 * b, 800) == free
                assert call(dtype, C, 400, X + 300 * b, 500) == inv


def test_router_gradients(rf):
    C, E, k, X = 8, 16, 2, 0x40000000
    far, n = P(0x10000000), C * E * 4

    def balance(d):
        return rf.lib().moe_balance_bwd(P(X), far, far, C, k, E, None, 1, None, 1, 0.1, far, P(d), 0, None)

    def route(d, idx=0x20000000, dw=0x30000000):
        return rf.lib().moe_route_bwd(P(X), P(idx), P(dw), C, k, E, None, P(d), 0, None)

    for d in (X, X + 4, X + n - 4, X - 4, X - n + 4):
        assert balance(d) == rf.MOE_ERR_INVALID_ARG
        assert route(d) == rf.MOE_ERR_INVALID_ARG
    for at in (0x50000000, 0x50000000 + n - 4, 0x50000000 - C * k * 4 + 4):
        assert route(0x50000000, dw=at) == rf.MOE_ERR_INVALID_ARG
        assert route(0x50000000, idx=at) == rf.MOE_ERR_INVALID_ARG
