"""Workspaces of the forward pass alone: what serving has to hold beside its adapters
and gated blocks.  Sizes and refusals on the CPU (every call ends at a check on the
host); calls in exactly that much memory on the GPU."""
import ctypes
import os

import pytest

P = ctypes.c_void_p
X, Y, FAR, WS, W = 0x40000000, 0x50000000, 0x10000000, 0x30000000, 0x70000000


@pytest.fixture(scope="module")
def rf():
    import routed_expert_fp4_amd as rf
    if not os.path.exists(rf.LIB_PATH):
        from routed_expert_fp4_amd import build
        build.build_library()
    rf.lib()
    return rf


def bank(rf, n, r, K, N, dtype=2):
    return rf.moe_adapter_bank(n, r, K, N, dtype, X, r * K, K, Y, N * r, r, FAR)


@pytest.mark.parametrize("C, n, r, K, N", [(1, 1024, 16, 7168, 3584), (64, 24, 32, 3584, 7168), (1024, 1024, 128, 7168, 7168),
                                           (4096, 1024, 64, 7168, 3584), (100000, 3, 8, 512, 512)])
def test_adapters_forward_takes_partial_sums_alone(rf, C, n, r, K, N):
    m = bank(rf, n, r, K, N)
    size = rf.lib().moe_adapter_fwd_workspace_size
    need = size(ctypes.byref(m), C)
    # ranges of 512 columns, or as many tokens as fill the card
    assert 0 < need <= min(C * -(-K // 512), max(C, 1 << 15)) * r * 4 + 256
    assert need == size(ctypes.byref(bank(rf, 1, r, K, N)), C)
    assert need < rf.lib().moe_adapter_workspace_size(ctypes.byref(m), C)
    sizes = [size(ctypes.byref(m), c) for c in list(range(1, 2200)) + [4096, 9000, 70000, 1 << 20]]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    for c in (0, -1, (1 << 20) + 1):
        assert size(ctypes.byref(m), c) == 0
    assert size(ctypes.byref(bank(rf, n, 129, K, N)), C) == 0


def test_adapter_refusals(rf):
    L, C, m = rf.lib(), 5, bank(rf, 3, 8, 64, 32)
    need = L.moe_adapter_fwd_workspace_size(ctypes.byref(m), C)
    pb, flag, space = L.moe_adapter_plan_size(C, 3), rf.MOE_WS_FORWARD, rf.MOE_ERR_WORKSPACE

    def fwd(ws, wb, y=0x21000000):
        return L.moe_adapter_fwd(ctypes.byref(m), P(W), pb, P(0x20000000), 64, C, None, 0, P(y), 32, None, 0.0, None, P(ws),
                                 wb, None)

    assert fwd(None, flag + need) == space and fwd(WS + 16, flag + need) == space
    assert fwd(WS, flag + need - 1) == space and fwd(WS, flag) == space
    assert fwd(WS, need) == space                          # not said to be of the forward pass
    for at in (X, Y, FAR, W, 0x20000000, 0x21000000, 0x21000000 - need + 256):
        assert fwd(at, flag + need) == rf.MOE_ERR_INVALID_ARG, hex(at)
    both = L.moe_adapter_workspace_size(ctypes.byref(m), C)
    assert L.moe_adapter_bwd(ctypes.byref(m), P(W), pb, P(0x20000000), 64, P(0x22000000), P(0x21000000), 32, C, None, 0,
                             P(0x23000000), 64, P(0x24000000), P(0x25000000), 0, 0.0, None, P(WS), flag + 2 * both,
                             None) == space


@pytest.mark.parametrize("H, I, dtype", [(7168, 4096, 2), (1001, 777, 1), (64, 12400, 3)])
def test_gated_block_forward_takes_less(rf, H, I, dtype):
    f = rf.moe_ffn(H, I, dtype, 1, X, H, Y, H)
    size, both = rf.lib().moe_ffn_fwd_workspace_size, rf.lib().moe_ffn_workspace_size
    for C in (1, 17, 32):
        assert size(ctypes.byref(f), C) == 256             # nothing is copied or split
    sizes = [size(ctypes.byref(f), c) for c in list(range(1, 1100)) + [4096, 9000]]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    for C in (33, 300, 4096):
        assert 256 < size(ctypes.byref(f), C) <= both(ctypes.byref(f), C)
    assert size(ctypes.byref(f), 4096) <= both(ctypes.byref(f), 4096) - 2 * 4096 * I * (2 if dtype > 1 else 1)
    for c in (0, (1 << 17) + 1):
        assert size(ctypes.byref(f), c) == 0
    assert size(ctypes.byref(rf.moe_ffn(0, I, dtype, 1, X, H, Y, H)), 5) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("C, K, N, n, r, xt", [(1, 7168, 300, 9, 16, "bf16"), (60, 3000, 700, 24, 32, "f16"),
                                               (333, 1099, 1001, 5, 24, "f32"), (1300, 2048, 96, 300, 64, "bf16")])
def test_adapters_in_it(C, K, N, n, r, xt):
    torch = pytest.importorskip("torch")
    import routed_expert_fp4_amd as rf
    from test_gpu_adapter import Case
    c = Case(C, K, N, n, r, xt, p=0.25)
    c.forward()
    y, hidden = c.y.clone(), c.hidden.clone()
    ws = rf.AdapterWorkspace(c.bank, C, backward=False)
    size = ws.tensor.numel()
    assert ws.nbytes == size < rf.AdapterWorkspace(c.bank, C).nbytes
    wide = torch.full((size + 4096,), 171, dtype=torch.uint8, device="cuda")
    ws.tensor = wide[:size]
    c.ws = ws
    c.y.fill_(9), c.hidden.fill_(9)
    c.forward()
    torch.cuda.synchronize()
    assert torch.equal(c.y, y) and torch.equal(c.hidden, hidden) and (wide[size:] == 171).all()
    # for fewer tokens too, and not for the gradients, nor for more tokens
    few = Case(max(1, C // 3), K, N, n, r, xt)
    few.forward()
    y = few.y.clone()
    few.ws = ws
    few.forward()
    torch.cuda.synchronize()
    assert torch.equal(few.y, y) and (wide[size:] == 171).all()
    with pytest.raises(rf.MoeError):
        c.backward()
    if C > 1:
        c.ws = rf.AdapterWorkspace(c.bank, C // 3, backward=False)
        with pytest.raises(rf.MoeError):
            c.forward()


@pytest.mark.gpu
@pytest.mark.parametrize("C, H, I, xt, pad", [(1, 1001, 130, "f16", 3), (32, 512, 300, "bf16", 0), (33, 12400, 300, "bf16", 1),
                                              (300, 1001, 777, "f32", 0), (700, 328, 200, "f16", 5)])
def test_gated_block_in_it(C, H, I, xt, pad):
    torch = pytest.importorskip("torch")
    import routed_expert_fp4_amd as rf
    from test_gpu_ffn import Case
    c = Case(C, H, I, xt, pad=pad)
    c.forward()
    want = [v.clone() for v in (c.h, c.gate, c.up)]
    ws = rf.FfnWorkspace(c.block, C, backward=False)
    wide = torch.full((ws.nbytes + 4096,), 171, dtype=torch.uint8, device="cuda")
    ws.tensor = wide[:ws.nbytes]
    c.ws = ws
    for v in (c.h, c.gate, c.up):
        v.fill_(9)
    c.forward()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((c.h, c.gate, c.up), want)) and (wide[ws.nbytes:] == 171).all()
    if xt != "f32":
        with pytest.raises(rf.MoeError):
            c.backward()
