"""The plain definitions against hand values, brute force and differences, and
the library's refusals of bad calls (no GPU)."""
import ctypes
import os

import numpy as np
import pytest

import load_ref as ref

FAKE = ctypes.c_void_p(0x20000)       # never dereferenced: validation fails first
OUT = ctypes.c_void_p(0x400000)
WS = ctypes.c_void_p(0x800000)


@pytest.fixture(scope="module")
def rf():
    import routed_expert_fp4_amd as rf
    if not os.path.exists(rf.LIB_PATH):
        from routed_expert_fp4_amd import build
        build.build_library()
    rf.lib()
    return rf


def test_quant_weights_by_hand():
    codes = np.array([[0x10, 0xF2]], np.uint8)                 # 0, 1, 2, 15
    W = ref.quant_weights(codes, np.array([[2.0]]), None, 4, 32)
    assert W.tolist() == [[-16.0, -14.0, -12.0, 14.0]]
    W = ref.quant_weights(codes, np.array([[2.0]]), np.array([[1]], np.uint8), 3, 32)
    assert W.tolist() == [[-2.0, 0.0, 2.0]]


def test_counts_by_hand():
    idx = np.array([[0, 2], [2, 1], [2, 9], [0, 0], [1, -1]])
    cnt, tok = ref.counts(idx, 3, seq=[0, 2, 2, 4], mask=[1, 1, 1, 0, 1], S=3)
    assert cnt.tolist() == [[1, 1, 2], [0, 0, 0], [0, 0, 1]] and tok.tolist() == [2, 0, 1]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_balanced_selection_has_loss_alpha(score):
    """Equal logits and equal counts: f = 1, P = 1 / E, loss = alpha."""
    E, k = 8, 2
    idx = np.array([[2 * t, 2 * t + 1] for t in range(4)])
    r = ref.balance(np.zeros((4, E)), idx, 0.25, score)
    assert abs(r["loss"] - 0.25) < 1e-15 and np.abs(r["dlogits"]).max() < 1e-17


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_balance_gradient_against_differences(score):
    rng = np.random.default_rng(3)
    C, E, k, S = 9, 7, 2, 3
    logits = rng.normal(0, 2, (C, E))
    idx = np.stack([rng.permutation(E)[:k] for _ in range(C)])
    seq, mask = [1, 4, 4, 8], [1, 1, 0, 1, 1, 1, 1, 1, 1]
    r = ref.balance(logits, idx, 0.7, score, seq, mask, S, grad=1.3)
    for t in range(C):
        for e in range(E):
            h = 1e-5
            up, dn = logits.copy(), logits.copy()
            up[t, e] += h
            dn[t, e] -= h
            num = 1.3 * (ref.balance(up, idx, 0.7, score, seq, mask, S)["loss"] -
                         ref.balance(dn, idx, 0.7, score, seq, mask, S)["loss"]) / (2 * h)
            assert abs(num - r["dlogits"][t, e]) < 1e-9


def test_route_gradient_against_differences():
    rng = np.random.default_rng(4)
    C, E, k = 5, 9, 4
    logits, dw = rng.normal(0, 2, (C, E)), rng.normal(0, 1, (C, k))
    idx = np.stack([rng.permutation(E)[:k] for _ in range(C)])
    idx[1, 2] = idx[1, 0]                                       # one expert twice
    idx[2, 1] = -1
    mask = [1, 1, 1, 0, 1]

    def value(l):
        v = 0.0
        for t in range(C):
            if mask[t]:
                on = [s for s in range(k) if idx[t, s] >= 0]
                s = 1 / (1 + np.exp(-l[t, idx[t, on]]))
                v += (s / s.sum() * dw[t, on]).sum()
        return v

    d = ref.route_grad(logits, idx, dw, mask)
    for t in range(C):
        for e in range(E):
            up, dn = logits.copy(), logits.copy()
            up[t, e] += 1e-5
            dn[t, e] -= 1e-5
            assert abs((value(up) - value(dn)) / 2e-5 - d[t, e]) < 1e-9


def test_shares_hold_where_sigmoids_underflow():
    l = np.array([-900.0, -901.0, -np.inf])
    p = ref.shares(l, "sigmoid")
    assert abs(p[0] / p[1] - np.e) < 1e-12 and p[2] == 0 and abs(p.sum() - 1) < 1e-15
    assert ref.shares(np.full(3, -np.inf), "softmax").tolist() == [0, 0, 0]


# ---------------------------------------------------------------------------
# Refusals
# ---------------------------------------------------------------------------
def _matrix(rf, **kw):
    m = rf.moe_quant_matrix(64, 256, 128, rf.MOE_DT_BF16, 0x100000, 128, 0x200000, 2, None, 0)
    for key, v in kw.items():
        setattr(m, key, v)
    return m


def test_quant_linear_rejects_bad_arguments(rf):
    L = rf.lib()
    n = L.moe_quant_workspace_size(ctypes.byref(_matrix(rf)), rf.MOE_DT_F32, 4)
    assert n >= 256
    size = lambda m, d=rf.MOE_DT_F32, C=4: L.moe_quant_workspace_size(ctypes.byref(m), d, C)  # noqa: E731
    assert size(_matrix(rf), d=0) == 0 and size(_matrix(rf), d=4) == 0
    assert size(_matrix(rf), C=0) == 0 and size(_matrix(rf), C=4097) == 0
    assert L.moe_quant_workspace_size(None, rf.MOE_DT_F32, 4) == 0

    def call(m=None, d=rf.MOE_DT_F32, x=FAKE, xp=256, C=4, y=OUT, yp=64, ws=WS, nb=None):
        m = _matrix(rf) if m is None else m
        return L.moe_quant_linear(ctypes.byref(m), d, x, xp, C, y, yp, 0, ws, n if nb is None else nb, None)

    inv, uns, wsp = rf.MOE_ERR_INVALID_ARG, rf.MOE_ERR_UNSUPPORTED, rf.MOE_ERR_WORKSPACE
    assert L.moe_quant_linear(None, rf.MOE_DT_F32, FAKE, 256, 4, OUT, 64, 0, WS, n, None) == inv
    for kw, want in [(dict(codes=None), inv), (dict(scales=None), inv), (dict(codes=0x100008), inv),
                     (dict(code_pitch=120), inv), (dict(code_pitch=112), inv), (dict(scale_pitch=1), inv),
                     (dict(scales=0x200001), inv), (dict(scale_dtype=rf.MOE_DT_F32, scales=0x200002), inv),
                     (dict(zeros=0x300000, zero_pitch=1), inv), (dict(rows=0), uns), (dict(cols=0), uns),
                     (dict(rows=rf.MOE_MAX_QUANT_ROWS + 1), uns), (dict(cols=rf.MOE_MAX_QUANT_COLS + 1), uns),
                     (dict(group=16), uns), (dict(group=96), uns), (dict(group=0), uns),
                     (dict(group=-128), uns), (dict(scale_dtype=9), uns)]:
        assert call(_matrix(rf, **kw)) == want, kw
    assert call(x=None) == inv and call(y=None) == inv and call(y=FAKE) == inv
    assert call(xp=255) == inv and call(yp=63) == inv
    assert call(x=ctypes.c_void_p(0x20002)) == inv and call(y=ctypes.c_void_p(0x400001)) == inv
    assert call(d=0) == uns and call(C=0) == uns and call(C=4097) == uns
    assert call(ws=None) == wsp and call(nb=n - 1) == wsp and call(ws=ctypes.c_void_p(0x800010)) == wsp


def test_router_load_rejects_bad_arguments(rf):
    L = rf.lib()
    inv, uns, wsp = rf.MOE_ERR_INVALID_ARG, rf.MOE_ERR_UNSUPPORTED, rf.MOE_ERR_WORKSPACE
    A, B, D, F = (ctypes.c_void_p(0x100000 * i) for i in (1, 2, 3, 5))
    big = rf.MOE_MAX_BATCH_TOKENS + 1

    def cnt(idx=FAKE, C=8, k=2, E=16, off=None, S=1, out=OUT):
        return L.moe_expert_counts(idx, C, k, E, off, S, None, out, None, 0, None)

    assert cnt(idx=None) == inv and cnt(out=None) == inv and cnt(S=2) == inv
    assert cnt(idx=ctypes.c_void_p(0x20002)) == inv and cnt(off=ctypes.c_void_p(0x20002)) == inv
    for kw in (dict(C=0), dict(C=big), dict(k=0), dict(k=33), dict(k=17), dict(E=0), dict(E=1025),
               dict(S=0), dict(S=65536, off=A)):
        assert cnt(**kw) == uns, kw

    n = L.moe_balance_workspace_size(8, 16, 1)
    assert n > 0 and L.moe_balance_workspace_size(0, 16, 1) == 0
    assert L.moe_balance_workspace_size(8, 1025, 1) == 0 and L.moe_balance_workspace_size(8, 16, 65536) == 0

    def fwd(logits=A, idx=B, C=8, k=2, E=16, off=None, S=1, score=1, c=D, t=F, p=OUT, l=FAKE, ws=WS, nb=n):
        return L.moe_balance_fwd(logits, idx, C, k, E, off, S, None, score, 0.1, c, t, p, l, ws, nb, None)

    for kw in (dict(logits=None), dict(idx=None), dict(c=None), dict(t=None), dict(p=None), dict(l=None),
               dict(S=3), dict(score=0), dict(score=3), dict(logits=ctypes.c_void_p(0x100002))):
        assert fwd(**kw) == inv, kw
    assert fwd(C=0) == uns and fwd(E=1025) == uns and fwd(k=17) == uns and fwd(S=0) == uns
    assert fwd(ws=None) == wsp and fwd(nb=n - 1) == wsp and fwd(ws=ctypes.c_void_p(0x800010)) == wsp
    assert fwd(C=4096) == wsp                                   # sized for 8 tokens

    def bwd(logits=A, c=D, t=F, C=8, k=2, E=16, off=None, S=1, score=2, g=FAKE, d=OUT):
        return L.moe_balance_bwd(logits, c, t, C, k, E, off, S, None, score, 0.1, g, d, 0, None)

    for kw in (dict(logits=None), dict(c=None), dict(t=None), dict(g=None), dict(d=None), dict(d=A),
               dict(S=2), dict(score=7), dict(d=ctypes.c_void_p(0x400002))):
        assert bwd(**kw) == inv, kw
    assert bwd(C=big) == uns and bwd(k=0) == uns

    def rb(logits=A, idx=B, dw=D, C=8, k=2, E=16, d=OUT):
        return L.moe_route_bwd(logits, idx, dw, C, k, E, None, d, 0, None)

    for kw in (dict(logits=None), dict(idx=None), dict(dw=None), dict(d=None), dict(d=A),
               dict(dw=ctypes.c_void_p(0x300002))):
        assert rb(**kw) == inv, kw
    assert rb(C=0) == uns and rb(k=17) == uns and rb(E=1025) == uns


def test_binding_rejects_host_tensors(rf):
    torch = pytest.importorskip("torch")
    idx = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        rf.moe_expert_counts(idx, 4, 8, 2, torch.zeros((1, 8), dtype=torch.int32))
    with pytest.raises(ValueError, match="device tensor"):
        rf.moe_route_bwd(torch.zeros(4, 8), idx, torch.zeros(4, 2), 4, 8, 2, torch.zeros(4, 8))
    with pytest.raises(ValueError, match="device tensor"):
        rf.QuantMatrix(torch.zeros((4, 16), dtype=torch.uint8), torch.zeros((4, 1)), 32, 32)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        rf._moe_dtype(torch.int32)
    with pytest.raises(ValueError, match="score"):
        rf._score("relu")
    with pytest.raises(rf.MoeError):
        rf.BalanceWorkspace(0, 8)
