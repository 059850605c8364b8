"""The 64-bit forms of dropout, adapters and the gated block against published
numbers, hand values and differences, and the refusals of their entry points (CPU:
every call ends at a check on the host)."""
import ctypes
import os

import numpy as np
import pytest

import dense_ref as ref

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def rf():
    import routed_expert_fp4_amd as rf
    if not os.path.exists(rf.LIB_PATH):
        from routed_expert_fp4_amd import build
        build.build_library()
    rf.lib()
    return rf


@pytest.mark.parametrize("key, counter, words", [
    ((0, 0), (0, 0, 0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 2, (0xFFFFFFFF,) * 4, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0xA4093822, 0x299F31D0), (0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_generator_gives_its_published_numbers(key, counter, words):
    assert [int(w) for w in ref.philox(key, counter)] == list(words)


def test_mask():
    m = ref.mask(12345, 678, 400, 1001, 0.25)
    assert set(np.unique(m)) == {0.0, 4 / 3}
    n = m.size                                             # five standard deviations
    assert abs((m == 0).sum() - n / 4) < 5 * np.sqrt(n * 3 / 16)
    assert (ref.mask(1, 2, 3, 5, 0.0) == 1).all() and (ref.mask(1, 2, 3, 5, 1.0) == 0).all()
    # a row's mask depends on its own place alone, and another offset gives another
    assert (ref.mask(12345, 678, 10, 1001, 0.25) == m[:10]).all()
    assert (ref.mask(12345, 678, 400, 17, 0.25) == m[:, :17]).all()
    assert (ref.mask(12345, 679, 400, 1001, 0.25) != m).mean() > 0.3
    assert (ref.mask(-5, -1, 4, 8, 0.5) == ref.mask((1 << 64) - 5, (1 << 64) - 1, 4, 8, 0.5)).all()


def test_adapter_gradients_against_differences():
    rng = np.random.default_rng(0)
    C, K, N, n, r = 5, 7, 6, 3, 2
    x, dy = rng.normal(size=(C, K)), rng.normal(size=(C, N))
    A, B, s = rng.normal(size=(n, r, K)), rng.normal(size=(n, N, r)), rng.uniform(0.5, 2, n)
    who, m = np.array([0, 2, -1, 0, 9]), ref.mask(3, 4, C, K, 0.4)

    def loss(x, A, B):
        return float((ref.adapters(x, who, A, B, s, m=m)[0] * dy).sum())

    t = ref.adapters(x, who, A, B, s, m=m)[1]
    grads = ref.adapter_grads(x, who, A, B, s, dy, t, m=m)
    assert (grads[1][1] == 0).all() and (grads[2][1] == 0).all() and (t[2] == 0).all()
    for at, g in enumerate(grads):
        args = [x, A, B]
        for i in np.ndindex(*g.shape):
            e = np.zeros(g.shape)
            e[i] = 1e-6
            d = (loss(*[v + e if k == at else v for k, v in enumerate(args)]) -
                 loss(*[v - e if k == at else v for k, v in enumerate(args)])) / 2e-6
            assert abs(d - g[i]) < 1e-7 * max(1, abs(d))


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_gated_gradients_against_differences(name):
    rng = np.random.default_rng(1)
    C, H, I = 4, 5, 3
    x, wg, wu, dh = rng.normal(size=(C, H)), rng.normal(size=(I, H)), rng.normal(size=(I, H)), rng.normal(size=(C, I))

    def loss(x, wg, wu):
        return float((ref.gated(name, x, wg, wu)[0] * dh).sum())

    _, g, u = ref.gated(name, x, wg, wu)
    for at, grad in enumerate(ref.gated_grads(name, x, wg, wu, g, u, dh)[:3]):
        args = [x, wg, wu]
        for i in np.ndindex(*grad.shape):
            e = np.zeros(grad.shape)
            e[i] = 1e-6
            d = (loss(*[v + e if k == at else v for k, v in enumerate(args)]) -
                 loss(*[v - e if k == at else v for k, v in enumerate(args)])) / 2e-6
            assert abs(d - grad[i]) < 1e-7 * max(1, abs(d))


def test_activations():
    assert ref.act("silu", np.array([0.0, 1.0]))[0] == pytest.approx([0.0, 1 / (1 + np.exp(-1.0))])
    assert ref.act("gelu", np.array([1.0]))[0] == pytest.approx([0.5 * (1 + np.tanh(ref.ROOT * 1.044715))])
    for name in ("silu", "gelu"):
        a, d = ref.act(name, np.array([-80.0, 80.0]))
        assert a == pytest.approx([0, 80], abs=1e-30) and d == pytest.approx([0, 1], abs=1e-30)


# refusals -----------------------------------------------------------------
X, Y, Z, W = 0x40000000, 0x50000000, 0x60000000, 0x70000000
FAR, WS = 0x10000000, 0x30000000


def test_dropout_refusals(rf):
    inv, uns = rf.MOE_ERR_INVALID_ARG, rf.MOE_ERR_UNSUPPORTED

    def call(dtype=2, x=X, xp=64, C=4, K=64, base=Z, bp=64, y=Y, yp=64, p=0.5, rng=FAR):
        return rf.lib().moe_dropout(dtype, P(x), xp, C, K, P(base), bp, P(y), yp, p, P(rng), None)

    for kw in (dict(dtype=0), dict(dtype=4), dict(C=0), dict(C=rf.MOE_MAX_BATCH_TOKENS + 1), dict(K=0),
               dict(K=rf.MOE_MAX_QUANT_COLS + 1), dict(xp=(1 << 24) + 1)):
        assert call(**kw) == uns, kw
    for kw in (dict(x=None), dict(y=None), dict(xp=63), dict(yp=63), dict(bp=63), dict(x=X + 1), dict(y=Y + 1),
               dict(p=-0.1), dict(p=1.1), dict(p=float("nan")), dict(rng=None), dict(rng=FAR + 4), dict(y=X + 2),
               dict(y=Z + 64), dict(x=Y, xp=128), dict(rng=Y)):
        assert call(**kw) == inv, kw
    assert call(dtype=1, x=X + 2) == inv


def bank(rf, n=3, r=8, K=64, N=32, dtype=2, a=X, b=Y, scales=FAR, **kw):
    m = rf.moe_adapter_bank(n, r, K, N, dtype, a, r * K, K, b, N * r, r, scales)
    for k, v in kw.items():
        setattr(m, k, v)
    return m


BAD_BANKS = [(dict(n=0), "uns"), (dict(n=1025), "uns"), (dict(r=0), "uns"), (dict(r=129), "uns"), (dict(K=0), "uns"),
             (dict(N=0), "uns"), (dict(K=(1 << 17) + 1), "uns"), (dict(dtype=0), "uns"), (dict(a=None), "inv"),
             (dict(b=None), "inv"), (dict(a=X + 1), "inv"), (dict(dtype=1, b=Y + 2), "inv"), (dict(a_pitch=63), "inv"),
             (dict(b_pitch=7), "inv"), (dict(a_stride=511), "inv"), (dict(b_stride=255), "inv"),
             (dict(a_pitch=(1 << 24) + 1, a_stride=1 << 30), "uns"), (dict(scales=FAR + 2), "inv")]


def test_adapter_refusals(rf):
    st = {"inv": rf.MOE_ERR_INVALID_ARG, "uns": rf.MOE_ERR_UNSUPPORTED}
    inv, uns, space = st["inv"], st["uns"], rf.MOE_ERR_WORKSPACE
    C, big = 5, 1 << 40
    L = rf.lib()
    plan_bytes = L.moe_adapter_plan_size(C, 3)
    assert plan_bytes % 256 == 0 and plan_bytes > 0
    for c, n in ((0, 3), (-1, 3), (rf.MOE_MAX_BATCH_TOKENS + 1, 3), (5, 0), (5, 1025)):
        assert L.moe_adapter_plan_size(c, n) == 0
        assert L.moe_adapter_plan(P(FAR), c, n, P(W), big, None) == uns
    assert L.moe_adapter_plan(None, C, 3, P(W), plan_bytes, None) == inv
    assert L.moe_adapter_plan(P(FAR + 2), C, 3, P(W), plan_bytes, None) == inv
    assert L.moe_adapter_plan(P(FAR), C, 3, None, plan_bytes, None) == space
    assert L.moe_adapter_plan(P(FAR), C, 3, P(W + 4), plan_bytes, None) == space
    assert L.moe_adapter_plan(P(FAR), C, 3, P(W), 64, None) == space
    assert L.moe_adapter_plan(P(W + 16), C, 3, P(W), plan_bytes, None) == inv

    def fwd(m, x=0x20000000, xp=64, C=C, base=None, bp=32, y=0x21000000, yp=32, hidden=None, p=0.0, rng=None, plan=W,
            pb=plan_bytes, ws=None, wb=0):
        return L.moe_adapter_fwd(ctypes.byref(m), P(plan), pb, P(x), xp, C, P(base), bp, P(y), yp, P(hidden), p, P(rng),
                                 P(ws), wb, None)

    def bwd(m, x=0x20000000, hidden=0x22000000, dy=0x21000000, C=C, base=None, dx=0x23000000, da=0x24000000,
            db=0x25000000, p=0.0, rng=None, ws=None, wb=0, xp=64, dp=32, dxp=64):
        return L.moe_adapter_bwd(ctypes.byref(m), P(W), plan_bytes, P(x), xp, P(hidden), P(dy), dp, C, P(base), 64, P(dx),
                                 dxp, P(da), P(db), 0, p, P(rng), P(ws), wb, None)

    for kw, want in BAD_BANKS:
        m = bank(rf, **kw)
        assert fwd(m) == st[want], kw
        assert bwd(m) == st[want], kw
        assert L.moe_adapter_workspace_size(ctypes.byref(m), C) == 0
    assert L.moe_adapter_fwd(None, P(W), plan_bytes, P(X), 64, C, None, 0, P(Y), 32, None, 0.0, None, None, 0, None) == inv
    m = bank(rf)
    need = L.moe_adapter_workspace_size(ctypes.byref(m), C)
    assert need > 0 and L.moe_adapter_workspace_size(ctypes.byref(m), 0) == 0
    assert fwd(m) == space and bwd(m) == space             # nothing else is wrong
    assert fwd(m, ws=WS, wb=need - 1) == space and fwd(m, ws=WS + 16, wb=need) == space
    assert fwd(m, plan=None) == space and fwd(m, pb=plan_bytes // 2) == space and fwd(m, plan=W + 16) == space
    for kw in (dict(C=0), dict(C=(1 << 20) + 1), dict(xp=(1 << 24) + 1)):
        assert fwd(m, **kw) == uns, kw
    for kw in (dict(x=None), dict(y=None), dict(x=0x20000001), dict(xp=63), dict(yp=31), dict(base=0x22000000, bp=31),
               dict(hidden=0x22000002), dict(p=2.0), dict(p=0.5), dict(p=0.5, rng=FAR + 4), dict(y=0x20000000),
               dict(base=0x21000002), dict(hidden=0x21000000), dict(hidden=0x20000000)):
        assert fwd(m, **kw) == inv, kw
    assert fwd(m, base=0x21000000) == space                # in place
    assert fwd(m, base=0x21000000, bp=40) == inv           # the same start, other rows
    for kw in (dict(dx=None, da=None, db=None), dict(dy=None), dict(x=None), dict(hidden=None), dict(da=0x24000002),
               dict(db=0x25000002), dict(dx=0x20000000), dict(dx=0x21000000), dict(da=0x20000000), dict(db=0x21000000),
               dict(da=0x22000000), dict(dx=0x24000000), dict(db=0x24000000), dict(base=0x23000002), dict(base=0x24000000),
               dict(p=0.5)):
        assert bwd(m, **kw) == inv, kw
    assert bwd(m, x=None, da=None) == space and bwd(m, hidden=None, db=None) == space
    # an adapter's tensors may not be overwritten
    assert fwd(m, y=X) == inv and fwd(m, hidden=Y) == inv
    assert bwd(m, dx=X) == inv and bwd(m, da=X) == inv and bwd(m, db=Y) == inv
    # nor the plan, nor anything by the workspace
    assert fwd(m, y=W) == inv and bwd(m, dx=W) == inv
    for at in (X, Y, FAR, W, 0x20000000, 0x21000000):
        assert fwd(m, ws=at, wb=need) == inv, hex(at)
    for at in (0x20000000, 0x21000000, 0x22000000, 0x23000000, 0x24000000, 0x25000000):
        assert bwd(m, ws=at, wb=need) == inv, hex(at)


def test_adapter_workspace_serves_fewer_tokens(rf):
    for kw in (dict(), dict(n=40, r=64, K=4096, N=3584), dict(n=1, r=16, K=7168, N=1000, dtype=1)):
        m = bank(rf, **kw)
        sizes = [rf.lib().moe_adapter_workspace_size(ctypes.byref(m), c) for c in list(range(1, 2200)) + [4096, 9000, 70000]]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), kw


def block(rf, H=64, I=32, dtype=2, act=1, wg=X, gp=None, wu=Y, up=None):
    return rf.moe_ffn(H, I, dtype, act, wg, H if gp is None else gp, wu, H if up is None else up)


def test_gated_block_refusals(rf):
    inv, uns, space = rf.MOE_ERR_INVALID_ARG, rf.MOE_ERR_UNSUPPORTED, rf.MOE_ERR_WORKSPACE
    L, C = rf.lib(), 5

    def fwd(f, x=0x20000000, xp=64, C=C, h=0x21000000, hp=32, gate=None, gp=32, up=None, upp=32, ws=None, wb=0):
        return L.moe_ffn_fwd(ctypes.byref(f), P(x), xp, C, P(h), hp, P(gate), gp, P(up), upp, P(ws), wb, None)

    def bwd(f, x=0x20000000, gate=0x21000000, up=0x22000000, dh=0x23000000, C=C, dx=0x24000000, gd=2, dwg=0x25000000,
            dwu=0x26000000, ws=None, wb=0, gp=32, dxp=64, dwp=64):
        return L.moe_ffn_bwd(ctypes.byref(f), P(x), 64, P(gate), gp, P(up), 32, P(dh), 32, C, P(dx), dxp, gd, P(dwg), dwp,
                             P(dwu), 64, 0, P(ws), wb, None)

    for kw, want in ((dict(H=0), uns), (dict(I=0), uns), (dict(H=(1 << 17) + 1), uns), (dict(dtype=4), uns),
                     (dict(act=0), uns), (dict(act=3), uns), (dict(wg=None), inv), (dict(wu=None), inv),
                     (dict(wg=X + 1), inv), (dict(gp=63), inv), (dict(up=63), inv), (dict(gp=(1 << 24) + 1), uns)):
        f = block(rf, **kw)
        assert fwd(f) == want and bwd(f) == want, kw
        assert L.moe_ffn_workspace_size(ctypes.byref(f), C) == 0
    f = block(rf)
    need = L.moe_ffn_workspace_size(ctypes.byref(f), C)
    assert need > 0 and L.moe_ffn_workspace_size(ctypes.byref(f), 0) == 0
    assert L.moe_ffn_workspace_size(ctypes.byref(f), (1 << 17) + 1) == 0
    assert fwd(f) == space and bwd(f) == space and fwd(f, ws=WS + 16, wb=need) == space
    for kw in (dict(C=0), dict(C=(1 << 17) + 1), dict(xp=(1 << 24) + 1)):
        assert fwd(f, **kw) == uns, kw
    for kw in (dict(x=None), dict(h=None), dict(x=0x20000001), dict(xp=63), dict(hp=31), dict(gate=0x22000000),
               dict(up=0x22000000), dict(gate=0x22000000, up=0x22000000), dict(h=0x20000000), dict(h=X), dict(h=Y),
               dict(gate=0x21000000, up=0x23000000), dict(gate=X, up=0x23000000)):
        assert fwd(f, **kw) == inv, kw
    for kw in (dict(dx=None, dwg=None, dwu=None), dict(dwg=None), dict(dwu=None), dict(x=None), dict(gate=None),
               dict(up=None), dict(dh=None), dict(gp=31), dict(dxp=63), dict(dwp=63), dict(dx=0x20000000),
               dict(dx=0x23000000), dict(dwg=X), dict(dwu=Y), dict(dwg=0x26000000), dict(dx=0x25000000),
               dict(dwg=0x21000000)):
        assert bwd(f, **kw) == inv, kw
    for at in (X, Y, 0x20000000, 0x21000000):
        assert fwd(f, ws=at, wb=need) == inv, hex(at)
    for at in (X, Y, 0x20000000, 0x21000000, 0x22000000, 0x23000000, 0x24000000, 0x25000000, 0x26000000):
        assert bwd(f, ws=at, wb=need) == inv, hex(at)
    assert bwd(f, gd=3) == uns and bwd(f, gd=1) == space and bwd(f, x=None, dwg=None, dwu=None) == space


def test_gated_block_workspace_serves_fewer_tokens(rf):
    for kw in (dict(), dict(H=7168, I=1536), dict(H=1001, I=777, dtype=1), dict(H=3584, I=4100, dtype=3)):
        f = block(rf, **kw)
        sizes = [rf.lib().moe_ffn_workspace_size(ctypes.byref(f), c) for c in list(range(1, 1100)) + [4096, 9000]]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), kw
