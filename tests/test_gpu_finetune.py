"""A fine-tuning step as a program makes it: a frozen 4-bit projection with an
adapter beside it, a gated block on what they give, and dropout on the residual;
forward and all gradients in fp32 against the same composed in 64 bits.  And a
serving step: the projection of a batch of requests with their adapters.

Tolerances: every stage is within fp32 sums (the stages' own tests); composed, the
relative 2-norm of an error stays under the sum of the stages' (walk of their
depths), which the factor of 8 covers for six stages."""
import numpy as np
import pytest

import dense_ref as ref
import load_ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if torch is not None:
    from dense_util import host


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import routed_expert_fp4_amd as rf
    rf.lib()
    torch.cuda.set_device(0)


def near(got, want, depth, what):
    r = np.linalg.norm(host(got) - want) / np.linalg.norm(want)
    assert r <= 8 * ref.walk(depth), f"{what}: {r:.2e}"


@pytest.mark.parametrize("C, K, N, I, n, r, p", [(37, 512, 320, 200, 2, 12, 0.25), (1100, 256, 192, 130, 1, 16, 0.1)])
def test_training_step(C, K, N, I, n, r, p):
    import routed_expert_fp4_amd as rf
    g = np.random.default_rng(C)
    cu = lambda a: torch.from_numpy(np.asarray(a, np.float32)).cuda()  # noqa: E731
    G = 64
    codes = torch.from_numpy(g.integers(0, 256, (N, K // 2), np.uint8)).cuda()
    scales = cu(g.uniform(0.004, 0.012, (N, K // G)))
    x, A, B = cu(g.normal(size=(C, K))), cu(g.normal(size=(n, r, K)) / np.sqrt(K)), cu(g.normal(size=(n, N, r)))
    s, who = cu(g.uniform(0.5, 1, n)), g.integers(0, n, C)
    wg, wu, wd = cu(g.normal(size=(I, N)) / np.sqrt(N)), cu(g.normal(size=(I, N)) / np.sqrt(N)), cu(g.normal(size=(N, I)))
    res, dout = cu(g.normal(size=(C, N))), cu(g.normal(size=(C, N)))
    rng_a, rng_d = (torch.tensor([11, o], dtype=torch.int64, device="cuda") for o in (0, 1))

    m = rf.QuantMatrix(codes, scales, K, G)
    qws, bank = rf.QuantWorkspace(m, C, torch.float32), rf.AdapterBank(A, B, s)
    plan, aws = rf.AdapterPlan(torch.from_numpy(who.astype(np.int32)).cuda(), n), rf.AdapterWorkspace(bank, C)
    block = rf.FfnBlock(wg, wu)
    fws = rf.FfnWorkspace(block, C)
    new = lambda *sh: torch.full(sh, float("nan"), device="cuda")  # noqa: E731
    y, hidden, h, gate, up, out = new(C, N), new(C, r), new(C, I), new(C, I), new(C, I), new(C, N)
    rf.moe_quant_linear(m, x, C, y, qws)
    rf.moe_adapter_fwd(bank, plan, x, C, y, aws, base=y, hidden=hidden, dropout=(p, rng_a))
    rf.moe_ffn_fwd(block, y, C, h, fws, gate, up)
    z = h @ wd.t()
    rf.moe_dropout(z, p, rng_d, out, base=res)
    # backward
    dz, dh, dy, dx = new(C, N), None, new(C, N), new(C, K)
    dA, dB, dwg, dwu = new(n, r, K), new(n, N, r), new(I, N), new(I, N)
    rf.moe_dropout(dout, p, rng_d, dz)
    dh = dz @ wd
    rf.moe_ffn_bwd(block, y, gate, up, dh, C, dy, dwg, dwu, fws)
    W = cu(load_ref.quant_weights(codes.cpu().numpy(), host(scales), None, K, G))
    rf.moe_adapter_bwd(bank, plan, x, hidden, dy, C, dx, dA, dB, aws, base=dy @ W, dropout=(p, rng_a))
    torch.cuda.synchronize()

    # the same in 64 bits, its gradients by autograd
    d = lambda t: t.double().cpu().requires_grad_(True)  # noqa: E731
    X, A6, B6, G6, U6 = d(x), d(A), d(B), d(wg), d(wu)
    m1, m2 = (torch.from_numpy(ref.mask(11, o, C, k, p)) for o, k in ((0, K), (1, N)))
    W6 = torch.from_numpy(load_ref.quant_weights(codes.cpu().numpy(), host(scales), None, K, G))
    sel = torch.from_numpy(who)
    t6 = torch.stack([A6[a] @ v for a, v in zip(who, X * m1)])
    y6 = X @ W6.t() + s.double().cpu()[sel][:, None] * torch.stack([B6[a] @ v for a, v in zip(who, t6)])
    h6 = torch.nn.functional.silu(y6 @ G6.t()) * (y6 @ U6.t())
    out6 = res.double().cpu() + (h6 @ wd.double().cpu().t()) * m2
    grads = torch.autograd.grad(out6, (X, A6, B6, G6, U6), dout.double().cpu())
    depth = K + 2 * N + 2 * I + C
    near(hidden, t6.detach().numpy(), depth, "hidden")
    near(y, y6.detach().numpy(), depth, "y")
    near(h, h6.detach().numpy(), depth, "h")
    near(out, out6.detach().numpy(), depth, "out")
    for name, got, want in zip(("dx", "dA", "dB", "dwg", "dwu"), (dx, dA, dB, dwg, dwu), grads):
        near(got, want.numpy(), depth, name)


@pytest.mark.parametrize("C", [1, 13, 200])
def test_serving_step(C):
    """One plan for two projections of a step."""
    import routed_expert_fp4_amd as rf
    g = np.random.default_rng(C)
    H, L, n, r, G = 768, 384, 9, 16, 128
    cu = lambda a: torch.from_numpy(np.asarray(a, np.float32)).cuda()  # noqa: E731
    who = g.integers(-1, n, C)
    plan = rf.AdapterPlan(torch.from_numpy(who.astype(np.int32)).cuda(), n)
    x = cu(g.normal(size=(C, H)))
    want = host(x)
    for K, N in ((H, L), (L, H)):
        codes = torch.from_numpy(g.integers(0, 256, (N, K // 2), np.uint8)).cuda()
        scales = cu(g.uniform(0.004, 0.012, (N, K // G)))
        A, B, s = cu(g.normal(size=(n, r, K)) / np.sqrt(K)), cu(g.normal(size=(n, N, r)) / 4), cu(g.uniform(0.5, 1, n))
        m, bank = rf.QuantMatrix(codes, scales, K, G), rf.AdapterBank(A, B, s)
        y = torch.empty((C, N), device="cuda")
        rf.moe_quant_linear(m, x, C, y, rf.QuantWorkspace(m, C, torch.float32))
        rf.moe_adapter_fwd(bank, plan, x, C, y, rf.AdapterWorkspace(bank, C), base=y)
        W = load_ref.quant_weights(codes.cpu().numpy(), host(scales), None, K, G)
        want = ref.adapters(want, who, host(A), host(B), host(s), want @ W.T)[0]
        near(y, want, 2 * (H + L), (K, N))
        x = y
