"""moe_quant_linear against the plain 64-bit product, through the C ABI.

Tolerance, element by element: a product passes at most 32 roundings inside
each matrix instruction of its group (four per 128 columns), one for the scale,
and one per group, slab and wave sum after it: under 160 + K / 32 roundings of
2^-24 against the sum of |x| |W|.  Activations held as fp16 terms keep 2^-23 of
an element and 2^-38 of the largest of their token.  The result is then rounded
to its type once (half a step: eps / 2).
"""
import numpy as np
import pytest

import load_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import routed_expert_fp4_amd as rf
    rf.lib()
    torch.cuda.set_device(0)


def make(C, N, K, G, xt="f32", st="bf16", zeros=False, seed=0, code_pad=0, x_pad=0, y_pad=0):
    """Device tensors of a case (wide ones sliced where a pad is given) and
    their float64 values."""
    rng = np.random.default_rng(seed)
    ng, pitch = -(-K // G), (-(-K // 2) + 15) // 16 * 16 + code_pad
    codes = torch.from_numpy(rng.integers(0, 256, (N, pitch), np.uint8)).cuda()
    scales = torch.from_numpy(rng.uniform(0.004, 0.012, (N, ng + 2)).astype(np.float32)).to(T[st]).cuda()[:, 1:1 + ng]
    z = torch.from_numpy(rng.integers(0, 16, (N, ng), np.uint8)).cuda() if zeros else None
    x = torch.from_numpy(rng.normal(0, 1, (C, K + x_pad)).astype(np.float32))
    x[:, ::97] *= 30.0
    x = x.to(T[xt]).cuda()[:, :K]
    y = torch.full((C, N + y_pad), 7.0, dtype=T[xt], device="cuda")
    return codes, scales, z, x, y


def expect(codes, scales, z, x, K, G):
    W = ref.quant_weights(codes.cpu().numpy(), scales.float().cpu().numpy(),
                          None if z is None else z.cpu().numpy(), K, G)
    xd = x.double().cpu().numpy()
    want = xd @ W.T
    size = np.abs(xd) @ np.abs(W).T
    few = np.abs(xd).max(axis=1, keepdims=True) * np.abs(W).sum(axis=1)[None, :]
    return want, (160 + K / 32 + 2) * ref.U * size + 2.0 ** -38 * few


def run(codes, scales, z, x, y, K, G, accumulate=False, stream=None):
    import routed_expert_fp4_amd as rf
    m = rf.QuantMatrix(codes, scales, K, G, z)
    ws = rf.QuantWorkspace(m, x.shape[0], x.dtype)
    rf.moe_quant_linear(m, x, x.shape[0], y, ws, accumulate=accumulate, stream=stream)
    torch.cuda.synchronize()
    return m, ws


def check(y, want, tol, what, rel=True):
    got = y.double().cpu().numpy()
    step = torch.finfo(y.dtype).eps / 2 * np.abs(want) + torch.finfo(y.dtype).smallest_normal * torch.finfo(y.dtype).eps
    bad = ~(np.abs(got - want) <= (tol + step) * 1.0001)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.abs(got - want).max():.3e}"
    if y.dtype == torch.float32 and rel:
        rel = np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-300)
        assert rel <= 2e-6, f"{what}: rel-L2 {rel:.2e}"


CASES = [
    # C, N, K, G, x, scales, zeros
    (1, 16, 32, 32, "f32", "f32", False),
    (1, 1, 1, 32, "f32", "f32", True),
    (1, 17, 31, 32, "bf16", "bf16", False),
    (2, 33, 33, 32, "f16", "f16", True),
    (3, 65, 127, 64, "f32", "f16", True),
    (4, 48, 128, 128, "bf16", "f32", True),
    (5, 130, 129, 128, "f32", "bf16", False),
    (1, 3584, 7168, 128, "f32", "bf16", False),
    (7, 1000, 3584, 32, "bf16", "f16", True),
    (8, 257, 2048, 64, "f16", "bf16", False),
    (9, 100, 4099, 64, "f32", "f32", True),
    (16, 1001, 4099, 128, "f32", "f16", True),
    (16, 320, 7168, 256, "f16", "f32", True),
    (13, 64, 1000, 1024, "bf16", "bf16", True),
    (17, 96, 512, 32, "f32", "bf16", True),
    (33, 272, 1056, 64, "bf16", "f32", False),
    (64, 130, 777, 128, "f16", "f16", True),
    (65, 513, 1100, 32, "f16", "bf16", True),
    (100, 260, 2050, 128, "f32", "f32", False),
    (129, 300, 640, 384, "bf16", "f16", True),
    (300, 129, 4096, 64, "f32", "f32", True),
    (4096, 40, 256, 32, "bf16", "bf16", False),
    # wider than a token's terms keep in registers or in LDS
    (20, 48, 8200, 32, "f32", "f32", True),
    (18, 33, 9001, 128, "bf16", "bf16", True),
    (1, 20, 12289, 128, "f32", "bf16", True),
    (1, 20, 24577, 64, "f16", "f16", False),
    # waves that share a row tile: eight, none, two; one or several slices to a
    # workgroup, ranges of slices
    (7, 7168, 3584, 32, "bf16", "f16", True),
    (7, 600, 5000, 64, "f32", "f32", True),
    (12, 9000, 1000, 64, "bf16", "bf16", True),
    (12, 9000, 2500, 32, "f16", "f16", False),
    (5, 20000, 2100, 128, "bf16", "f32", True),
    (6, 4096, 8192, 128, "bf16", "bf16", False),
    (16, 130, 8195, 32, "bf16", "f32", True),
    (12, 4000, 4096, 64, "f32", "bf16", True),
    (3, 33000, 2100, 256, "f32", "f16", True),
    # one token: eight, four, two and one wave to a row tile
    (1, 5000, 640, 128, "bf16", "f32", True),
    (1, 9000, 700, 64, "f32", "f16", False),
    (1, 17000, 300, 32, "f16", "bf16", True),
    (1, 40000, 260, 128, "f32", "bf16", True),
    # the larger matrix tile
    (300, 16384, 272, 32, "f32", "bf16", True),
    (520, 8200, 300, 128, "bf16", "f32", True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_against_the_definition(case):
    C, N, K, G, xt, st, zeros = case
    say(f"[quant] {case}")
    codes, scales, z, x, y = make(C, N, K, G, xt, st, zeros, seed=N)
    run(codes, scales, z, x, y, K, G)
    want, tol = expect(codes, scales, z, x, K, G)
    check(y, want, tol, case)


@pytest.mark.parametrize("C", [1, 6, 16, 70])
@pytest.mark.parametrize("xt", ["f32", "bf16", "f16"])
def test_slices_of_wider_tensors(C, xt):
    """Odd pitches of x and y, padded rows of codes, scales from the middle of
    a table; what is behind a row stays as it was and is not read."""
    N, K, G = 75, 333, 64
    codes, scales, z, x, y = make(C, N, K, G, xt, "f16", True, 5, 48, 3, 5)
    want, tol = expect(codes, scales, z, x, K, G)
    wide = x._base if x._base is not None else x
    wide[:, K:] = float("nan")
    run(codes, scales, z, x, y[:, :N], K, G)
    check(y[:, :N], want, tol, (C, xt))
    assert bool((y[:, N:] == 7.0).all())


@pytest.mark.parametrize("C", [1, 5, 40])
@pytest.mark.parametrize("xt", ["f32", "bf16", "f16"])
def test_accumulate(C, xt):
    N, K, G = 100, 500, 128
    codes, scales, z, x, y = make(C, N, K, G, xt, "f32", False, 6)
    old = torch.randn((C, N), device="cuda").to(T[xt])
    y.copy_(old)
    run(codes, scales, z, x, y, K, G, accumulate=True)
    want, tol = expect(codes, scales, z, x, K, G)
    want = want + old.double().cpu().numpy()
    check(y, want, tol + ref.U * np.abs(want), (C, xt))


@pytest.mark.parametrize("C", [1, 4, 16, 48])
@pytest.mark.parametrize("size", [1e-41, 1e-30, 1e4, 1e30])
def test_activations_of_any_magnitude(C, size):
    """fp32 activations far from 1, tokens of different magnitudes together."""
    N, K, G = 40, 640, 64
    codes, scales, z, x, y = make(C, N, K, G, "f32", "f32", True, 7)
    x = x * size
    x[C - 1] /= 3e5
    run(codes, scales, z, x, y, K, G)
    want, tol = expect(codes, scales, z, x, K, G)
    # subnormal sums: each rounding is off by up to half the smallest subnormal
    check(y, want, tol + (162 + K / 32) * 2.0 ** -150, (C, size), rel=size > 1e-38)


@pytest.mark.parametrize("C", [1, 3, 16, 20])
@pytest.mark.parametrize("xt", ["f32", "bf16", "f16"])
def test_infinities_and_nan_stay_in_their_token(C, xt):
    N, K, G = 64, 512, 128
    codes, scales, z, x, y = make(C, N, K, G, xt, "f32", False, 8)
    codes |= 0x11                                   # no code is 8: no weight is 0
    x[0, 100] = float("inf")
    if C > 1:
        x[1, 7] = float("nan")
    run(codes, scales, z, x, y, K, G)
    W = ref.quant_weights(codes.cpu().numpy(), scales.float().cpu().numpy(), None, K, G)
    sign = np.where(W[:, 100] > 0, np.inf, -np.inf)
    assert np.array_equal(y[0].double().cpu().numpy(), sign)
    if C > 1:
        assert bool(torch.isnan(y[1]).all())
    if C > 2:
        want, tol = expect(codes, scales, None, x[2:], K, G)
        check(y[2:], want, tol, (C, xt))


def test_constant_sign_activations_lose_nothing():
    """All activations positive: sums of q alone would be far larger than the
    result."""
    for C in (1, 8, 32):
        codes, scales, z, x, y = make(C, 128, 4096, 128, "f32", "f32", False, 9)
        x = x.abs() + 1
        run(codes, scales, z, x, y, 4096, 128)
        want, tol = expect(codes, scales, z, x, 4096, 128)
        check(y, want, tol, C)


@pytest.mark.parametrize("C", [1, 16, 64])
def test_repeats_are_identical_and_streams_are_kept(C):
    import routed_expert_fp4_amd as rf
    N, K, G = 512, 2048, 64
    codes, scales, z, x, y = make(C, N, K, G, "f32", "bf16", True, 10)
    m, ws = run(codes, scales, z, x, y, K, G)
    first = y.clone()
    side = torch.cuda.Stream()
    for _ in range(3):
        y2 = torch.full_like(y, float("nan"))
        torch.cuda.synchronize()
        rf.moe_quant_linear(m, x, C, y2, ws, stream=side)
        side.synchronize()
        assert torch.equal(first, y2)


@pytest.mark.parametrize("C", [1, 16, 64])
def test_captured_into_a_graph(C):
    import routed_expert_fp4_amd as rf
    N, K, G = 384, 1536, 32
    codes, scales, z, x, y = make(C, N, K, G, "bf16", "f16", True, 11)
    m, ws = run(codes, scales, z, x, y, K, G)
    graph = torch.cuda.CUDAGraph()
    y2 = torch.zeros_like(y)
    with torch.cuda.graph(graph):
        rf.moe_quant_linear(m, x, C, y2, ws)
    for r in range(4):
        x.copy_(torch.randn_like(x) * (r + 1))
        y2.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        rf.moe_quant_linear(m, x, C, y, ws)
        torch.cuda.synchronize()
        assert torch.equal(y, y2), r


@pytest.mark.parametrize("C", [1, 24])
def test_codes_past_four_gigabytes(C):
    """Row offsets that pass 32 bits."""
    import routed_expert_fp4_amd as rf
    N, K, G, pitch = 70000, 256, 128, 65536
    say(f"[quant] {N} rows of pitch {pitch}")
    codes = torch.empty((N, pitch), dtype=torch.uint8, device="cuda")
    codes[:, :128] = torch.randint(0, 256, (N, 128), dtype=torch.uint8, device="cuda")
    scales = torch.full((N, 2), 0.5, device="cuda")
    x = torch.randn((C, K), device="cuda")
    y = torch.zeros((C, N), device="cuda")
    m = rf.QuantMatrix(codes, scales, K, G)
    rf.moe_quant_linear(m, x, C, y, rf.QuantWorkspace(m, C, x.dtype))
    torch.cuda.synchronize()
    at = torch.tensor([0, 1, 32767, 32768, 65535, 65536, N - 2, N - 1], device="cuda")
    want, tol = expect(codes[at, :128].contiguous(), scales[at], None, x, K, G)
    check(y[:, at], want, tol, "rows")
    del codes, m
    torch.cuda.empty_cache()


def test_one_workspace_for_several_shapes():
    """Every path in turn over one workspace, twice: none leaves anything
    behind that another takes for its own."""
    import routed_expert_fp4_amd as rf
    shapes = [(16, 300, 4100, 64, "f32"), (80, 500, 1300, 128, "f32"), (1, 900, 700, 32, "bf16"),
              (5, 2000, 3000, 128, "bf16"), (33, 260, 2050, 64, "f16"), (9, 64, 9000, 32, "f16")]
    work = []
    for j, (C, N, K, G, xt) in enumerate(shapes):
        codes, scales, z, x, y = make(C, N, K, G, xt, "f16", True, 20 + j)
        m = rf.QuantMatrix(codes, scales, K, G, z)
        work.append((m, x, y, rf.QuantWorkspace(m, C, x.dtype), expect(codes, scales, z, x, K, G)))
    ws = max((w[3] for w in work), key=lambda w: w.nbytes)
    for _ in range(2):
        for (m, x, y, _, (want, tol)), shape in zip(work, shapes):
            y.fill_(float("nan"))
            rf.moe_quant_linear(m, x, x.shape[0], y, ws)
            check(y, want, tol, shape)


def test_refused_tensors():
    import routed_expert_fp4_amd as rf
    codes, scales, z, x, y = make(4, 32, 128, 64, "f32", "f32", True, 1)
    m = rf.QuantMatrix(codes, scales, 128, 64, z)
    ws = rf.QuantWorkspace(m, 4, x.dtype)
    for bad_x, bad_y in [(x[:, ::2], y), (x, y.half()), (x[:3], y), (x, y.t()), (x.t().contiguous().t(), y),
                         (x.cpu(), y), (x, y.cpu()), (x[:1].expand(4, 128), y), (x.int(), y)]:
        with pytest.raises(ValueError):
            rf.moe_quant_linear(m, bad_x, 4, bad_y, ws)
    with pytest.raises(ValueError):
        rf.QuantMatrix(codes, scales, 300, 64)                  # too few bytes a row
    with pytest.raises(ValueError):
        rf.QuantMatrix(codes, scales[:, :1], 128, 64)
    short = torch.zeros(16 * 3 + 8, dtype=torch.uint8, device="cuda").as_strided((4, 8), (16, 1))
    with pytest.raises(ValueError):
        rf.QuantMatrix(short, scales[:4], 16, 32)               # last row's 16 bytes not readable
    with pytest.raises(rf.MoeError):
        rf.QuantWorkspace(m, 4097, x.dtype)
