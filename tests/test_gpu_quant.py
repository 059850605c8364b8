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
    (20, 40, 16500, 64, "f32", "f32", True),
    (19, 30, 17001, 128, "bf16", "bf16", False),
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


@pytest.mark.parametrize("C", [1, 5, 40, 70])
@pytest.mark.parametrize("K,G", [(33, 32), (65, 64), (200, 64), (300, 128)])
def test_infinite_scales_stay_in_their_row(C, K, G):
    """A row whose last, partial group has an infinite scale: its results are
    infinite (NaN where the group's sum is 0), and no other row changes."""
    codes, scales, z, x, y = make(C, 50, K, G, "f32", "f32", False, 51)
    codes |= 0x11                                   # no code is 8: no weight is 0
    x[:, K // G * G:] = x[:, K // G * G:].abs() + 1
    codes[7] = 0xFF                                 # every weight 7 scales
    scales[7, -1] = float("inf")
    scales[9, 0] = float("nan")
    run(codes, scales, z, x, y, K, G)
    assert bool((y[:, 7] == float("inf")).all()) and bool(torch.isnan(y[:, 9]).all())
    rows = [n for n in range(50) if n not in (7, 9)]
    want, tol = expect(codes[rows], scales[rows], None, x, K, G)
    check(y[:, rows], want, tol, (C, K, G))


@pytest.mark.parametrize("C", [1, 7, 16, 50])
@pytest.mark.parametrize("G", [32, 64, 128])
def test_every_zero_point(C, G):
    """Zero points are bytes: all 256 of them, not the codes' range alone."""
    N, K = 64, 1000
    codes, scales, z, x, y = make(C, N, K, G, "f32", "f16", True, 52)
    z.copy_((torch.arange(z.numel(), device="cuda") % 256).to(torch.uint8).view(z.shape))
    run(codes, scales, z, x, y, K, G)
    want, tol = expect(codes, scales, z, x, K, G)
    check(y, want, tol, (C, G), rel=False)


@pytest.mark.parametrize("C", [1, 9, 40])
def test_two_streams_at_once(C):
    """Calls that overlap, each stream with a workspace of its own."""
    import routed_expert_fp4_amd as rf
    codes, scales, z, x, y = make(C, 2000, 4000, 128, "f32", "bf16", True, 53)
    m, _ = run(codes, scales, z, x, y, 4000, 128)
    lanes = []
    for _ in range(3):
        lanes.append((torch.cuda.Stream(), torch.zeros_like(y), rf.QuantWorkspace(m, C, x.dtype)))
    torch.cuda.synchronize()
    for _ in range(10):
        for stream, out, ws in lanes:
            rf.moe_quant_linear(m, x, C, out, ws, stream=stream)
    torch.cuda.synchronize()
    for _, out, _ in lanes:
        assert torch.equal(out, y)


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


def test_largest_matrix_and_row():
    """The most rows a matrix may have, and the most columns."""
    import routed_expert_fp4_amd as rf
    N, K = rf.MOE_MAX_QUANT_ROWS, 40
    for C in (1, 2, 18):
        say(f"[quant] {N} rows, {C} tokens")
        codes, scales, z, x, y = make(C, 64, K, 32, "bf16", "bf16", True, 30)
        copies = N // 64
        many = [t.repeat(copies, 1) for t in (codes, scales, z)]
        y = torch.full((C, N), float("nan"), dtype=x.dtype, device="cuda")
        run(*many, x, y, K, 32)
        want, tol = expect(codes, scales, z, x, K, 32)
        check(y[:, :64], want, tol, C)
        assert bool((y.reshape(C, copies, 64) == y[:, None, :64]).all())
    K = rf.MOE_MAX_QUANT_COLS
    for C, xt in ((1, "f32"), (9, "bf16"), (33, "f16")):
        say(f"[quant] {K} columns, {C} tokens")
        codes, scales, z, x, y = make(C, 37, K, 64, xt, "f32", True, 31)
        run(codes, scales, z, x, y, K, 64)
        want, tol = expect(codes, scales, z, x, K, 64)
        check(y, want, tol, C, rel=False)


@pytest.mark.parametrize("C", [3, 21])
def test_largest_pitches(C):
    """Rows of x and y 2^24 elements apart, rows of codes, scales and zero
    points 2^22."""
    N, K, G = 20, 200, 64
    codes, scales, z, x, y = make(C, N, K, G, "f32", "f32", True, 32)
    want, tol = expect(codes, scales, z, x, K, G)

    def spread(t, pitch):
        behind = float("nan") if t.is_floating_point() else 255
        wide = torch.full((t.shape[0], pitch), behind, dtype=t.dtype, device="cuda")[:, :t.shape[1]]
        wide.copy_(t)
        return wide

    codes, scales, z = (spread(t, 1 << 22) for t in (codes, scales, z))
    x, y = spread(x, 1 << 24), spread(y, 1 << 24)
    run(codes, scales, z, x, y, K, G)
    check(y, want, tol, C)
    torch.cuda.empty_cache()


def test_scales_past_two_gigabytes_of_a_workgroup():
    """The larger matrix tile's 256 rows of fp32 scales, 2^22 elements apart."""
    C, N, K, G = 4096, 512, 160, 32
    codes, scales, z, x, y = make(C, N, K, G, "f32", "f32", False, 33)
    # what lies between the rows of scales is no number
    wide = torch.full((N, 1 << 22), float("nan"), device="cuda")[:, :scales.shape[1]]
    wide.copy_(scales)
    run(codes, wide, z, x, y, K, G)
    at = torch.arange(0, C, 97)
    want, tol = expect(codes, scales, z, x[at], K, G)
    check(y[at], want, tol, "wide")
    del wide
    torch.cuda.empty_cache()


@pytest.mark.parametrize("seed", range(48))
def test_drawn_calls(seed):
    """Sizes, types, pitches, alignments and accumulation drawn together."""
    rng = np.random.default_rng(1000 + seed)
    C = int(rng.choice([1, 2, 4, 8, 11, 16, 17, 40, 64, 100, 200, 600]))
    N, K = int(rng.integers(1, 1200)), int(rng.integers(1, 5000))
    if rng.random() < 0.4:
        K = max(32, K // 128 * 128)
    G = int(rng.choice([32, 64, 128, 256, 640]))
    xt, st = (str(rng.choice(["f32", "bf16", "f16"])) for _ in range(2))
    zeros, acc = bool(rng.random() < 0.5), bool(rng.random() < 0.3)
    pads = [int(rng.choice([0, 0, 1, 3, 8])) for _ in range(2)]
    say(f"[quant] C={C} N={N} K={K} G={G} x={xt} scales={st} zeros={zeros} accumulate={acc} pads={pads}")
    codes, scales, z, x, y = make(C, N, K, G, xt, st, zeros, seed, 16 * int(rng.integers(0, 3)), *pads)
    shift = int(rng.integers(0, 4))                 # x from any element on
    flat = torch.zeros(x.numel() + C * pads[0] + 8, dtype=x.dtype, device="cuda")
    moved = flat[shift:].as_strided(x.shape, (K + pads[0], 1), shift)
    moved.copy_(x)
    y.copy_(torch.randn(y.shape, device="cuda"))
    old, part = y.clone(), y[:, :N]
    run(codes, scales, z, moved, part, K, G, accumulate=acc)
    want, tol = expect(codes, scales, z, x, K, G)
    if acc:
        want = want + old[:, :N].double().cpu().numpy()
        tol = tol + ref.U * np.abs(want)
    check(part, want, tol, seed, rel=False)
    assert torch.equal(y[:, N:], old[:, N:])


@pytest.mark.parametrize("C", [1, 12, 40])
def test_two_graphs_share_a_workspace(C):
    """Two captured calls of different shapes over one workspace, replayed in
    turn with eager calls between them."""
    import routed_expert_fp4_amd as rf
    calls = []
    for j, (N, K, G) in enumerate(((300, 4100, 64), (700, 1300, 128))):
        codes, scales, z, x, y = make(C, N, K, G, "f32", "f16", True, 40 + j)
        m = rf.QuantMatrix(codes, scales, K, G, z)
        calls.append([m, x, y, expect(codes, scales, z, x, K, G)])
    ws = max((rf.QuantWorkspace(m, C, x.dtype) for m, x, _, _ in calls), key=lambda w: w.nbytes)
    for call in calls:
        m, x, y, _ = call
        rf.moe_quant_linear(m, x, C, y, ws)
        torch.cuda.synchronize()
        call.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(call[4]):
            rf.moe_quant_linear(m, x, C, y, ws)
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for j in order:
            m, x, y, (want, tol), graph = calls[j]
            y.fill_(float("nan"))
            graph.replay()
            check(y, want, tol, (C, order, j))
            y.fill_(float("nan"))
            rf.moe_quant_linear(m, x, C, y, ws)
            check(y, want, tol, (C, order, j))


@pytest.mark.parametrize("C", [1, 5, 16])
def test_together_as_a_latent_layer(C):
    """A latent layer whose dense steps are held in 4 bits: router, routed_down
    by the dense product, routed experts, RMS norm, routed_up by the dense
    product onto the shared experts' sum; against moe_latent_layer_fwd with the
    same weights in bf16 (integers times powers of two: exact) and the oracle.
    Bars as for the layer itself, whose experts both share."""
    import oracle
    import routed_expert_fp4_amd as rf
    import synth
    from gpu_util import assert_close, cached_bank, to_dev
    oracle.build()
    wl = synth.LatentWorkload("lat_quant", synth.FMT_MX, 64, 8, 1024, 512, 512, 2, 1024, C, gamma_scale=2.0 ** 17)
    Wr, x, _, _, gamma = synth.latent_inputs(wl, 0, C=C)
    rng = np.random.default_rng(50)
    mats, bits = [], []
    for N, K, G in ((wl.L, wl.H, 128), (wl.H, wl.L, 32)):
        codes = rng.integers(0, 256, (N, K // 2), np.uint8)
        scales = np.ldexp(1.0, rng.integers(-9, -6, (N, K // G))).astype(np.float32)
        zeros = rng.integers(6, 10, (N, K // G), np.uint8)
        W = ref.quant_weights(codes, scales, zeros, K, G).astype(np.float32)
        b = W.view(np.uint32)
        assert not (b & 0xFFFF).any()
        bits.append((b >> 16).astype(np.uint16))
        mats.append(rf.QuantMatrix(to_dev(codes), to_dev(scales), K, G, to_dev(zeros)))
    routed, shared = cached_bank(wl.routed_bank()), cached_bank(wl.shared_bank())
    gd, xd, wd = to_dev(gamma), to_dev(x), to_dev(Wr)

    layer = rf.LatentLayer(wd, to_dev(bits[0].view(np.int16)), gd, wl.eps, to_dev(bits[1].view(np.int16)),
                           routed, shared)
    whole = torch.empty((C, wl.H), device="cuda")
    chosen = torch.empty((C, wl.k), dtype=torch.int32, device="cuda")
    rf.moe_latent_layer_fwd(layer, xd, C, wl.k, whole, chosen, None, rf.LatentWorkspace(layer, wl.k, C))

    logits = torch.empty((C, wl.E), device="cuda")
    idx, w = torch.empty_like(chosen), torch.empty((C, wl.k), device="cuda")
    rf.moe_route(xd, wd, logits, C, wl.H, wl.E, wl.k, idx, w, rf.Workspace(wl.E, wl.H, 512, wl.k, C))
    lat, mixed = torch.empty((C, wl.L), device="cuda"), torch.empty((C, wl.L), device="cuda")
    out = torch.empty((C, wl.H), device="cuda")
    ws = max((rf.QuantWorkspace(m, C, torch.float32) for m in mats), key=lambda s: s.nbytes)
    rf.moe_quant_linear(mats[0], xd, C, lat, ws)
    rf.moe_expert_fwd(routed, lat, C, wl.k, idx, w, mixed, rf.Workspace(routed.E, wl.L, routed.I, wl.k, C))
    normed = gd * mixed / torch.sqrt((mixed * mixed).mean(dim=1, keepdim=True) + wl.eps)
    every = torch.arange(shared.E, dtype=torch.int32, device="cuda").repeat(C, 1)
    rf.moe_expert_fwd(shared, xd, C, shared.E, every, torch.ones((C, shared.E), device="cuda"), out,
                      rf.Workspace(shared.E, wl.H, shared.I, shared.E, C))
    before = out.clone()
    rf.moe_quant_linear(mats[1], normed.contiguous(), C, out, ws, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(idx, chosen)
    assert float((out - before).norm()) > 0.1 * float(before.norm())     # the routed part counts
    assert_close(out.cpu().numpy(), whole.cpu().numpy(), f"against the bf16 layer, C={C}")
    want = oracle.latent_layer(wl, Wr, x, bits[0], bits[1], gamma, idx=idx.cpu().numpy())
    assert_close(out.cpu().numpy(), want["out"], f"against the oracle, C={C}")


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
