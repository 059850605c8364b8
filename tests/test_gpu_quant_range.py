"""moe_quant_linear where scales are very large and activations very small:
every finite result is finite, on every path, whatever the type.

Tolerance as in test_gpu_quant.
"""
import numpy as np
import pytest

from gpu_util import say
from test_gpu_quant import check, expect, make, run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def extreme(C, N, K, G, xt, st="f32", seed=3):
    """Activations near 1e-33, every third row's scales near 1e36: results from
    1e-33 to 1e6.  Raised to just below 2^15, as the matrix cores take them, the
    activations' products with these scales pass the largest fp32."""
    codes, scales, z, x, y = make(C, N, K, G, xt, st, True, seed)
    scales[::3] *= 1e38
    x *= 1e-33
    return codes, scales, z, x, y


@pytest.mark.parametrize("C,N,K", [(1, 48, 640), (1, 700, 7168), (3, 48, 640), (8, 200, 4099), (16, 48, 4100),
                                   (16, 9000, 1000), (40, 48, 640), (70, 90, 4099), (520, 4000, 300)])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("xt,st", [("f32", "f32"), ("bf16", "bf16")])
def test_large_scales_and_small_activations(C, N, K, G, xt, st):
    say(f"[quant] {C} x {N} x {K}, groups of {G}, {xt}")
    codes, scales, z, x, y = extreme(C, N, K, G, xt, st)
    want, tol = expect(codes, scales, z, x, K, G)
    assert np.abs(want).max() < 1e10                         # far inside fp32
    run(codes, scales, z, x, y, K, G)
    # rows of ordinary scales have results near 1e-33: each element has its own bound
    check(y, want, tol, (C, N, K, G, xt), rel=False)


@pytest.mark.parametrize("C", [1, 5, 16, 40])
def test_added_to_what_is_there(C):
    codes, scales, z, x, y = extreme(C, 60, 700, 64, "f32")
    old = torch.randn((C, 60), device="cuda") * 1e4
    y.copy_(old)
    run(codes, scales, z, x, y, 700, 64, accumulate=True)
    want, tol = expect(codes, scales, z, x, 700, 64)
    want = want + old.double().cpu().numpy()
    check(y, want, tol + 2.0 ** -24 * np.abs(want), C, rel=False)


@pytest.mark.parametrize("C", [2, 16, 40])
def test_beside_tokens_that_are_not_finite(C):
    """The NaN token's results are NaN, and no other token changes."""
    codes, scales, z, x, y = extreme(C, 60, 700, 64, "f32")
    x[1, 300] = float("nan")
    run(codes, scales, z, x, y, 700, 64)
    assert bool(torch.isnan(y[1]).all())
    rows = [t for t in range(C) if t != 1]
    want, tol = expect(codes, scales, z, x[rows], 700, 64)
    check(y[rows], want, tol, C, rel=False)


@pytest.mark.parametrize("C", [1, 5, 16, 40])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_results_past_the_largest_number(C, xt):
    """What no fp32 holds is infinite, with its sign."""
    codes, scales, z, x, y = make(C, 48, 300, 128, xt, "f32", False, 4)
    codes |= 0x11                                            # no weight is 0
    scales[::2] *= 1e38
    x = (x.abs() + 1) * 1e4
    codes[0::4] = 0xFF                                       # every weight 7 scales
    codes[2::4] = 0x11                                       # every weight -7 scales
    run(codes, scales, z, x, y, 300, 128)
    assert bool((y[:, 0::4] == float("inf")).all()) and bool((y[:, 2::4] == float("-inf")).all())
    want, tol = expect(codes[1::2], scales[1::2], None, x, 300, 128)
    check(y[:, 1::2], want, tol, C, rel=False)


@pytest.mark.parametrize("C", [1, 5, 16, 40, 200])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_an_infinite_scale_multiplies_its_groups_sum(C, G, xt):
    """Beside finite groups, and beside very large ones: the infinity of the
    group's sum, with its sign, and a NaN scale's row is NaN."""
    N, K = 60, 700
    codes, scales, z, x, y = make(C, N, K, G, xt, "f32", True, 5)
    scales[1::5] *= 1e38                                     # left the range without an infinity too
    x *= 1e-33
    scales[2::5, 3] = float("inf")
    scales[1::5, 2] = float("-inf")
    scales[3::5, 1] = float("nan")
    run(codes, scales, z, x, y, K, G)
    got, xd = y.double().cpu().numpy(), x.double().cpu().numpy()
    q = np.empty((N, 2 * codes.shape[1]))
    c = codes.cpu().numpy()
    q[:, 0::2], q[:, 1::2] = c & 15, c >> 4
    for first, g, sign in ((2, 3, 1.0), (1, 2, -1.0)):
        at = slice(g * G, (g + 1) * G)
        w = q[first::5, at] - z.cpu().numpy()[first::5, g:g + 1]
        sums = xd[:, at] @ w.T
        # a sum within its own roundings of zero may have either sign, or be zero
        clear = np.abs(sums) > 170 * 2.0 ** -24 * (np.abs(xd[:, at]) @ np.abs(w).T)
        assert clear.mean() > 0.9                            # of twelve rows at least eleven
        assert np.array_equal(got[:, first::5][clear], (sign * np.sign(sums) * np.inf)[clear])
        assert not np.isfinite(got[:, first::5]).any()
    assert np.isnan(got[:, 3::5]).all()
    rows = [n for n in range(N) if n % 5 not in (1, 2, 3)]
    want, tol = expect(codes[rows], scales[rows], z[rows], x, K, G)
    check(y[:, rows], want, tol, (C, G, xt), rel=False)


@pytest.mark.parametrize("C", [1, 7, 16, 40])
def test_captured_into_a_graph(C):
    import routed_expert_fp4_amd as rf
    N, K, G = 300, 2100, 64
    codes, scales, z, x, y = extreme(C, N, K, G, "f32")
    m, ws = run(codes, scales, z, x, y, K, G)
    graph, again = torch.cuda.CUDAGraph(), torch.zeros_like(y)
    with torch.cuda.graph(graph):
        rf.moe_quant_linear(m, x, C, again, ws)
    for r in range(4):
        x.copy_(torch.randn_like(x) * 1e-33)
        again.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        rf.moe_quant_linear(m, x, C, y, ws)
        torch.cuda.synchronize()
        assert torch.equal(y, again) and bool(torch.isfinite(y).all()), r
