"""moe_dropout against its definition, through the C ABI.  The mask is equal; a
kept value is multiplied by a factor rounded once, the product and the sum with
base round once each in fp32 (3 roundings of 2^-24 of the terms), and the result is
rounded to its type."""
import numpy as np
import pytest

import dense_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if torch is not None:
    from dense_util import T, check, device, host, untouched


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import routed_expert_fp4_amd as rf
    rf.lib()
    torch.cuda.set_device(0)


def rng_of(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("C, K, p, xt, pad, off", [
    (1, 1, 0.5, "f32", 0, 0), (1, 8, 0.0, "bf16", 0, 0), (3, 7, 1.0, "f16", 1, 3), (5, 9, 0.1, "bf16", 0, 1),
    (17, 1000, 0.9, "f32", 3, 1), (64, 4099, 0.05, "f16", 5, 0), (300, 3584, 0.1, "bf16", 0, 0), (2000, 77, 0.3, "f32", 0, 0),
    (2, 131072, 0.5, "f16", 0, 0), (5, 40, 1e-6, "f32", 0, 0), (5, 40, 2 ** -16, "f32", 0, 0), (40000, 3, 0.5, "bf16", 2, 1)])
@pytest.mark.parametrize("with_base", [False, True])
def test_against_the_definition(C, K, p, xt, pad, off, with_base):
    import routed_expert_fp4_amd as rf
    say(f"[dropout] {C} {K} {p} {xt} {pad} {off} {with_base}")
    g = np.random.default_rng(C + K)
    x, y = device(g.normal(size=(C, K)), T[xt], pad, off), device(np.full((C, K), np.nan), T[xt], pad + 1, off)
    base = device(g.normal(size=(C, K)), T[xt], off, pad) if with_base else None
    seed, offset = int(g.integers(-2 ** 62, 2 ** 62)), int(g.integers(-2 ** 62, 2 ** 62))
    rf.moe_dropout(x, p, rng_of(seed, offset), y, base=base)
    torch.cuda.synchronize()
    m = ref.mask(seed, offset, C, K, p)
    kept = host(x) * m
    want = kept + (host(base) if with_base else 0)
    check(y, want, 3 * ref.U * (np.abs(kept) + np.abs(want)), 3, "y")
    if not with_base and p < 1:
        assert ((host(y) == 0) == (kept == 0)).all()
    assert untouched(y, y)


def test_dropped_infinities_and_places():
    import routed_expert_fp4_amd as rf
    C, K = 9, 333
    x = torch.full((C, K), float("inf"), device="cuda")
    x[::2] = float("nan")
    m = ref.mask(7, 8, C, K, 0.6)
    y = torch.empty_like(x)
    rf.moe_dropout(x, 0.6, rng_of(7, 8), y)
    got = host(y)
    assert (got[m == 0] == 0).all() and np.isinf(got[1::2][m[1::2] > 0]).all() and np.isnan(got[::2][m[::2] > 0]).all()
    # in place, over x and over base
    a = torch.randn(C, K, device="cuda")
    want = torch.empty_like(a)
    rf.moe_dropout(a, 0.6, rng_of(7, 8), want, base=a)
    rf.moe_dropout(a, 0.6, rng_of(7, 8), a, base=a)
    assert torch.equal(a, want)


def test_the_backward_pass_is_the_same_call():
    import routed_expert_fp4_amd as rf
    C, K, p = 33, 520, 0.25
    x, dy = torch.randn(C, K, device="cuda"), torch.randn(C, K, device="cuda")
    r, dx = rng_of(-3, 1 << 40), torch.empty(C, K, device="cuda")
    rf.moe_dropout(dy, p, r, dx)
    # against differences of sum(dy * dropout(x)): the function is linear
    y0, y1, e = torch.empty_like(x), torch.empty_like(x), torch.randn(C, K, device="cuda")
    rf.moe_dropout(x, p, r, y0)
    rf.moe_dropout(x + e, p, r, y1)
    lhs = ((y1.double() - y0.double()) * dy.double()).sum()
    rhs = (dx.double() * e.double()).sum()
    size = (dx.double().abs() * (x.double().abs() + e.double().abs())).sum()
    assert abs(lhs - rhs) <= 8 * ref.U * size


def test_captured_calls_take_the_offset_at_replay():
    import routed_expert_fp4_amd as rf
    C, K, p = 70, 640, 0.5
    x, y, r = torch.randn(C, K, device="cuda"), torch.empty(C, K, device="cuda"), rng_of(1, 0)
    rf.moe_dropout(x, p, r, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rf.moe_dropout(x, p, r, y)
    for offset in (5, 6, 5):
        r[1] = offset
        y.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(y)
        rf.moe_dropout(x, p, r, want)
        assert torch.equal(y, want)
        assert ((host(y) == 0) == (ref.mask(1, offset, C, K, p) == 0)).all()


def test_rows_past_two_gigabytes():
    import routed_expert_fp4_amd as rf
    C, K = 40000, 32768
    x = torch.ones((C, K), dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    rf.moe_dropout(x, 0.5, rng_of(9, 9), y)
    torch.cuda.synchronize()
    for c in (0, 32767, 32768, C - 1):
        row = host(y[c])
        w = ref.philox((9, 0), (np.full(K // 8, 9, np.uint64), np.zeros(K // 8, np.uint64), np.arange(K // 8, dtype=np.uint64),
                                np.full(K // 8, c, np.uint64)))
        h = np.stack([v >> np.uint64(s) & np.uint64(0xFFFF) for v in w for s in (0, 16)], axis=1).reshape(-1)
        assert (row == np.where(h >= 32768, 2.0, 0.0)).all()


def test_python_refusals():
    import routed_expert_fp4_amd as rf
    x, r = torch.randn(4, 16, device="cuda"), rng_of(1, 2)
    y = torch.empty_like(x)
    for args in ((x[0], 0.5, r, y), (x, 0.5, r.int(), y), (x, 0.5, r[:1], y), (x, 0.5, r, y.half()), (x, 0.5, r, y[:3]),
                 (x, 0.5, r, y.t().contiguous().t()), (x.cpu(), 0.5, r, y), (x.double(), 0.5, r, y)):
        with pytest.raises(ValueError):
            rf.moe_dropout(*args)
    for args in ((x, 0.5, None, y), (x, -1.0, r, y), (x, 1.5, r, y), (x[:2], 0.5, r, x[1:3])):
        with pytest.raises(rf.MoeError):
            rf.moe_dropout(*args)
