"""Infinite gates, for both activations: act is infinite with slope 1 at +inf, and 0
with slope 0 at -inf.  They come of infinities in x or the weights, and in fp16 of
gates beyond 65504, which the forward pass keeps as infinities."""
import numpy as np
import pytest

from gpu_util import say
from test_gpu_ffn import Case

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import routed_expert_fp4_amd as rf
    rf.lib()
    torch.cuda.set_device(0)


# few tokens, whole tiles, and ranges of the sum that are joined
SHAPES = [(5, 200, 96), (80, 201, 96), (40, 12400, 300), (300, 64, 40)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("xt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_forward(shape, xt, act):
    say(f"[infinite gates] {shape} {xt} {act}")
    c = Case(*shape, xt, act)
    c.forward()
    h = c.h.clone()
    # one unit's gates: the sign of x decides, u is finite
    c.wg[3, 5] = INF
    c.forward()
    torch.cuda.synchronize()
    x, u, got = c.x[:, 5].float(), c.up[:, 3].float(), c.h[:, 3].float()
    assert (x != 0).all() and (u != 0).all() and torch.isfinite(u).all()
    up = x > 0
    assert torch.equal(c.gate[:, 3].float(), torch.where(up, INF, -INF))
    assert torch.equal(got[up], torch.where(u[up] > 0, INF, -INF)) and (got[~up] == 0).all()
    c.h[:, 3] = h[:, 3]
    assert torch.equal(c.h, h)
    # one token's: g and u both infinite
    c.wg[3, 5] = 0
    c.x[2, 7] = -INF
    c.forward()
    torch.cuda.synchronize()
    g, u = -c.wg[:, 7].float() * INF, -c.wu[:, 7].float() * INF
    assert torch.equal(c.gate[2].float().nan_to_num(7, INF, -INF), g.nan_to_num(7, INF, -INF))
    want = torch.where(g > 0, u, float("nan"))             # 0 times an infinity
    assert torch.equal(c.h[2].float().nan_to_num(7, INF, -INF), want.nan_to_num(7, INF, -INF))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("xt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C", [5, 300])
def test_backward(C, xt, act):
    c = Case(C, 200, 96, xt, act)
    c.forward()
    names = ("dx", "dwg", "dwu")

    def grads(gate):
        c.gate[2, 7] = gate
        c.backward()
        torch.cuda.synchronize()
        return {k: getattr(c, k).clone() for k in names}

    far, inf = grads(-6e4), grads(-INF)
    assert all(torch.isfinite(far[k].float()).all() for k in names)
    for k in names:
        assert torch.equal(far[k], inf[k]), (k, "-inf")
    far, inf = grads(100.0), grads(INF)
    # dg = dh u is finite, du infinite
    eps = torch.finfo(c.t).eps if xt == "f16" else 0.0     # the finite gate may set the call's power of two
    at = {"dx": 2, "dwg": None, "dwu": 7}
    for k in names:
        a, b = far[k].float(), inf[k].float()
        keep = torch.arange(a.shape[0], device="cuda") != (-1 if at[k] is None else at[k])
        assert torch.isfinite(b[keep]).all(), k
        assert ((a - b)[keep].abs() <= eps * a[keep].abs() + (6e-8 if eps else 0)).all(), (k, "+inf")
        if at[k] is not None:
            assert not torch.isfinite(b[at[k]]).any(), k
