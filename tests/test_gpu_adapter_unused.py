"""An adapter that no token uses: zero gradients, whatever its slot of the bank holds,
and no effect on the others."""
import numpy as np
import pytest

from test_gpu_adapter import Case

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import routed_expert_fp4_amd as rf
    rf.lib()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("xt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C, p", [(9, 0.0), (70, 0.25), (1100, 0.0)])
def test_an_unused_slot(xt, C, p):
    c = Case(C, 136, 72, 5, 9, xt, who="skew", p=p)
    who = np.where(c.who == 3, 0, c.who)
    c.dev_who.copy_(torch.from_numpy(who.astype(np.int32)))
    c.plan.update(c.dev_who)
    c.forward()
    c.backward()
    names = ("y", "hidden", "dx", "dA", "dB")
    want = [getattr(c, k).clone() for k in names]
    assert (c.dA[3] == 0).all() and (c.dB[3] == 0).all()
    for bad in (float("nan"), float("inf"), -float("inf")):
        c.A[3], c.B[3], c.s[3] = bad, bad, bad
        for k in names:
            getattr(c, k).fill_(9)
        c.forward()
        c.backward()
        torch.cuda.synchronize()
        for k, w in zip(names, want):
            assert torch.equal(getattr(c, k), w), (k, bad)
        c.dA.fill_(2), c.dB.fill_(3)
        c.backward(accumulate=True)
        torch.cuda.synchronize()
        assert (c.dA[3] == 2).all() and (c.dB[3] == 3).all(), bad
