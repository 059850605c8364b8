"""fp16 adapters whose ranks are of very different size.  t and u enter y and dx as two
fp16 terms under a power of two per token that puts its largest at 2^14 or more: the
first leaves 2^(k-11) of a value in [2^k, 2^(k+1)), the second half a step of that,
2^-23 of the value, or, where fp16 has no normals left, 2^-25 beside 2^14: 2^-39 of the
token's largest.  Where B is large against a small t that shows in y."""
import numpy as np
import pytest

import dense_ref as ref
from test_gpu_adapter import Case, sum_over

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if torch is not None:
    from dense_util import check, host


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import routed_expert_fp4_amd as rf
    rf.lib()
    torch.cuda.set_device(0)


def held(v):
    """What the two terms of values of one token (a row) may be off."""
    return np.maximum(2.0 ** -23 * np.abs(v), 2.0 ** -39 * np.abs(v).max(axis=1, keepdims=True))


@pytest.mark.parametrize("C", [7, 60, 1100])
@pytest.mark.parametrize("r", [9, 33, 70])
@pytest.mark.parametrize("span", [8, 20, 32])
def test_ranks_of_different_size(C, r, span):
    c = Case(C, 256, 200, 3, r, "f16", base=False)
    # A's rows over 2^span, B's columns the other way, so that the products are alike
    size = 2.0 ** np.round(np.linspace(span / 2 - 4, -span / 2 - 4, r))
    g = np.random.default_rng(r + span)
    put = lambda a: torch.from_numpy(a.astype(np.float32)).to(c.t).cuda()  # noqa: E731
    c.A.copy_(put(np.clip(g.normal(size=(3, r, 256)), -3, 3) * size[None, :, None]))
    c.B.copy_(put(np.clip(g.normal(size=(3, 200, r)), -3, 3) * (2.0 ** -8 / size)[None, None, :]))
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    x, who, A, B, s = c.values()
    y, t = ref.adapters(x, who, A, B, s)
    d = c.K + 64
    tt = ref.sums(ref.adapters(np.abs(x), who, np.abs(A), np.abs(B), s)[1], d) + held(t)
    check(c.y, y, sum_over(who, np.abs(B), s, tt) + ref.sums(sum_over(who, np.abs(B), s, np.abs(t)), 2 * r + 64), 0, "y",
          rel=False)
    dy, hidden = host(c.dy), host(c.hidden)
    dx = ref.adapter_grads(x, who, A, B, s, dy, hidden)[0]
    tol = np.zeros_like(dx)
    for a in range(3):
        rows = np.flatnonzero(who == a)
        u = s[a] * (dy[rows] @ B[a])
        mag = s[a] * (np.abs(dy[rows]) @ np.abs(B[a]))
        tol[rows] = (ref.sums(mag, c.N + 64) + (held(u) if len(rows) else 0)) @ np.abs(A[a]) \
            + ref.sums(np.abs(u) @ np.abs(A[a]), 2 * r + 64)
    check(c.dx, dx, tol, 0, "dx", rel=False)
    # the gradients' terms: 2^-22 of a product is the most that what is left out can be
    dA, dB = ref.adapter_grads(x, who, A, B, s, dy, hidden)[1:]
    aA, aB = ref.adapter_grads(np.abs(x), who, np.abs(A), np.abs(B), s, np.abs(dy), np.abs(hidden))[1:]
    check(c.dA, dA, ref.sums(aA, c.N + C + 192) + 2.0 ** -22 * aA, 0, "dA", rel=False)
    check(c.dB, dB, ref.sums(aB, C + 192) + 2.0 ** -22 * aB, 0, "dB", rel=False)
