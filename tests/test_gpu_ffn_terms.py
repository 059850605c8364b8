"""The gated block's gradients of 16-bit tensors carry the rounding of their results
and no other that counts: dg and du enter the matrix products in two terms.

Tolerances: of a value in [2^k, 2^(k+1)) a first bf16 term leaves 2^(k-8) at most and
a second half a step of that, 2^(k-17): 2^-17 of the value.  fp16: 2^(k-11), 2^(k-23),
or, where that has no normals left, half of 2^-24; under one power of two for the call,
that puts its largest finite value at 2^14 or more, 2^-39 of that.  An activation and
its slope are some 32 fp32 roundings of their terms, and a sum of n products of two
terms each passes at most 2 n roundings of 2^-24 of the magnitudes summed (64 more
where ranges are joined)."""
import numpy as np
import pytest

import dense_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if torch is not None:
    from dense_util import T, check, device, host


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import routed_expert_fp4_amd as rf
    rf.lib()
    torch.cuda.set_device(0)


class Case:
    def __init__(self, C, H, I, xt, act="silu", dh=1.0, up=1.0, w=1.0, grad=None, seed=0):
        import routed_expert_fp4_amd as rf
        g = np.random.default_rng(seed + C + H + I)
        self.C, self.H, self.I, self.t, self.act = C, H, I, T[xt], act
        put = lambda a: device(a, self.t)  # noqa: E731
        self.x = put(g.normal(size=(C, H)))
        self.wg, self.wu = put(w * g.normal(size=(I, H)) / np.sqrt(H)), put(w * g.normal(size=(I, H)) / np.sqrt(H))
        self.gate, self.up = put(1.5 * g.normal(size=(C, I))), put(up * g.normal(size=(C, I)))
        self.dh = put(dh * np.clip(g.normal(size=(C, I)), -3, 3))      # 6e4 at dh = 2e4: finite in fp16
        new = lambda *s, t=self.t: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
        self.dx, self.dwg, self.dwu = new(C, H), new(I, H, t=grad or self.t), new(I, H, t=grad or self.t)
        self.block = rf.FfnBlock(self.wg, self.wu, act)
        self.ws = rf.FfnWorkspace(self.block, C)
        self.ws.tensor.fill_(255)

    def backward(self, accumulate=False):
        import routed_expert_fp4_amd as rf
        rf.moe_ffn_bwd(self.block, self.x, self.gate, self.up, self.dh, self.C, self.dx, self.dwg, self.dwu, self.ws,
                       accumulate=accumulate)
        torch.cuda.synchronize()

    def wanted(self):
        """{name: (value, tolerance)} in 64 bits, and dg and du."""
        x, wg, wu, dh, g, u = (host(v) for v in (self.x, self.wg, self.wu, self.dh, self.gate, self.up))
        dx, dwg, dwu, dg, du = ref.gated_grads(self.act, x, wg, wu, g, u, dh)
        most = max(np.abs(v[np.isfinite(v)]).max() for v in (dg, du))
        slope = ref.act(self.act, g)[1]
        z = 1.0 if self.act == "silu" else 2 * ref.ROOT * (1 + 3 * 0.044715 * g * g)
        e = np.abs(g) * z / (2 + 2 * np.cosh(np.minimum(np.abs(g * z), 300)))
        fp32 = 32 * ref.U
        if self.t == torch.float32:
            held = lambda v: 0.0 * v  # noqa: E731
        elif self.t == torch.bfloat16:
            held = lambda v: 2.0 ** -17 * np.abs(v)  # noqa: E731
        else:
            held = lambda v: np.maximum(2.0 ** -23 * np.abs(v), 2.0 ** -39 * most)  # noqa: E731
        tdg = held(dg) + fp32 * np.abs(dh * u) * (np.abs(slope) + 2 * e)
        tdu = held(du) + fp32 * np.abs(dh * g)
        ag, au = np.abs(dg) + tdg, np.abs(du) + tdu
        x = np.abs(x)
        tol = (tdg @ np.abs(wg) + tdu @ np.abs(wu) + ref.sums(ag @ np.abs(wg) + au @ np.abs(wu), 4 * self.I + 64),
               tdg.T @ x + ref.sums(ag.T @ x, 2 * self.C + 64), tdu.T @ x + ref.sums(au.T @ x, 2 * self.C + 64))
        return dict(zip(("dx", "dwg", "dwu"), zip((dx, dwg, dwu), tol))), dg, du

    def check(self, what, of=("dx", "dwg", "dwu")):
        want, dg, du = self.wanted()
        for k in of:
            got = getattr(self, k)
            check(got, want[k][0], want[k][1], 0, f"{what}: {k}", rel=False)
        return want, dg, du


SHAPES = [
    # C, H, I: every path of the product, and ends of rows inside a step
    (1, 1, 1), (3, 40, 31), (33, 130, 33), (40, 1000, 1), (65, 777, 129), (129, 1024, 256), (200, 520, 72), (500, 4096, 64),
    (130, 72, 3000), (300, 24604, 36), (40, 12400, 300), (257, 6300, 520), (1000, 12300, 264),
]


@pytest.mark.parametrize("xt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_every_element(shape, xt):
    say(f"[ffn terms] {shape} {xt}")
    c = Case(*shape, xt, "gelu" if shape[0] % 2 else "silu")
    c.backward()
    c.check((shape, xt))


@pytest.mark.parametrize("xt", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(96, 512, 640), (700, 328, 200), (512, 3584, 1024)])
def test_results_are_rounded_once(shape, xt):
    """The 2-norm of the errors is that of the 64-bit results' own rounding, within a
    twentieth.  (dg and du rounded to the type themselves made it 1.4 times that.)"""
    c = Case(*shape, xt)
    c.backward()
    want = c.wanted()[0]
    for k in ("dx", "dwg", "dwu"):
        w = torch.from_numpy(want[k][0])
        once = np.linalg.norm(host(w.to(c.t).cuda()) - want[k][0])
        off = np.linalg.norm(host(getattr(c, k)) - want[k][0])
        assert off <= 1.05 * once, f"{shape} {xt} {k}: {off / once:.3f} times the rounding"


@pytest.mark.parametrize("xt", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(96, 256, 160), (300, 300, 400)])
def test_gradients_in_fp32_of_16_bit_weights(shape, xt):
    c = Case(*shape, xt, grad=torch.float32)
    c.backward()
    want = c.check((shape, xt))[0]
    for k in ("dwg", "dwu"):
        w = want[k][0]
        r = np.linalg.norm(host(getattr(c, k)) - w) / np.linalg.norm(w)
        # what the terms leave, as often up as down, and fp32 sums
        assert r <= (2.0 ** -17 if xt == "bf16" else 2.0 ** -23) + ref.walk(2 * c.C + 96), f"{shape} {xt} {k}: {r:.2e}"


def test_products_beyond_the_range_of_fp16():
    """dg and du where fp16 itself would hold infinities, or zeros; the results are in
    its range (dx by small weights) or in fp32."""
    for dh, up, w in ((2e4, 300.0, 2.0 ** -12), (6e-5, 2e-4, 16.0), (1.0, 1e-6, 1.0)):
        for C in (40, 300):
            c = Case(C, 200, 96, "f16", dh=dh, up=up, w=w, grad=torch.float32)
            c.backward()
            want, dg, _ = c.check((dh, up, C))
            if dh > 1:
                assert np.abs(dg).max() > 65504 and np.abs(want["dx"][0]).max() < 60000
            elif dh < 1e-3:
                assert np.median(np.abs(dg)) < 2.0 ** -25


def test_tokens_of_very_different_gradients():
    """A token at 2^-20 of the largest keeps its bits."""
    for xt in ("bf16", "f16"):
        c = Case(64, 200, 96, xt, grad=torch.float32)
        c.dh[::2] *= 2.0 ** -10
        c.up[::2] *= 2.0 ** -10
        c.backward()
        want = c.check(xt)[0]
        w = want["dx"][0][::2]
        assert np.abs(host(c.dx)[::2] - w).max() <= 2.0 ** -8 * np.abs(w).max()


def test_a_gradient_that_is_not_finite_stays_alone():
    """An infinite or NaN dh spoils its own token's dx and its own unit's rows."""
    for xt in ("f32", "bf16", "f16"):
        for bad in (float("inf"), float("nan")):
            for C in (20, 300):
                c = Case(C, 200, 96, xt)
                c.dh[4, 7] = bad
                c.backward()
                c.dh[4, 7] = 0
                want = c.wanted()[0]
                for k, at in (("dx", 4), ("dwg", 7), ("dwu", 7)):
                    got, w, t = getattr(c, k).clone(), want[k][0], want[k][1]
                    assert not torch.isfinite(got[at].float()).any(), (xt, bad, C, k)
                    keep = np.arange(w.shape[0]) != at
                    check(got[torch.from_numpy(keep).cuda()], w[keep], t[keep], 0, f"{xt} {bad} {C} {k}", rel=False)


@pytest.mark.parametrize("xt", ["bf16", "f16", "f32"])
def test_sums_that_are_added_to(xt):
    for grad in (None, torch.float32):
        c = Case(140, 200, 96, xt, grad=grad)
        c.dx.fill_(1), c.dwg.fill_(2), c.dwu.fill_(3)
        c.backward(accumulate=True)
        want = c.wanted()[0]
        for k, was in (("dx", 1), ("dwg", 2), ("dwu", 3)):
            w = was + want[k][0]
            check(getattr(c, k), w, want[k][1] + 2 * ref.U * np.abs(w), 0, f"{xt} {grad} {k}", rel=False)


def test_each_replay_of_a_captured_call_takes_its_own_power_of_two():
    """Gradients of other sizes on every replay, eager calls on another workspace
    between them."""
    for C in (6, 300):
        c, other = Case(C, 200, 96, "f16", grad=torch.float32), Case(C, 200, 96, "f16", dh=100.0)
        c.backward()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            import routed_expert_fp4_amd as rf
            rf.moe_ffn_bwd(c.block, c.x, c.gate, c.up, c.dh, C, c.dx, c.dwg, c.dwu, c.ws)
        dh = c.dh.clone()
        for size in (1.0, 2.0 ** -10, 2.0 ** 12, 1.0, 0.0):
            c.dh.copy_(dh * size)
            for v in (c.dx, c.dwg, c.dwu):
                v.fill_(9)
            graph.replay()
            torch.cuda.synchronize()
            got = [v.clone() for v in (c.dx, c.dwg, c.dwu)]
            c.check((C, size))
            other.backward()
            c.backward()
            assert all(torch.equal(a, b) for a, b in zip(got, (c.dx, c.dwg, c.dwu)))
