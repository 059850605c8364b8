"""moe_ffn_fwd and moe_ffn_bwd against the plain 64-bit definition, through the C ABI.

Tolerances: a sum over n products on the matrix cores passes at most n roundings,
and 64 more where waves and ranges are joined, each of 2^-24 of the magnitudes
summed; an activation and its slope are some 32 fp32 roundings of their terms (the
exponential's argument, up to 88 in magnitude there, costs the most where the
result is smallest).  g's and u's errors enter h through the activation, whose slope
is below 1.13.  dg and du are rounded to the type (half a step), and so is every
result."""
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


class Case:
    def __init__(self, C, H, I, xt, act="silu", pad=0, off=0, seed=0):
        import routed_expert_fp4_amd as rf
        g = np.random.default_rng(seed + C + H + I)
        self.C, self.H, self.I, self.t, self.act = C, H, I, T[xt], act
        x = g.normal(size=(C, H))
        x[:, ::41] *= 6
        self.x = device(x, self.t, pad, off)
        self.wg = device(1.5 * g.normal(size=(I, H)) / np.sqrt(H), self.t, pad, off)
        self.wu = device(g.normal(size=(I, H)) / np.sqrt(H), self.t, off, pad)
        self.dh = device(g.normal(size=(C, I)), self.t, pad, off)
        nan = lambda *s, t=self.t: device(np.full(s, np.nan), t, off, pad)  # noqa: E731
        self.h, self.gate, self.up = nan(C, I), nan(C, I), nan(C, I)
        self.dx, self.dwg, self.dwu = nan(C, H), nan(I, H), nan(I, H)
        self.block = rf.FfnBlock(self.wg, self.wu, act)
        self.ws = rf.FfnWorkspace(self.block, C)
        self.ws.tensor.fill_(255)

    def forward(self, keep=True):
        import routed_expert_fp4_amd as rf
        rf.moe_ffn_fwd(self.block, self.x, self.C, self.h, self.ws, *((self.gate, self.up) if keep else ()))

    def backward(self, accumulate=False):
        import routed_expert_fp4_amd as rf
        rf.moe_ffn_bwd(self.block, self.x, self.gate, self.up, self.dh, self.C, self.dx, self.dwg, self.dwu, self.ws,
                       accumulate=accumulate)

    def check_forward(self, what, keep=True):
        x, wg, wu = host(self.x), host(self.wg), host(self.wu)
        h, g, u = ref.gated(self.act, x, wg, wu)
        d = self.H + 64
        tg, tu = ref.sums(np.abs(x) @ np.abs(wg).T, d), ref.sums(np.abs(x) @ np.abs(wu).T, d)
        a = np.abs(ref.act(self.act, g)[0])
        # a single h is as far off, relative to itself, as |g| roundings of g make it where
        # g is far below 0 (g = -40: 40 * 2^-24 = 2.4e-6); many together are not
        check(self.h, h, 1.13 * tg * (np.abs(u) + tu) + a * tu + 32 * ref.U * np.abs(g * u), d, f"{what}: h",
              rel=h.size >= 256)
        if keep:
            check(self.gate, g, tg, d, f"{what}: gate")
            check(self.up, u, tu, d, f"{what}: up")
        for v in (self.h, self.gate, self.up):
            assert untouched(v, v)

    def check_backward(self, what, was=None, of=("dx", "dwg", "dwu")):
        x, wg, wu, dh = host(self.x), host(self.wg), host(self.wu), host(self.dh)
        g, u = host(self.gate), host(self.up)
        want = dict(zip(("dx", "dwg", "dwu"), ref.gated_grads(self.act, x, wg, wu, g, u, dh)))
        dg, du = ref.gated_grads(self.act, x, wg, wu, g, u, dh)[3:]
        eps = torch.finfo(self.t).eps / 2
        tiny = 2 * eps * torch.finfo(self.t).smallest_normal
        a, slope = ref.act(self.act, g)
        z = 1.0 if self.act == "silu" else 2 * ref.ROOT * (1 + 3 * 0.044715 * g * g)
        e = np.abs(g) * z / (2 + 2 * np.cosh(np.minimum(np.abs(g * z), 300)))
        tdg = eps * np.abs(dg) + tiny + 32 * ref.U * np.abs(dh * u) * (np.abs(slope) + 2 * e)
        tdu = eps * np.abs(du) + tiny + 32 * ref.U * np.abs(dh) * np.abs(g)
        ax, ag, au = (np.abs(dg) + tdg) @ np.abs(wg) + (np.abs(du) + tdu) @ np.abs(wu), (np.abs(dg) + tdg).T @ np.abs(x), \
            (np.abs(du) + tdu).T @ np.abs(x)
        tol = {"dx": tdg @ np.abs(wg) + tdu @ np.abs(wu) + ref.sums(ax, 2 * self.I + 64),
               "dwg": tdg.T @ np.abs(x) + ref.sums(ag, self.C + 64), "dwu": tdu.T @ np.abs(x) + ref.sums(au, self.C + 64)}
        for k in of:
            w, t = want[k], tol[k]
            if was is not None:
                w = w + was[k]
                t = t + 2 * ref.U * np.abs(w)
            # a result of fp32 from 16-bit operands is held element by element
            check(getattr(self, k), w, t, 2 * self.I + self.C, f"{what}: {k}",
                  rel=was is None and getattr(self, k).dtype == self.t, steps=3)
            assert untouched(getattr(self, k), getattr(self, k))


CASES = [
    # C, H, I, type, activation
    (1, 1, 1, "f32", "silu"), (1, 64, 8, "bf16", "silu"), (1, 7168, 40, "bf16", "gelu"), (1, 1001, 130, "f16", "silu"),
    (2, 65, 9, "f32", "gelu"), (15, 513, 33, "bf16", "silu"), (16, 512, 100, "f16", "gelu"), (17, 511, 64, "f32", "silu"),
    (32, 4099, 17, "bf16", "silu"), (33, 128, 64, "bf16", "silu"), (33, 130, 66, "f16", "gelu"), (40, 1000, 1, "f32", "silu"),
    (64, 2048, 192, "bf16", "gelu"), (65, 777, 129, "f16", "silu"), (129, 1024, 256, "bf16", "silu"),
    (200, 520, 72, "f32", "gelu"), (300, 1001, 777, "f32", "silu"), (128, 8, 8, "f16", "silu"), (257, 64, 1000, "bf16", "gelu"),
    (500, 4096, 64, "f16", "silu"), (130, 72, 3000, "bf16", "silu"),
    # the larger tile: of the forward product, of dx, of the weights' gradients
    (300, 64, 12400, "bf16", "silu"), (290, 100, 12400, "f32", "gelu"), (300, 24600, 40, "f16", "gelu"),
    (300, 24604, 36, "f32", "silu"), (40, 12400, 300, "bf16", "silu"), (257, 6300, 520, "f16", "silu"),
    (1000, 12300, 264, "bf16", "gelu"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_against_the_definition(case):
    say(f"[ffn] {case}")
    c = Case(*case)
    c.forward()
    torch.cuda.synchronize()
    c.check_forward(case)
    c.backward()
    torch.cuda.synchronize()
    c.check_backward(case)


@pytest.mark.parametrize("C", [3, 30, 70, 300])
@pytest.mark.parametrize("xt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad, off", [(8, 0), (8, 8), (3, 1), (0, 2)])
def test_slices_of_wider_tensors(C, xt, pad, off):
    say(f"[ffn] {C} {xt} {pad} {off}")
    c = Case(C, 200, 144, xt, pad=pad, off=off)
    c.forward(keep=False)
    torch.cuda.synchronize()
    c.check_forward("slices", keep=False)
    c.forward()
    torch.cuda.synchronize()
    c.check_forward("slices")
    c.backward()
    torch.cuda.synchronize()
    c.check_backward("slices")


def test_matrices_of_different_pitches():
    """w_gate and w_up as views of wider tensors of different widths, and the gradients
    too."""
    import routed_expert_fp4_amd as rf
    for C, H, I, xt in ((5, 256, 96, "bf16"), (90, 256, 200, "f16"), (300, 512, 320, "f32"), (300, 24600, 40, "bf16")):
        c = Case(C, H, I, xt)
        for wide, name in ((64, "wu"), (40, "dwu"), (24, "x"), (88, "dx"), (16, "up")):
            setattr(c, name, device(host(getattr(c, name)), c.t, wide))
        c.block = rf.FfnBlock(c.wg, c.wu)
        c.forward()
        torch.cuda.synchronize()
        c.check_forward((C, H, I, xt))
        c.backward()
        torch.cuda.synchronize()
        c.check_backward((C, H, I, xt))


def test_every_shape_of_call():
    import routed_expert_fp4_amd as rf
    for C, H, I in ((20, 256, 96), (300, 300, 400)):
        c = Case(C, H, I, "bf16")
        c.forward()
        h = c.h.clone()
        c.forward(keep=False)
        assert torch.equal(c.h, h)
        c.backward()
        want = {k: getattr(c, k).clone() for k in ("dx", "dwg", "dwu")}
        c.dx.zero_()
        rf.moe_ffn_bwd(c.block, None, c.gate, c.up, c.dh, C, c.dx, None, None, c.ws)
        assert torch.equal(c.dx, want["dx"])
        c.dwg.zero_(), c.dwu.zero_()
        rf.moe_ffn_bwd(c.block, c.x, c.gate, c.up, c.dh, C, None, c.dwg, c.dwu, c.ws)
        assert torch.equal(c.dwg, want["dwg"]) and torch.equal(c.dwu, want["dwu"])
        # sums that are added to
        was = {k: host(v) for k, v in want.items()}
        c.backward(accumulate=True)   # dx was left as want["dx"]
        c.check_backward("accumulate", was)
        # weight gradients in fp32, written and added to
        c.dwg, c.dwu = torch.full((I, H), float("nan"), device="cuda"), torch.full((I, H), float("nan"), device="cuda")
        c.backward()
        c.check_backward("fp32", of=("dwg", "dwu"))
        was = {"dwg": host(c.dwg), "dwu": host(c.dwu)}
        c.backward(accumulate=True)
        c.check_backward("fp32 accumulate", was, of=("dwg", "dwu"))


def test_far_gates():
    """Gates where the sigmoid is 0 or 1, and where its argument leaves fp32."""
    import routed_expert_fp4_amd as rf
    for xt in ("f32", "bf16"):
        for act in ("silu", "gelu"):
            c = Case(70, 64, 64, xt, act)
            c.forward()
            v = torch.tensor([-3e38, -1e20, -200.0, -90.0, -30.0, -1e-30, 0.0, 1e-30, 30.0, 90.0, 200.0, 1e4], device="cuda")
            c.gate[:, :12] = v.to(c.t)
            c.up[:, :12] = 0.5
            c.backward()
            torch.cuda.synchronize()
            assert torch.isfinite(c.dx.float()).all() and torch.isfinite(c.dwg.float()).all()
            c.gate[:, :2] = -60.0     # the largest gradients themselves are 64-bit's to say where it can
            c.backward()
            torch.cuda.synchronize()
            c.check_backward(f"far gates {act}")


def test_a_row_that_is_not_finite_stays_alone():
    for xt in ("f32", "bf16", "f16"):
        for C, H in ((9, 200), (80, 201), (300, 200)):
            c = Case(C, H, 96, xt)
            c.forward()
            h = c.h.clone()
            c.x[4, 7] = float("nan")
            c.forward()
            same = torch.ones(C, dtype=torch.bool)
            same[4] = False
            assert torch.equal(c.h[same], h[same]) and torch.isnan(c.h[4].float()).all(), (xt, C)


def test_what_lies_behind_rows_has_no_effect():
    """Padded rows (NaN between them) give the same bits as packed ones of the same
    alignment."""
    for xt in ("bf16", "f32"):
        for C in (20, 140):
            a, b = Case(C, 256, 128, xt), Case(C, 256, 128, xt, pad=64)
            for c in (a, b):
                c.forward()
                c.backward()
            for k in ("h", "gate", "up", "dx", "dwg", "dwu"):
                assert torch.equal(getattr(a, k), getattr(b, k)), (xt, C, k)


def test_workspace_of_more_tokens_and_calls_on_streams():
    import routed_expert_fp4_amd as rf
    big, small = Case(700, 328, 200, "bf16"), Case(50, 328, 200, "bf16", "gelu")
    small.ws = rf.FfnWorkspace(small.block, 700)
    small.ws.tensor.fill_(255)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for c, s in ((big, s1), (small, s2)):
        with torch.cuda.stream(s):
            c.forward()
            c.backward()
    torch.cuda.synchronize()
    for c in (big, small):
        c.check_forward("streams")
        c.check_backward("streams")


def test_a_captured_step_replayed():
    for C in (6, 90, 400):
        c = Case(C, 256, 192, "bf16")
        c.forward()
        c.backward()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.forward()
            c.backward()
        names = ("h", "gate", "up", "dx", "dwg", "dwu")
        for k in range(3):
            g = np.random.default_rng(k)
            c.x.copy_(torch.from_numpy(g.normal(size=(C, 256))).to(c.x))
            c.dh.copy_(torch.from_numpy(g.normal(size=(C, 192))).to(c.dh))
            for n in names:
                getattr(c, n).fill_(9)
            graph.replay()
            torch.cuda.synchronize()
            got = [getattr(c, n).clone() for n in names]
            c.forward()
            c.backward()
            torch.cuda.synchronize()
            assert all(torch.equal(a, getattr(c, n)) for a, n in zip(got, names)), (C, k)


def test_tensors_past_two_gigabytes():
    import routed_expert_fp4_amd as rf
    # rows of x 16 MB apart: 300 of them pass 4 GB
    C, H, I, pitch = 300, 96, 64, 1 << 23
    c = Case(C, H, I, "bf16")
    far = torch.zeros((C, pitch), dtype=torch.bfloat16, device="cuda")[:, :H]
    far.copy_(c.x)
    c.forward()
    h = c.h.clone()
    rf.moe_ffn_fwd(c.block, far, C, c.h, c.ws)
    assert torch.equal(c.h, h)
    c.backward()
    dwg = c.dwg.clone()
    rf.moe_ffn_bwd(c.block, far, c.gate, c.up, c.dh, C, None, c.dwg, c.dwu, c.ws)
    assert torch.equal(c.dwg, dwg)


def test_python_refusals():
    import routed_expert_fp4_amd as rf
    c = Case(10, 64, 48, "bf16")
    for args in ((c.wg, c.wu[:5]), (c.wg, c.wu.half()), (c.wg, c.wu, "relu"), (c.wg[0], c.wu), (c.wg.cpu(), c.wu),
                 (c.wg.t(), c.wu.t())):
        with pytest.raises(ValueError):
            rf.FfnBlock(*args)
    with pytest.raises(rf.MoeError):
        rf.FfnWorkspace(c.block, 0)
    big = Case(300, 64, 48, "bf16")
    with pytest.raises(rf.MoeError):
        rf.moe_ffn_fwd(big.block, big.x, 300, big.h, c.ws)
    with pytest.raises(rf.MoeError):
        rf.moe_ffn_fwd(c.block, c.x, 10, c.h, c.ws, gate=c.gate)
    for args in ((c.x.half(), 10, c.h, c.ws), (c.x, 9, c.h, c.ws), (c.x, 10, c.h[:, :40], c.ws), (c.x, 10, c.h, None)):
        with pytest.raises(ValueError):
            rf.moe_ffn_fwd(c.block, *args)
    with pytest.raises(ValueError):
        rf.moe_ffn_bwd(c.block, c.x, c.gate, c.up, c.dh, 10, c.dx, c.dwg, c.dwu.float(), c.ws)
    with pytest.raises(rf.MoeError):
        rf.moe_ffn_bwd(c.block, c.x, c.gate, c.up, c.dh, 10, c.dx, c.dwg.half(), c.dwu.half(), c.ws)
    with pytest.raises(rf.MoeError):
        rf.moe_ffn_bwd(c.block, None, c.gate, c.up, c.dh, 10, c.dx, c.dwg, c.dwu, c.ws)
