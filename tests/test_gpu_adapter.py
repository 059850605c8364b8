"""moe_adapter_fwd and moe_adapter_bwd against the plain 64-bit definition, through
the C ABI.

Tolerances: a sum over n products on the matrix cores passes at most n roundings
(and a few more where waves, ranges and chunks are joined: 64 covers them), each of
2^-24 of the magnitudes summed; a factor or a piece's left-out products one more.
t's error enters y through B, u's enters dx and da, on top of their own sums.  The
result is rounded to its type once."""
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
    """Device tensors and their float64 values."""

    def __init__(self, C, K, N, n, r, xt, who="mixed", pad=0, off=0, p=0.0, base=True, scales=True, seed=0):
        import routed_expert_fp4_amd as rf
        g = np.random.default_rng(seed + C + K + N + n + r)
        self.C, self.K, self.N, self.n, self.r, self.t, self.p = C, K, N, n, r, T[xt], p
        x = g.normal(size=(C, K))
        x[:, ::37] *= 8
        self.x = device(x, self.t, pad, off)
        self.A = device(g.normal(size=(n, r, K)) / np.sqrt(K), self.t, pad, off)
        self.B = device(g.normal(size=(n, N, r)) / np.sqrt(r), self.t, off, pad)
        self.s = torch.from_numpy(g.uniform(0.5, 2, n).astype(np.float32)).cuda() if scales else None
        self.base = device(g.normal(size=(C, N)), self.t, pad, 0) if base else None
        self.dy = device(g.normal(size=(C, N)), self.t, off, pad)
        self.dbase = device(g.normal(size=(C, K)), self.t, pad, 0) if base else None
        w = {"mixed": g.integers(-1, n + 1, C), "one": np.full(C, n - 1), "none": np.full(C, -1),
             "skew": np.floor(n * g.random(C) ** 3).astype(int)}[who]
        self.who = w
        self.dev_who = torch.from_numpy(w.astype(np.int32)).cuda()
        self.y = device(np.full((C, N), np.nan), self.t, pad, off)
        self.dx = device(np.full((C, K), np.nan), self.t, pad, off)
        self.hidden = torch.full((C, r), float("nan"), device="cuda")
        self.dA = torch.full((n, r, K), float("nan"), device="cuda")
        self.dB = torch.full((n, N, r), float("nan"), device="cuda")
        seed, offset = int(g.integers(-2 ** 62, 2 ** 62)), int(g.integers(-2 ** 62, 2 ** 62))
        self.rng = torch.tensor([seed, offset], dtype=torch.int64, device="cuda")
        self.mask = ref.mask(seed, offset, C, K, p) if p else None
        self.drop = (p, self.rng) if p else None
        self.bank = rf.AdapterBank(self.A, self.B, self.s)
        self.plan = rf.AdapterPlan(self.dev_who, n)
        self.ws = rf.AdapterWorkspace(self.bank, C)
        self.ws.tensor.fill_(255)                          # NaN in every type

    def forward(self):
        import routed_expert_fp4_amd as rf
        rf.moe_adapter_fwd(self.bank, self.plan, self.x, self.C, self.y, self.ws, base=self.base, hidden=self.hidden,
                           dropout=self.drop)

    def backward(self, accumulate=False):
        import routed_expert_fp4_amd as rf
        rf.moe_adapter_bwd(self.bank, self.plan, self.x, self.hidden, self.dy, self.C, self.dx, self.dA, self.dB, self.ws,
                           base=self.dbase, dropout=self.drop, accumulate=accumulate)

    def values(self):
        s = host(self.s) if self.s is not None else np.ones(self.n)
        return host(self.x), self.who, host(self.A), host(self.B), s

    def check_forward(self, what):
        x, who, A, B, s = self.values()
        base = host(self.base) if self.base is not None else None
        y, t = ref.adapters(x, who, A, B, s, base, self.mask)
        d = self.K + 64
        tt = ref.sums(ref.adapters(np.abs(x), who, np.abs(A), np.abs(B), s, None, self.mask)[1], d)
        check(self.hidden, t, tt, d, f"{what}: hidden")
        ty = sum_over(who, np.abs(B), s, tt) + ref.sums(sum_over(who, np.abs(B), s, np.abs(t)), self.r + 64) + ref.U * np.abs(y)
        check(self.y, y, ty, d, f"{what}: y")
        assert untouched(self.y, self.y)

    def check_backward(self, what, was=None):
        x, who, A, B, s = self.values()
        dy, t = host(self.dy), host(self.hidden)
        dbase = host(self.dbase) if self.dbase is not None else None
        dx, dA, dB = ref.adapter_grads(x, who, A, B, s, dy, t, dbase, self.mask)
        ax, aA, aB = ref.adapter_grads(np.abs(x), who, np.abs(A), np.abs(B), s, np.abs(dy), np.abs(t), None, self.mask)
        d = self.N + self.r + 128
        check(self.dx, dx, ref.sums(ax, d) + ref.U * np.abs(dx), d, f"{what}: dx")
        tA, tB = ref.sums(aA, self.N + self.C + 192), ref.sums(aB, self.C + 192)
        if was is not None:
            dA, dB = dA + was[0], dB + was[1]
            tA, tB = tA + 2 * ref.U * np.abs(dA), tB + 2 * ref.U * np.abs(dB)
        check(self.dA, dA, tA, self.N + self.C + 192, f"{what}: dA")
        check(self.dB, dB, tB, self.C + 192, f"{what}: dB")
        assert untouched(self.dx, self.dx)


def sum_over(who, B, s, t):
    out = np.zeros((t.shape[0], B.shape[1]))
    for a in range(B.shape[0]):
        rows = np.flatnonzero(who == a)
        out[rows] = s[a] * (t[rows] @ B[a].T)
    return out


CASES = [
    # C, K, N, n, r, type
    (1, 1, 1, 1, 1, "f32"), (1, 64, 48, 1, 16, "bf16"), (1, 7, 130, 3, 5, "f16"), (2, 65, 128, 4, 17, "bf16"),
    (16, 512, 512, 1, 16, "f16"), (17, 513, 511, 2, 24, "f32"), (33, 1000, 300, 5, 33, "bf16"), (64, 768, 640, 24, 32, "f16"),
    (100, 2050, 129, 7, 64, "f32"), (100, 300, 2049, 7, 65, "bf16"), (40, 260, 260, 3, 128, "f16"), (40, 260, 260, 3, 127, "f32"),
    (300, 128, 96, 300, 8, "bf16"), (5, 100, 90, 1024, 3, "f32"), (1024, 200, 150, 3, 20, "f16"), (1025, 200, 150, 3, 20, "f16"),
    (1500, 333, 257, 1, 16, "bf16"), (2100, 130, 600, 4, 64, "f32"), (2500, 96, 72, 9, 100, "bf16"), (1300, 72, 200, 2, 128, "f16"),
    (1200, 3584, 100, 2, 48, "bf16"), (9000, 40, 24, 3, 8, "f32"), (1100, 64, 64, 2, 128, "f32"), (20000, 16, 16, 2, 4, "bf16"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_against_the_definition(case, p):
    say(f"[adapter] {case} {p}")
    c = Case(*case, p=p)
    c.forward()
    torch.cuda.synchronize()
    c.check_forward(case)
    c.backward()
    torch.cuda.synchronize()
    c.check_backward(case)


@pytest.mark.parametrize("who", ["one", "none", "skew"])
@pytest.mark.parametrize("C", [21, 1111])
@pytest.mark.parametrize("xt", ["f32", "bf16", "f16"])
def test_shares_of_adapters_and_slices_of_wider_tensors(who, C, xt):
    say(f"[adapter] {who} {C} {xt}")
    c = Case(C, 203, 171, 6, 12, xt, who=who, pad=3, off=1, p=0.5, base=C > 100, scales=C > 100)
    c.forward()
    torch.cuda.synchronize()
    c.check_forward(who)
    if who == "none":
        want = host(c.base) if c.base is not None else 0
        assert (host(c.y) == want).all() and (host(c.hidden) == 0).all()
    c.backward()
    torch.cuda.synchronize()
    c.check_backward(who)


def test_every_shape_of_call():
    """dx, da and db alone and together give the same bits; so do sums added to."""
    import routed_expert_fp4_amd as rf
    for C in (50, 1200):
        c = Case(C, 300, 280, 4, 16, "bf16", p=0.1)
        c.forward()
        c.backward()
        want = [v.clone() for v in (c.dx, c.dA, c.dB)]
        for has in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1), (1, 0, 1)):
            c.dx.zero_(), c.dA.zero_(), c.dB.zero_()
            rf.moe_adapter_bwd(c.bank, c.plan, c.x if has[1] else None, c.hidden if has[2] else None, c.dy, C,
                               c.dx if has[0] else None, c.dA if has[1] else None, c.dB if has[2] else None, c.ws,
                               base=c.dbase if has[0] else None, dropout=c.drop)
            for got, w, h in zip((c.dx, c.dA, c.dB), want, has):
                assert torch.equal(got, w if h else torch.zeros_like(w)), (C, has)
        was = host(c.dA), host(c.dB)
        c.dA.copy_(want[1]), c.dB.copy_(want[2])
        was = host(c.dA), host(c.dB)
        c.backward(accumulate=True)
        c.check_backward("accumulate", was)
        # in place over base, and repeated: the same bits
        y = c.y.clone()
        c.base.copy_(c.base)
        rf.moe_adapter_fwd(c.bank, c.plan, c.x, C, c.base, c.ws, base=c.base, dropout=c.drop)
        assert torch.equal(c.base, y)


def test_a_row_that_is_not_finite_stays_alone():
    for xt in ("f32", "bf16", "f16"):
        for C in (40, 1100):
            c = Case(C, 200, 150, 2, 20, xt, who="skew")
            c.forward()
            want = c.y.clone()
            c.x[3, 5] = float("inf")
            c.x[7, 150] = float("nan")
            c.forward()
            same = torch.ones(C, dtype=torch.bool)
            same[3] = same[7] = False
            assert torch.equal(c.y[same], want[same]), (xt, C)
            assert not torch.isfinite(c.y[7].float()).any() and torch.isnan(c.y[7].float()).all()
            bad = c.y[3].float()
            assert not torch.isfinite(bad).any(), (xt, C)
            # an adapter's NaN reaches its own tokens alone
            c.x[3, 5], c.x[7, 150] = 0.0, 0.0
            c.forward()
            want = c.y.clone()
            c.A[1, 0, 0] = float("nan")
            c.forward()
            mine = torch.from_numpy(c.who == 1)
            assert torch.equal(c.y[~mine], want[~mine]) and torch.isnan(c.y[mine].float()).all()


def test_an_infinity_reaches_its_own_sums_and_no_others():
    """One token, one adapter: u and the outer products are single terms.  fp32 keeps
    the infinity's sign; the 16-bit types, whose operands enter in pieces, make it an
    infinity or NaN."""
    for xt in ("f32", "bf16", "f16"):
        c = Case(1, 32, 32, 1, 1, xt, who="one", base=False, scales=False)
        c.forward()
        c.x.fill_(1.0)
        c.x[0, 3] = float("inf")
        c.A.fill_(0.5), c.B.fill_(0.25), c.dy.fill_(1.0)
        c.hidden.fill_(2.0)
        c.backward()
        d = host(c.dA)[0, 0]
        assert (np.delete(d, 3) == 8.0).all() and not np.isfinite(d[3]) and (host(c.dB) == 2).all()
        assert xt != "f32" or d[3] == np.inf
        c.hidden.fill_(-float("inf"))
        c.backward()
        assert not np.isfinite(host(c.dB)).any() and (xt != "f32" or (host(c.dB) == -np.inf).all())


def test_another_batch_on_one_plan_and_a_plan_of_another_batch():
    import routed_expert_fp4_amd as rf
    c = Case(30, 64, 64, 3, 8, "f32")
    other = Case(30, 64, 64, 3, 8, "f32", who="skew", seed=5)
    plan = c.plan
    plan.update(other.dev_who)
    other.plan = plan
    other.forward()
    torch.cuda.synchronize()
    other.check_forward("updated plan")
    with pytest.raises(ValueError):
        rf.moe_adapter_fwd(c.bank, plan, c.x[:20], 20, c.y[:20], c.ws)
    # past the binding: a plan's own sizes are what counts, and nothing is written
    small = rf.AdapterPlan(c.dev_who[:20].contiguous(), 3)
    big = torch.zeros(plan.tensor.numel(), dtype=torch.int32, device="cuda")
    big[:small.tensor.numel()] = small.tensor
    small.C, small.tensor, small.nbytes = 30, big, plan.nbytes
    c.y.fill_(5.0)
    rf.moe_adapter_fwd(c.bank, small, c.x, 30, c.y, c.ws)
    assert (host(c.y) == 5).all()


def test_workspace_of_more_tokens_and_calls_on_streams():
    import routed_expert_fp4_amd as rf
    big = Case(1200, 260, 300, 4, 16, "bf16")
    small = Case(70, 260, 300, 4, 16, "bf16", p=0.3)
    small.ws = rf.AdapterWorkspace(big.bank, 1200)
    small.ws.tensor.fill_(255)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        big.forward()
        big.backward()
    with torch.cuda.stream(s2):
        small.forward()
        small.backward()
    torch.cuda.synchronize()
    for c in (big, small):
        c.check_forward("streams")
        c.check_backward("streams")


def test_a_captured_step_replayed():
    for C in (48, 1200):
        c = Case(C, 320, 256, 4, 16, "bf16", p=0.25)
        c.forward()
        c.backward()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.plan.update(c.dev_who)
            c.forward()
            c.backward()
        for k in range(3):
            g = np.random.default_rng(k)
            c.x.copy_(torch.from_numpy(g.normal(size=(C, 320))).to(c.x))
            c.who = g.integers(-1, 5, C)
            c.dev_who.copy_(torch.from_numpy(c.who.astype(np.int32)))
            c.rng[1] = k
            c.mask = ref.mask(int(c.rng[0]), k, C, 320, 0.25)
            for v in (c.y, c.dx, c.hidden, c.dA, c.dB):
                v.fill_(9)
            graph.replay()
            torch.cuda.synchronize()
            got = [v.clone() for v in (c.y, c.hidden, c.dx, c.dA, c.dB)]
            c.plan.update(c.dev_who)
            c.forward()
            c.backward()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, (c.y, c.hidden, c.dx, c.dA, c.dB))), (C, k)
            assert (host(c.hidden[torch.from_numpy((c.who < 0) | (c.who >= 4))]) == 0).all()


def test_dropout_inside_is_dropout_outside():
    import routed_expert_fp4_amd as rf
    for xt, C in (("f32", 60), ("bf16", 1100)):
        c = Case(C, 240, 200, 3, 16, xt, p=0.5)            # a factor of 2: exact in every type
        c.forward()
        xd, y = torch.empty_like(c.x), torch.empty_like(c.y)
        rf.moe_dropout(c.x, 0.5, c.rng, xd)
        h = torch.empty_like(c.hidden)
        rf.moe_adapter_fwd(c.bank, c.plan, xd, C, y, c.ws, base=c.base, hidden=h)
        assert torch.equal(h, c.hidden) and torch.equal(y, c.y)


def test_columns_past_two_gigabytes():
    """Tokens whose rows lie far apart, and a bank whose adapters do."""
    import routed_expert_fp4_amd as rf
    C, K, N, r, pitch = 400, 64, 48, 8, 1 << 23
    x = torch.zeros((C, pitch), dtype=torch.bfloat16, device="cuda")[:, :K]
    x.copy_(torch.randn(C, K, device="cuda"))
    A = torch.zeros((3, 1 << 30), dtype=torch.bfloat16, device="cuda").as_strided((3, r, K), (1 << 30, K, 1))
    A.copy_(torch.randn(3, r, K, device="cuda"))
    B = torch.randn(3, N, r, device="cuda").bfloat16()
    who = np.arange(C) % 3
    bank = rf.AdapterBank(A, B)
    plan = rf.AdapterPlan(torch.from_numpy(who.astype(np.int32)).cuda(), 3)
    y = torch.empty((C, N), dtype=torch.bfloat16, device="cuda")
    rf.moe_adapter_fwd(bank, plan, x, C, y, rf.AdapterWorkspace(bank, C))
    want, t = ref.adapters(host(x), who, host(A), host(B), np.ones(3))
    size, _ = ref.adapters(np.abs(host(x)), who, np.abs(host(A)), np.abs(host(B)), np.ones(3))
    check(y, want, ref.sums(size, K + r + 128), K, "far rows")


def test_python_refusals():
    import routed_expert_fp4_amd as rf
    c = Case(10, 64, 48, 2, 8, "f32")
    A, B = c.A.contiguous(), c.B.contiguous()
    for args in ((A, B[:1]), (A, B.half()), (A, B[:, :, :4]), (A[0], B), (A.cpu(), B), (A, B, c.s.half()), (A, B, c.s[:1]),
                 (A.transpose(1, 2), B), (A[:0], B[:0]), (A.double(), B.double())):
        with pytest.raises((ValueError, rf.MoeError)):
            rf.AdapterBank(*args)
    with pytest.raises(rf.MoeError):
        rf.AdapterPlan(c.dev_who, 2000)
    with pytest.raises(ValueError):
        rf.AdapterPlan(c.dev_who.long(), 2)
    with pytest.raises(rf.MoeError):
        rf.AdapterWorkspace(c.bank, 0)
    big = Case(10, 64, 48, 40, 8, "f32")
    for kw in (dict(x=c.x.half()), dict(x=c.x[:9]), dict(y=c.y[:, :40]), dict(ws=None), dict(hidden=c.hidden.half()),
               dict(plan=big.plan), dict(base=c.base[:5]), dict(dropout=(0.5, c.rng.int()))):
        a = dict(dict(x=c.x, y=c.y, ws=c.ws, hidden=c.hidden, plan=c.plan, base=c.base, dropout=None), **kw)
        with pytest.raises(ValueError):
            rf.moe_adapter_fwd(c.bank, a["plan"], a["x"], 10, a["y"], a["ws"], a["base"], a["hidden"], a["dropout"])
    with pytest.raises(rf.MoeError):                       # a workspace of fewer tokens
        rf.moe_adapter_fwd(big.bank, big.plan, big.x, 10, big.y, rf.AdapterWorkspace(rf.AdapterBank(A[:1], B[:1]), 1))
    for kw in (dict(dA=c.dA[:1]), dict(dB=c.dB.half()), dict(dy=c.dy[:, 1:])):
        a = dict(dict(dA=c.dA, dB=c.dB, dy=c.dy), **kw)
        with pytest.raises(ValueError):
            rf.moe_adapter_bwd(c.bank, c.plan, c.x, c.hidden, a["dy"], 10, c.dx, a["dA"], a["dB"], c.ws)
