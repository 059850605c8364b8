"""Counts, balance loss and router gradients against the plain 64-bit
definitions, through the C ABI.

Tolerances.  A share is an exponential (2 units), 1 + u, a reciprocal, a
product (1 unit each), divided by a sum of E / 64 + 6 additions, of numbers of
one sign; the exponent's own rounding adds its magnitude (the logits' range R)
in units of 2^-24 where a row is shifted by its largest: relative error at most
(E / 64 + 16 + R) 2^-24.  P adds the tokens of a slot, four waves, the slots in
16 strands and those strands: TB / 4 + slots / 16 + 24 additions, also of one
sign.  The gradient multiplies p sigmoid(-l) with g - p . g, whose two terms
carry the error of g (8 roundings) and of the dot (E / 64 + 8 additions).
"""
import numpy as np
import pytest

import load_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = ref.U


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import routed_expert_fp4_amd as rf
    rf.lib()
    torch.cuda.set_device(0)


def dev(a, dtype):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def make(C, E, k, S=1, mask=False, seed=0, scale=2.0):
    rng = np.random.default_rng(seed)
    logits = (rng.normal(0, scale, (C, E)) + rng.normal(0, 0.7, E)).astype(np.float32)
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    seq = None
    if S > 1:
        seq = np.sort(rng.integers(0, C + 1, S + 1)).astype(np.int32)
        seq[-1] = C - C // 10
        seq = np.minimum.accumulate(seq[::-1])[::-1].copy()
    m = (rng.random(C) < 0.8).astype(np.uint8) if mask else None
    return logits, idx, seq, m


def rng_of(l):
    f = l[np.isfinite(l)]
    return float(f.max() - f.min()) if f.size else 0.0


def tol_p(E, l):
    return (E / 64 + 16 + rng_of(l)) * U


def fwd(logits, idx, E, alpha, score, seq, mask, S, ws=None):
    import routed_expert_fp4_amd as rf
    C, k = idx.shape
    t = dict(logits=dev(logits, torch.float32), idx=dev(idx, torch.int32), seq=dev(seq, torch.int32),
             mask=dev(mask, torch.uint8),
             counts=torch.full((S, E), -7, dtype=torch.int32, device="cuda"),
             tokens=torch.full((S,), -7, dtype=torch.int32, device="cuda"),
             probs=torch.full((S, E), float("nan"), device="cuda"),
             loss=torch.full((1,), float("nan"), device="cuda"))
    ws = ws or rf.BalanceWorkspace(C, E, S)
    rf.moe_balance_fwd(t["logits"], t["idx"], C, E, k, alpha, t["counts"], t["tokens"], t["probs"],
                       t["loss"], ws, score=score, seq_offsets=t["seq"], S=S, token_mask=t["mask"])
    torch.cuda.synchronize()
    return t, ws


def bwd(t, C, E, k, alpha, grad, score, S, dlogits, accumulate=False):
    import routed_expert_fp4_amd as rf
    rf.moe_balance_bwd(t["logits"], t["counts"], t["tokens"], C, E, k, alpha, dev(np.array([grad]), torch.float32),
                       dlogits, score=score, seq_offsets=t["seq"], S=S, token_mask=t["mask"],
                       accumulate=accumulate)
    torch.cuda.synchronize()


def grad_tol(r, logits, alpha, grad, score, seq, mask, S, E, k):
    """Element by element: what the gradient's roundings may come to."""
    tol = np.zeros_like(r["dlogits"])
    for s, rows in enumerate(ref.sequences(logits.shape[0], seq, mask, S)):
        if not rows:
            continue
        g = abs(grad) * alpha / (S * len(rows)) * E * r["counts"][s] / (k * len(rows))
        for t in rows:
            p = ref.shares(logits[t].astype(np.float64), score)
            n = np.exp(ref.log_sigmoid(-logits[t].astype(np.float64))) if score == "sigmoid" else 1.0
            unit = 2 * tol_p(E, logits[t]) + (E / 64 + 20) * U
            tol[t] = unit * p * n * (g + p @ g) + 1e-44
    return tol


CASES = [
    # C, E, k, S, mask
    (1, 1, 1, 1, False),
    (1, 8, 2, 1, False),
    (1, 896, 16, 1, False),
    (3, 17, 5, 1, True),
    (7, 448, 16, 1, False),
    (16, 896, 16, 1, False),
    (17, 255, 8, 3, True),
    (64, 256, 8, 1, False),
    (65, 257, 32, 5, True),
    (100, 1024, 32, 1, True),
    (200, 60, 4, 40, False),
    (333, 1023, 3, 7, True),
    (1000, 100, 10, 1, True),
    (1025, 64, 6, 13, False),
    (2048, 896, 16, 1, False),
    (3001, 448, 8, 2, True),
    (17000, 36, 4, 9, True),
    (32, 100, 7, 1, True),
    (33, 100, 7, 1, True),
]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_balance_against_the_definition(case, score):
    C, E, k, S, masked = case
    say(f"[balance] {case} {score}")
    logits, idx, seq, mask = make(C, E, k, S, masked, seed=C)
    alpha, grad = 0.02, -1.7
    t, _ = fwd(logits, idx, E, alpha, score, seq, mask, S)
    r = ref.balance(logits, idx, alpha, score, seq, mask, S, grad)
    assert np.array_equal(t["counts"].cpu().numpy(), r["counts"])
    assert np.array_equal(t["tokens"].cpu().numpy(), r["tokens"])
    # tokens per slot: at least 8, at most 32 up to 16384 tokens, then 2 C / 1024
    slot = 8 if C <= 8192 else 2 * C / 1024
    tp = tol_p(E, logits) + (max(4, slot / 8) + (C / slot + S) / 16 + 24) * U
    got = t["probs"].double().cpu().numpy()
    assert (np.abs(got - r["probs"]) <= tp * r["probs"] + 1e-44).all(), np.abs(got - r["probs"]).max()
    tl = tp + (8 + 6 + S * E / 64 / 1024 + 12) * U
    assert abs(float(t["loss"]) - r["loss"]) <= tl * r["loss"] + 1e-44
    d = torch.full((C, E), 5.0, device="cuda")
    bwd(t, C, E, k, alpha, grad, score, S, d)
    got = d.double().cpu().numpy()
    inside = np.zeros(C, bool)
    inside[0 if seq is None else seq[0]: C if seq is None else seq[-1]] = True
    assert (got[~inside] == 5.0).all()
    tol = grad_tol(r, logits, alpha, grad, score, seq, mask, S, E, k)
    bad = ~(np.abs(got - r["dlogits"]) <= tol)[inside]
    assert not bad.any(), f"{bad.sum()} of {bad.size} off"
    # added to what is there: one more rounding
    base = torch.randn((C, E), device="cuda") * float(np.abs(r["dlogits"]).max() + 1e-9)
    d2 = base.clone()
    bwd(t, C, E, k, alpha, grad, score, S, d2, accumulate=True)
    want = base.double().cpu().numpy() + np.where(inside[:, None], r["dlogits"], 0)
    assert (np.abs(d2.double().cpu().numpy() - want) <= tol + U * np.abs(want) * 1.01).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_masked_and_outside_tokens_are_not_read(score):
    C, E, k, S = 90, 130, 6, 4
    logits, idx, _, mask = make(C, E, k, 1, True, seed=5)
    seq = np.array([3, 20, 20, 61, 80], np.int32)               # one is empty
    clean = ref.balance(logits, idx, 0.1, score, seq, mask, S)
    dead = np.ones(C, bool)
    for rows in ref.sequences(C, seq, mask, S):
        dead[rows] = False
    logits[dead] = np.nan
    idx[dead] = 2 ** 30
    t, _ = fwd(logits, idx, E, 0.1, score, seq, mask, S)
    assert np.array_equal(t["counts"].cpu().numpy(), clean["counts"])
    assert np.array_equal(t["tokens"].cpu().numpy(), clean["tokens"])
    assert abs(float(t["loss"]) - clean["loss"]) <= 100 * U * clean["loss"]
    d = torch.full((C, E), 5.0, device="cuda")
    bwd(t, C, E, k, 0.1, 1.0, score, S, d)
    got = d.cpu().numpy()
    assert (got[:3] == 5.0).all() and (got[80:] == 5.0).all()
    inner = dead.copy()
    inner[:3] = inner[80:] = False
    assert (got[inner] == 0.0).all() and np.isfinite(got[3:80]).all()


@pytest.mark.parametrize("C", [5, 32, 33, 700])
def test_one_sequence_by_its_offsets(C):
    """One sequence that does not begin at the first token nor end at the last."""
    E, k = 70, 6
    logits, idx, _, mask = make(C, E, k, 1, True, seed=12)
    seq = np.array([1, C - 2], np.int32)
    r = ref.balance(logits, idx, 0.1, "sigmoid", seq, mask, 1)
    t, _ = fwd(logits, idx, E, 0.1, "sigmoid", seq, mask, 1)
    assert np.array_equal(t["counts"].cpu().numpy(), r["counts"]) and int(t["tokens"]) == r["tokens"][0]
    tp = tol_p(E, logits) + (4 + (C / 8 + 1) / 16 + 24) * U
    assert (np.abs(t["probs"].double().cpu().numpy() - r["probs"]) <= tp * r["probs"] + 1e-44).all()
    assert abs(float(t["loss"]) - r["loss"]) <= (tp + 30 * U) * r["loss"] + 1e-44
    d = torch.full((C, E), 5.0, device="cuda")
    bwd(t, C, E, k, 0.1, 1.0, "sigmoid", 1, d)
    got = d.double().cpu().numpy()
    assert (got[:1] == 5.0).all() and (got[C - 2:] == 5.0).all()
    tol = grad_tol(r, logits, 0.1, 1.0, "sigmoid", seq, mask, 1, E, k)
    assert (np.abs(got - r["dlogits"]) <= tol)[1:C - 2].all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_no_token_at_all(score):
    C, E, k, S = 12, 40, 4, 3
    logits, idx, _, _ = make(C, E, k)
    for seq, mask, s in [(np.zeros(S + 1, np.int32), None, S), (None, np.zeros(C, np.uint8), 1),
                         (np.full(S + 1, C, np.int32), None, S)]:
        t, _ = fwd(logits, idx, E, 0.1, score, seq, mask, s)
        assert not t["counts"].any() and not t["tokens"].any() and not t["probs"].any()
        assert float(t["loss"]) == 0.0
        d = torch.full((C, E), 5.0, device="cuda")
        bwd(t, C, E, k, 0.1, 1.0, score, s, d)
        assert bool((d == (0.0 if seq is None else 5.0)).all())


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E", [40, 300])
def test_logits_at_the_edges(score, E):
    """Rows of -inf, of one finite logit, far below zero (every sigmoid
    underflows), far above, of mixed extremes; a NaN row spoils only itself."""
    C, k = 8, 3
    logits, idx, _, _ = make(C, E, k, seed=9)
    logits[0] = -np.inf
    logits[1] = -np.inf
    logits[1, 7] = 3.0
    logits[2] -= 2000.0
    logits[3] += 90.0
    logits[4, ::2] = -3e38
    logits[5, 1::2] = -np.inf
    logits[6] -= 70.0
    r = ref.balance(logits, idx, 0.3, score)
    t, _ = fwd(logits, idx, E, 0.3, score, None, None, 1)
    tp = (E / 64 + 16 + 2200) * U
    assert (np.abs(t["probs"].double().cpu().numpy() - r["probs"]) <= tp * r["probs"] + 1e-37).all()
    assert abs(float(t["loss"]) - r["loss"]) <= 2 * tp * r["loss"]
    d = torch.full((C, E), 5.0, device="cuda")
    bwd(t, C, E, k, 0.3, 1.0, score, 1, d)
    got = d.double().cpu().numpy()
    assert np.isfinite(got).all() and not got[0].any()
    g = 0.3 * E * r["counts"][0] / (k * C * C)
    assert (np.abs(got - r["dlogits"]) <= 3 * tp * g.max()).all()
    logits[7, 3] = np.nan
    t, _ = fwd(logits, idx, E, 0.3, score, None, None, 1)
    assert np.isnan(float(t["loss"]))
    bwd(t, C, E, k, 0.3, 1.0, score, 1, d)
    got2 = d.double().cpu().numpy()
    assert np.isnan(got2[7]).all() and np.isfinite(got2[:7]).all()


def test_gradient_against_differences_of_the_loss():
    """The library's own loss: differences along random directions."""
    C, E, k, S = 40, 64, 4, 3
    logits, idx, seq, mask = make(C, E, k, S, True, seed=2)
    rng = np.random.default_rng(1)
    for score in ("sigmoid", "softmax"):
        t, ws = fwd(logits, idx, E, 1.0, score, seq, mask, S)
        d = torch.zeros((C, E), device="cuda")
        bwd(t, C, E, k, 1.0, 1.0, score, S, d)
        for _ in range(3):
            v = rng.normal(0, 1, (C, E)).astype(np.float32)
            h = np.float32(2.0 ** -4)
            a, _ = fwd(logits + h * v, idx, E, 1.0, score, seq, mask, S, ws)
            b, _ = fwd(logits - h * v, idx, E, 1.0, score, seq, mask, S, ws)
            num = (float(a["loss"]) - float(b["loss"])) / (2 * float(h))
            want = float((d.double().cpu().numpy() * v).sum())
            # a difference of two losses near 1, each within 200 roundings, and
            # a third-order term of h^2 times the sum of shares' curvature
            assert abs(num - want) <= 200 * U * 2 / (2 * float(h)) + float(h) ** 2 * 0.5 * np.abs(d.cpu().numpy()).sum()


def test_unaligned_and_odd_rows():
    """A slice of logits that starts at any element."""
    import routed_expert_fp4_amd as rf
    for E in (63, 64, 450):
        C, k = 21, 4
        logits, idx, _, _ = make(C, E, k, seed=E)
        flat = torch.zeros(C * E + 8, device="cuda")
        r = ref.balance(logits, idx, 0.1, "sigmoid")
        for shift in (1, 2, 3):
            view = flat[shift:shift + C * E].view(C, E)
            view.copy_(torch.from_numpy(logits))
            t, ws = fwd(logits, idx, E, 0.1, "sigmoid", None, None, 1)
            t["logits"] = view
            t["loss"].zero_()
            rf.moe_balance_fwd(view, t["idx"], C, E, k, 0.1, t["counts"], t["tokens"], t["probs"], t["loss"], ws)
            assert abs(float(t["loss"]) - r["loss"]) <= 100 * U * r["loss"]
            out = torch.zeros(C * E + 8, device="cuda")
            d = out[shift:shift + C * E].view(C, E)
            bwd(t, C, E, k, 0.1, 1.0, "sigmoid", 1, d)
            tol = grad_tol(r, logits, 0.1, 1.0, "sigmoid", None, None, 1, E, k)
            assert (np.abs(d.double().cpu().numpy() - r["dlogits"]) <= tol).all()
            assert not out[:shift].any() and not out[shift + C * E:].any()
            dw = torch.randn((C, k), device="cuda")
            rf.moe_route_bwd(view, t["idx"], dw, C, E, k, d)
            rr = ref.route_grad(logits, idx, dw.double().cpu().numpy())
            assert np.abs(d.double().cpu().numpy() - rr).max() <= 200 * U * np.abs(rr).max()


def test_bad_offsets_stay_inside_the_batch():
    """Offsets outside [0, C] or falling are clipped: nothing outside the
    tensors is read or written, and every count stays within the batch."""
    C, E, k, S = 50, 33, 4, 5
    logits, idx, _, _ = make(C, E, k, seed=3)
    for seq in ([-5, 10, 900, 20, 2 ** 31 - 1, 40], [50, 40, 30, 20, 10, 0], [-2 ** 31] * 6, [7] * 6):
        t, _ = fwd(logits, idx, E, 0.1, "sigmoid", np.array(seq, np.int32), None, S)
        d = torch.zeros((C, E), device="cuda")
        bwd(t, C, E, k, 0.1, 1.0, "sigmoid", S, d)
        assert bool((t["tokens"] >= 0).all()) and bool((t["tokens"] <= C).all())
        import routed_expert_fp4_amd as rf
        cnt = torch.zeros((S, E), dtype=torch.int32, device="cuda")
        rf.moe_expert_counts(t["idx"], C, E, k, cnt, seq_offsets=t["seq"], S=S)
        assert int(cnt.max()) <= C * k


@pytest.mark.parametrize("C,E,k,S,masked", [(1, 1, 1, 1, False), (7, 448, 16, 1, False), (50, 9, 9, 6, True),
                                            (5000, 896, 16, 1, True), (9001, 100, 7, 3, False),
                                            (600, 1024, 32, 600, False)])
def test_counts(C, E, k, S, masked):
    import routed_expert_fp4_amd as rf
    say(f"[counts] {C} {E} {k} {S}")
    _, idx, seq, mask = make(C, E, k, S, masked, seed=C + 1)
    idx[0, 0] = -3
    idx[C // 2, k - 1] = E
    if k > 1:
        idx[C - 1, 1] = idx[C - 1, 0]
    want, tok = ref.counts(idx, E, seq, mask, S)
    cnt = torch.full((S, E), 9, dtype=torch.int32, device="cuda")
    tk = torch.full((S,), 9, dtype=torch.int32, device="cuda")
    i, s, m = dev(idx, torch.int32), dev(seq, torch.int32), dev(mask, torch.uint8)
    for round_ in range(3):                       # written, then added to twice
        rf.moe_expert_counts(i, C, E, k, cnt, tk, seq_offsets=s, S=S, token_mask=m, accumulate=round_ > 0)
        assert np.array_equal(cnt.cpu().numpy(), want * (round_ + 1))
        assert np.array_equal(tk.cpu().numpy(), tok * (round_ + 1))
    cnt.fill_(4)
    rf.moe_expert_counts(i, C, E, k, cnt, None, seq_offsets=s, S=S, token_mask=m)
    assert np.array_equal(cnt.cpu().numpy(), want)


@pytest.mark.parametrize("C,E,k,masked", [(1, 1, 1, False), (1, 896, 16, False), (5, 8, 8, True), (64, 448, 8, True),
                                          (33, 1023, 32, False), (301, 65, 3, True)])
def test_route_gradient(C, E, k, masked):
    import routed_expert_fp4_amd as rf
    logits, idx, _, mask = make(C, E, k, 1, masked, seed=C + 2)
    rng = np.random.default_rng(C)
    dw = rng.normal(0, 1, (C, k)).astype(np.float32)
    if k > 2:
        idx[0, 2] = idx[0, 0]                     # one expert twice
        idx[C - 1, 1] = E + 5                     # outside: skipped
    if C > 4:
        logits[1] = -np.inf                       # no weight at all
        logits[2] -= 500.0                        # every sigmoid underflows
        logits[3] += 100.0
    r = ref.route_grad(logits, idx, dw, mask)
    if mask is not None:
        logits[mask == 0] = np.nan
        idx[mask == 0] = 2 ** 30
    l, i, g, m = dev(logits, torch.float32), dev(idx, torch.int32), dev(dw, torch.float32), dev(mask, torch.uint8)
    d = torch.full((C, E), 5.0, device="cuda")
    rf.moe_route_bwd(l, i, g, C, E, k, d, token_mask=m)
    # w: 16 roundings, the shift up to 500 * 2^-24 (and the range); the dot k / 64 + 6; duplicates k
    live = logits[np.isfinite(logits)]
    unit = (2 * (40 + 4 * (np.abs(live).max() if live.size else 0)) + 2 * k) * U
    size = np.abs(dw).max(axis=1, keepdims=True) * 2
    p = np.zeros((C, E))
    for t in range(C):
        for s in range(k):
            if (mask is None or mask[t]) and 0 <= idx[t, s] < E:
                on = [idx[t, q] for q in range(k) if 0 <= idx[t, q] < E]
                w = ref.shares(logits[t, on].astype(np.float64), "sigmoid")
                neg = np.exp(ref.log_sigmoid(-logits[t, idx[t, s]].astype(np.float64)))
                p[t, idx[t, s]] += w[on.index(idx[t, s])] * neg
    tol = unit * p * size + 1e-37
    got = d.double().cpu().numpy()
    assert (np.abs(got - r) <= tol).all(), np.abs(got - r).max()
    base = torch.randn((C, E), device="cuda")
    d2 = base.clone()
    rf.moe_route_bwd(l, i, g, C, E, k, d2, token_mask=m, accumulate=True)
    want = base.double().cpu().numpy() + r
    assert (np.abs(d2.double().cpu().numpy() - want) <= tol + U * np.abs(want) * 1.01).all()
    again = torch.full((C, E), -1.0, device="cuda")
    rf.moe_route_bwd(l, i, g, C, E, k, again, token_mask=m)
    assert torch.equal(d, again)


def test_captured_into_a_graph_and_repeated():
    """Forward and both backward calls in one graph, replayed with eager work
    between; two graphs over one workspace, replayed in turn."""
    import routed_expert_fp4_amd as rf
    C, E, k, S = 300, 200, 8, 4
    logits, idx, seq, mask = make(C, E, k, S, True, seed=6)
    t, ws = fwd(logits, idx, E, 0.1, "sigmoid", seq, mask, S)
    grad, dw = torch.ones(1, device="cuda"), torch.randn((C, k), device="cuda")

    def step(o):
        rf.moe_balance_fwd(t["logits"], t["idx"], C, E, k, 0.1, o["counts"], o["tokens"], o["probs"], o["loss"],
                           ws, seq_offsets=t["seq"], S=S, token_mask=t["mask"])
        rf.moe_balance_bwd(t["logits"], o["counts"], o["tokens"], C, E, k, 0.1, grad, o["d"],
                           seq_offsets=t["seq"], S=S, token_mask=t["mask"])
        rf.moe_route_bwd(t["logits"], t["idx"], dw, C, E, k, o["d"], token_mask=t["mask"], accumulate=True)
        rf.moe_expert_counts(t["idx"], C, E, k, o["c2"], seq_offsets=t["seq"], S=S, token_mask=t["mask"])

    def outs():
        return dict(counts=torch.zeros((S, E), dtype=torch.int32, device="cuda"),
                    c2=torch.zeros((S, E), dtype=torch.int32, device="cuda"),
                    tokens=torch.zeros(S, dtype=torch.int32, device="cuda"),
                    probs=torch.zeros((S, E), device="cuda"), loss=torch.zeros(1, device="cuda"),
                    d=torch.zeros((C, E), device="cuda"))

    eager, a, b = outs(), outs(), outs()
    step(eager)
    torch.cuda.synchronize()
    graphs = []
    for o in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(o)
        graphs.append((g, o))
    for r in range(4):
        t["logits"].copy_(torch.randn((C, E), device="cuda") * (1 + r))
        step(eager)
        for g, o in graphs:
            for v in o.values():
                v.fill_(3)
            g.replay()
        torch.cuda.synchronize()
        for _, o in graphs:
            for n in eager:
                rows = slice(int(seq[0]), int(seq[-1])) if n == "d" else slice(None)
                assert torch.equal(eager[n][rows], o[n][rows]), (r, n)


def test_a_large_batch():
    """More logits than 32-bit offsets reach: 2^31 of them, tokens at both ends
    checked."""
    import routed_expert_fp4_amd as rf
    E, k = 1024, 4
    C = (1 << 20)
    say(f"[balance] {C} tokens of {E} experts")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    logits = torch.empty((C, E), device="cuda")
    for lo in range(0, C, 1 << 16):
        logits[lo:lo + (1 << 16)].normal_(0, 2, generator=g)
    idx = torch.randint(0, E, (C, k), dtype=torch.int32, device="cuda", generator=g)
    counts, tokens = torch.zeros((1, E), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    probs, loss = torch.zeros((1, E), device="cuda"), torch.zeros(1, device="cuda")
    ws = rf.BalanceWorkspace(C, E)
    rf.moe_balance_fwd(logits, idx, C, E, k, 1.0, counts, tokens, probs, loss, ws)
    assert torch.equal(counts[0].long(), torch.bincount(idx.reshape(-1).long(), minlength=E))
    c2 = torch.zeros_like(counts)
    rf.moe_expert_counts(idx, C, E, k, c2)
    assert torch.equal(counts, c2) and int(tokens) == C
    want = torch.zeros(E, dtype=torch.float64, device="cuda")
    for lo in range(0, C, 1 << 16):
        s = torch.sigmoid(logits[lo:lo + (1 << 16)].double())
        want += (s / s.sum(1, keepdim=True)).sum(0)
    want /= C
    # 1024 tokens a slot over eight waves, 1024 slots over 16 strands
    tol = (E / 64 + 16 + 24 + 128 + 64 + 24) * U
    assert float(((probs[0].double() - want).abs() / want).max()) <= tol
    d = torch.empty((C, E), device="cuda")
    rf.moe_balance_bwd(logits, counts, tokens, C, E, k, 1.0, torch.ones(1, device="cuda"), d)
    dr = torch.empty((C, E), device="cuda")
    dw = torch.randn((C, k), device="cuda", generator=g)
    rf.moe_route_bwd(logits, idx, dw, C, E, k, dr)
    for lo in (0, C // 2 - 4, C - 8):
        at = slice(lo, lo + 8)
        l = logits[at].double().cpu().numpy()
        f = E * counts[0].cpu().numpy() / (k * C)
        gg = f / C
        for j in range(8):
            p = ref.shares(l[j], "sigmoid")
            n = np.exp(ref.log_sigmoid(-l[j]))
            w = p * (gg - p @ gg) * n
            tol = (2 * tol_p(E, l[j]) + (E / 64 + 20) * U) * p * n * (gg + p @ gg) + 1e-44
            assert (np.abs(d[lo + j].double().cpu().numpy() - w) <= tol).all()
        rr = ref.route_grad(l, idx[at].cpu().numpy(), dw[at].double().cpu().numpy())
        assert np.abs(dr[at].double().cpu().numpy() - rr).max() <= 400 * U * np.abs(dw[at].cpu().numpy()).max()
    del logits, d, dr
    torch.cuda.empty_cache()


@pytest.mark.parametrize("seed", range(24))
def test_drawn_calls(seed):
    """Batches, sequences, padding and alignment drawn together: the counts by
    both entry points, the loss, and both gradients added into one tensor on
    another stream."""
    import routed_expert_fp4_amd as rf
    rng = np.random.default_rng(2000 + seed)
    C, E = int(np.exp(rng.uniform(0, np.log(3000)))), int(rng.integers(1, 1025))
    k = int(rng.integers(1, min(E, 32) + 1))
    S = int(rng.integers(1, min(C, 50) + 1))
    score, masked = str(rng.choice(["sigmoid", "softmax"])), bool(rng.random() < 0.5)
    say(f"[balance] C={C} E={E} k={k} S={S} {score} masked={masked}")
    logits, idx, seq, mask = make(C, E, k, S, masked, seed=seed)
    alpha, grad = 0.3, 0.9
    t, ws = fwd(logits, idx, E, alpha, score, seq, mask, S)
    r = ref.balance(logits, idx, alpha, score, seq, mask, S, grad)
    cnt = torch.full((S, E), 9, dtype=torch.int32, device="cuda")
    rf.moe_expert_counts(t["idx"], C, E, k, cnt, seq_offsets=t["seq"], S=S, token_mask=t["mask"])
    assert torch.equal(cnt, t["counts"])
    assert np.array_equal(t["counts"].cpu().numpy(), r["counts"])
    assert np.array_equal(t["tokens"].cpu().numpy(), r["tokens"])
    # at most 32 tokens a slot, eight waves; slots of 8 or more tokens in 16 strands
    tp = tol_p(E, logits) + (4 + (C / 8 + S) / 16 + 24) * U
    assert (np.abs(t["probs"].double().cpu().numpy() - r["probs"]) <= tp * r["probs"] + 1e-44).all()
    assert abs(float(t["loss"]) - r["loss"]) <= (tp + (26 + S * E / 64 / 1024) * U) * r["loss"] + 1e-44
    # from any element on
    off = int(rng.integers(0, 4))
    moved = torch.zeros(C * E + 4, device="cuda")[off:off + C * E].view(C, E)
    moved.copy_(t["logits"])
    d = torch.zeros(C * E + 4, device="cuda")[off:off + C * E].view(C, E)
    dw = rng.normal(0, alpha / C, (C, k)).astype(np.float32)
    dwd, one = dev(dw, torch.float32), dev(np.array([grad]), torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    rf.moe_route_bwd(moved, t["idx"], dwd, C, E, k, d, token_mask=t["mask"], stream=side)
    side.synchronize()
    first = d.clone()
    torch.cuda.synchronize()
    rf.moe_balance_bwd(moved, t["counts"], t["tokens"], C, E, k, alpha, one, d, score=score, seq_offsets=t["seq"],
                       S=S, token_mask=t["mask"], accumulate=True, stream=side)
    side.synchronize()
    route = ref.route_grad(logits, idx, dw, mask)
    size = np.abs(dw).max(axis=1, keepdims=True) * 2
    # weights and slopes of at most 1: 40 roundings, the shift by the range, the sums over k
    tol = (2 * (40 + 4 * np.abs(logits).max()) + 2 * k) * U * size
    assert (np.abs(first.double().cpu().numpy() - route) <= tol + 1e-37).all()
    inside = np.zeros(C, bool)
    inside[0 if seq is None else seq[0]: C if seq is None else seq[-1]] = True
    want = first.double().cpu().numpy() + np.where(inside[:, None], r["dlogits"], 0)
    tol = grad_tol(r, logits, alpha, grad, score, seq, mask, S, E, k) + U * np.abs(want) * 1.01
    assert (np.abs(d.double().cpu().numpy() - want) <= tol).all()


def test_most_sequences():
    """65535 sequences of none to three tokens each."""
    import routed_expert_fp4_amd as rf
    S, E, k = rf.MOE_MAX_SEQUENCES, 24, 3
    rng = np.random.default_rng(9)
    seq = np.concatenate([[0], np.cumsum(rng.integers(0, 4, S))]).astype(np.int32)
    C = int(seq[-1])
    say(f"[balance] {C} tokens in {S} sequences")
    logits, idx, _, _ = make(C, E, k, seed=9)
    t, _ = fwd(logits, idx, E, 0.7, "softmax", seq, None, S)
    owner = np.repeat(np.arange(S), np.diff(seq))
    counts = np.zeros((S, E), np.int64)
    np.add.at(counts, (owner[:, None], idx), 1)
    assert np.array_equal(t["counts"].cpu().numpy(), counts)
    n = np.diff(seq)
    assert np.array_equal(t["tokens"].cpu().numpy(), n)
    e = np.exp(logits.astype(np.float64) - logits.max(axis=1, keepdims=True))
    p = e / e.sum(axis=1, keepdims=True)
    P = np.zeros((S, E))
    np.add.at(P, owner, p)
    at = np.maximum(n, 1)[:, None]
    P /= at
    tp = tol_p(E, logits) + 28 * U
    assert (np.abs(t["probs"].double().cpu().numpy() - P) <= tp * P + 1e-44).all()
    f = E * counts / (k * at)
    loss = 0.7 / S * (f * P).sum()
    assert abs(float(t["loss"]) - loss) <= (tp + (26 + S / 1024) * U) * loss
    d = torch.full((C, E), 5.0, device="cuda")
    bwd(t, C, E, k, 0.7, 1.0, "softmax", S, d)
    g = (0.7 / S / at * f)[owner]
    want = p * (g - (p * g).sum(axis=1, keepdims=True))
    tol = (2 * tol_p(E, logits) + (E / 64 + 20) * U) * p * (g + (p * g).sum(axis=1, keepdims=True)) + 1e-44
    assert (np.abs(d.double().cpu().numpy() - want) <= tol).all()
    cnt = torch.full((S, E), 9, dtype=torch.int32, device="cuda")
    tk = torch.full((S,), 9, dtype=torch.int32, device="cuda")
    rf.moe_expert_counts(t["idx"], C, E, k, cnt, tk, seq_offsets=t["seq"], S=S)
    assert torch.equal(cnt, t["counts"]) and torch.equal(tk, t["tokens"])


@pytest.mark.parametrize("C,k,S", [(600, 16, 2), (3000, 32, 40), (40000, 16, 3), (70000, 32, 1), (20000, 32, 700)])
def test_counts_of_uneven_sequences(C, k, S):
    """Nearly all tokens in one sequence, written and added up."""
    import routed_expert_fp4_amd as rf
    E = 64
    rng = np.random.default_rng(C)
    idx = rng.integers(0, E, (C, k)).astype(np.int32)
    seq = np.sort(rng.integers(0, min(C, 2 * S), S + 1)).astype(np.int32)
    seq[0], seq[-1] = 1, C - 1
    seq = None if S == 1 else np.maximum.accumulate(seq)
    say(f"[counts] {C} {k} {S}")
    want, tok = ref.counts(idx, E, seq, None, S)
    i, s = dev(idx, torch.int32), dev(seq, torch.int32)
    cnt = torch.full((S, E), 9, dtype=torch.int32, device="cuda")
    tk = torch.full((S,), 9, dtype=torch.int32, device="cuda")
    for round_ in range(2):
        rf.moe_expert_counts(i, C, E, k, cnt, tk, seq_offsets=s, S=S, accumulate=round_ > 0)
        assert np.array_equal(cnt.cpu().numpy(), want * (round_ + 1))
        assert np.array_equal(tk.cpu().numpy(), tok * (round_ + 1))


def test_together_as_a_calibration_step_uses_them():
    """The router's logits and selection from moe_route, the counts and the
    balance loss over them, both gradients into one dlogits."""
    import routed_expert_fp4_amd as rf
    C, H, E, k = 33, 256, 64, 8
    rng = np.random.default_rng(8)
    x = dev(rng.normal(0, 1, (C, H)), torch.float32)
    Wr = dev(rng.normal(0, 0.1, (E, H)), torch.float32)
    logits = torch.empty((C, E), device="cuda")
    idx = torch.empty((C, k), dtype=torch.int32, device="cuda")
    w = torch.empty((C, k), device="cuda")
    rf.moe_route(x, Wr, logits, C, H, E, k, idx, w, rf.Workspace(E, H, 32, k, C))
    ln, ix = logits.cpu().numpy(), idx.cpu().numpy()
    t, _ = fwd(ln, ix, E, 0.05, "sigmoid", None, None, 1)
    dw = dev(rng.normal(0, 1, (C, k)), torch.float32)
    d = torch.empty((C, E), device="cuda")
    rf.moe_route_bwd(logits, idx, dw, C, E, k, d)
    bwd(t, C, E, k, 0.05, 1.0, "sigmoid", 1, d, accumulate=True)
    r = ref.balance(ln, ix, 0.05, "sigmoid")
    want = r["dlogits"] + ref.route_grad(ln, ix, dw.double().cpu().numpy())
    assert np.array_equal(t["counts"].cpu().numpy(), r["counts"])
    assert np.abs(d.double().cpu().numpy() - want).max() <= 200 * U * np.abs(want).max()


def test_refused_tensors():
    import routed_expert_fp4_amd as rf
    C, E, k = 8, 16, 2
    idx = torch.zeros((C, k), dtype=torch.int32, device="cuda")
    cnt = torch.zeros((1, E), dtype=torch.int32, device="cuda")
    for kw in (dict(counts=cnt.long()), dict(counts=cnt[:, :8]), dict(counts=cnt.cpu()),
               dict(topk_idx=idx.long()), dict(topk_idx=idx.t().contiguous().t()), dict(token_mask=cnt[0, :8].bool()),
               dict(seq_offsets=cnt[0, :3])):
        with pytest.raises(ValueError):
            rf.moe_expert_counts(**{**dict(topk_idx=idx, C=C, E=E, k=k, counts=cnt), **kw})
    with pytest.raises(rf.MoeError):
        rf.moe_expert_counts(idx, C, E, k, torch.zeros((2, E), dtype=torch.int32, device="cuda"), S=2)
    logits = torch.zeros((C, E), device="cuda")
    with pytest.raises(rf.MoeError):
        rf.moe_route_bwd(logits, idx, torch.zeros((C, k), device="cuda"), C, E, k, logits)
    with pytest.raises(ValueError):
        rf.moe_route_bwd(logits, idx, torch.zeros((C, k), device="cuda"), C, E, k, logits.half())
