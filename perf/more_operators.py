"""Measured cases of the adapter, gated-block and dropout operators.

Three operators and their gradients: low-rank adapters of many requests beside a
shared projection (moe_adapter_fwd, moe_adapter_bwd), the gated feed-forward
block in 16- and 32-bit weights (moe_ffn_fwd, moe_ffn_bwd) and dropout whose
mask is formed anew from a counter wherever it is needed (moe_dropout, and
inside the adapters' training calls).  `own` chooses between their plain form,
written in elementary torch operations, and the library's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _adapter(C, K, N, n, r, x, idle=False, pad=0):
    """y = base + s B (A x) for C tokens of requests that use n adapters of rank
    r beside a projection from K to N; `idle`: some tokens have no adapter;
    `pad`: unused elements behind each row of x and of y."""
    return {"op": "adapter", "C": C, "K": K, "N": N, "n": n, "r": r, "x": x, "idle": idle, "pad": pad}


def _tune(C, K, N, n, r, x, p):
    """The same forward with dropout p of its input, and all of its gradients."""
    return {"op": "tune", "C": C, "K": K, "N": N, "n": n, "r": r, "x": x, "p": p}


def _ffn(op, C, H, I, x, act="silu"):
    """h = act(x Wg^T) * (x Wu^T) for C tokens ("ffn"), or its gradients from
    what the forward pass kept ("ffn_bwd")."""
    return {"op": op, "C": C, "H": H, "I": I, "x": x, "act": act}


def _dropout(C, K, x, p):
    """y = base + dropout(x)."""
    return {"op": "dropout", "C": C, "K": K, "x": x, "p": p}


def listed():
    return [
        # one decoded token beside routed_down: launch latency
        dict(_adapter(1, 7168, 3584, 8, 16, "bf16"), name="adapter, one token"),
        # a decode batch of many requests beside routed_up, some without adapter
        dict(_adapter(64, 3584, 7168, 24, 32, "f16", True), name="adapters, decode batch"),
        # odd sizes, rows of a wider tensor, fp32 activations
        dict(_adapter(333, 4099, 1001, 5, 24, "f32", True, 5), name="adapters, odd sizes"),
        # a prefill chunk of several requests
        dict(_adapter(4096, 7168, 3584, 8, 64, "bf16"), name="adapters, chunk"),
        # a fine-tuning step of one adapter beside a frozen projection
        dict(_tune(2048, 7168, 3584, 1, 16, "bf16", 0.05), name="tune, one adapter"),
        # several adapters trained in one packed batch
        dict(_tune(8192, 3584, 7168, 4, 64, "f16", 0.1), name="tune, packed"),
        # a shared expert's width, one decoded token: the weights' stream
        dict(_ffn("ffn", 1, 7168, 1536, "bf16"), name="gated block, one token"),
        # the same block over a prefill chunk: the compute-bound end
        dict(_ffn("ffn", 2048, 7168, 4096, "bf16"), name="gated block, chunk"),
        # its gradients for a training batch: the largest
        dict(_ffn("ffn_bwd", 4096, 7168, 4096, "bf16"), name="gated block, backward"),
        # odd sizes, fp32, the other activation
        dict(_ffn("ffn_bwd", 300, 1001, 777, "f32", "gelu"), name="gated block, backward odd"),
        # the residual of a few tokens: launch latency
        dict(_dropout(7, 3584, "f32", 0.1), name="dropout, seven tokens"),
        # the residual stream of a training batch
        dict(_dropout(16384, 7168, "bf16", 0.1), name="dropout, 16k tokens"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _width(rng, lo, hi):
    """A row's length: half of them multiples of 64, the others as they come."""
    v = _log(rng, lo, hi)
    return max(64, v // 64 * 64) if rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["adapter", "adapter", "tune", "ffn", "ffn_bwd", "dropout"])
    x = rng.choice(["f32", "bf16", "f16"])
    if op in ("adapter", "tune"):
        K, N = _width(rng, 48, 7168), _width(rng, 48, 7168)
        n, r = _log(rng, 1, 48), rng.choice([4, 8, 16, 24, 32, 64, rng.randint(1, 64)])
        C = _log(rng, 1, 4096 if op == "adapter" else 8192)
        if op == "tune":
            return _tune(C, K, N, min(n, 8), r, x, rng.choice([0.0, 0.05, 0.1, 0.5]))
        return _adapter(C, K, N, n, r, x, rng.random() < 0.5, rng.choice([0, 0, 3, 8]))
    if op == "dropout":
        K = _width(rng, 16, 16384)
        return _dropout(_log(rng, 1, max(1, 16384 * 3584 // K)), K, x, rng.choice([0.0, 0.05, 0.1, 0.5, 0.9]))
    # fp32 runs at a sixteenth of the 16-bit types' rate
    most = 2048 * 4096 * (1 if x == "f32" else 7)
    H, I = _width(rng, 64, 7168), _width(rng, 64, 4096)
    C = _log(rng, 1, max(1, min(4096, most * 1024 // (H * I))))
    return _ffn(op, C, H, I, x, rng.choice(["silu", "silu", "gelu"]))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _activations(g, C, K, t, pad=0):
    """Hidden states: a few channels are much larger than the others."""
    x = torch.randn((C, K + pad), generator=g, device="cuda")
    x *= 1 + 7 * (torch.rand((K + pad,), generator=g, device="cuda") < 0.004)
    return x.to(t)[:, :K]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    state = {"case": case}
    t, C = DTYPES[case["x"]], case["C"]

    def normal(*shape, scale=1.0, t=t):
        return (scale * torch.randn(shape, generator=g, device=dev)).to(t)

    if "p" in case:
        # a seed and an offset, on the device as a training loop keeps them
        state["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device=dev, dtype=torch.int64)
    if case["op"] in ("adapter", "tune"):
        K, N, n, r, pad = case["K"], case["N"], case["n"], case["r"], case.get("pad", 0)
        state["x"] = _activations(g, C, K, t, pad)
        state["A"] = normal(n, r, K, scale=K ** -0.5)
        state["B"] = normal(n, N, r, scale=r ** -0.5)
        state["scales"] = 0.5 + torch.rand((n,), generator=g, device=dev)
        # every adapter is used where there are tokens enough, some by far more
        # tokens than others, and requests' tokens lie anywhere in the batch
        who = torch.floor(n * torch.rand((C,), generator=g, device=dev) ** 2).to(torch.int32)
        order = torch.randperm(C, generator=g, device=dev)
        who[order[:min(n, C)]] = torch.arange(min(n, C), dtype=torch.int32, device=dev)
        if case.get("idle"):
            who[order[min(n, C):][: C // 10]] = -1
        state["who"] = who
        state["base"] = normal(C, N + pad)[:, :N]
        state["y"] = torch.zeros((C, N + pad), dtype=t, device=dev)[:, :N]
        if case["op"] == "tune":
            state["hidden"] = torch.zeros((C, r), device=dev)
            state["dy"], state["dbase"] = normal(C, N, scale=0.01), normal(C, K, scale=0.01)
            state["dx"] = torch.zeros((C, K), dtype=t, device=dev)
            state["dA"], state["dB"] = torch.zeros((n, r, K), device=dev), torch.zeros((n, N, r), device=dev)
        if own:
            import routed_expert_fp4_amd as rf
            state["bank"] = rf.AdapterBank(state["A"], state["B"], state["scales"])
            state["plan"] = rf.AdapterPlan(state["who"], n)
            state["ws"] = rf.AdapterWorkspace(state["bank"], C)
        return state
    if case["op"] == "dropout":
        K = case["K"]
        state["x"], state["base"] = _activations(g, C, K, t), normal(C, K)
        state["y"] = torch.zeros((C, K), dtype=t, device=dev)
        return state
    H, I = case["H"], case["I"]
    state["x"] = _activations(g, C, H, t)
    state["wg"], state["wu"] = normal(I, H, scale=H ** -0.5), normal(I, H, scale=H ** -0.5)
    if case["op"] == "ffn":
        state["h"] = torch.zeros((C, I), dtype=t, device=dev)
    else:
        state["gate"], state["up"] = normal(C, I, scale=1.5), normal(C, I, scale=1.5)
        state["dh"] = normal(C, I, scale=0.01)
        state["dx"] = torch.zeros((C, H), dtype=t, device=dev)
        state["dwg"], state["dwu"] = torch.zeros_like(state["wg"]), torch.zeros_like(state["wu"])
    if own:
        import routed_expert_fp4_amd as rf
        state["block"] = rf.FfnBlock(state["wg"], state["wu"], case["act"])
        state["ws"] = rf.FfnWorkspace(state["block"], C)
    return state


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    case = state["case"]
    op, C = case["op"], case["C"]
    if own:
        import routed_expert_fp4_amd as rf
        if op in ("adapter", "tune"):
            # the batch's order by adapter, made of its tokens in every pass (a program's
            # further projections of the step take the same one)
            state["plan"].update(state["who"])
        if op == "adapter":
            rf.moe_adapter_fwd(state["bank"], state["plan"], state["x"], C, state["y"], state["ws"],
                               base=state["base"])
            return state["y"]
        if op == "tune":
            drop = (case["p"], state["rng"])
            rf.moe_adapter_fwd(state["bank"], state["plan"], state["x"], C, state["y"], state["ws"],
                               base=state["base"], hidden=state["hidden"], dropout=drop)
            rf.moe_adapter_bwd(state["bank"], state["plan"], state["x"], state["hidden"], state["dy"], C,
                               state["dx"], state["dA"], state["dB"], state["ws"], base=state["dbase"],
                               dropout=drop)
            return {n: state[n] for n in ("y", "dx", "dA", "dB")}
        if op == "dropout":
            rf.moe_dropout(state["x"], case["p"], state["rng"], state["y"], base=state["base"])
            return state["y"]
        if op == "ffn":
            rf.moe_ffn_fwd(state["block"], state["x"], C, state["h"], state["ws"])
            return state["h"]
        rf.moe_ffn_bwd(state["block"], state["x"], state["gate"], state["up"], state["dh"], C, state["dx"],
                       state["dwg"], state["dwu"], state["ws"])
        return {n: state[n] for n in ("dx", "dwg", "dwu")}
    if op == "adapter":
        return _plain_adapter(state)[0]
    if op == "tune":
        return _plain_tune(state)
    if op == "dropout":
        keep, scale = _plain_keep(state["rng"], C, case["K"], case["p"])
        x = torch.where(keep, state["x"].float() * scale, 0.0)
        return (state["base"].float() + x).to(state["x"].dtype)
    return _plain_ffn(state) if op == "ffn" else _plain_ffn_bwd(state)


def _plain_keep(rng, C, K, p):
    """The mask [C][K] of Philox 4x32 in ten rounds: element (c, k) takes 16 bits
    of the four words of counter (offset, k // 8, c) under the seed, the low half
    of word (k % 8) // 2 for even k and the high half for odd, and is kept where
    they are at least 65536 p; and what kept elements are multiplied by."""
    drop = int(round(p * 65536))
    if drop == 0:
        return torch.ones((C, K), dtype=torch.bool, device=rng.device), 1.0
    low = 0xFFFFFFFF
    nb = -(-K // 8)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    a = (rng[1] & low).expand(C, nb)
    b = ((rng[1] >> 32) & low).expand(C, nb)
    c = torch.arange(nb, device=rng.device).expand(C, nb)
    d = torch.arange(C, device=rng.device)[:, None].expand(C, nb)
    for _ in range(10):
        # products of 32 bits wrap as int64 where they pass 63 bits: their bits are right
        u, v = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = ((v >> 32) & low) ^ b ^ k0, v & low, ((u >> 32) & low) ^ d ^ k1, u & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    h = torch.stack((a & 0xFFFF, a >> 16, b & 0xFFFF, b >> 16, c & 0xFFFF, c >> 16, d & 0xFFFF, d >> 16), dim=2)
    return (h >= drop).reshape(C, nb * 8)[:, :K], (65536 / (65536 - drop) if drop < 65536 else 0.0)


def _plain_adapter(state, x=None):
    """y = base + s_a B_a (A_a x), all adapters' rows in one product and each
    token's own taken from it; also each token's row of A x among all adapters'."""
    A, B, who = state["A"].float(), state["B"].float(), state["who"].long()
    n, r, K = A.shape
    x = state["x"].float() if x is None else x
    mine = who[:, None] == torch.arange(n, device=who.device)
    t = torch.where(mine[:, :, None], (x @ A.reshape(n * r, K).t()).reshape(-1, n, r), 0.0)
    y = (t * state["scales"][None, :, None]).reshape(-1, n * r) @ B.permute(0, 2, 1).reshape(n * r, -1)
    return (state["base"].float() + y).to(state["x"].dtype), t, mine


def _plain_tune(state):
    """With u = s_a B_a^T dy: dB_a = sum dy (s_a A_a x)^T, dA_a = sum u x^T over a's
    tokens, dx = A_a^T u through the mask."""
    case = state["case"]
    keep, scale = _plain_keep(state["rng"], case["C"], case["K"], case["p"])
    x = torch.where(keep, state["x"].float() * scale, 0.0)
    y, t, mine = _plain_adapter(state, x)
    A, B, s, dy = state["A"].float(), state["B"].float(), state["scales"][None, :, None], state["dy"].float()
    n, r, K = A.shape
    u = (dy @ B.permute(0, 2, 1).reshape(n * r, -1).t()).reshape(-1, n, r)
    u = torch.where(mine[:, :, None], u * s, 0.0).reshape(-1, n * r)
    dB = ((t * s).reshape(-1, n * r).t() @ dy).reshape(n, r, -1).permute(0, 2, 1).contiguous()
    dx = torch.where(keep, (u @ A.reshape(n * r, K)) * scale, 0.0)
    return {"y": y, "dx": (state["dbase"].float() + dx).to(y.dtype), "dA": (u.t() @ x).reshape(n, r, K), "dB": dB}


_ROOT = math.sqrt(2 / math.pi)


def _plain_ffn(state):
    x = state["x"].float()
    g, u = x @ state["wg"].float().t(), x @ state["wu"].float().t()
    if state["case"]["act"] == "silu":
        h = g / (1 + torch.exp(-g)) * u
    else:
        h = g / (1 + torch.exp(-2 * _ROOT * (g + 0.044715 * g * g * g))) * u
    return h.to(state["x"].dtype)


def _plain_ffn_bwd(state):
    """du = dh act(g), dg = dh u act'(g); dx = dg Wg + du Wu, dW = d^T x."""
    t = state["x"].dtype
    g, u, dh, x = state["gate"].float(), state["up"].float(), state["dh"].float(), state["x"].float()
    if state["case"]["act"] == "silu":
        s = 1 / (1 + torch.exp(-g))
        a, slope = g * s, s * (1 + g * (1 - s))
    else:
        s = 1 / (1 + torch.exp(-2 * _ROOT * (g + 0.044715 * g * g * g)))
        a, slope = g * s, s + g * s * (1 - s) * 2 * _ROOT * (1 + 3 * 0.044715 * g * g)
    dg, du = dh * u * slope, dh * a
    dx = dg @ state["wg"].float() + du @ state["wu"].float()
    return {"dx": dx.to(t), "dwg": (dg.t() @ x).to(t), "dwu": (du.t() @ x).to(t)}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    b, C = {"f32": 4, "bf16": 2, "f16": 2}[case["x"]], case["C"]
    if case["op"] in ("adapter", "tune"):
        K, N, r, used = case["K"], case["N"], case["r"], min(case["n"], C)
        bank = used * (r * (K + N) * b + 4)
        if case["op"] == "adapter":
            return {"bytes": C * (K + 2 * N) * b + 4 * C + bank, "flops": 2 * C * r * (K + N)}
        # x, base, dy and dx's base in, y and dx out, gradients in fp32
        return {"bytes": C * (3 * K + 3 * N) * b + 4 * C + bank + 4 * case["n"] * r * (K + N),
                "flops": 6 * C * r * (K + N)}
    if case["op"] == "dropout":
        return {"bytes": 3 * C * case["K"] * b, "flops": C * case["K"] * 20}
    H, I = case["H"], case["I"]
    if case["op"] == "ffn":
        return {"bytes": (2 * H * I + C * (H + I)) * b, "flops": 4 * C * H * I}
    return {"bytes": (4 * H * I + C * (2 * H + 3 * I)) * b, "flops": 8 * C * H * I}


# ---------------------------------------------------------------------------
# In 64 bits, from the definitions
# ---------------------------------------------------------------------------
def _exact_mask(rng, C, K, p):
    """The same mask from products formed of 16-bit halves, as multipliers."""
    drop = int(round(p * 65536))
    if drop == 0:
        return torch.ones((1, 1), dtype=torch.float64, device=rng.device)
    seed, off = (int(v) % (1 << 64) for v in rng.cpu().tolist())
    keys = [((seed + i * 0x9E3779B9) % (1 << 32), ((seed >> 32) + i * 0xBB67AE85) % (1 << 32)) for i in range(10)]

    def high_low(v, m):
        a, b, e, f = v // 65536, v % 65536, m >> 16, m & 65535
        mid = a * f + (b * f) // 65536
        cross = b * e + mid % 65536
        return a * e + mid // 65536 + cross // 65536, (cross % 65536) * 65536 + (b * f) % 65536

    nb = (K + 7) // 8
    out = torch.empty((C, nb, 8), dtype=torch.float64, device=rng.device)
    step = max(1, (1 << 24) // nb)
    for lo in range(0, C, step):
        rows = torch.arange(lo, min(C, lo + step), device=rng.device)
        w = [torch.full((len(rows), nb), off % (1 << 32), device=rng.device),
             torch.full((len(rows), nb), off >> 32, device=rng.device),
             torch.arange(nb, device=rng.device).repeat(len(rows), 1), rows[:, None].repeat(1, nb)]
        for k0, k1 in keys:
            h0, l0 = high_low(w[0], 0xD2511F53)
            h1, l1 = high_low(w[2], 0xCD9E8D57)
            w = [h1 ^ w[1] ^ k0, l1, h0 ^ w[3] ^ k1, l0]
        for j in range(8):
            out[lo:lo + len(rows), :, j] = (w[j // 2] // 65536 ** (j % 2) % 65536 >= drop).double()
    return out.reshape(C, -1)[:, :K] * (65536 / (65536 - drop) if drop < 65536 else 0.0)


def exact(case, seed):
    state = prepare(case, seed)
    x = state["x"].double()
    C = case["C"]
    mask = _exact_mask(state["rng"], C, case["K"], case["p"]) if "p" in case else None
    if case["op"] == "dropout":
        return state["base"].double() + x * mask
    if case["op"] in ("adapter", "tune"):
        train = case["op"] == "tune"
        y = state["base"].double()
        xd = x * mask if train else x
        dx = state["dbase"].double() if train else None
        dA = torch.zeros(state["A"].shape, dtype=torch.float64, device=x.device)
        dB = torch.zeros(state["B"].shape, dtype=torch.float64, device=x.device)
        for a in range(case["n"]):
            rows = torch.nonzero(state["who"] == a).reshape(-1)
            if not len(rows):
                continue
            W = state["scales"][a].double() * (state["B"][a].double() @ state["A"][a].double())
            y[rows] += xd[rows] @ W.t()
            if train:
                dy = state["dy"][rows].double()
                G = (dy.t() @ xd[rows]) * state["scales"][a].double()      # the product's own gradient
                dA[a], dB[a] = state["B"][a].double().t() @ G, G @ state["A"][a].double().t()
                dx[rows] += (dy @ W) * (mask[rows] if mask.shape[0] > 1 else mask)
        return {"y": y, "dx": dx, "dA": dA, "dB": dB} if train else y
    act = torch.nn.functional.silu if case["act"] == "silu" else (
        lambda v: torch.nn.functional.gelu(v, approximate="tanh"))
    wg, wu = state["wg"].double(), state["wu"].double()
    if case["op"] == "ffn":
        return act(x @ wg.t()) * (x @ wu.t())
    g = state["gate"].double().requires_grad_(True)
    u = state["up"].double().requires_grad_(True)
    dg, du = torch.autograd.grad(act(g) * u, (g, u), state["dh"].double())
    return {"dx": dg @ wg + du @ wu, "dwg": dg.t() @ x, "dwu": du.t() @ x}
