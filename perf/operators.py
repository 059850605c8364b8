"""Measured cases of the router-load and 4-bit dense operators.

Four operators: the 4-bit group-scaled matrix-vector product (moe_quant_linear),
the per-expert counts of a selection (moe_expert_counts), the balance loss with
its gradient (moe_balance_fwd / moe_balance_bwd) and the gradient of the
renormalised routing weights (moe_route_bwd).  `own` chooses between their
plain form, written in elementary torch operations, and the library's calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _q4(C, N, K, G, x, scales, zeros, pad=0):
    """x [C][K] times a matrix [N][K] of 4-bit codes, one scale (and zero point
    where `zeros`) per G codes of a row; `pad`: unused elements behind each row
    of x and of y, as in a slice of a wider tensor."""
    return {"op": "q4", "C": C, "N": N, "K": K, "G": G, "x": x, "scales": scales, "zeros": zeros,
            "pad": pad}


def _router(op, C, E, k, S, masked, score="sigmoid"):
    """C tokens over E experts, top-k, packed as S sequences of different
    lengths; `masked`: some tokens are padding."""
    return {"op": op, "C": C, "E": E, "k": k, "S": S, "masked": masked, "score": score}


def listed():
    return [
        # routed_down of the K3 latent layer, one decoded token, fp32 activations
        dict(_q4(1, 3584, 7168, 128, "f32", "bf16", False), name="q4 latent down, one token"),
        # routed_up for seven drafted tokens, small groups with zero points
        dict(_q4(7, 7168, 3584, 32, "bf16", "f16", True), name="q4 latent up, seven tokens"),
        # odd sizes, rows of a wider tensor, a full decode batch
        dict(_q4(16, 1001, 4099, 64, "f32", "f32", True, 5), name="q4 odd sizes, 16 tokens"),
        # an output head over a large vocabulary, one token: the largest stream
        dict(_q4(1, 65536, 7168, 128, "bf16", "bf16", False), name="q4 head, one token"),
        # routed_down for one prefill chunk: the compute-bound end
        dict(_q4(2048, 3584, 7168, 128, "bf16", "bf16", True), name="q4 latent down, chunk"),
        # load statistics of one verification step
        dict(_router("counts", 7, 448, 16, 1, False), name="counts, seven tokens"),
        # load statistics of a calibration batch, by sequence
        dict(_router("counts", 65536, 896, 16, 61, True), name="counts, 64k tokens"),
        # the loss on one decode batch: launch latency
        dict(_router("balance", 16, 896, 16, 1, False), name="balance, 16 tokens"),
        # one prefill chunk as a single sequence
        dict(_router("balance", 2048, 896, 16, 1, False), name="balance, chunk"),
        # a packed calibration batch with padding
        dict(_router("balance", 65536, 448, 8, 37, True, "softmax"), name="balance, packed 64k"),
        # gradients of the routing weights of one prefill chunk
        dict(_router("route_bwd", 2048, 896, 16, 1, False), name="route weights, chunk"),
        # and of a padded calibration batch
        dict(_router("route_bwd", 40001, 448, 8, 1, True), name="route weights, 40k tokens"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["q4", "q4", "q4", "counts", "balance", "balance", "route_bwd"])
    if op == "q4":
        C = _log(rng, 1, 2048)
        N = _log(rng, 16, 65536)
        # at most the largest stream's codes and the chunk's products
        most = min(65536 * 7168 // N, 2048 * 3584 * 7168 // (C * N), 14336)
        N, K = (N, _log(rng, 33, most)) if most >= 64 else (256, 1024)
        if rng.random() < 0.5:
            K = max(32, K // 32 * 32)
        return _q4(C, N, K, rng.choice([32, 64, 128, 256]), rng.choice(["f32", "bf16", "f16"]),
                   rng.choice(["f32", "bf16", "f16"]), rng.random() < 0.5,
                   rng.choice([0, 0, 3, 8]))
    E = rng.choice([_log(rng, 8, 1024), 448, 896])
    k = rng.randint(2, max(2, min(E // 4, 32)))    # k = E leaves nothing to balance
    C = _log(rng, 1, 65536 * 448 // max(E, 448))
    return _router(op, C, E, k, 1 if op == "route_bwd" else min(_log(rng, 1, 128), C),
                   C >= 8 and rng.random() < 0.5, rng.choice(["sigmoid", "softmax"]))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    state = {"case": case}
    if case["op"] == "q4":
        C, N, K, G = case["C"], case["N"], case["K"], case["G"]
        ng, t = -(-K // G), DTYPES[case["x"]]
        pitch = (-(-K // 2) + 15) // 16 * 16       # rows of codes start 16-byte aligned
        state["codes"] = torch.randint(0, 256, (N, pitch), generator=g, device=dev, dtype=torch.uint8)
        # a group's scale is its range over 15: about 0.02 * 6 / 15 for N(0, 0.02^2) weights
        s = 0.008 * (0.6 + 0.8 * torch.rand((N, ng), generator=g, device=dev))
        state["scales"] = s.to(DTYPES[case["scales"]])
        state["zeros"] = (torch.randint(5, 11, (N, ng), generator=g, device=dev, dtype=torch.uint8)
                          if case["zeros"] else None)
        # activations with a few large channels, as hidden states have them
        x = torch.randn((C, K + case["pad"]), generator=g, device=dev)
        x *= 1 + 15 * (torch.rand((K + case["pad"],), generator=g, device=dev) < 0.004)
        state["x"] = x.to(t)[:, :K]
        state["y"] = torch.zeros((C, N + case["pad"]), dtype=t, device=dev)[:, :N]
        if own:
            import routed_expert_fp4_amd as rf
            state["m"] = rf.QuantMatrix(state["codes"], state["scales"], K, G, state["zeros"])
            state["ws"] = rf.QuantWorkspace(state["m"], C, t)
        return state

    C, E, k, S = case["C"], case["E"], case["k"], case["S"]
    # logits of x ~ N(0, 1), W_r ~ N(0, 0.02^2) at H = 7168, and popular experts
    logits = 1.7 * torch.randn((C, E), generator=g, device=dev)
    logits += 0.7 * torch.randn((E,), generator=g, device=dev)
    state["logits"] = logits
    state["idx"] = torch.topk(logits, k, dim=1).indices.to(torch.int32).contiguous()
    # sequences of different lengths; the last tokens are behind every sequence
    state["seq"] = None
    if S > 1:
        cuts = np.sort(np.random.RandomState(seed % (1 << 31)).randint(0, C - C // 50 + 1, S + 1))
        cuts[0], cuts[S] = 0, C - C // 50
        state["seq"] = torch.from_numpy(cuts.astype(np.int32)).to(dev)
    state["mask"] = ((torch.rand((C,), generator=g, device=dev) < 0.9).to(torch.uint8)
                     if case["masked"] else None)
    if case["op"] == "route_bwd":
        state["dw"] = torch.randn((C, k), generator=g, device=dev)
    else:
        state["counts"] = torch.zeros((S, E), dtype=torch.int32, device=dev)
        state["tokens"] = torch.zeros((S,), dtype=torch.int32, device=dev)
    if case["op"] == "balance":
        state["alpha"] = 0.01
        state["grad"] = 0.5 + torch.rand((1,), generator=g, device=dev)
        state["probs"] = torch.zeros((S, E), device=dev)
        state["loss"] = torch.zeros((1,), device=dev)
    if case["op"] != "counts":
        state["dlogits"] = torch.zeros((C, E), device=dev)
    if own and case["op"] == "balance":
        import routed_expert_fp4_amd as rf
        state["ws"] = rf.BalanceWorkspace(C, E, S)
    return state


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import routed_expert_fp4_amd as rf
        if op == "q4":
            rf.moe_quant_linear(state["m"], state["x"], case["C"], state["y"], state["ws"])
            return state["y"]
        C, E, k, S = case["C"], case["E"], case["k"], case["S"]
        if op == "counts":
            rf.moe_expert_counts(state["idx"], C, E, k, state["counts"], state["tokens"],
                                 seq_offsets=state["seq"], S=S, token_mask=state["mask"])
            return {"counts": state["counts"], "tokens": state["tokens"]}
        if op == "balance":
            rf.moe_balance_fwd(state["logits"], state["idx"], C, E, k, state["alpha"],
                               state["counts"], state["tokens"], state["probs"], state["loss"],
                               state["ws"], score=case["score"], seq_offsets=state["seq"], S=S,
                               token_mask=state["mask"])
            rf.moe_balance_bwd(state["logits"], state["counts"], state["tokens"], C, E, k,
                               state["alpha"], state["grad"], state["dlogits"],
                               score=case["score"], seq_offsets=state["seq"], S=S,
                               token_mask=state["mask"])
            return {n: state[n] for n in ("counts", "tokens", "probs", "loss", "dlogits")}
        rf.moe_route_bwd(state["logits"], state["idx"], state["dw"], C, E, k, state["dlogits"],
                         token_mask=state["mask"])
        return state["dlogits"]
    if op == "q4":
        return _plain_q4(state)
    if op == "counts":
        seq, live = _plain_sequences(state)
        return _plain_counts(state, seq, live)
    if op == "balance":
        return _plain_balance(state)
    return _plain_route_bwd(state)


def _plain_q4(state):
    """y = x W^T with W[n][k] = s[n][g] (q[n][k] - z[n][g]), g = k // G."""
    case, codes = state["case"], state["codes"]
    K, G = case["K"], case["G"]
    q = torch.stack((codes & 15, codes >> 4), dim=2).reshape(codes.shape[0], -1)[:, :K].float()
    z = state["zeros"].float() if state["zeros"] is not None else torch.full_like(state["scales"], 8, dtype=torch.float32)
    g = torch.arange(K, device=q.device) // G
    w = (q - z[:, g]) * state["scales"].float()[:, g]
    return (state["x"].float() @ w.t()).to(state["x"].dtype)


def _plain_sequences(state):
    """(sequence of each token, whether the token counts)."""
    C = state["case"]["C"]
    live = torch.ones((C,), dtype=torch.bool, device=state["idx"].device)
    seq = torch.zeros((C,), dtype=torch.int64, device=state["idx"].device)
    if state["seq"] is not None:
        t = torch.arange(C, device=seq.device)
        seq = torch.searchsorted(state["seq"].long(), t, right=True) - 1
        live = (seq >= 0) & (seq < state["case"]["S"])
        seq = seq.clamp(0, state["case"]["S"] - 1)
    if state["mask"] is not None:
        live = live & (state["mask"] != 0)
    return seq, live


def _plain_counts(state, seq, live):
    case = state["case"]
    S, E, k = case["S"], case["E"], case["k"]
    at = (seq[:, None] * E + state["idx"].long()).reshape(-1)
    one = live.to(torch.int32)
    counts = torch.zeros((S * E,), dtype=torch.int32, device=at.device)
    counts.index_add_(0, at, one[:, None].expand(-1, k).reshape(-1))
    tokens = torch.zeros((S,), dtype=torch.int32, device=at.device).index_add_(0, seq, one)
    return {"counts": counts.reshape(S, E), "tokens": tokens}


def _plain_balance(state):
    """loss = alpha / S * sum_s sum_e f[s][e] P[s][e], f = E counts / (k T_s),
    P = the mean over the sequence's T_s tokens of the normalised scores."""
    case, logits = state["case"], state["logits"]
    S, E, k = case["S"], case["E"], case["k"]
    seq, live = _plain_sequences(state)
    out = _plain_counts(state, seq, live)
    if case["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-logits))
        p = s / s.sum(dim=1, keepdim=True)
        slope = 1 / (1 + torch.exp(logits))        # 1 - s without its cancellation
    else:
        s = torch.exp(logits - logits.max(dim=1, keepdim=True).values)
        p = s / s.sum(dim=1, keepdim=True)
        slope = None
    n = out["tokens"].float()
    per = torch.where(n > 0, 1 / n.clamp(min=1), torch.zeros_like(n))
    probs = torch.zeros((S, E), device=p.device).index_add_(0, seq, p * live[:, None]) * per[:, None]
    f = out["counts"].float() * per[:, None] * (E / k)
    loss = (state["alpha"] / S) * (f * probs).sum().reshape(1)
    g = (state["grad"] * (state["alpha"] / S) * per[:, None] * f)[seq]
    d = p * (g - (p * g).sum(dim=1, keepdim=True))
    if slope is not None:
        d = d * slope
    return dict(out, probs=probs, loss=loss, dlogits=d * live[:, None])


def _plain_route_bwd(state):
    """w = sigmoid(l) / sum of the k chosen; the gradient of its sum against dw."""
    case, at = state["case"], state["idx"].long()
    l = torch.gather(state["logits"], 1, at)
    s = 1 / (1 + torch.exp(-l))
    w = s / s.sum(dim=1, keepdim=True)
    d = w / (1 + torch.exp(l)) * (state["dw"] - (w * state["dw"]).sum(dim=1, keepdim=True))
    if state["mask"] is not None:
        d = d * (state["mask"] != 0)[:, None]
    return torch.zeros((case["C"], case["E"]), device=d.device).scatter_(1, at, d)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if case["op"] == "q4":
        C, N, K = case["C"], case["N"], case["K"]
        ng = -(-K // case["G"])
        return {"bytes": N * -(-K // 2) + N * ng * (size[case["scales"]] + int(case["zeros"])) +
                C * (K + N) * size[case["x"]],
                "flops": 2 * C * N * K}
    C, E, k, S = case["C"], case["E"], case["k"], case["S"]
    out = 4 * S * (E + 1)
    if case["op"] == "counts":
        return {"bytes": 4 * C * k + C * case["masked"] + out, "flops": C * k}
    if case["op"] == "balance":
        # logits and selection in, the gradient and the statistics out
        return {"bytes": 8 * C * E + 4 * C * k + C * case["masked"] + 2 * out, "flops": 20 * C * E}
    # of the logits only the chosen ones are needed
    return {"bytes": 4 * C * E + 12 * C * k + C * case["masked"], "flops": 20 * C * k}


# ---------------------------------------------------------------------------
# In 64 bits, from the definitions
# ---------------------------------------------------------------------------
def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "q4":
        K, G = case["K"], case["G"]
        x = state["x"].double()
        y = torch.zeros((case["C"], case["N"]), dtype=torch.float64, device=x.device)
        for lo in range(0, K, G):                  # one group of columns at a time
            hi, j = min(K, lo + G), lo // G
            b = state["codes"][:, lo // 2:(hi + 1) // 2].to(torch.int64)
            xg = x[:, lo:hi]
            even, odd = xg[:, 0::2], xg[:, 1::2]
            part = even @ (b % 16).double().t()
            part += odd @ torch.div(b[:, :odd.shape[1]], 16, rounding_mode="floor").double().t()
            z = 8.0 if state["zeros"] is None else state["zeros"][:, j].double()
            y += state["scales"][:, j].double() * (part - z * xg.sum(dim=1, keepdim=True))
        return y
    C, E, k, S = case["C"], case["E"], case["k"], case["S"]
    idx = state["idx"].cpu().numpy().astype(np.int64)
    keep = np.ones(C, bool) if state["mask"] is None else state["mask"].cpu().numpy() != 0
    cuts = [0, C] if state["seq"] is None else state["seq"].cpu().numpy().tolist()
    logits = state["logits"].double()
    if case["op"] == "route_bwd":
        leaf = logits.clone().requires_grad_(True)
        s = torch.sigmoid(torch.gather(leaf, 1, state["idx"].long()))
        w = s / s.sum(dim=1, keepdim=True)
        live = torch.from_numpy(keep).to(w.device)
        (w * state["dw"].double())[live].sum().backward()
        return leaf.grad
    counts, tokens = np.zeros((S, E), np.int32), np.zeros((S,), np.int32)
    rows = []
    for s in range(S):
        at = np.arange(cuts[s], cuts[s + 1])
        at = at[keep[cuts[s]:cuts[s + 1]]]
        rows.append(torch.from_numpy(at).to(logits.device))
        counts[s] = np.bincount(idx[at].reshape(-1), minlength=E)
        tokens[s] = len(at)
    if case["op"] == "counts":
        return {"counts": counts, "tokens": tokens}
    leaf = logits.clone().requires_grad_(True)
    probs = torch.zeros((S, E), dtype=torch.float64, device=leaf.device)
    loss = torch.zeros((1,), dtype=torch.float64, device=leaf.device)
    total = loss
    for s in range(S):
        if tokens[s]:
            l = leaf[rows[s]]
            q = torch.log_softmax(l, 1) if case["score"] == "softmax" else torch.log_softmax(
                torch.nn.functional.logsigmoid(l), 1)
            P = torch.exp(q).mean(dim=0)
            probs[s] = P.detach()
            f = torch.from_numpy(counts[s].astype(np.float64)).to(P.device) * E / (k * float(tokens[s]))
            total = total + state["alpha"] / S * (f * P).sum()
    if total.requires_grad:
        (total * state["grad"].double()).sum().backward()
    return {"counts": counts, "tokens": tokens, "probs": probs, "loss": total.detach(),
            "dlogits": leaf.grad if leaf.grad is not None else torch.zeros_like(logits)}
