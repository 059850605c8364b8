"""Plain 64-bit definitions of the dense 4-bit product, the counts, the balance
loss and the router gradients, for the tests of the library's kernels."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24                        # half a step of fp32, relative


def quant_weights(codes, scales, zeros, K, G):
    """W [N][K] float64 of uint8 codes [N][>= K / 2], scales [N][groups] and
    zeros [N][groups] (None: 8)."""
    q = np.empty((codes.shape[0], 2 * codes.shape[1]))
    q[:, 0::2] = codes & 15
    q[:, 1::2] = codes >> 4
    g = np.arange(K) // G
    z = 8.0 if zeros is None else zeros[:, g].astype(np.float64)
    return scales.astype(np.float64)[:, g] * (q[:, :K] - z)


def sequences(C, seq, mask, S):
    """The live tokens of each sequence, in order."""
    seq = [0, C] if seq is None else [int(v) for v in seq]
    live = np.ones(C, bool) if mask is None else np.asarray(mask) != 0
    return [[t for t in range(seq[s], seq[s + 1]) if live[t]] for s in range(S)]


def counts(idx, E, seq=None, mask=None, S=1):
    C = idx.shape[0]
    out, tok = np.zeros((S, E), np.int64), np.zeros(S, np.int64)
    for s, rows in enumerate(sequences(C, seq, mask, S)):
        tok[s] = len(rows)
        for t in rows:
            for e in idx[t]:
                if 0 <= e < E:
                    out[s, e] += 1
    return out, tok


def log_sigmoid(l):
    with np.errstate(all="ignore"):
        return np.where(l >= 0, -np.log1p(np.exp(-np.abs(l))), l - np.log1p(np.exp(-np.abs(l))))


def shares(l, score):
    """One token's logits [E] as shares; a row of -inf has none."""
    v = log_sigmoid(l) if score == "sigmoid" else np.asarray(l, np.float64)
    m = np.max(v)
    if m == -np.inf:
        return np.zeros_like(v)
    with np.errstate(all="ignore"):
        p = np.exp(v - m)
        return p / p.sum()


def balance(logits, idx, alpha, score, seq=None, mask=None, S=1, grad=1.0):
    """counts, tokens, probs, loss and the gradient of grad * loss."""
    C, E = logits.shape
    k = idx.shape[1]
    cnt, tok = counts(idx, E, seq, mask, S)
    probs, d = np.zeros((S, E)), np.zeros((C, E))
    loss = 0.0
    for s, rows in enumerate(sequences(C, seq, mask, S)):
        if not rows:
            continue
        T = len(rows)
        f = E * cnt[s] / (k * T)
        p = {t: shares(logits[t].astype(np.float64), score) for t in rows}
        probs[s] = sum(p.values()) / T
        loss += alpha / S * float(f @ probs[s])
        g = grad * alpha / (S * T) * f
        for t in rows:
            d[t] = p[t] * (g - p[t] @ g)
            if score == "sigmoid":
                d[t] *= np.exp(log_sigmoid(-logits[t].astype(np.float64)))
    return dict(counts=cnt, tokens=tok, probs=probs, loss=loss, dlogits=d)


def route_grad(logits, idx, dw, mask=None):
    C, E = logits.shape
    d = np.zeros((C, E))
    for t in range(C):
        if mask is not None and not mask[t]:
            continue
        slots = [s for s in range(idx.shape[1]) if 0 <= idx[t, s] < E]
        if not slots:
            continue
        l = logits[t, idx[t, slots]].astype(np.float64)
        w = shares(l, "sigmoid")
        dl = w * np.exp(log_sigmoid(-l)) * (dw[t, slots] - w @ dw[t, slots].astype(np.float64))
        for j, s in enumerate(slots):
            d[t, idx[t, s]] += dl[j]
    return d
