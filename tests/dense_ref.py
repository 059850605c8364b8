"""Plain 64-bit definitions of dropout's mask, the adapters and the gated block,
for the tests of the library's kernels."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24                        # half a step of fp32, relative


def philox(key, counter):
    """Philox 4x32, ten rounds: key [2], counter [4] of Python integers (or uint64
    arrays) below 2^32."""
    k0, k1 = (np.uint64(k) for k in key)
    w = [np.asarray(c, np.uint64) for c in counter]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p, q = w[0] * np.uint64(0xD2511F53), w[2] * np.uint64(0xCD9E8D57)
        w = [(q >> np.uint64(32)) ^ w[1] ^ k0, q & low, (p >> np.uint64(32)) ^ w[3] ^ k1, p & low]
        k0, k1 = (k0 + np.uint64(0x9E3779B9)) & low, (k1 + np.uint64(0xBB67AE85)) & low
    return w


def mask(seed, offset, C, K, p):
    """What element (c, k) is multiplied by: 0, or 1 / (1 - p')."""
    drop = int(round(p * 65536))
    if drop == 0:
        return np.ones((C, K))
    seed, offset, low = seed % (1 << 64), offset % (1 << 64), 0xFFFFFFFF
    nb = -(-K // 8)
    block, row = np.arange(nb, dtype=np.uint64)[None, :], np.arange(C, dtype=np.uint64)[:, None]
    z = np.zeros((C, nb), np.uint64)
    w = philox((seed & low, seed >> 32), (z + np.uint64(offset & low), z + np.uint64(offset >> 32), z + block, z + row))
    h = np.stack([v >> np.uint64(s) & np.uint64(0xFFFF) for v in w for s in (0, 16)], axis=2).reshape(C, nb * 8)[:, :K]
    return np.where(h >= drop, 65536 / max(65536 - drop, 1), 0.0) if drop < 65536 else np.zeros((C, K))


def dropped(x, m):
    """x through the mask; a dropped element is 0 whatever it holds."""
    return np.where(m > 0, x * np.where(m > 0, m, 1.0), 0.0) if m is not None else x


def adapters(x, who, A, B, s, base=None, m=None):
    """(y, t): t_c = A_a d(x_c), y_c = base_c + s_a B_a t_c."""
    C, n = x.shape[0], A.shape[0]
    xd = dropped(x, m)
    y = np.zeros((C, B.shape[1])) if base is None else base.copy()
    t = np.zeros((C, A.shape[1]))
    for a in range(n):
        rows = np.flatnonzero(who == a)
        t[rows] = xd[rows] @ A[a].T
        y[rows] += s[a] * (t[rows] @ B[a].T)
    return y, t


def adapter_grads(x, who, A, B, s, dy, t, base=None, m=None):
    """(dx, dA, dB) from t as given."""
    xd = dropped(x, m)
    dx = np.zeros(x.shape) if base is None else base.copy()
    dA, dB = np.zeros(A.shape), np.zeros(B.shape)
    for a in range(A.shape[0]):
        rows = np.flatnonzero(who == a)
        u = s[a] * (dy[rows] @ B[a])
        g = u @ A[a]
        dx[rows] += g if m is None else dropped(g, m[rows])
        dA[a], dB[a] = u.T @ xd[rows], s[a] * (dy[rows].T @ t[rows])
    return dx, dA, dB


ROOT = np.sqrt(2 / np.pi)


def act(name, g):
    """act(g) and its slope."""
    z = g if name == "silu" else 2 * ROOT * (g + 0.044715 * g ** 3)
    dz = 1.0 if name == "silu" else 2 * ROOT * (1 + 3 * 0.044715 * g * g)
    with np.errstate(over="ignore"):
        s, c = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
    return g * s, s + g * dz * s * c


def gated(name, x, wg, wu):
    g, u = x @ wg.T, x @ wu.T
    return act(name, g)[0] * u, g, u


def gated_grads(name, x, wg, wu, g, u, dh):
    """(dx, dwg, dwu, dg, du)."""
    a, slope = act(name, g)
    du, dg = dh * a, dh * u * slope
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dg, du


# how far results may be off ------------------------------------------------
def sums(terms, depth):
    """A sum of `depth` roundings against the sum of its terms' magnitudes."""
    return depth * U * terms


def walk(depth):
    """The relative 2-norm of many such sums' errors: each of the roundings is off by
    half a step at most and as often up as down."""
    return 2 * np.sqrt(depth) * U
