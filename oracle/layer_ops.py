"""fp64 restatement of the 8-bit projection steps and the gated linear recurrence (numpy).

Test infrastructure only: the definitions written out, and the error bounds that fp32
arithmetic with the documented cast points obeys.  Nothing here is shared with the kernels.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126


def e4m3(z):
    """z rounded to the nearest e4m3 value (ties to even, saturating at +-448; NaN stays)."""
    z = np.asarray(z, np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        e = np.floor(np.log2(np.maximum(np.abs(z), 2.0 ** -6)))
        step = 2.0 ** (np.minimum(e, 8) - 3)
        return np.clip(np.round(z / step) * step, -E4M3_MAX, E4M3_MAX)


def block_scales(v, block_rows):
    """The scale of each block_rows x 128 block of v [R, C]."""
    R, C = v.shape
    rb, cb = -(-R // block_rows), -(-C // BLOCK)
    s = np.empty((rb, cb))
    for i in range(rb):
        for j in range(cb):
            s[i, j] = np.abs(v[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]).max()
    return np.maximum(s / E4M3_MAX, SCALE_MIN)


def expand_scales(s, block_rows, R, C):
    """Scales per element."""
    return np.repeat(np.repeat(s, block_rows, 0)[:R], BLOCK, 1)[:, :C]


def quantize(v, block_rows):
    """(q, scale) of v [R, C] in fp64."""
    v = np.asarray(v, np.float64)
    s = block_scales(v, block_rows)
    return e4m3(v / expand_scales(s, block_rows, *v.shape)), s


def rmsnorm(x, residual=None, gain=None, eps=1e-6):
    """(n, r): the normalised rows and the sum they come from."""
    r = np.asarray(x, np.float64)
    if residual is not None:
        r = r + np.asarray(residual, np.float64)
    n = r / np.sqrt((r * r).mean(1, keepdims=True) + eps)
    return (n if gain is None else n * np.asarray(gain, np.float64)), r


def projection(a, sa, w, sw):
    """(y, sum of magnitudes) of the product of two dequantised operands."""
    a, w = np.asarray(a, np.float64), np.asarray(w, np.float64)
    a = a * expand_scales(np.asarray(sa, np.float64), 1, *a.shape)
    w = w * expand_scales(np.asarray(sw, np.float64), BLOCK, *w.shape)
    return a @ w.T, np.abs(a) @ np.abs(w).T


def decay(gate, logits):
    """(a, d log a / d gate)."""
    g = np.asarray(gate, np.float64)
    if not logits:
        return np.exp(g), np.ones_like(g)
    a = 1 / (1 + np.exp(np.minimum(g, 700)))
    return a, -1 / (1 + np.exp(np.minimum(-g, 700)))


def recurrence(x, gate, cu, h0=None, logits=False, c=2.0 ** -20):
    """(y, h_final, bound): bound[t] is how far fp32 arithmetic may take h_t.

    A step h = fl(a h + x) with a of relative error d adds at most a d |h| + 2^-24 |h_t| to the
    error carried on, a E.  a d is at most 2^-21: the exponential is good to 2^-22 and its
    argument to 2^-23 |gate|, with a |gate| < 0.37 for both forms of a <= 1, and the reciprocal
    of the logit form to 2^-22.  Joining segments rounds their maps once more each, of the same
    size.  Both together stay under c times M_t, the recurrence of the magnitudes."""
    x = np.asarray(x, np.float64)
    a, _ = decay(gate, logits)
    y, E = np.zeros_like(x), np.zeros_like(x)
    N, C = len(cu) - 1, x.shape[1]
    fin, fin_e = np.zeros((N, C)), np.zeros((N, C))
    for n in range(N):
        h = np.zeros(C) if h0 is None else np.asarray(h0[n], np.float64)
        M, e = np.abs(h), np.zeros(C)
        for t in range(cu[n], cu[n + 1]):
            h, M = a[t] * h + x[t], a[t] * M + np.abs(x[t])
            e = a[t] * e + c * M
            y[t], E[t] = h, e
        fin[n], fin_e[n] = h, e
    return y, fin, E, fin_e


def recurrence_grad(dy, gate, y, cu, h0=None, dh_final=None, logits=False, c=2.0 ** -20):
    """(dx, dgate, dh0) and their bounds, from the same argument run backwards."""
    dy, y = np.asarray(dy, np.float64), np.asarray(y, np.float64)
    a, w = decay(gate, logits)
    dx, dg = np.zeros_like(dy), np.zeros_like(dy)
    ex, eg = np.zeros_like(dy), np.zeros_like(dy)
    N, C = len(cu) - 1, dy.shape[1]
    dh0, eh = np.zeros((N, C)), np.zeros((N, C))
    for n in range(N):
        u = np.zeros(C) if dh_final is None else np.asarray(dh_final[n], np.float64)
        M, e = np.abs(u), np.zeros(C)
        first = np.zeros(C) if h0 is None else np.asarray(h0[n], np.float64)
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            G, MG = dy[t] + u, np.abs(dy[t]) + M
            dx[t], ex[t] = G, e + c * MG
            u, M, e = a[t] * G, a[t] * MG, a[t] * (e + c * MG) + c * a[t] * MG
            h = y[t - 1] if t > cu[n] else first
            dg[t] = u * h * w[t]
            eg[t] = (e + 2 * c * M) * np.abs(h * w[t])
        dh0[n], eh[n] = u, e
    return dx, dg, dh0, ex, eg, eh
