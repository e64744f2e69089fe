"""Plain fp64 NumPy forms of the experts' gated feed-forward block for
training, its backward pass, and rows kept in 8 bits.

Written from the formulas, expert by expert; shares no code with the GPU path.
Rows behind the last computed pair are taken from the buffers handed in.
"""
from __future__ import annotations

import numpy as np

BLOCK = 64
SMALL = 2.0 ** -100


def sigmoid(z):
    return 0.5 * (1.0 + np.tanh(0.5 * np.asarray(z, np.float64)))


def pack8(v):
    """(codes, scale) of rows [n][cols] in blocks of 64 columns."""
    v = np.asarray(v, np.float64)
    n, cols = v.shape
    blocks = -(-cols // BLOCK)
    codes, scale = np.zeros((n, cols)), np.zeros((n, blocks))
    for b in range(blocks):
        c = slice(b * BLOCK, min(cols, (b + 1) * BLOCK))
        for i in range(n):
            part = v[i, c]
            if not np.isfinite(part).all():
                scale[i, b] = np.nan
                continue
            top = np.abs(part).max()
            if top >= SMALL:
                scale[i, b] = top / 127
                codes[i, c] = np.rint(part * 127 / top)      # part * 127 is exact: ties are ties
    return codes, scale


def unpack8(codes, scale):
    cols = codes.shape[1]
    return codes * np.repeat(scale, BLOCK, axis=1)[:, :cols]


def segments(offsets, perm, k):
    """(expert, rows, their tokens) of every expert with rows."""
    for e in range(len(offsets) - 1):
        if offsets[e + 1] > offsets[e]:
            r = slice(int(offsets[e]), int(offsets[e + 1]))
            yield e, r, np.asarray(perm)[r] // k


def forward(x, wg, wu, wd, offsets, perm, k, P):
    """(y, g, u): [P][H], [P][I], [P][I]; zeros behind the last row."""
    y, g, u = np.zeros((P, x.shape[1])), np.zeros((P, wg.shape[1])), np.zeros((P, wg.shape[1]))
    for e, r, t in segments(offsets, perm, k):
        g[r], u[r] = x[t] @ wg[e].T, x[t] @ wu[e].T
        y[r] = (g[r] * sigmoid(g[r]) * u[r]) @ wd[e].T
    return y, g, u


def gated_grad(g, u, da):
    """a = SiLU(g) u and the gradients of g and u."""
    s = sigmoid(g)
    return g * s * u, da * u * s * (1 + g * (1 - s)), da * g * s


def backward(x, wg, wu, wd, offsets, perm, k, g, u, dy):
    """(dx, dW_g, dW_u, dW_d)."""
    dx = np.zeros((len(g), wd.shape[1]))
    dwg, dwu, dwd = (np.zeros(w.shape) for w in (wg, wu, wd))
    for e, r, t in segments(offsets, perm, k):
        a, dg, du = gated_grad(g[r], u[r], dy[r] @ wd[e])
        dx[r] = dg @ wg[e] + du @ wu[e]
        dwg[e], dwu[e], dwd[e] = dg.T @ x[t], du.T @ x[t], dy[r].T @ a
    return dx, dwg, dwu, dwd
