"""Activation operators of the oracle, in float64 from their definitions:
8-bit checkpoints, layer / RMS norm with its backward pass, and the weight
gradient of a linear layer.

TEST INFRASTRUCTURE ONLY (see ``oracle.gift``).  Sources: GIFT 阅读笔记,
§前置知识 Eq. (4) (A = E[a a^T] and W_g = delta^T a from the layer's input a),
and "FP8 到底是什么" for the code formats.

Reading taken here for the checkpoint: one scale per token and 32 columns, a
power of two 2^(e - 127), e the smallest integer >= 32 with
amax <= FMAX 2^(e - 127); a block with an Inf or NaN has e = 255 and codes
0x7F, values NaN.
"""
from __future__ import annotations

import numpy as np

from . import fp8

BLOCK = 32


def ckpt_save(x: np.ndarray, fmt: str):
    """codes uint8 [T][32 nb] and exponents int [T][nb] of x [T][d]."""
    x = np.asarray(x, np.float64)
    T, d = x.shape
    nb = -(-d // BLOCK)
    v = np.zeros((T, nb * BLOCK))
    v[:, :d] = x
    v = v.reshape(T, nb, BLOCK)
    bad = ~np.isfinite(v).all(2)
    amax = np.where(bad, 1.0, np.abs(np.where(np.isfinite(v), v, 0)).max(2))
    e = np.full((T, nb), 32)
    while True:                       # the definition, one step at a time
        over = amax > np.ldexp(fp8.FMAX[fmt], e - 127)
        if not over.any():
            break
        e = e + over
    with np.errstate(invalid="ignore", under="ignore"):
        q = np.ldexp(v, (127 - e)[:, :, None]).astype(np.float32)
    codes = fp8.encode(np.where(bad[:, :, None], np.float32(0), q), fmt)
    codes = np.where(bad[:, :, None], np.uint8(0x7F), codes)
    return codes.reshape(T, nb * BLOCK), np.where(bad, 255, e)


def ckpt_values(codes, e, d, fmt):
    v = fp8.decode(codes, fmt) * np.repeat(np.ldexp(1.0, e - 127), BLOCK, axis=1)
    return v[:, :d]


def exponent_layout(e):
    """[T][nb] -> uint8 [ceil(T / 8)][nb][8] (zero past T)."""
    T, nb = e.shape
    out = np.zeros((-(-T // 8), nb, 8), np.uint8)
    for t in range(T):
        out[t // 8, :, t % 8] = e[t]
    return out


def norm_forward(x, weight, bias, eps, kind):
    x = np.asarray(x, np.float64)
    mean = x.mean(1) if kind == "layer" else np.zeros(x.shape[0])
    c = x - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(1) + eps)
    y = c * rstd[:, None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def norm_backward(dy, x, mean, rstd, weight, kind):
    dy = np.asarray(dy, np.float64)
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * (1.0 if weight is None else weight)
    dx = g - xh * (g * xh).mean(1)[:, None]
    if kind == "layer":
        dx = dx - g.mean(1)[:, None]
    return dx * rstd[:, None], (dy * xh).sum(0), dy.sum(0)


def weight_grad(delta, a, alpha):
    return alpha * (np.asarray(delta, np.float64).T @ np.asarray(a, np.float64))
