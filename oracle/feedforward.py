"""Gated feed-forward block and dropout of the oracle, in float64 from their
definitions.

TEST INFRASTRUCTURE ONLY (see ``oracle.gift``).  Philox4x32-10 is written from
its description (Salmon et al., "Parallel random numbers: as easy as 1, 2,
3", SC 2011) in Python integers and pinned by the known answers published
with it.
"""
from __future__ import annotations

import math

import numpy as np
from scipy import special

M = (1 << 32) - 1


def philox(ctr, key):
    c, k = [int(v) for v in ctr], [int(v) for v in key]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & M, (a >> 32) ^ c[3] ^ k[1], a & M]
        k = [(k[0] + 0x9E3779B9) & M, (k[1] + 0xBB67AE85) & M]
    return c


def threshold(p):
    """round(65536 p), ties to even."""
    return round(65536 * p)


def kept(T, d, p, seed, offset):
    """Boolean [T][d].  The rounds of philox(), on arrays of words."""
    nb = -(-d // 8)
    u = np.uint64
    c = [np.arange(nb, dtype=u)[None, :], np.arange(T, dtype=u)[:, None], u(offset & M), u(offset >> 32)]
    c = [np.broadcast_to(v, (T, nb)).copy() for v in c]
    k = [seed & M, seed >> 32]
    for _ in range(10):
        a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(b >> u(32)) ^ c[1] ^ u(k[0]), b & u(M), (a >> u(32)) ^ c[3] ^ u(k[1]), a & u(M)]
        k = [(k[0] + 0x9E3779B9) & M, (k[1] + 0xBB67AE85) & M]
    bits = np.stack([v for w in c for v in (w & u(0xFFFF), w >> u(16))], axis=2).reshape(T, nb * 8)
    return bits[:, :d] >= u(threshold(p))


def factor(T, d, drop):
    """What dropout multiplies each element by; drop: (p, seed, offset) or None."""
    if drop is None:
        return np.ones((T, d))
    thr = threshold(drop[0])
    return np.where(kept(T, d, *drop), 65536.0 / max(65536 - thr, 1), 0.0)


def apply(x, f):
    """Dropped elements are zero whatever they held."""
    return np.where(f == 0, 0.0, x * np.where(f == 0, 1.0, f))


def act(z, kind):
    """act(z) and act'(z)."""
    z = np.asarray(z, np.float64)
    if kind == "relu":
        return np.maximum(z, 0), (z > 0).astype(np.float64)
    if kind == "sigmoid":
        s = special.expit(z)
        return s, s * special.expit(-z)
    if kind == "silu":
        s = special.expit(z)
        return z * s, s + z * s * special.expit(-z)
    if kind == "gelu":
        n = special.ndtr(z)
        return z * n, n + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        k = 2 * math.sqrt(2 / math.pi)
        w = k * (z + 0.044715 * z ** 3)
        s = special.expit(w)
        return z * s, s + z * s * special.expit(-w) * k * (1 + 3 * 0.044715 * z ** 2)
    raise ValueError(kind)


def glu_forward(x, wg, wu, kind, f):
    """h, z, u with dropout's factors f [T][f]."""
    z, u = x @ wg.T, x @ wu.T
    return apply(act(z, kind)[0] * u, f), z, u


def glu_gradients(dh, z, u, kind, f):
    """dgate, dup."""
    e = apply(dh, f)
    a, da = act(z, kind)
    return e * u * da, e * a
