"""The activations of the gated block and their derivatives over the whole
range of a type: the tails, where both tend to zero, and values whose squares
and cubes pass fp32's largest number.

Tolerances.  U = 2^-24 is fp32's half step.  A value or derivative is a sum of
terms of which each is off relative to itself: by (32 + 8 z^2 + 2 |z|^3) U, for
  * some ten operations and hardware functions (1 ulp each): under 24 U;
  * the normal tail's polynomial, 8 U (4.4e-7);
  * an argument off by 4 U of itself, which moves e^-w by 4 |w| U: w = z (silu,
    sigmoid), z^2 / 2 (gelu) or 1.6 |z| + 0.0714 |z|^3 (gelu_tanh).
The terms are the derivative's own (terms() below), not larger ones.  A
logistic value or exponential below 2^-126 may be zero: 2^-126 times what
multiplies it is added."""
import math

import numpy as np
import pytest
import torch
from scipy import special

from oracle import feedforward as F
from test_gpu_feedforward import ACTS, DEV, DT, U, check, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    import fac_whitening_amd as fw
    return fw


def relative(z):
    z = np.abs(z)
    return (32 + 8 * z ** 2 + 2 * z ** 3) * U


def lost(z):
    """What a number below 2^-126, taken as zero, is multiplied by at most."""
    z = np.abs(z)
    return 2.0 ** -126 * (1 + 1.6 * z * (1 + 0.135 * z ** 2))


def terms(z, act):
    """Magnitudes that act'(z) adds."""
    s, q = special.expit(z), special.expit(-z)
    if act == "relu":
        return (z > 0) * 1.0
    if act == "sigmoid":
        return s * q
    if act == "silu":
        return s + np.abs(z) * s * q
    if act == "gelu":
        return special.ndtr(z) + np.abs(z) * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    k = 2 * math.sqrt(2 / math.pi)
    w = k * (z + 0.044715 * z ** 3)
    s, q = special.expit(w), special.expit(-w)
    return s + np.abs(z) * s * q * k * (1 + 3 * 0.044715 * z ** 2)


def derivatives(fw, z, act, form):
    """act'(z) and act(z) of a row z, from the gradient pass ("pass") or the few-token form ("tokens")."""
    n, t = z.numel(), z.dtype
    z = z.view(1, n)
    one = torch.ones_like(z)
    kw = {}
    if form == "tokens":
        kw = dict(w_gate=torch.zeros(n, 8, dtype=t, device=DEV), w_up=torch.zeros(n, 8, dtype=t, device=DEV))
    dx, dgate, dup = fw.glu_backward(one, z, one, act=act, **kw)
    torch.cuda.synchronize()
    assert (dx is None) == (form == "pass")
    return dgate, dup


def values(fw, z, act, form):
    """act(z) and z from the forward pass: tokens of two numbers, z and 1 ("tiles"), or one token and weights of z."""
    n, t = z.numel(), z.dtype
    one, unit = torch.ones_like(z), torch.eye(2, dtype=t, device=DEV)
    rows = torch.stack([z, one], 1)
    if form == "tiles":
        h, gate, up = fw.glu_forward(rows, unit[:1], unit[1:], act, keep=True)
    else:
        h, gate, up = fw.glu_forward(torch.ones(1, 2, dtype=t, device=DEV), rows * unit[0], rows * unit[1], act, keep=True)
    torch.cuda.synchronize()
    assert (f64(up) == 1).all()
    return h.view(1, n), gate.view(1, n)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("form", ["pass", "tokens"])
def test_derivatives_in_the_tails(fw, act, form):
    z = torch.cat([torch.linspace(-30, 30, 6001, device=DEV), torch.linspace(-3, 3, 1001, device=DEV)])
    Z = f64(z).reshape(1, -1)
    a, da = F.act(Z, act)
    dgate, dup = derivatives(fw, z, act, form)
    check(dgate, da, relative(Z) * terms(Z, act) + lost(Z), act + " derivative")
    check(dup, a, relative(Z) * np.abs(a) + lost(Z) * np.abs(Z), act)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("form", ["tiles", "tokens"])
def test_values_in_the_tails(fw, act, form):
    z = torch.linspace(-30, 30, 4001, device=DEV)
    Z = f64(z).reshape(1, -1)
    h, gate = values(fw, z, act, form)
    assert np.array_equal(f64(gate), Z)
    a = F.act(Z, act)[0]
    check(h, a, relative(Z) * np.abs(a) + lost(Z) * (1 + np.abs(Z)), act)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("act", ACTS)
def test_large_values(fw, act, dtype):
    """Far from zero an activation is z, 1 or 0 and its derivative 1 or 0, also where z^2 or z^3 is infinite in fp32."""
    v = [1e4, 1e7, 1e10, 1e13, 1e18, 1.8e19, 1.9e19, 1e25, 1e30, 1e38, 3e38]
    z = torch.tensor([s * x for x in v * 7 for s in (1.0, -1.0)], device=DEV).to(DT[dtype])
    Z = f64(z).reshape(1, -1)
    with np.errstate(over="ignore"):
        a, da = F.act(Z, act)
    for form in ("pass", "tokens"):
        dgate, dup = derivatives(fw, z, act, form)
        assert np.array_equal(f64(dgate), da), (form, f64(dgate)[0, :22])
        assert np.array_equal(f64(dup), a), (form, f64(dup)[0, :22])
    for form in ("tiles", "tokens"):
        h, gate = values(fw, z, act, form)
        assert np.array_equal(f64(gate), Z), form
        assert np.array_equal(f64(h), a), (form, f64(h)[0, :22])
