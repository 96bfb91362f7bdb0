"""The activations of the gated block and their derivatives where squares and
cubes of their arguments pass fp32's largest number."""
import numpy as np
import pytest
import torch

from oracle import feedforward as F
from test_gpu_feedforward import ACTS, DEV, DT, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    import fac_whitening_amd as fw
    return fw


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
