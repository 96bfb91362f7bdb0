"""The gated block, its backward pass and the weight gradient in every form of
their kernels (tests/product_forms.py lists the sizes and a host test holds
them to it): dense operands with dropout and kept products, and operands of
one nonzero a row or column, whose outputs are single products.

A single product of 16-bit numbers is exact in fp32.  One of fp32 numbers is
off by 3.2 U of itself at most, U = 2^-24:
  * what the three largest of nine plane products leave out: each number is
    b0 + b1 + b2, |b1| <= 2^-8, |b2| <= 2^-17 of the power of two below it, so
    a1 b2 + a2 b1 + a2 b2 stay below 2^-24 |a b|;
  * the six that are added are exact (8 by 8 bits), every other product is
    zero, and of the sums only the last is as large as the result: off by its
    last bit at most, 2 U, and the five before it, below 2^-7 of it, by 0.08 U.
The values below have three planes of full size: leaving out or doubling any
of the six moves more than 999 of 1000 results past the bound."""
import numpy as np
import pytest
import torch

from oracle import feedforward as F
from product_forms import FORMS
from test_gpu_feedforward import (ACTS, DEV, DT, OFFSET, SEED, U, act_error, chain, check, draw, f64, gradients_reference,
                                  half_step)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    import fac_whitening_amd as fw
    return fw


def sizes(op, *types):
    return [pytest.param(t, *s, id=f"{t}-{'x'.join(map(str, s))}-{form.replace(' ', '-')}")
            for o, u, s, form in FORMS if o == op for t in (["bf16", "fp16"] if u == "16" else [u]) if t in types]


ALL = ("bf16", "fp16", "fp32")


def mm(a, b):
    """a b^T in float64, on the GPU."""
    return (a.double() @ b.double().t()).cpu().numpy()


# -- dense ---------------------------------------------------------------------

@pytest.mark.parametrize("dtype,T,d,f", sizes("forward", *ALL))
def test_forward(fw, T, d, f, dtype):
    act = ACTS[(T + f) % 5]
    x, wg, wu = draw(T, d, dtype, 1), draw(f, d, dtype, 2, 1.5 * d ** -0.5), draw(f, d, dtype, 3, d ** -0.5)
    drop = (0.2, SEED, OFFSET + 7)
    h, gate, up = fw.glu_forward(x, wg, wu, act, keep=True, drop=fw.Dropout(*drop))
    alone = fw.glu_forward(x, wg, wu, act, drop=fw.Dropout(*drop))[0]
    whole = fw.glu_forward(x, wg, wu, act)[0]
    torch.cuda.synchronize()
    t, c, k = DT[dtype], chain(d, dtype), F.factor(T, f, drop)
    z, u = mm(x, wg), mm(x, wu)
    ez, eu = c * mm(x.abs(), wg.abs()) + 1e-37, c * mm(x.abs(), wu.abs()) + 1e-37
    check(gate, z, half_step(t, z) * 1.01 + ez, "gate")
    check(up, u, half_step(t, u) * 1.01 + eu, "up")
    a = F.act(z, act)[0]
    eh = (1.2 * ez + act_error(z) * np.abs(a)) * (np.abs(u) + eu) + np.abs(a) * eu + 4 * U * np.abs(a * u) + 1e-37
    check(whole, a * u, half_step(t, a * u) * 1.01 + eh, "h")
    want = F.apply(a * u, k)
    check(h, want, half_step(t, want) * 1.01 + k * eh, "h with dropout")
    assert not f64(h)[k == 0].any()
    assert torch.equal(alone, h)


@pytest.mark.parametrize("dtype,T,d,f", sizes("dx", *ALL))
def test_backward(fw, T, d, f, dtype):
    act = ACTS[(T + d) % 5]
    dh, gate, up = draw(T, f, dtype, 1, 0.2), draw(T, f, dtype, 2, 1.5), draw(T, f, dtype, 3)
    wg, wu = draw(f, d, dtype, 4, f ** -0.5), draw(f, d, dtype, 5, f ** -0.5)
    drop = (0.2, SEED, OFFSET)
    dx, dgate, dup = fw.glu_backward(dh, gate, up, wg, wu, act, fw.Dropout(*drop))
    torch.cuda.synchronize()
    (rz, tz), (ru, tu) = gradients_reference(dh, gate, up, act, F.factor(T, f, drop), dtype)
    check(dgate, rz, tz, "dgate")
    check(dup, ru, tu, "dup")
    want = mm(dgate, wg.t()) + mm(dup, wu.t())
    mag = mm(dgate.abs(), wg.abs().t()) + mm(dup.abs(), wu.abs().t())
    check(dx, want, half_step(DT[dtype], want) * 1.01 + chain(2 * f, dtype) * mag + 1e-37, "dx")


@pytest.mark.parametrize("dtype,T,d,f", sizes("wgrad", *ALL))
def test_weight_gradient(fw, T, d, f, dtype):
    delta, x = draw(T, f, dtype, 1, 0.05), draw(T, d, dtype, 2)
    W = fw.weight_grad(delta, x, alpha=0.5)
    torch.cuda.synchronize()
    want, mag = 0.5 * mm(delta.t(), x.t()), 0.5 * mm(delta.abs().t(), x.abs().t())
    check(W, want, chain(T, dtype) * mag + 1e-37, "W")
    both = fw.weight_grad(delta, x, alpha=1.0, out=W, accumulate=True)
    check(both, 3 * want, (chain(T, dtype) + 2 * U) * 3 * mag + 1e-37, "accumulated")


# -- single products -------------------------------------------------------------

def full(rows, cols, dtype, seed):
    """Numbers of every bit: fp32 ones with three planes of full size (see above)."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def pick(n):
        return torch.randint(0, n, (rows, cols), generator=g, device=DEV).double()

    def sign():
        return 2 * pick(2) - 1
    v = 1 + pick(128) / 128
    if dtype == "fp16":
        v = v + pick(8) / 1024
    if dtype == "fp32":
        v = v + sign() * 2.0 ** -9 * (1 + pick(128) / 128) + sign() * 2.0 ** -18 * (1 + pick(32) / 32)
    v = v * sign() * torch.exp2(pick(7) - 3)
    out = v.to(DT[dtype])
    assert torch.equal(out.double(), v)
    return out


def places(n, length, first):
    """For each of n rows a place on an axis, spread over all of it."""
    return (torch.arange(n, device=DEV) * 7919 + first) % length


def one_a_row(rows, cols, dtype, seed, first):
    """[rows][cols] with one nonzero a row, its places and values."""
    v, at = full(rows, 1, dtype, seed), places(rows, cols, first)
    out = torch.zeros(rows, cols, dtype=DT[dtype], device=DEV)
    out[torch.arange(rows, device=DEV), at] = v[:, 0]
    return out, at, v[:, 0].double()


def single(got, want, what):
    off = (got.double() - want).abs() / want.abs()
    bound = 3.2 * U if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2 * 1.01
    assert (want != 0).all() and off.max() <= bound, (what, off.max().item() / U, int((off > bound).sum()))


@pytest.mark.parametrize("dtype,T,d,f", sizes("forward", *ALL))
def test_forward_of_single_products(fw, T, d, f, dtype):
    for sparse in ("weights", "x"):
        if sparse == "weights":
            x = full(T, d, dtype, 1)
            wg, ag, vg = one_a_row(f, d, dtype, 2, 5)
            wu, au, vu = one_a_row(f, d, dtype, 3, 11)
            z, u = x.double()[:, ag] * vg, x.double()[:, au] * vu
        else:
            x, at, v = one_a_row(T, d, dtype, 1, 3)
            wg, wu = full(f, d, dtype, 2), full(f, d, dtype, 3)
            z, u = v[:, None] * wg.double().t()[at], v[:, None] * wu.double().t()[at]
        h, gate, up = fw.glu_forward(x, wg, wu, "relu", keep=True)
        torch.cuda.synchronize()
        single(gate, z, "gate, one of " + sparse)
        single(up, u, "up, one of " + sparse)
        if dtype == "fp32":
            assert torch.equal(h, gate.clamp(min=0) * up)
        else:                       # (the products are exact in fp32)
            assert torch.equal(h, (z.float().clamp(min=0) * u.float()).to(h.dtype))


@pytest.mark.parametrize("dtype,T,d,f", sizes("dx", *ALL))
def test_dx_of_single_products(fw, T, d, f, dtype):
    rows, cols = torch.arange(T, device=DEV), torch.arange(d, device=DEV)
    # columns of the weights with one nonzero: of Wg's for even columns, of Wu's for odd ones
    w, at, v = one_a_row(d, f, dtype, 4, 3)
    w = w.t().contiguous()
    even = (cols % 2 == 0).to(w.dtype)
    dh, gate, up = full(T, f, dtype, 1), full(T, f, dtype, 2).abs(), full(T, f, dtype, 3)
    dx, dgate, dup = fw.glu_backward(dh, gate, up, w * even, w * (1 - even), "relu")
    torch.cuda.synchronize()
    if dtype == "fp32":
        assert torch.equal(dgate, dh * up) and torch.equal(dup, dh * gate)
    single(dx, torch.where(cols % 2 == 0, dgate[:, at].double(), dup[:, at].double()) * v, "dx, one of the weights")
    # rows of the gradients with one nonzero: of dup's for even rows (u = 0), of dgate's for odd ones (gelu(0) = 0)
    dh, at, _ = one_a_row(T, f, dtype, 1, 5)
    gate, up = full(T, f, dtype, 2).abs(), full(T, f, dtype, 3)
    up[rows % 2 == 0] = 0
    gate[rows % 2 == 1] = 0
    wg, wu = full(f, d, dtype, 4), full(f, d, dtype, 5)
    dx, dgate, dup = fw.glu_backward(dh, gate, up, wg, wu, "gelu")
    torch.cuda.synchronize()
    assert not dgate[rows % 2 == 0].any() and not dup[rows % 2 == 1].any()
    z, u = dgate.double()[rows, at][:, None] * wg.double()[at], dup.double()[rows, at][:, None] * wu.double()[at]
    single(dx, z + u, "dx, one of the gradients")


@pytest.mark.parametrize("dtype,T,d,f", sizes("wgrad", *ALL))
def test_weight_gradient_of_single_products(fw, T, d, f, dtype):
    bound = 3.2 * U if dtype == "fp32" else 0
    for sparse in ("delta", "x"):
        if sparse == "delta":
            delta, at, v = one_a_row(f, T, dtype, 1, 3)
            delta, x = delta.t().contiguous(), full(T, d, dtype, 2)
            want = v[:, None] * x.double()[at]
        else:
            x, at, v = one_a_row(d, T, dtype, 1, 3)
            x, delta = x.t().contiguous(), full(T, f, dtype, 2)
            want = delta.double()[at].t() * v
        W = fw.weight_grad(delta, x)
        torch.cuda.synchronize()
        off = ((W.double() - want).abs() / want.abs()).max().item()
        assert off <= bound, (sparse, off / U)
