"""What the products of the gated block and of the weight gradient keep of
small numbers.

16-bit operands enter whole, subnormal ones too.  An fp32 operand is the sum
of three bf16 numbers, of which 2^-133 is the smallest: numbers whose last bit
is not below that lose nothing, of others (all are below 2^-110) what lies
under it is dropped, less than 2^-133 of each.  The other side is scaled up
here, so that the results are normal fp32 numbers."""
import numpy as np
import pytest
import torch

from product_forms import FORMS
from test_gpu_feedforward import DEV, DT, chain, check, draw, f64, half_step
from test_gpu_product_forms import full, mm, one_a_row, single

pytestmark = pytest.mark.gpu
LAST = 2.0 ** -133
BIG = 2.0 ** 40


@pytest.fixture(scope="module")
def fw():
    import fac_whitening_amd as fw
    return fw


def scaled(t, e):
    return (t.double() * 2.0 ** e).to(t.dtype)


FORWARD = [(5, 72, 264), (20, 1001, 700), (65, 130, 96), (300, 72, 6144), (1537, 72, 2731)]
DX = [(3, 200, 700), (16, 1001, 2731), (65, 72, 96), (8200, 1032, 96)]
WGRAD = [(65, 72, 96), (65, 130, 6144), (4300, 130, 2731)]


def test_sizes_are_of_different_forms():
    for op, mine in (("forward", FORWARD), ("dx", DX), ("wgrad", WGRAD)):
        forms = [form for o, t, s, form in FORMS if o == op and t == "fp32" and s in mine]
        assert len(forms) == len(mine)


@pytest.mark.parametrize("T,d,f", FORWARD)
def test_tiny_fp32_operands_of_the_forward(fw, T, d, f):
    x, wg, wu = draw(T, d, "fp32", 1), draw(f, d, "fp32", 2), draw(f, d, "fp32", 3)
    for e in (-112, -118, -126, -133, -140):
        for tiny in ("weights", "x"):
            a, b = (x * BIG, scaled(wg, e)) if tiny == "weights" else (scaled(x, e), wg * BIG)
            u = scaled(wu, e) if tiny == "weights" else wu * BIG
            _, gate, up = fw.glu_forward(a, b, u, "relu", keep=True)
            torch.cuda.synchronize()
            for got, w, what in ((gate, b, "gate"), (up, u, "up")):
                other = f64(a).__abs__().sum(1)[:, None] if tiny == "weights" else f64(w).__abs__().sum(1)[None, :]
                want = mm(a, w)
                check(got, want, half_step(torch.float32, want) + chain(d, "fp32") * mm(a.abs(), w.abs()) + LAST * other,
                      (what, tiny, e))
    # with their last bit at 2^-133 (the values end 26 bits below 1)
    wg, at, v = one_a_row(f, d, "fp32", 2, 5)
    x = full(T, d, "fp32", 1)
    _, gate, _ = fw.glu_forward(x * BIG, scaled(wg, -107), scaled(wg, -107), "relu", keep=True)
    single(gate, x.double()[:, at] * v * 2.0 ** (40 - 107), "tiny weights")
    _, gate, _ = fw.glu_forward(scaled(x, -107), wg * BIG, wg * BIG, "relu", keep=True)
    single(gate, x.double()[:, at] * v * 2.0 ** (40 - 107), "tiny x")


@pytest.mark.parametrize("T,d,f", DX)
def test_tiny_fp32_operands_of_dx(fw, T, d, f):
    dh, gate, up = draw(T, f, "fp32", 1), draw(T, f, "fp32", 2), draw(T, f, "fp32", 3)
    wg, wu = draw(f, d, "fp32", 4), draw(f, d, "fp32", 5)
    for e in (-112, -118, -126, -133, -140):
        for tiny in ("weights", "gradients"):
            by = (BIG, None) if tiny == "weights" else (None, BIG)
            g = dh * by[0] if by[0] else scaled(dh, e)
            a, b = (w * by[1] if by[1] else scaled(w, e) for w in (wg, wu))
            dx, dgate, dup = fw.glu_backward(g, gate, up, a, b, "relu")
            torch.cuda.synchronize()
            want = mm(dgate, a.t()) + mm(dup, b.t())
            mag = mm(dgate.abs(), a.abs().t()) + mm(dup.abs(), b.abs().t())
            if tiny == "weights":
                other = (f64(dgate).__abs__() + f64(dup).__abs__()).sum(1)[:, None]
            else:
                other = (f64(a).__abs__() + f64(b).__abs__()).sum(0)[None, :]
            check(dx, want, half_step(torch.float32, want) + chain(2 * f, "fp32") * mag + LAST * other, (tiny, e))


@pytest.mark.parametrize("T,d,f", WGRAD)
def test_tiny_fp32_operands_of_the_weight_gradient(fw, T, d, f):
    delta, x = draw(T, f, "fp32", 1), draw(T, d, "fp32", 2)
    for e in (-112, -118, -126, -133, -140):
        for a, b in ((scaled(delta, e), x * BIG), (delta * BIG, scaled(x, e))):
            W = fw.weight_grad(a, b)
            torch.cuda.synchronize()
            small, other = (a, f64(b).__abs__().sum(0)[None, :]) if a.abs().max() < 1 else (b, f64(a).__abs__().sum(0)[:, None])
            want = mm(a.t(), b.t())
            check(W, want, half_step(torch.float32, want) + chain(T, "fp32") * mm(a.abs().t(), b.abs().t()) + LAST * other, e)


def patterns(rows, dtype, seed):
    """Finite nonzero numbers of every exponent, half of them subnormal."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    mant = 7 if dtype == "bf16" else 10
    top = 60 if dtype == "bf16" else 31          # (bf16: up to 2^-67, the other side is 2^60)
    e = torch.randint(1, top, (rows,), generator=g, device=DEV) * torch.randint(0, 2, (rows,), generator=g, device=DEV)
    bits = (e << mant) | torch.randint(1, 1 << mant, (rows,), generator=g, device=DEV)
    bits |= torch.randint(0, 2, (rows,), generator=g, device=DEV) << 15
    return bits.to(torch.uint16).view(DT[dtype])


def rounded(got, want, what):
    """Within half a step, and at least the largest number where want is."""
    most = float(torch.finfo(got.dtype).max)
    fits = np.abs(want) < most
    check(torch.where(torch.from_numpy(fits).to(DEV), got, 0), np.where(fits, want, 0.0), half_step(got.dtype, want) * 1.01, what)
    beyond = f64(got)[~fits]
    assert (np.abs(beyond) >= most).all() and (np.sign(beyond) == np.sign(want[~fits])).all(), what


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,d,f", [(5, 72, 264), (20, 1001, 700), (65, 72, 96), (300, 72, 6144), (1537, 520, 2731)])
def test_subnormal_16_bit_operands(fw, T, d, f, dtype):
    big = 2.0 ** 60 if dtype == "bf16" else 1.0
    other, t = full(T, d, dtype, 1) * big, DT[dtype]
    w, at, _ = one_a_row(f, d, dtype, 2, 5)
    v = patterns(f, dtype, 3)
    w[torch.arange(f, device=DEV), at] = v
    assert (v.double().abs() < torch.finfo(t).tiny).sum() > f // 4
    _, gate, up = fw.glu_forward(other, w, w, "relu", keep=True)
    torch.cuda.synchronize()
    want = f64(other)[:, at.cpu().numpy()] * f64(v)
    rounded(gate, want, "gate")
    assert torch.equal(gate, up)
    # the same rows as gradients of d tokens: fp32 outputs, exact
    delta, x = w.t().contiguous(), full(d, 136, dtype, 4) * big
    W = fw.weight_grad(delta, x)
    assert torch.equal(W.double(), v.double()[:, None] * x.double()[at])
    # and as hidden units whose gradients dx adds: u = 1, relu' = 1, so dgate is dh
    one = torch.ones(T, d, dtype=t, device=DEV)
    dh = other
    zero = torch.zeros_like(w.t()).contiguous()
    dx, dgate, dup = fw.glu_backward(dh, one, one, w.t().contiguous(), zero, "relu")
    torch.cuda.synchronize()
    assert torch.equal(dgate, dh) and torch.equal(dup, dh)
    rounded(dx, want, "dx")
