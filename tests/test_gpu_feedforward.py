"""Gated feed-forward block, dropout and the weight gradient from a whole
activation on the GPU, against their float64 oracle.

Tolerances.  U = 2^-24 is fp32's half step, u half a step of the output type
(finfo.eps / 2).  A value is off by its own rounding, u |value|, and by the
fp32 arithmetic before it.
  * A product over K: 16-bit operands multiply exactly, and a sum takes at
    most K / 4 + 64 fp32 additions in a chain (the matrix instruction adds at
    least four products at once; pieces are joined), so it is off by at most
    (K / 4 + 64) U times the sum of |a| |b|.  An fp32 operand is three bf16
    numbers, six of the nine products are added: a chain of 6 K / 4 + 64, and
    what is left out is below 4 U of |a| |b|.
  * act(z) by exp, erfc and a few operations: relative to |act| (for the
    derivative, to the magnitudes it adds) each operation is off by 2 U, the
    library functions by 4 U; an argument off by 4 U of itself moves exp(w) by
    4 |w| U and erfc by 2 z^2 of that.  (32 + 8 z^2 + 2 |z|^3) U covers all five.
  * act moves by at most 1.2 times its argument (1.13 is the largest slope)."""
import numpy as np
import pytest
import torch

from oracle import activation as A
from oracle import feedforward as F

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTS = ["silu", "gelu", "gelu_tanh", "relu", "sigmoid"]
SEED, OFFSET = 0xFEDCBA9876543210, 0x8000000180000003


@pytest.fixture(scope="module")
def fw():
    import fac_whitening_amd as fw
    return fw


def f64(t):
    return t.detach().cpu().double().numpy()


def half_step(t, v):
    """Half a step of type t at v (of a subnormal number at least)."""
    i = torch.finfo(t)
    return i.eps / 2 * np.maximum(np.abs(v), i.tiny)


def chain(K, dtype):
    return (6 * K / 4 + 68) * U if dtype == "fp32" else (K / 4 + 64) * U


def act_error(z):
    z = np.minimum(np.abs(z), 20)
    return (32 + 8 * z ** 2 + 2 * z ** 3) * U


def strided(T, n, dtype, ld=None, off=0):
    """A [T][n] view with leading dimension ld that starts off elements into its buffer."""
    ld = n if ld is None else ld
    buf = torch.full((off + max(T, 1) * ld,), 777.0, dtype=dtype, device=DEV)
    return torch.as_strided(buf, (T, n), (ld, 1), off)


def untouched(*views):
    """Nothing was written outside the views of strided()."""
    for v in views:
        base = v._base if v._base is not None else v
        mask = torch.ones_like(base, dtype=torch.bool)
        torch.as_strided(mask, v.shape, v.stride(), v.storage_offset()).fill_(False)
        assert (base[mask] == 777.0).all()


def draw(T, n, dtype, seed, scale=1.0, ld=None, off=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    out = strided(T, n, DT[dtype], ld, off)
    out.copy_((torch.randn(T, n, generator=g, device=DEV) * scale).to(DT[dtype]))
    return out


def check(got, want, tol, what):
    bad = ~(np.abs(f64(got) - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4], float(np.nanmax(np.abs(f64(got) - want) / tol)))


# -- dropout -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,d,ld,off,p", [(1, 1, None, 0, 0.5), (1, 1536, None, 0, 0.1), (3, 7, None, 1, 0.3), (9, 8, 24, 8, 0.25),
                                          (17, 100, 107, 3, 0.9), (300, 257, None, 0, 0.1), (5, 4096, 4100, 4, 0.05),
                                          (2000, 40, None, 0, 2.0 ** -16), (33, 1023, None, 1, 65535 / 65536)])
def test_dropout(fw, T, d, ld, off, p, dtype):
    print(f"[dropout {T}x{d} ld {ld} off {off} p {p} {dtype}]", flush=True)
    t = DT[dtype]
    x, r = draw(T, d, dtype, T + d, 1.0, ld, off), draw(T, d, dtype, T + d + 1, 2.0, None if ld is None else ld + 1, off)
    drop = fw.Dropout(p, SEED, OFFSET)
    f = F.factor(T, d, (p, SEED, OFFSET))
    y = fw.dropout_forward(x, drop, residual=r, out=strided(T, d, t, ld, off))
    z = fw.dropout_forward(x, drop)
    dx = fw.dropout_backward(x, drop, dx=strided(T, d, t, ld, off))
    torch.cuda.synchronize()
    v = F.apply(f64(x), f)
    # the scale as an fp32 number, the product, the sum: three roundings
    with np.errstate(over="ignore"):
        check(z, v, half_step(t, v) * 1.01 + 3 * U * np.abs(v), "no residual")
    w = v + f64(r)
    check(y, w, half_step(t, w) * 1.01 + 3 * U * (np.abs(v) + np.abs(f64(r))), "residual")
    assert torch.equal(dx, z) and (f64(z)[f == 0] == 0).all()
    untouched(y, dx)
    # in place, over the input and over the residual
    a, b = x.clone(), r.clone()
    assert torch.equal(fw.dropout_forward(a, drop, residual=r, out=a), y)
    assert torch.equal(fw.dropout_forward(x, drop, residual=b, out=b), y)


def test_dropout_ends_and_masked_values(fw):
    """p = 0 and 1; what is dropped is zero whatever it held."""
    T, d = 40, 200
    x = draw(T, d, "bf16", 3)
    assert torch.equal(fw.dropout_forward(x, fw.Dropout(0.0, 1)), x)
    assert torch.equal(fw.dropout_forward(x, fw.Dropout(1e-6, 1)), x)          # rounds to 0
    one = fw.Dropout(1.0, 1)
    assert (fw.dropout_forward(torch.full_like(x, float("nan")), one) == 0).all()
    assert torch.equal(fw.dropout_forward(x, one, residual=x), x)
    k = F.kept(T, d, 0.5, 7, 0)
    y = fw.dropout_forward(torch.full_like(x, float("inf")), fw.Dropout(0.5, 7))
    assert np.array_equal(f64(y), np.where(k, np.inf, 0.0))
    z = torch.empty(0, d, dtype=torch.bfloat16, device=DEV)
    assert fw.dropout_forward(z, one).shape == (0, d)


def test_dropout_counter_in_a_graph(fw):
    """Replays draw by the counter's value at the time."""
    T, d = 64, 96
    x = torch.ones(T, d, device=DEV)
    counter = torch.zeros(1, dtype=torch.int64, device=DEV)
    drop = fw.Dropout(0.5, 9, offset=(1 << 64) - 2, counter=counter)
    y = torch.empty_like(x)
    fw.dropout_forward(x, drop, out=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fw.dropout_forward(x, drop, out=y)
        counter.add_(1)
    for n in range(5):                    # the sum wraps past 64 bits
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(f64(y), 2.0 * F.kept(T, d, 0.5, 9, ((1 << 64) - 2 + n) % (1 << 64))), n
        x.mul_(1.0).sum().item()
    assert counter.item() == 5


# -- gated feed-forward: forward -------------------------------------------------

def forward_reference(x, wg, wu, act, f, dtype):
    """h, z, u in float64 and what they may be off by."""
    X, G, W = f64(x), f64(wg), f64(wu)
    t = DT[dtype]
    h, z, u = F.glu_forward(X, G, W, act, f)
    c = chain(X.shape[1], dtype)
    ez, eu = c * (np.abs(X) @ np.abs(G).T) + 1e-37, c * (np.abs(X) @ np.abs(W).T) + 1e-37
    a = np.abs(F.act(z, act)[0])
    ea = 1.2 * ez + act_error(z) * a
    eh = np.abs(f) * (ea * (np.abs(u) + eu) + a * eu + 4 * U * a * np.abs(u)) + 1e-37
    return (h, half_step(t, h) * 1.01 + eh), (z, half_step(t, z) * 1.01 + ez), (u, half_step(t, u) * 1.01 + eu)


SHAPES = [(1, 1, 1, 0), (1, 64, 256, 0), (1, 1536, 520, 0), (2, 7, 5, 1), (3, 1001, 77, 0), (5, 33, 31, 3), (8, 128, 64, 0),
          (16, 64, 96, 0), (16, 1000, 200, 8), (17, 100, 130, 1), (31, 260, 300, 0), (32, 512, 384, 0), (33, 257, 129, 0),
          (64, 512, 256, 0), (65, 72, 1000, 0), (100, 96, 72, 4), (128, 640, 128, 0), (130, 300, 260, 0), (200, 1001, 333, 1),
          (257, 513, 255, 0), (300, 256, 512, 0), (515, 1536, 264, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,d,f,off", SHAPES)
def test_glu_forward(fw, T, d, f, off, dtype):
    act = ACTS[(T + d + f) % 5]
    print(f"[glu_forward {T}x{d}x{f} off {off} {dtype} {act}]", flush=True)
    t = DT[dtype]
    ld = None if off == 0 else d + off
    x = draw(T, d, dtype, T + d, 1.0, ld, off)
    wg, wu = (draw(f, d, dtype, T + f + i, 1.5 * d ** -0.5, ld, off) for i in range(2))
    wg.mul_(1.5)
    wide = None if off == 0 else 2 * f + off
    h = strided(T, f, t, wide, off)
    gate, up = strided(T, f, t, wide, off), strided(T, f, t, wide, off)
    fw.glu_forward(x, wg, wu, act, out=h, gate=gate, up=up)
    torch.cuda.synchronize()
    (rh, th), (rz, tz), (ru, tu) = forward_reference(x, wg, wu, act, np.ones((T, f)), dtype)
    check(gate, rz, tz, "gate")
    check(up, ru, tu, "up")
    check(h, rh, th, "h")
    untouched(h, gate, up)
    # dropout on the way, no pre-activations, a checkpoint beside it
    drop = (0.25, SEED, OFFSET + T)
    ck = fw.ActCheckpoint(T, f, "e4m3", device=DEV)
    h2, none, none2 = fw.glu_forward(x, wg, wu, act, drop=fw.Dropout(*drop), ckpt=ck, out=strided(T, f, t, wide, off))
    torch.cuda.synchronize()
    assert none is None and none2 is None
    k = F.factor(T, f, drop)
    (rh, th), _, _ = forward_reference(x, wg, wu, act, k, dtype)
    check(h2, rh, th, "h with dropout")
    assert (f64(h2)[k == 0] == 0).all()
    untouched(h2)
    codes, e = A.ckpt_save(f64(h2), "e4m3")
    assert np.array_equal(ck.codes.cpu().numpy(), codes)
    got = ck.bscales.cpu().numpy()
    assert all(np.array_equal(got[i // 8, :, i % 8], e[i]) for i in range(T))


@pytest.mark.parametrize("act", ACTS)
def test_glu_activations_over_their_range(fw, act):
    """z from -40 to 40 through a product of one term, fp32: act's own accuracy, u = 1."""
    n = 4001
    z = torch.linspace(-40, 40, n, device=DEV).view(n, 1)
    one = torch.ones(1, 1, device=DEV)
    for w, f in ((one, None), (torch.ones(2, 1, device=DEV), None)):
        # u = 1: w_up . x with a second column
        x = torch.cat([z, torch.ones_like(z)], 1)
        wg, wu = torch.tensor([[1.0, 0.0]], device=DEV), torch.tensor([[0.0, 1.0]], device=DEV)
        h, gate, up = fw.glu_forward(x, wg, wu, act, keep=True)
    Z = f64(z)
    assert np.array_equal(f64(gate), Z) and (f64(up) == 1).all()
    a, da = F.act(Z, act)
    check(h, a, (act_error(Z) + U) * np.abs(a) + 1e-37, act)
    dx, dgate, dup = fw.glu_backward(torch.ones_like(h), gate, up, act=act)
    assert dx is None
    mag = np.abs(da) + np.abs(a) + np.abs(Z) * np.exp(-np.abs(Z) / 2) + np.exp(-np.abs(Z))
    check(dgate, da, act_error(Z) * mag + 1e-37, act + " derivative")
    assert torch.equal(dup, h)


def test_glu_forward_weights_as_halves_of_one(fw):
    T, d, f = 70, 192, 160
    x, w = draw(T, d, "bf16", 1), draw(2 * f, d, "bf16", 2, d ** -0.5)
    a = fw.glu_forward(x, w[:f], w[f:], keep=True)
    b = fw.glu_forward(x, w[:f].clone(), w[f:].clone(), keep=True)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    # h alone is the same with and without the pre-activations
    assert torch.equal(fw.glu_forward(x, w[:f], w[f:])[0], a[0])


@pytest.mark.parametrize("T", [1, 20, 300])
def test_glu_forward_nonfinite_stays_in_its_row_or_column(fw, T):
    d, f = 200, 150
    for dtype in DT:
        x, wg, wu = draw(T, d, dtype, 1), draw(f, d, dtype, 2, 0.1), draw(f, d, dtype, 3, 0.1)
        wg[7, 3] = float("nan")
        wu[9, 5] = float("inf")
        if T > 1:
            x[T // 2, 11] = float("nan")
        h = f64(fw.glu_forward(x, wg, wu)[0])
        assert np.isnan(h[:, 7]).all()
        # (an infinity in an fp32 operand may give NaN)
        assert not np.isfinite(h[:, 9]).any() or (f64(x)[:, 5] == 0).any()
        rows, cols = np.ones(T, bool), np.ones(f, bool)
        cols[[7, 9]] = False
        if T > 1:
            rows[T // 2] = False
            assert np.isnan(h[T // 2]).all()
        assert np.isfinite(h[rows][:, cols]).all()


# -- gated feed-forward: backward ------------------------------------------------

def gradients_reference(dh, gate, up, act, f, dtype):
    """dgate and dup in float64 and what they may be off by."""
    t = DT[dtype]
    D, Z, W = f64(dh), f64(gate), f64(up)
    dz, du = F.glu_gradients(D, Z, W, act, f)
    a, da = F.act(Z, act)
    e = np.abs(F.apply(D, f))
    mag = np.abs(da) + np.abs(a) + np.abs(Z) * np.exp(-np.abs(Z) / 2) + np.exp(-np.abs(Z))
    tz = e * np.abs(W) * (act_error(Z) * mag + 6 * U * np.abs(da))
    tu = e * (act_error(Z) + 6 * U) * np.abs(a)
    return (dz, half_step(t, dz) * 1.01 + tz + 1e-37), (du, half_step(t, du) * 1.01 + tu + 1e-37)


def check_dx(dx, dgate, dup, wg, wu, dtype):
    """dx is the product of the rounded gradients."""
    t = DT[dtype]
    Z, W, G, V = f64(dgate), f64(dup), f64(wg), f64(wu)
    want = Z @ G + W @ V
    mag = np.abs(Z) @ np.abs(G) + np.abs(W) @ np.abs(V)
    check(dx, want, half_step(t, want) * 1.01 + chain(2 * Z.shape[1], dtype) * mag + 1e-37, "dx")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,d,f,off", SHAPES)
def test_glu_backward(fw, T, d, f, off, dtype):
    act = ACTS[(T + d + 2 * f) % 5]
    print(f"[glu_backward {T}x{d}x{f} off {off} {dtype} {act}]", flush=True)
    t = DT[dtype]
    ldw, ldf = (None, None) if off == 0 else (d + off, f + off)
    dh = draw(T, f, dtype, T, 0.2, ldf, off)
    gate, up = draw(T, f, dtype, T + 1, 1.5, ldf, off), draw(T, f, dtype, T + 2, 1.0, ldf, off)
    wg, wu = (draw(f, d, dtype, T + f + i, f ** -0.5, ldw, off) for i in range(2))
    drop = None if T % 2 else (0.1, SEED, OFFSET)
    dx, dgate, dup = fw.glu_backward(dh, gate, up, wg, wu, act, None if drop is None else fw.Dropout(*drop),
                                     dx=strided(T, d, t, ldw, off), dgate=strided(T, f, t, ldf, off),
                                     dup=strided(T, f, t, ldf, off))
    torch.cuda.synchronize()
    (rz, tz), (ru, tu) = gradients_reference(dh, gate, up, act, F.factor(T, f, drop), dtype)
    check(dgate, rz, tz, "dgate")
    check(dup, ru, tu, "dup")
    check_dx(dx, dgate, dup, wg, wu, dtype)
    untouched(dx, dgate, dup)


def test_glu_backward_in_place_and_without_dx(fw):
    T, d, f = 90, 128, 200
    dh, gate, up = (draw(T, f, "bf16", i) for i in range(3))
    wg, wu = draw(f, d, "bf16", 4, 0.1), draw(f, d, "bf16", 5, 0.1)
    want = fw.glu_backward(dh, gate, up, wg, wu, "gelu")
    none, dgate, dup = fw.glu_backward(dh, gate, up, act="gelu")
    assert none is None and torch.equal(dgate, want[1]) and torch.equal(dup, want[2])
    for over in ((0, 1), (1, 2), (2, 1), (1, 0)):
        a = [dh.clone(), gate.clone(), up.clone()]
        got = fw.glu_backward(*a, wg, wu, "gelu", dgate=a[over[0]], dup=a[over[1]])
        assert all(torch.equal(p, q) for p, q in zip(got, want)), over
    # both gradients as halves of one matrix
    both = torch.empty(T, 2 * f, dtype=torch.bfloat16, device=DEV)
    got = fw.glu_backward(dh, gate, up, wg, wu, "gelu", dgate=both[:, :f], dup=both[:, f:])
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_no_rows(fw):
    d, f = 64, 96
    for dtype, t in DT.items():
        x, h = torch.empty(0, d, dtype=t, device=DEV), torch.empty(0, f, dtype=t, device=DEV)
        wg, wu = draw(f, d, dtype, 1), draw(f, d, dtype, 2)
        ck = fw.ActCheckpoint(0, f, device=DEV)
        out = fw.glu_forward(x, wg, wu, keep=True, ckpt=ck, drop=fw.Dropout(0.1, 1))
        assert all(o.shape == (0, f) for o in out)
        dx, dgate, dup = fw.glu_backward(h, h, h, wg, wu)
        assert dx.shape == (0, d) and dgate.shape == (0, f) and dup.shape == (0, f)
        W = fw.weight_grad(h, x)
        assert W.shape == (f, d) and (W == 0).all()
        W.fill_(3.0)
        fw.weight_grad(h, x, out=W, accumulate=True)
        assert (W == 3.0).all()


def test_gradients_against_differences(fw):
    """Directional differences of the fp32 forward against the backward.  Their truncation is what the float64 oracle
    shows at the same step; the forward's own error, divided by the step, is the rest."""
    T, d, f, e = 12, 40, 56, 2.0 ** -6
    x, wg, wu = draw(T, d, "fp32", 1), draw(f, d, "fp32", 2, d ** -0.5), draw(f, d, "fp32", 3, d ** -0.5)
    dh = draw(T, f, "fp32", 4)
    v, vg, vu = draw(T, d, "fp32", 5), draw(f, d, "fp32", 6, d ** -0.5), draw(f, d, "fp32", 7, d ** -0.5)
    drop = (0.25, 3, 4)
    k = F.factor(T, f, drop)
    for act in ("silu", "gelu", "gelu_tanh", "sigmoid"):
        h, gate, up = fw.glu_forward(x, wg, wu, act, keep=True, drop=fw.Dropout(*drop))
        dx, dgate, dup = fw.glu_backward(dh, gate, up, wg, wu, act, fw.Dropout(*drop))
        dwg, dwu = fw.weight_grad(dgate, x), fw.weight_grad(dup, x)
        slope = (f64(dx) * f64(v)).sum() + (f64(dwg) * f64(vg)).sum() + (f64(dwu) * f64(vu)).sum()
        got, ref, noise = [], [], 0.0
        for s in (e, -e):
            a = (x + s * v, wg + s * vg, wu + s * vu)
            hs = fw.glu_forward(*a, act, drop=fw.Dropout(*drop))[0]
            got.append((f64(dh) * f64(hs)).sum())
            (rh, th), _, _ = forward_reference(*a, act, k, "fp32")
            ref.append((f64(dh) * rh).sum())
            noise += (np.abs(f64(dh)) * th).sum() / (2 * e)
        num, true = (got[0] - got[1]) / (2 * e), (ref[0] - ref[1]) / (2 * e)
        assert abs(num - true) <= noise
        Z, W = f64(x) @ f64(wg).T, f64(x) @ f64(wu).T
        dz, du = F.glu_gradients(f64(dh), Z, W, act, k)
        exact = ((dz @ f64(wg) + du @ f64(wu)) * f64(v)).sum() + (dz.T @ f64(x) * f64(vg)).sum() + (
            du.T @ f64(x) * f64(vu)).sum()
        assert abs(slope - num) <= abs(exact - true) + 2 * noise, (act, slope, num, exact, true, noise)


# -- weight gradient from a whole activation -------------------------------------

def check_wgrad(W, delta, x, alpha, dtype, old=None):
    D, X = f64(delta), f64(x)
    want, mag = alpha * (D.T @ X), abs(alpha) * (np.abs(D).T @ np.abs(X))
    if old is not None:
        want, mag = want + old, mag + np.abs(old)
    check(W, want, chain(D.shape[0], dtype) * mag + 1e-37, "W")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,m,d,off", [(1, 1, 1, 0), (1, 64, 256, 0), (7, 3, 5, 1), (31, 4, 33, 0), (32, 5, 64, 2), (33, 129, 127, 0),
                                       (64, 256, 256, 0), (100, 255, 257, 3), (1000, 64, 256, 0), (515, 300, 700, 1),
                                       (2048, 520, 264, 0), (1537, 131, 1001, 0), (640, 512, 768, 8)])
def test_weight_grad_from_x(fw, T, m, d, off, dtype):
    print(f"[wgrad_x T {T} {m}x{d} off {off} {dtype}]", flush=True)
    delta = draw(T, m, dtype, T + m, 0.05, None if off == 0 else m + off, off)
    x = draw(T, d, dtype, T + d, 1.0, None if off == 0 else d + off, off)
    W = strided(m, d, torch.float32, d + 3, 1)
    fw.weight_grad(delta, x, alpha=1.0 / T, out=W)
    torch.cuda.synchronize()
    check_wgrad(W, delta, x, float(np.float32(1.0 / T)), dtype)
    untouched(W)
    old = f64(W)
    fw.weight_grad(delta, x, alpha=-0.5, out=W, accumulate=True)
    torch.cuda.synchronize()
    check_wgrad(W, delta, x, -0.5, dtype, old)
    untouched(W)


def test_weight_grad_from_x_exact_integers(fw):
    """Small integers: every product and sum is exact in fp32, whatever the order."""
    g = torch.Generator(device=DEV).manual_seed(3)
    for T, m, d in ((700, 300, 520), (4096, 256, 512)):
        for t in DT.values():
            x = torch.randint(-8, 9, (T, d), generator=g, device=DEV).to(t)
            delta = torch.randint(-100, 101, (T, m), generator=g, device=DEV).to(t)
            assert np.array_equal(f64(fw.weight_grad(delta, x)), f64(delta).T @ f64(x))


def test_weight_grad_of_both_forms_agree(fw):
    """From a checkpoint and from the values that it stands for."""
    T, m, d = 900, 200, 320
    delta, x = draw(T, m, "bf16", 1), draw(T, d, "bf16", 2)
    ck = fw.ActCheckpoint(T, d, device=DEV).save(x)
    a, b = f64(fw.weight_grad(delta, ck)), f64(fw.weight_grad(delta, ck.restore(torch.bfloat16)))
    mag = np.abs(f64(delta)).T @ np.abs(f64(ck.restore(torch.float32)))
    assert (np.abs(a - b) <= 2 * chain(T, "bf16") * mag).all()


# -- together ----------------------------------------------------------------------

class Block:
    """Norm, gated block with hidden dropout, down projection, residual dropout; their backward passes and the
    weight gradients of both projections."""

    def __init__(self, fw, T, d, f, dtype="bf16"):
        self.fw, self.T = fw, T
        self.x, self.dout = draw(T, d, dtype, 1), draw(T, d, dtype, 2, 0.1)
        self.w, self.wd = draw(2 * f, d, dtype, 3, d ** -0.5), draw(d, f, dtype, 4, f ** -0.5)
        self.gamma = torch.ones(d, dtype=DT[dtype], device=DEV)
        self.f = f
        self.ck = fw.ActCheckpoint(T, f, device=DEV)
        self.counter = torch.zeros(1, dtype=torch.int64, device=DEV)
        self.hidden = fw.Dropout(0.1, 11, 0, self.counter)
        self.resid = fw.Dropout(0.2, 12, 0, self.counter)
        self.dgu = torch.empty(T, 2 * f, dtype=DT[dtype], device=DEV)

    def step(self):
        fw, f = self.fw, self.f
        y, _, rstd = fw.norm_forward(self.x, self.gamma, kind="rms")
        h, gate, up = fw.glu_forward(y, self.w[:f], self.w[f:], keep=True, drop=self.hidden, ckpt=self.ck)
        o = h.float() @ self.wd.float().t()
        out = fw.dropout_forward(o.to(self.x.dtype), self.resid, residual=self.x)
        do = fw.dropout_backward(self.dout, self.resid)
        dwd = fw.weight_grad(do, self.ck, 1.0 / self.T)
        dh = (do.float() @ self.wd.float()).to(do.dtype)
        dy, _, _ = fw.glu_backward(dh, gate, up, self.w[:f], self.w[f:], drop=self.hidden, dgate=self.dgu[:, :f],
                                   dup=self.dgu[:, f:])
        dw = fw.weight_grad(self.dgu, y, 1.0 / self.T)
        dx, dgamma, _ = fw.norm_backward(dy, self.x, None, rstd, self.gamma, kind="rms")
        return out, dx, dgamma, dw, dwd, h, self.dgu


def test_block_on_a_stream_and_in_a_graph(fw):
    b = Block(fw, 300, 192, 320)
    want = {}
    for n in range(3):
        b.counter.fill_(n)
        want[n] = [v.clone() for v in b.step()]
    assert not torch.equal(want[0][5], want[1][5])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.counter.fill_(1)
        got = b.step()
        side.synchronize()
        assert all(torch.equal(g, v) for g, v in zip(got, want[1]))
    b.counter.zero_()
    b.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = b.step()
    for n in (0, 1, 2, 0, 1):
        for v in got:
            v.zero_()
        b.counter.fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, v) for g, v in zip(got, want[n])), n
        b.x.mul_(1.0).sum().item()
        b.dout.clone()


def test_block_against_the_oracle(fw):
    """dx of the whole chain in fp32: every operator within its own bound, so the chain is compared loosely but over
    all of its parts (fp32 sums of up to a few hundred terms through six operators: 1e-4 of the largest magnitude)."""
    T, d, f = 48, 64, 96
    b = Block(fw, T, d, f, "fp32")
    out, dx, dgamma, dw, dwd, h, dgu = b.step()
    X, W, V = f64(b.x), f64(b.w), f64(b.wd)
    y, mean, rstd = A.norm_forward(X, np.ones(d), None, 1e-5, "rms")
    kh, kr = F.factor(T, f, (0.1, 11, 0)), F.factor(T, d, (0.2, 12, 0))
    H, z, u = F.glu_forward(y, W[:f], W[f:], "silu", kh)
    want_out = F.apply(H @ V.T, kr) + X
    do = F.apply(f64(b.dout), kr)
    dz, du = F.glu_gradients(do @ V, z, u, "silu", kh)
    dy = dz @ W[:f] + du @ W[f:]
    rdx, rdg, _ = A.norm_backward(dy, X, mean, rstd, np.ones(d), "rms")
    codes, e = A.ckpt_save(f64(h), "e4m3")
    for got, want in ((out, want_out), (h, H), (dx, rdx), (dgamma, rdg), (dw, np.concatenate([dz, du], 1).T @ y / T),
                      (dwd, do.T @ A.ckpt_values(codes, e, f, "e4m3") / T)):
        assert np.abs(f64(got) - want).max() <= 1e-4 * np.abs(want).max()


def test_calls_repeat_bit_for_bit(fw):
    T, d, f = 700, 328, 1100
    for dtype in DT:
        x, dh = draw(T, d, dtype, 1), draw(T, f, dtype, 2)
        wg, wu = draw(f, d, dtype, 3, 0.05), draw(f, d, dtype, 4, 0.05)
        drop = fw.Dropout(0.1, 5)
        first = None
        for _ in range(3):
            h, gate, up = fw.glu_forward(x, wg, wu, keep=True, drop=drop)
            out = (h, gate, up, *fw.glu_backward(dh, gate, up, wg, wu, drop=drop), fw.weight_grad(dh, x))
            first = first or out
            assert all(torch.equal(a, b) for a, b in zip(out, first))


def test_given_stream_owns_what_it_allocates(fw):
    """Calls on another stream than the current one: outputs and workspaces are that stream's."""
    T, d, f = 600, 301, 501          # rows that the workspace holds anew
    x, dh = draw(T, d, "bf16", 1), draw(T, f, "bf16", 2)
    wg, wu = draw(f, d, "bf16", 3, 0.05), draw(f, d, "bf16", 4, 0.05)
    h, gate, up = fw.glu_forward(x, wg, wu, keep=True)
    want = (h, gate, up, *fw.glu_backward(dh, gate, up, wg, wu), fw.weight_grad(dh, x))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        h2, gate2, up2 = fw.glu_forward(x, wg, wu, keep=True, stream=s)
        got = (h2, gate2, up2, *fw.glu_backward(dh, gate2, up2, wg, wu, stream=s), fw.weight_grad(dh, x, stream=s))
        junk = [torch.full((1 << 18,), 5.0, device=DEV) for _ in range(8)]    # the current stream's allocations
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del junk


def test_workspace_too_small_is_refused(fw):
    """Where a call needs a workspace, one byte less is an error before anything is enqueued."""
    T, d, f = 200, 301, 333
    x, wg, wu = draw(T, d, "fp32", 1), draw(f, d, "fp32", 2), draw(f, d, "fp32", 3)
    n = fw._lib.gift_glu_workspace_bytes(T, d, f, fw.FP32, 0)
    if n:
        h = torch.full((T, f), 5.0, device=DEV)
        with pytest.raises(fw.GiftError):
            fw.glu_forward(x, wg, wu, out=h, work=torch.empty(n - 1, dtype=torch.uint8, device=DEV))
        torch.cuda.synchronize()
        assert (h == 5.0).all()
