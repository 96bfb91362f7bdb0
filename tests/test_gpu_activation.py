"""Activation operators on the GPU against their float64 oracle: 8-bit
checkpoints (bit for bit), layer / RMS norm forward and backward (from the
input and from its checkpoint), the weight gradient, their use together,
on a side stream and in a graph.

Tolerances.  u = 2^-24 is fp32's half step, u_t half a step of the output type
(finfo.eps / 2).  A value is off by its own rounding, u_t |value|, and by the
fp32 arithmetic before it: each sum of the forward and backward runs over at
most 41 additions in a chain (32 elements of a lane, 6 lane exchanges, 7
waves), and a handful of roundings follow, so 100 u times the magnitudes that
are added bounds the forward, 200 u the backward (two such sums meet there).
Parameter gradients up to 4096 rows: 8 rows of a workgroup, 4 waves, 16
partials in a thread and 32 threads are 60 additions: 100 u.  The weight
gradient's products are exact; its chain is at most T / 4 + 64 additions."""
import numpy as np
import pytest
import torch

from oracle import activation as A

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def fw():
    import fac_whitening_amd as fw
    return fw


def u_of(t):
    return torch.finfo(t).eps / 2


def f64(t):
    return t.detach().cpu().double().numpy()


def strided(T, n, dtype, ld=None, off=0):
    """A [T][n] view with leading dimension ld that starts off elements into its buffer."""
    ld = n if ld is None else ld
    buf = torch.full((off + max(T, 1) * ld,), 777.0, dtype=dtype, device=DEV)
    return torch.as_strided(buf, (T, n), (ld, 1), off)


def draw(T, n, dtype, seed, scale=1.0, ld=None, off=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    v = torch.randn(T, n, generator=g, device=DEV) * torch.exp(torch.randn(T, 1, generator=g, device=DEV)) * scale
    out = strided(T, n, dtype, ld, off)
    out.copy_((v + 0.5).to(dtype))
    return out


# -- checkpoints -------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,d,ld,off", [(1, 1, None, 0), (3, 7, None, 1), (8, 32, 40, 0), (9, 33, None, 0),
                                        (17, 100, 107, 3), (5, 2048, None, 0), (20, 2081, 2090, 1), (70, 257, None, 0)])
def test_checkpoint_bits(fw, T, d, ld, off, dtype, fmt):
    print(f"[ckpt {T}x{d} ld {ld} off {off} {dtype} {fmt}]", flush=True)
    x = draw(T, d, DT[dtype], 1 + T + d, 3.0, ld, off)
    x[T // 2, :] *= 1e-3
    if d >= 40:
        x[0, :33] = 0
        x[T - 1, 32:40] = torch.tensor([448.0, 449.0, -57344.0, 3e-5, -0.0, 2e-8, 240.0, 17.0]).to(x)
    ck = fw.ActCheckpoint(T, d, fmt, device=DEV)
    ck.codes.fill_(0xAA)
    ck.bscales.fill_(0xAA)
    ck.save(x)
    torch.cuda.synchronize()
    codes, e = A.ckpt_save(f64(x), fmt)
    assert np.array_equal(ck.codes.cpu().numpy(), codes)
    lay, got = A.exponent_layout(e), ck.bscales.cpu().numpy()
    for t in range(T):
        assert np.array_equal(got[t // 8, :, t % 8], lay[t // 8, :, t % 8])
    want = A.ckpt_values(codes, e, d, fmt)
    for o in ("bf16", "fp32", "fp16"):
        out = strided(T, d, DT[o], None if ld is None else ld + 2, off)
        ck.restore(out=out)
        torch.cuda.synchronize()
        with np.errstate(over="ignore"):
            w = want.astype(np.float16).astype(np.float64) if o == "fp16" else want
        assert np.array_equal(f64(out), w), o
        base = out._base if out._base is not None else out
        mask = torch.ones_like(base, dtype=torch.bool)
        torch.as_strided(mask, out.shape, out.stride(), out.storage_offset()).fill_(False)
        assert (base[mask] == 777.0).all()          # nothing outside the rows


def test_checkpoint_extremes(fw):
    fi = torch.finfo(torch.float32)
    x = torch.zeros(4, 96, device=DEV)
    x[0, 3], x[0, 40] = float("inf"), float("nan")
    x[1, :32] = fi.max / 2
    x[1, 32:64] = fi.tiny
    x[1, 64:] = 2.0 ** -100
    x[2, :32] = torch.linspace(-3e-30, 3e-30, 32)
    x[3, :32] = -float("inf")
    for fmt in ("e4m3", "e5m2"):
        ck = fw.ActCheckpoint(4, 96, fmt, device=DEV).save(x)
        codes, e = A.ckpt_save(f64(x), fmt)
        torch.cuda.synchronize()
        assert np.array_equal(ck.codes.cpu().numpy(), codes)
        assert np.array_equal(ck.bscales.cpu().numpy()[0, :, :4].T, e)
        assert np.array_equal(f64(ck.restore(torch.float32)), A.ckpt_values(codes, e, 96, fmt), equal_nan=True)


# -- norms ---------------------------------------------------------------------

SHAPES = [(1, 1, None, 0), (5, 3, None, 1), (33, 64, None, 0), (17, 128, 131, 0), (9, 129, None, 0), (7, 512, 520, 0),
          (10, 1023, None, 1), (1, 1536, None, 0), (70, 1536, 1540, 4), (6, 2047, None, 0), (5, 2049, 2055, 1),
          (9, 4096, None, 0), (3, 6144, None, 0), (3, 8191, None, 0), (2, 12288, None, 0), (3, 16384, None, 0),
          (2, 16383, None, 1)]


def _params(d, dtype, kind, wdtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    wt = torch.float32 if wdtype == "fp32" else DT[dtype]
    w = (1 + 0.3 * torch.randn(d, generator=g, device=DEV)).to(wt)
    b = torch.randn(d, generator=g, device=DEV).to(wt) if kind == "layer" else None
    return (None, None) if wdtype is None else (w, b)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "same"), ("bf16", "fp32"), ("fp16", "same"), ("fp32", "same"),
                                          ("bf16", None)])
@pytest.mark.parametrize("T,d,ld,off", SHAPES)
def test_norm_against_oracle(fw, T, d, ld, off, dtype, wdtype, kind):
    print(f"[norm {T}x{d} ld {ld} off {off} {dtype} w {wdtype} {kind}]", flush=True)
    eps, t = 1e-5, DT[dtype]
    x = draw(T, d, t, 7 * T + d, 1.0, ld, off)
    dy = draw(T, d, t, 9 * T + d, 0.1, None if ld is None else ld + 1, off)
    w, b = _params(d, dtype, kind, wdtype, d)
    ck = fw.ActCheckpoint(T, d, "e4m3", device=DEV)
    y, mean, rstd = fw.norm_forward(x, w, b, eps, kind, ckpt=ck, out=strided(T, d, t, ld, off))
    y2, mean2, rstd2 = fw.norm_forward(x, w, b, eps, kind)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(rstd, rstd2)
    X, W, B = f64(x), None if w is None else f64(w), None if b is None else f64(b)
    ry, rm, rr = A.norm_forward(X, W, B, eps, kind)
    aw = np.ones(d) if W is None else np.abs(W)
    spread = np.abs(X).mean(1)[:, None]
    tol = u_of(t) * np.abs(ry) + 100 * U * (aw * (np.abs(X - rm[:, None]) + spread) * rr[:, None] +
                                            (0 if B is None else np.abs(B)))
    tol = np.maximum(tol, torch.finfo(t).tiny)
    assert (np.abs(f64(y) - ry) <= tol).all()
    if kind == "layer":
        assert (np.abs(f64(mean) - rm) <= 100 * U * spread[:, 0]).all()
    else:
        assert mean is None
    var = 1 / rr ** 2
    assert (np.abs(f64(rstd) - rr) <= 100 * U * rr * (1 + spread[:, 0] ** 2 * 100 * U / var)).all()
    codes, e = A.ckpt_save(X, "e4m3")
    assert np.array_equal(ck.codes.cpu().numpy(), codes)
    got = ck.bscales.cpu().numpy()
    assert all(np.array_equal(got[i // 8, :, i % 8], e[i]) for i in range(T))
    # backward, from the input and from its checkpoint, with the forward's own mean and rstd
    M = np.zeros(T) if mean is None else f64(mean)
    for src, XS in ((x, X), (ck, A.ckpt_values(codes, e, d, "e4m3"))):
        dx, dw, db = fw.norm_backward(dy, src, mean, rstd, w, kind, dx=strided(T, d, t, ld, off))
        torch.cuda.synchronize()
        _check_backward(dx, dw, db, f64(dy), XS, M, f64(rstd), W, kind, t)


def _check_backward(dx, dw, db, DY, X, M, R, W, kind, t):
    rdx, rdw, rdb = A.norm_backward(DY, X, M, R, W, kind)
    g = np.abs(DY * (1.0 if W is None else W))
    xh = (X - M[:, None]) * R[:, None]
    mag = g + g.mean(1)[:, None] + np.abs(xh) * (g * np.abs(xh)).mean(1)[:, None]
    tol = np.maximum(u_of(t) * np.abs(rdx) + 200 * U * R[:, None] * mag, torch.finfo(t).tiny)
    assert (np.abs(f64(dx) - rdx) <= tol).all()
    assert (np.abs(f64(dw) - rdw) <= 100 * U * np.abs(DY * xh).sum(0) + 1e-37).all()
    if kind == "layer":
        assert (np.abs(f64(db) - rdb) <= 100 * U * np.abs(DY).sum(0) + 1e-37).all()
    else:
        assert db is None


@pytest.mark.parametrize("T,d", [(4096, 96), (2000, 512), (4096, 1536), (700, 4096)])
def test_norm_backward_many_rows(fw, T, d):
    """More row groups than one workgroup takes at once; parameter gradients over all of them."""
    x, dy = draw(T, d, torch.bfloat16, 3), draw(T, d, torch.bfloat16, 4)
    w, b = _params(d, "bf16", "layer", "same", 5)
    _, mean, rstd = fw.norm_forward(x, w, b)
    dx, dw, db = fw.norm_backward(dy, x, mean, rstd, w)
    torch.cuda.synchronize()
    _check_backward(dx, dw, db, f64(dy), f64(x), f64(mean), f64(rstd), f64(w), "layer", torch.bfloat16)


def test_norm_rows_past_the_partials(fw):
    """Every workgroup takes several row groups (T over 8 x 512), compared
    with the sums of two halves: chains of at most T / 2048 + 60 additions."""
    T, d = 9001, 200
    x, dy = draw(T, d, torch.float32, 13), draw(T, d, torch.float32, 14)
    _, mean, rstd = fw.norm_forward(x)
    dx, dw, db = fw.norm_backward(dy, x, mean, rstd)
    torch.cuda.synchronize()
    _check_backward(dx, dw, db, f64(dy), f64(x), f64(mean), f64(rstd), None, "layer", torch.float32)


def test_norm_edge_rows(fw):
    """Constant rows (no variance), zero rows, rows with an Inf or NaN: the
    others are not touched by them."""
    T, d = 24, 300
    x = draw(T, d, torch.float32, 21)
    x[2], x[5] = 4.0, 0.0
    x[7, 11], x[9, 250] = float("inf"), float("nan")
    for kind in ("layer", "rms"):
        y, mean, rstd = fw.norm_forward(x, kind=kind)
        with np.errstate(invalid="ignore"):
            ry, rm, rr = A.norm_forward(f64(x), None, None, 1e-5, kind)
        good = [i for i in range(T) if i not in (7, 9)]
        assert np.allclose(f64(y)[good], ry[good], rtol=0, atol=2e-4)
        assert np.isnan(f64(y)[9]).all() and np.isnan(f64(y)[7, 11])
        if kind == "layer":
            assert (f64(y)[2] == 0).all() and np.isnan(f64(y)[7]).all()
        assert (f64(y)[5] == 0).all()
        dy = draw(T, d, torch.float32, 22)
        dx, dw, db = fw.norm_backward(dy, x, mean, rstd, kind=kind)
        assert torch.isfinite(dx[good]).all() and not torch.isfinite(dx[[7, 9]]).all()


def test_norm_in_place_and_accumulate(fw):
    T, d = 37, 1000
    x, dy = draw(T, d, torch.bfloat16, 31), draw(T, d, torch.bfloat16, 32)
    w, b = _params(d, "bf16", "layer", "fp32", 33)
    y, mean, rstd = fw.norm_forward(x, w, b)
    dx, dw, db = fw.norm_backward(dy, x, mean, rstd, w)
    z = x.clone()
    fw.norm_forward(z, w, b, out=z)
    assert torch.equal(z, y)
    g = dy.clone()
    dw2, db2 = torch.full_like(dw, 2.0), torch.full_like(db, -1.0)
    fw.norm_backward(g, x, mean, rstd, w, dx=g, dweight=dw2, dbias=db2, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(g, dx) and torch.equal(dw2, dw + 2.0) and torch.equal(db2, db - 1.0)
    # one gradient alone, or none
    dw3 = torch.empty_like(dw)
    fw.norm_backward(dy, x, mean, rstd, w, dweight=dw3)
    assert torch.equal(dw3, dw)


def test_no_rows(fw):
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    ck = fw.ActCheckpoint(0, 64, device=DEV)
    y, mean, rstd = fw.norm_forward(x, ckpt=ck)
    dx, dw, db = fw.norm_backward(x, ck, mean, rstd)
    assert y.shape == (0, 64) and dx.shape == (0, 64)
    assert (dw == 0).all() and (db == 0).all()
    W = fw.weight_grad(torch.empty(0, 40, dtype=torch.float32, device=DEV), ck)
    assert W.shape == (40, 64) and (W == 0).all()
    W.fill_(3.0)
    fw.weight_grad(torch.empty(0, 40, dtype=torch.float32, device=DEV), ck, out=W, accumulate=True)
    assert (W == 3.0).all()
    assert ck.restore().shape == (0, 64)


# -- weight gradient -------------------------------------------------------------

def _ckpt(fw, T, d, fmt, seed):
    x = draw(T, d, torch.bfloat16, seed)
    ck = fw.ActCheckpoint(T, d, fmt, device=DEV).save(x)
    torch.cuda.synchronize()
    return ck, f64(ck.restore(torch.float32))


def _check_wgrad(W, DELTA, a, alpha, T, old=None):
    ref = A.weight_grad(DELTA, a, alpha)
    mag = abs(alpha) * (np.abs(DELTA).T @ np.abs(a))
    if old is not None:
        ref, mag = ref + old, mag + np.abs(old)
    tol = (T / 4 + 64) * U * mag
    assert (np.abs(W - ref) <= tol + 1e-37).all(), float((np.abs(W - ref) / (tol + 1e-37)).max())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,m,d,ld,off", [
    (1, 1, 1, None, 0), (1, 64, 256, None, 0), (7, 3, 5, None, 1), (31, 4, 33, None, 0), (32, 5, 64, 9, 2),
    (33, 129, 127, None, 0), (64, 256, 256, None, 0), (100, 255, 257, 261, 3), (1000, 64, 256, None, 0),
    (515, 300, 700, None, 1), (2048, 520, 264, None, 0), (1537, 131, 1001, None, 0)])
def test_weight_grad_against_oracle(fw, T, m, d, ld, off, dtype):
    print(f"[wgrad T {T} {m}x{d} ld {ld} off {off} {dtype}]", flush=True)
    fmt = "e5m2" if (T + m) % 2 else "e4m3"
    ck, a = _ckpt(fw, T, d, fmt, T + d)
    ck.bscales.view(-1)  # exponents past T may hold anything
    if T % 8:
        ck.bscales[-1, :, T % 8:] = 255
    delta = draw(T, m, DT[dtype], T + m, 0.01, ld, off)
    W = strided(m, d, torch.float32, d + 3, 1)
    fw.weight_grad(delta, ck, alpha=1.0 / T, out=W)
    torch.cuda.synchronize()
    _check_wgrad(f64(W), f64(delta), a, float(np.float32(1.0 / T)), T)
    mask = torch.ones_like(W._base, dtype=torch.bool)
    torch.as_strided(mask, W.shape, W.stride(), W.storage_offset()).fill_(False)
    assert (W._base[mask] == 777.0).all()
    old = W.clone()
    fw.weight_grad(delta, ck, alpha=-0.5, out=W, accumulate=True)
    torch.cuda.synchronize()
    _check_wgrad(f64(W), f64(delta), a, -0.5, T, f64(old))


def test_weight_grad_exact_integers(fw):
    """Small integers: every product and sum is exact in fp32, whatever the order."""
    g = torch.Generator(device=DEV).manual_seed(3)
    for T, m, d in ((700, 300, 520), (4096, 256, 512)):
        x = torch.randint(-8, 9, (T, d), generator=g, device=DEV).to(torch.bfloat16)
        ck = fw.ActCheckpoint(T, d, "e4m3", device=DEV).save(x)
        for t in DT.values():
            delta = torch.randint(-100, 101, (T, m), generator=g, device=DEV).to(t)
            W = fw.weight_grad(delta, ck)
            assert np.array_equal(f64(W), f64(delta).T @ f64(x))


def test_weight_grad_keeps_all_bits_of_delta(fw):
    """One token: W is the outer product, exact up to fp32's rounding for any 24-bit delta."""
    m, d = 200, 300
    x = draw(1, d, torch.bfloat16, 5)
    ck = fw.ActCheckpoint(1, d, "e4m3", device=DEV).save(x)
    a = f64(ck.restore(torch.float32))
    for t in (torch.float32, torch.float16):
        delta = draw(1, m, t, 6)
        W = f64(fw.weight_grad(delta, ck))
        ref = f64(delta).T @ a
        assert (np.abs(W - ref) <= 4 * U * np.abs(ref)).all()


def test_weight_grad_nonfinite(fw):
    T, m, d = 100, 140, 300
    x = draw(T, d, torch.float32, 41)
    x[50, 70] = float("nan")
    ck = fw.ActCheckpoint(T, d, "e4m3", device=DEV).save(x)
    for t in DT.values():
        delta = draw(T, m, t, 42)
        delta[20, 7] = float("inf")
        delta[21, 9] = float("nan")
        W = f64(fw.weight_grad(delta, ck))
        cols = np.zeros(d, bool)
        cols[64:96] = True                       # the block of the NaN
        assert np.isnan(W[:, cols]).all() and np.isnan(W[9]).all() and not np.isfinite(W[7]).any()
        rest = np.ones(m, bool)
        rest[[7, 9]] = False
        assert np.isfinite(W[rest][:, ~cols]).all()


# -- together ----------------------------------------------------------------------

def _step(fw, x, w, b, dy, delta, L, bufs):
    """norm (input kept in 8 bits) -> its backward; weight gradient from a
    checkpoint of the layer's input -> encoded gradient."""
    ck, ckx, work, W, codes, scales = bufs
    y, mean, rstd = fw.norm_forward(x, w, b, ckpt=ckx)
    ck.save(y)
    fw.weight_grad(delta, ck, alpha=1.0 / x.shape[0], out=W, work=work)
    dx, dw, db = fw.norm_backward(dy, ckx, mean, rstd, w)
    L.encode(W, codes=codes, scales=scales)
    return y, dx, dw, db, W, codes, scales


def test_step_on_a_stream_and_in_a_graph(fw):
    T, m, d = 520, 264, 512
    args = (draw(T, d, torch.bfloat16, 51), *_params(d, "bf16", "layer", "same", 52), draw(T, d, torch.bfloat16, 53),
            draw(T, m, torch.bfloat16, 54, 0.01))
    L = fw.Layer(m, d, "euclid", device=DEV)
    bufs = (fw.ActCheckpoint(T, d, device=DEV), fw.ActCheckpoint(T, d, device=DEV),
            torch.empty(int(fw._lib.gift_weight_grad_workspace_bytes(T, m, d, fw.BF16)), dtype=torch.uint8, device=DEV),
            torch.empty(m, d, device=DEV), torch.empty(m, d, dtype=torch.uint8, device=DEV),
            torch.empty(1, device=DEV))
    want = [v.clone() for v in _step(fw, *args, L, bufs)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _step(fw, *args, L, bufs)
        side.synchronize()
        assert all(torch.equal(g, v) for g, v in zip(got, want))
    # the activation operators in a graph, replayed with eager work between
    x, w, b, dy, delta = args
    ck, ckx, work, W, _, _ = bufs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, mean, rstd = fw.norm_forward(x, w, b, ckpt=ckx)
        ck.save(y)
        fw.weight_grad(delta, ck, alpha=1.0 / T, out=W, work=work)
        dx, dw, db = fw.norm_backward(dy, ckx, mean, rstd, w)
    for _ in range(4):
        for v in (y, dx, dw, db, W, work):
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, v) for g, v in zip((y, dx, dw, db, W), want))
        torch.cuda.synchronize()
        x.mul_(1.0).sum().item()


def test_calls_repeat_bit_for_bit(fw):
    T, m, d = 3000, 400, 1100
    x, dy, delta = draw(T, d, torch.bfloat16, 61), draw(T, d, torch.bfloat16, 62), draw(T, m, torch.bfloat16, 63)
    ck = fw.ActCheckpoint(T, d, device=DEV).save(x)
    first = None
    for _ in range(3):
        y, mean, rstd = fw.norm_forward(x)
        out = (y, mean, rstd, *fw.norm_backward(dy, ck, mean, rstd), fw.weight_grad(delta, ck))
        if first is None:
            first = out
        assert all(torch.equal(a, b) for a, b in zip(out, first))


def test_given_stream_owns_what_it_allocates(fw):
    """A call on another stream than the current one: outputs and workspace
    are that stream's."""
    T, d = 600, 768
    x, dy = draw(T, d, torch.bfloat16, 71), draw(T, d, torch.bfloat16, 72)
    y, mean, rstd = fw.norm_forward(x)
    dx, dw, db = fw.norm_backward(dy, x, mean, rstd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        y2, mean2, rstd2 = fw.norm_forward(x, stream=s)
        dx2, dw2, db2 = fw.norm_backward(dy, x, mean2, rstd2, stream=s)
        junk = [torch.full((512 * 2 * d,), 5.0, device=DEV) for _ in range(4)]    # the current stream's allocations
        s.synchronize()
        assert torch.equal(y2, y) and torch.equal(dx2, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
        del junk
