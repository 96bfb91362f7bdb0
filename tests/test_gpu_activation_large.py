"""Activation operators where their kernels change form: weight gradients with
whole, split and many tiles, rows past 4 GiB, outputs larger than the caches,
every lane group of the norm's backward with many rows, gradients against
differences, split tiles in a graph, and the MLP example.

Tolerances are those of test_gpu_activation.py: fp32 chains of at most T / 4 +
64 additions in the weight gradient, 100 half steps of fp32 for a parameter
gradient of up to 4096 rows."""
import numpy as np
import pytest
import torch

from oracle import activation as A
from tests.test_gpu_activation import DEV, DT, U, _check_backward, _ckpt, _params, draw, f64, strided, u_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    import fac_whitening_amd as fw
    return fw


def _wgrad64(delta, ck, alpha):
    """alpha delta^T a and its magnitudes in 64 bits, on the device."""
    D, a = delta.double(), ck.restore(torch.float32).double()
    return alpha * torch.mm(D.t().contiguous(), a), abs(alpha) * torch.mm(D.abs().t().contiguous(), a.abs())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,m,d,ld,off", [
    (700, 1030, 2100, None, 0),        # tiles cross both edges
    (2048, 1536, 6144, None, 0),       # 144 tiles of 256 x 256: split in several levels
    (1100, 2560, 8200, 2563, 1),       # whole rounds and split tiles, rows of odd length
    (130, 4104, 4100, None, 0),        # few tokens, many tiles
    (9000, 264, 511, None, 0),         # few tiles, many tokens
    (4099, 9, 40, 11, 3)])             # a single tile narrower than its chunks
def test_weight_grad_tiles(fw, T, m, d, ld, off, dtype):
    fmt = "e5m2" if (T + m) % 4 == 2 else "e4m3"
    print(f"[wgrad T {T} {m}x{d} ld {ld} off {off} {dtype} {fmt}]", flush=True)
    ck = fw.ActCheckpoint(T, d, fmt, device=DEV).save(draw(T, d, torch.bfloat16, T + d))
    if T % 8:
        ck.bscales[-1, :, T % 8:] = 255
    delta = draw(T, m, DT[dtype], T + m, 0.01, ld, off)
    W = strided(m, d, torch.float32, d + 5, 3)
    fw.weight_grad(delta, ck, alpha=1.0 / T, out=W)
    ref, mag = _wgrad64(delta, ck, float(np.float32(1.0 / T)))
    assert ((W.double() - ref).abs() <= (T / 4 + 64) * U * mag + 1e-37).all()
    mask = torch.ones_like(W._base, dtype=torch.bool)
    torch.as_strided(mask, W.shape, W.stride(), W.storage_offset()).fill_(False)
    assert (W._base[mask] == 777.0).all()
    old = W.double()
    fw.weight_grad(delta, ck, alpha=0.25, out=W, accumulate=True)
    ref, mag = _wgrad64(delta, ck, 0.25)
    assert ((W.double() - ref - old).abs() <= (T / 4 + 64) * U * (mag + old.abs()) + 1e-37).all()


def test_weight_grad_nonfinite_in_split_tiles(fw):
    T, m, d = 1000, 1536, 6144
    x = draw(T, d, torch.float32, 3)
    x[990, 5000] = float("nan")
    ck = fw.ActCheckpoint(T, d, "e4m3", device=DEV).save(x)
    for t in DT.values():
        delta = draw(T, m, t, 4)
        delta[3, 700], delta[999, 1500] = -float("inf"), float("nan")
        W = fw.weight_grad(delta, ck)
        bad = torch.zeros(m, d, dtype=torch.bool, device=DEV)
        bad[:, 5000 // 32 * 32:5000 // 32 * 32 + 32] = True
        bad[700] = bad[1500] = True
        assert torch.equal(~torch.isfinite(W), bad)
        # an infinity times a finite value keeps its sign
        a = ck.restore(torch.float32)[3]
        ok = torch.isfinite(a) & (a != 0) & ~torch.isnan(W[700])
        assert ok.sum() > d - 40 - (a == 0).sum() and (W[700][ok] == -torch.sign(a[ok]) * float("inf")).all()


def test_weight_grad_rows_past_4_gib(fw):
    """Codes of more than 4 GiB; all but a few tokens are zero, so W is exact."""
    T, m, d = (1 << 21) + 43, 24, 2080
    ck = fw.ActCheckpoint(T, d, "e4m3", device=DEV)
    ck.codes.zero_()
    ck.bscales.fill_(127)
    rows = [0, 70000, T - 50, T - 2, T - 1]
    x = torch.randint(-8, 9, (len(rows), d), device=DEV).to(torch.bfloat16)
    for t in (torch.bfloat16, torch.float32):
        delta = torch.ones(T, m, dtype=t, device=DEV)
        D = torch.randint(-9, 10, (len(rows), m), device=DEV)
        for i, r in enumerate(rows):
            delta[r] = D[i].to(t)
            ck.codes[r, :d] = x[i].to(torch.float8_e4m3fn).view(torch.uint8)
        W = fw.weight_grad(delta, ck)
        assert torch.equal(W.double(), D.double().t().contiguous() @ x.double())


def test_rows_past_4_gib(fw):
    """The last rows of a tensor of more than 4 GiB as in a small call."""
    T, d = 1 << 20, 2080
    x = torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
    x[-9:] = draw(9, d, torch.bfloat16, 1)
    x[-9 - 8:-9] = 1.0
    ck, small = fw.ActCheckpoint(T, d, device=DEV), fw.ActCheckpoint(16, d, device=DEV)
    y, mean, rstd = fw.norm_forward(x, kind="rms", ckpt=ck)
    y2, _, rstd2 = fw.norm_forward(x[-16:], kind="rms", ckpt=small)
    assert torch.equal(y[-16:], y2) and torch.equal(rstd[-16:], rstd2)
    assert torch.equal(ck.codes[-16:], small.codes) and torch.equal(ck.bscales[-2:], small.bscales)
    ck.codes.zero_()
    ck.bscales.zero_()
    ck.save(x)
    assert torch.equal(ck.codes[-16:], small.codes) and torch.equal(ck.bscales[-2:], small.bscales)
    back = ck.restore()
    assert torch.equal(back[-16:], small.restore())
    del y
    dx, dw, _ = fw.norm_backward(x, ck, None, rstd, kind="rms")
    dx2, _, _ = fw.norm_backward(x[-16:], small, None, rstd2, kind="rms")
    assert torch.equal(dx[-16:], dx2)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_outputs_larger_than_the_caches(fw, dtype):
    """Over 32 MiB the outputs are written another way: the same values."""
    T, d = 9001, 2049 if dtype == "bf16" else 2056
    x = draw(T, d, DT[dtype], 5, 2.0)
    ck = fw.ActCheckpoint(T, d, "e5m2", device=DEV)
    y, mean, rstd = fw.norm_forward(x, ckpt=ck)
    back = ck.restore(DT[dtype])
    ck2 = fw.ActCheckpoint(T, d, "e5m2", device=DEV).save(x)
    assert torch.equal(ck.codes, ck2.codes)
    dx, dw, db = fw.norm_backward(x, ck, mean, rstd)
    for r in (0, 4000, T - 24):
        part = fw.ActCheckpoint(24, d, "e5m2", device=DEV)
        y2, mean2, rstd2 = fw.norm_forward(x[r:r + 24], ckpt=part)
        assert torch.equal(y[r:r + 24], y2) and torch.equal(mean[r:r + 24], mean2)
        assert torch.equal(back[r:r + 24], part.restore(DT[dtype])) and torch.equal(ck.codes[r:r + 24], part.codes)
        dx2, _, _ = fw.norm_backward(x[r:r + 24], part, mean2, rstd2)
        assert torch.equal(dx[r:r + 24], dx2)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", [(4096, 100), (4090, 1024), (4096, 1500), (4001, 2000), (1100, 5000), (1101, 8192),
                                 (1100, 9000), (600, 16384)])
def test_norm_backward_lane_groups(fw, T, d, dtype, kind):
    print(f"[norm backward {T}x{d} {dtype} {kind}]", flush=True)
    x, dy = draw(T, d, DT[dtype], T), draw(T, d, DT[dtype], d, 0.1)
    w, b = _params(d, dtype, kind, "same", 5)
    ck = fw.ActCheckpoint(T, d, device=DEV)
    _, mean, rstd = fw.norm_forward(x, w, b, kind=kind, ckpt=ck)
    M = np.zeros(T) if mean is None else f64(mean)
    for src in (x, ck):
        X = f64(x) if src is x else f64(ck.restore(torch.float32))
        dx, dw, db = fw.norm_backward(dy, src, mean, rstd, w, kind)
        _check_backward(dx, dw, db, f64(dy), X, M, f64(rstd), f64(w), kind, DT[dtype])


@pytest.mark.parametrize("T,d", [(1000, 4096), (1024, 520), (300, 12288)])
def test_norm_backward_in_place_with_few_rows(fw, T, d):
    """dx written over dy or over x: the parameter gradients still come from the
    old values."""
    x, dy = draw(T, d, torch.bfloat16, 1), draw(T, d, torch.bfloat16, 2)
    w, b = _params(d, "bf16", "layer", "same", 3)
    _, mean, rstd = fw.norm_forward(x, w, b)
    dx, dw, db = fw.norm_backward(dy, x, mean, rstd, w)
    M = f64(mean)
    _check_backward(dx, dw, db, f64(dy), f64(x), M, f64(rstd), f64(w), "layer", torch.bfloat16)
    for over_x in (False, True):
        X, G = x.clone(), dy.clone()
        dx2, dw2, db2 = fw.norm_backward(G, X, mean, rstd, w, dx=X if over_x else G)
        _check_backward(dx2, dw2, db2, f64(dy), f64(x), M, f64(rstd), f64(w), "layer", torch.bfloat16)
    ck = fw.ActCheckpoint(T, d, device=DEV).save(x)
    G = dy.clone()
    dx3, dw3, db3 = fw.norm_backward(G, ck, mean, rstd, w, dx=G)
    _check_backward(dx3, dw3, db3, f64(dy), f64(ck.restore(torch.float32)), M, f64(rstd), f64(w), "layer",
                    torch.bfloat16)


def test_rms_bias_gradient_when_given(fw):
    T, d = 600, 1000
    x, dy = draw(T, d, torch.bfloat16, 8), draw(T, d, torch.bfloat16, 9)
    _, _, rstd = fw.norm_forward(x, kind="rms")
    dx, dw, none = fw.norm_backward(dy, x, None, rstd, kind="rms")
    assert none is None
    db = torch.full((d,), 3.0, device=DEV)
    dx2, dw2, db2 = fw.norm_backward(dy, x, None, rstd, kind="rms", dbias=db)
    assert db2 is db and torch.equal(dx, dx2) and torch.equal(dw, dw2)
    D = f64(dy)
    assert (np.abs(f64(db) - D.sum(0)) <= 100 * U * np.abs(D).sum(0)).all()


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_gradient_against_differences(fw, kind):
    """The kernel's gradients against central differences of the 64-bit forward.
    h = 1e-5: differences are off by h^2 times third derivatives (below 1e-8
    here) and 1e-16 / h of rounding; the kernel by 200 half steps of fp32 times
    magnitudes below 10: 2e-4 covers both."""
    T, d, eps, h = 3, 70, 1e-3, 1e-5
    x, dy = draw(T, d, torch.float32, 1, 0.5), draw(T, d, torch.float32, 2, 0.5)
    w, b = _params(d, "fp32", kind, "same", 3)
    _, mean, rstd = fw.norm_forward(x, w, b, eps, kind)
    dx, dw, db = fw.norm_backward(dy, x, mean, rstd, w, kind)
    X, D, W, B = f64(x), f64(dy), f64(w), None if b is None else f64(b)

    def loss(X, W, B):
        return (A.norm_forward(X, W, B, eps, kind)[0] * D).sum()

    checks = [(X, dx, lambda v: loss(v, W, B)), (W, dw, lambda v: loss(X, v, B))]
    if B is not None:
        checks.append((B, db, lambda v: loss(X, W, v)))
    for arr, grad, f in checks:
        for i in list(np.ndindex(arr.shape))[::7]:
            p, q = arr.copy(), arr.copy()
            p[i] += h
            q[i] -= h
            assert abs((f(p) - f(q)) / (2 * h) - f64(grad)[i]) <= 2e-4, i


def test_weight_grad_against_differences(fw):
    """Loss sum_t delta_t . (W a_t): linear, so a difference is exact but for rounding."""
    T, m, d, h = 90, 33, 70, 0.5
    ck, a = _ckpt(fw, T, d, "e4m3", 1)
    delta = draw(T, m, torch.float32, 2)
    dW, D = f64(fw.weight_grad(delta, ck)), f64(delta)
    W = np.random.default_rng(0).standard_normal((m, d))
    mag = np.abs(D).T @ np.abs(a)
    for i, j in [(0, 0), (32, 69), (7, 31), (8, 32), (20, 50)]:
        P, Q = W.copy(), W.copy()
        P[i, j] += h
        Q[i, j] -= h
        diff = ((D * (a @ P.T)).sum() - (D * (a @ Q.T)).sum()) / (2 * h)
        total = (np.abs(D) * (np.abs(a) @ np.abs(W).T)).sum()
        assert abs(diff - dW[i, j]) <= (T / 4 + 64) * U * mag[i, j] + 1e-12 * total


def test_split_tiles_in_a_graph(fw):
    """Both launches of a split product, replayed with other work between."""
    T, m, d = 4096, 512, 2048
    ck = fw.ActCheckpoint(T, d, device=DEV).save(draw(T, d, torch.bfloat16, 1))
    delta = draw(T, m, torch.bfloat16, 2)
    want = fw.weight_grad(delta, ck)
    work = torch.empty(fw._lib.gift_weight_grad_workspace_bytes(T, m, d, fw.BF16), dtype=torch.uint8, device=DEV)
    assert work.numel() > 4 * m * d                     # its tiles are split
    W = torch.empty_like(want)
    fw.weight_grad(delta, ck, out=W, work=work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fw.weight_grad(delta, ck, out=W, work=work)
    for k in range(4):
        W.zero_()
        work.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(W, want), k
        assert torch.equal(fw.weight_grad(delta, ck), want)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_mlp_example(fw, kind):
    """The example's gradients against 64-bit ones from exact activations:
    8-bit activations are off by at most 2^-4 of each value, so sums over many
    tokens by far less than 5 %."""
    from examples.mlp_block_step import Block
    T, width, hidden = 1000, 256, 520
    b = Block(width, hidden, T, kind)
    x, dout = draw(T, width, torch.bfloat16, 1), draw(T, width, torch.bfloat16, 2, 0.1)
    out = b.forward(x)
    g = b.backward(dout)
    decoded = b.exchange()
    torch.cuda.synchronize()
    X, D, w1, w2 = f64(x), f64(dout), f64(b.w1), f64(b.w2)
    y, mean, rstd = A.norm_forward(X, f64(b.gamma), None if b.beta is None else f64(b.beta), 1e-5, kind)
    h = np.maximum(y @ w1.T, 0)
    dh = (D @ w2) * (h > 0)
    dxn, dgam, dbet = A.norm_backward(dh @ w1, X, mean, rstd, f64(b.gamma), kind)

    def rel(got, ref):
        return np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)

    assert rel(out, X + h @ w2.T) < 0.01
    assert rel(g["dw1"], dh.T @ y / T) < 0.05 and rel(g["dw2"], D.T @ h / T) < 0.05
    assert rel(g["dx"], dxn + D) < 0.05 and rel(g["dgamma"], dgam) < 0.05
    assert g["dbeta"] is None if kind == "rms" else rel(g["dbeta"], dbet) < 0.05
    for m, w in zip(decoded, (g["dw1"], g["dw2"])):
        assert rel(m, f64(w)) < 0.05                    # E4M3 per tensor
    assert b.kept_bytes() < 0.6 * 2 * T * (2 * width + hidden)
