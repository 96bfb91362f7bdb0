"""The gated block, dropout and the whole-activation weight gradient where the
size or the operands choose another form: few tokens in place, one tile split
over many workgroups, tiles of both sizes, rows past 4 GiB, rows far apart."""
import numpy as np
import pytest
import torch

from oracle import feedforward as F
from test_gpu_feedforward import (DEV, DT, OFFSET, SEED, chain, check, check_dx, check_wgrad, draw, f64, forward_reference,
                                  gradients_reference, half_step, strided, untouched)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    import fac_whitening_amd as fw
    return fw


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 5, 16, 32])
def test_few_tokens_in_place(fw, T, dtype):
    """Outputs over inputs give what separate ones give, within both bounds; dx over dh too."""
    d, f = 256, 700
    dh, gate, up = (draw(T, f, dtype, i) for i in range(3))
    wg, wu = draw(f, d, dtype, 4, 0.1), draw(f, d, dtype, 5, 0.1)
    drop = (0.2, SEED, OFFSET)
    (rz, tz), (ru, tu) = gradients_reference(dh, gate, up, "silu", F.factor(T, f, drop), dtype)
    for over in (None, (0, 1), (1, 2), (2, 1)):
        a = [dh.clone(), gate.clone(), up.clone()]
        kw = {} if over is None else dict(dgate=a[over[0]], dup=a[over[1]])
        dx, dgate, dup = fw.glu_backward(*a, wg, wu, drop=fw.Dropout(*drop), **kw)
        torch.cuda.synchronize()
        check(dgate, rz, tz, "dgate")
        check(dup, ru, tu, "dup")
        check_dx(dx, dgate, dup, wg, wu, dtype)
    a = [dh.clone(), gate.clone(), up.clone()]
    flat = a[0].view(-1)[:T * d].view(T, d)
    dx, dgate, dup = fw.glu_backward(*a, wg, wu, drop=fw.Dropout(*drop), dx=flat)
    torch.cuda.synchronize()
    check(dgate, rz, tz, "dgate")
    check_dx(dx, dgate, dup, wg, wu, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,d,f", [(1, 91, 9001), (3, 1000, 513), (40, 64, 8200), (64, 130, 4097), (33, 1, 300), (20, 9, 257)])
def test_one_tile_over_many_workgroups(fw, T, d, f, dtype):
    """A long sum behind few outputs: slabs and pieces of it, joined in order."""
    print(f"[bwd {T}x{d}x{f} {dtype}]", flush=True)
    dh, gate, up = (draw(T, f, dtype, i, 0.5) for i in range(3))
    wg, wu = draw(f, d, dtype, 4, f ** -0.5), draw(f, d, dtype, 5, f ** -0.5)
    first = None
    for _ in range(2):
        dx, dgate, dup = fw.glu_backward(dh, gate, up, wg, wu, "gelu_tanh", dx=strided(T, d, DT[dtype], d + 3, 1))
        torch.cuda.synchronize()
        (rz, tz), (ru, tu) = gradients_reference(dh, gate, up, "gelu_tanh", np.ones((T, f)), dtype)
        check(dgate, rz, tz, "dgate")
        check(dup, ru, tu, "dup")
        check_dx(dx, dgate, dup, wg, wu, dtype)
        untouched(dx)
        first = dx if first is None else first
        assert torch.equal(dx, first)
    x = draw(T, d, dtype, 6)
    W = fw.weight_grad(dh, x)
    check_wgrad(W, dh, x, 1.0, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d,f", [(2100, 320, 1100), (4300, 128, 700), (1024, 2100, 640)])
def test_large_tiles(fw, T, d, f, dtype):
    print(f"[large {T}x{d}x{f} {dtype}]", flush=True)
    x, wg, wu = draw(T, d, dtype, 1), draw(f, d, dtype, 2, d ** -0.5), draw(f, d, dtype, 3, d ** -0.5)
    drop = (0.1, SEED, 7)
    h, gate, up = fw.glu_forward(x, wg, wu, "gelu", keep=True, drop=fw.Dropout(*drop))
    (rh, th), (rz, tz), (ru, tu) = forward_reference(x, wg, wu, "gelu", F.factor(T, f, drop), dtype)
    check(h, rh, th, "h")
    check(gate, rz, tz, "gate")
    check(up, ru, tu, "up")
    dh = draw(T, f, dtype, 4, 0.1)
    dx, dgate, dup = fw.glu_backward(dh, gate, up, wg, wu, "gelu", fw.Dropout(*drop))
    check_dx(dx, dgate, dup, wg, wu, dtype)
    old = torch.ones(f, d, device=DEV)
    check_wgrad(fw.weight_grad(dgate, x, 0.5, out=old, accumulate=True), dgate, x, 0.5, dtype, np.ones((f, d)))


def test_rows_past_4_gib(fw):
    """Offsets of the last rows pass 32 bits (x and the gradients 4.6 GB each)."""
    T, d, f = 1_100_000, 2048, 16
    x = torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
    x[-200:] = draw(200, d, "bf16", 1)
    w = draw(2 * f, d, "bf16", 2, d ** -0.5)
    h, gate, up = fw.glu_forward(x, w[:f], w[f:], keep=True)
    (rh, th), (rz, tz), _ = forward_reference(x[-200:], w[:f], w[f:], "silu", np.ones((200, f)), "bf16")
    check(h[-200:], rh, th, "h")
    check(gate[-200:], rz, tz, "gate")
    assert (h[:-200] == 0).all()
    dh = torch.ones_like(h)
    dx, dgate, dup = fw.glu_backward(dh, gate, up, w[:f], w[f:])
    check_dx(dx[-200:], dgate[-200:], dup[-200:], w[:f], w[f:], "bf16")
    # a gradient that only the last rows make: the chain over the zeros in front adds nothing
    W = fw.weight_grad(dgate, x)
    check_wgrad(W, dgate[-200:], x[-200:], 1.0, "bf16")
    # dropout, the last rows
    drop = fw.Dropout(0.5, SEED, OFFSET)
    y = fw.dropout_forward(dx, drop, residual=x)
    t0 = T - 3
    kept = np.zeros((3, d), bool)
    for t in range(3):
        for c in range(d // 8):
            b = F.philox((c, t0 + t, OFFSET & F.M, OFFSET >> 32), (SEED & F.M, SEED >> 32))
            kept[t, 8 * c:8 * c + 8] = [(b[i // 2] >> 16 * (i % 2)) & 0xFFFF >= 32768 for i in range(8)]
    want = np.where(kept, 2 * f64(dx[t0:]), 0.0) + f64(x[t0:])
    check(y[t0:], want, half_step(torch.bfloat16, want) * 1.01 + 1e-6 * np.abs(f64(x[t0:])), "y")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_far_apart(fw, dtype):
    """Rows more than 4 MB apart, which the products lay out anew, and just below."""
    T, d, f = 70, 64, 48
    size = 2 if dtype == "bf16" else 4
    for ld in ((1 << 22) // size, (1 << 22) // size + 8):
        buf = torch.empty((T - 1) * ld + d, dtype=DT[dtype], device=DEV)
        x = torch.as_strided(buf, (T, d), (ld, 1))
        x.copy_(draw(T, d, dtype, 1))
        w = draw(2 * f, d, dtype, 2, d ** -0.5)
        h, gate, up = fw.glu_forward(x, w[:f], w[f:], keep=True)
        (rh, th), _, _ = forward_reference(x, w[:f], w[f:], "silu", np.ones((T, f)), dtype)
        check(h, rh, th, "h")
        check_wgrad(fw.weight_grad(h, x), h, x, 1.0, dtype)
        del buf, x


def test_weights_and_gradients_with_strides_of_their_own(fw):
    """Separate weights and gradients whose rows are different distances apart."""
    T, d, f = 150, 96, 120
    wg, wu = draw(f, d, "bf16", 1, 0.1, d + 8), draw(f, d, "bf16", 2, 0.1, d + 32)
    dh, gate, up = (draw(T, f, "bf16", i) for i in range(3))
    dx, dgate, dup = fw.glu_backward(dh, gate, up, wg, wu, dgate=strided(T, f, torch.bfloat16, f + 8),
                                     dup=strided(T, f, torch.bfloat16, f + 40))
    torch.cuda.synchronize()
    check_dx(dx, dgate, dup, wg, wu, "bf16")
    x = draw(T, d, "bf16", 5)
    h, gate, up = fw.glu_forward(x, wg, wu, keep=True)
    (rh, th), _, _ = forward_reference(x, wg, wu, "silu", np.ones((T, f)), "bf16")
    check(h, rh, th, "h")


def test_largest_fp32_values(fw):
    """Values beyond the largest bf16 number split without an overflow."""
    big = torch.finfo(torch.float32).max
    for T in (1, 70):
        x = torch.full((T, 8), 0.0, device=DEV)
        x[:, 0] = big
        w = torch.zeros(32, 8, device=DEV)
        w[:, 0] = 2.0 ** -127
        h, gate, up = fw.glu_forward(x, w[:16], w[16:], act="relu", keep=True)
        want = float(np.float64(big) * 2.0 ** -127)
        assert np.allclose(f64(gate), want, rtol=2.0 ** -20, atol=0)


def test_two_graphs_with_one_workspace_each(fw):
    """Captured calls keep their own workspaces: replays in turn do not disturb each other."""
    T, d, f = 200, 301, 333
    sets = []
    for k in range(2):
        x, wg, wu = draw(T, d, "fp32", 10 * k + 1), draw(f, d, "fp32", 10 * k + 2, 0.1), draw(f, d, "fp32", 10 * k + 3, 0.1)
        want = [v.clone() for v in fw.glu_forward(x, wg, wu, keep=True)]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = fw.glu_forward(x, wg, wu, keep=True)
        sets.append((g, got, want, x, wg, wu))
    for _ in range(3):
        for g, got, want, *_ in sets:
            for v in got:
                v.zero_()
            g.replay()
        torch.cuda.synchronize()
        for g, got, want, *_ in sets:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
