"""The gated block and the weight gradient on operands of more than 2^32
elements, which are read where they lie."""
import numpy as np
import pytest
import torch

from test_gpu_feedforward import DEV, check, check_dx, check_wgrad, draw, f64, forward_reference, gradients_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    import fac_whitening_amd as fw
    return fw


def test_more_than_2_to_the_32_elements(fw):
    """x, dgate and dup of 4.5e9 elements each, all zero but a few rows at the start and the end."""
    T, n, f = 2_200_000, 2048, 16
    x = torch.zeros(T, n, dtype=torch.bfloat16, device=DEV)
    some = torch.cat([torch.arange(150, device=DEV), torch.arange(T - 150, T, device=DEV)])
    x[some] = draw(300, n, "bf16", 1)
    w = draw(2 * f, n, "bf16", 2, n ** -0.5)
    print("[forward]", flush=True)
    h, gate, up = fw.glu_forward(x, w[:f], w[f:], "gelu", keep=True)
    (rh, th), (rz, tz), _ = forward_reference(x[some], w[:f], w[f:], "gelu", np.ones((300, f)), "bf16")
    check(h[some], rh, th, "h")
    check(gate[some], rz, tz, "gate")
    assert not h[150:-150].any()
    print("[weight gradient]", flush=True)
    W = fw.weight_grad(x, x[:, :64].contiguous())          # delta of more than 2^32 elements
    check_wgrad(W, x[some], x[some][:, :64], 1.0, "bf16")
    print("[backward]", flush=True)
    dx, dgate, dup = fw.glu_backward(h, gate, up, w[:f], w[f:], "gelu", dx=x)   # (dx of more than 2^32 elements)
    check_dx(dx[some], dgate[some], dup[some], w[:f], w[f:], "bf16")
    assert not dx[150:-150].any()


@pytest.mark.parametrize("T", [3, 80])
def test_weights_of_more_than_2_to_the_32_elements(fw, T):
    """[f][d] of 2^32 + 2^22 elements, of which every 4096th row is not zero: forward and backward, few tokens and tiles."""
    d, f = 2056, 1 << 21
    wg = torch.zeros(f, d, dtype=torch.bfloat16, device=DEV)
    wu = torch.zeros(f, d, dtype=torch.bfloat16, device=DEV)
    rows = torch.arange(4095, f, 4096, device=DEV)          # the last one among them
    wg[rows], wu[rows] = draw(len(rows), d, "bf16", 1, d ** -0.5), draw(len(rows), d, "bf16", 2, d ** -0.5)
    x = draw(T, d, "bf16", 3)
    print("[forward]", flush=True)
    h, gate, up = fw.glu_forward(x, wg, wu, keep=True)
    (rh, th), (rz, tz), (ru, tu) = forward_reference(x, wg[rows], wu[rows], "silu", np.ones((T, len(rows))), "bf16")
    check(h[:, rows], rh, th, "h")
    check(gate[:, rows], rz, tz, "gate")
    check(up[:, rows], ru, tu, "up")
    assert torch.count_nonzero(gate).item() <= T * len(rows)
    print("[backward]", flush=True)
    gate[:, rows] += 0.5
    up[:, rows] += 0.5
    dh = torch.ones_like(h)
    dx, dgate, dup = fw.glu_backward(dh, gate, up, wg, wu)
    (rz, tz), (ru, tu) = gradients_reference(dh[:, rows], gate[:, rows], up[:, rows], "silu", np.ones((T, len(rows))), "bf16")
    check(dgate[:, rows], rz, tz, "dgate")
    check(dup[:, rows], ru, tu, "dup")
    check_dx(dx, dgate[:, rows], dup[:, rows], wg[rows], wu[rows], "bf16")
