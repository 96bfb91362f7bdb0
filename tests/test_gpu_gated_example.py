"""The gated block's example: it runs, and its gradients are the formula's."""
import numpy as np
import pytest
import torch

from oracle import activation as A
from oracle import feedforward as F

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def f64(t):
    return t.detach().cpu().double().numpy()


def test_gated_block_step():
    """Each gradient against float64 on the same parameters, masks and kept values.  Every tensor that passes between the
    operators is rounded to bf16 (2^-9 of a value at most, random), and h to 8 bits where dw2 reads it from its
    checkpoint (2^-4 at most, which the oracle applies as well): along the longest path six roundings meet, so 6 2^-9
    of the gradient's norm bounds what they add."""
    from examples.gated_block_step import GatedBlock
    T, d, f, p = 200, 128, 320, 0.1
    b = GatedBlock(d, f, T, "silu", p)
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(T, d, generator=g, device=DEV).bfloat16()
    dout = (0.1 * torch.randn(T, d, generator=g, device=DEV)).bfloat16()
    for n in range(2):
        out = b.forward(x)
        grads = {k: f64(v) for k, v in b.backward(dout).items()}
        mean = b.exchange()
        torch.cuda.synchronize()
        assert b.step.item() == n + 1
        X, W, V = f64(x), f64(b.w1), f64(b.w2)
        kh, ko = F.factor(T, f, (p, 1, n)), F.factor(T, d, (p, 2, n))
        y, m, rstd = A.norm_forward(X, np.ones(d), None, 1e-5, "rms")
        h, z, u = F.glu_forward(y, W[:f], W[f:], "silu", kh)
        do = F.apply(f64(dout), ko)
        dz, du = F.glu_gradients(do @ V, z, u, "silu", kh)
        rdx, rdg, _ = A.norm_backward(dz @ W[:f] + du @ W[f:], X, m, rstd, np.ones(d), "rms")
        codes = b.ck_h.restore(torch.float32)
        want = {"dx": rdx + f64(dout), "dgamma": rdg, "dw1": np.concatenate([dz, du], 1).T @ y / T,
                "dw2": do.T @ f64(codes) / T}
        for k, w in want.items():
            assert np.linalg.norm(grads[k] - w) <= 6 * 2.0 ** -9 * np.linalg.norm(w), k
        o = F.apply(h @ V.T, ko) + X
        assert np.linalg.norm(f64(out) - o) <= 6 * 2.0 ** -9 * np.linalg.norm(o)
        # the payloads' round trip: E4M3 rounds by 2^-4 of a value at most
        for got, k in zip(mean, ("dw1", "dw2")):
            assert np.linalg.norm(f64(got) - grads[k]) <= 2.0 ** -4 * np.linalg.norm(grads[k])
