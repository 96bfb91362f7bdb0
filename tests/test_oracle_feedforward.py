"""The oracle's generator against the published known answers, its array form
against the scalar one, and its derivatives against differences."""
import numpy as np
import pytest

from oracle import feedforward as F


@pytest.mark.parametrize("ctr,key,want", [
    ((0,) * 4, (0,) * 2, (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((F.M,) * 4, (F.M,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_philox_known_answers(ctr, key, want):
    assert tuple(F.philox(ctr, key)) == want


def test_kept_is_philox_by_place():
    p, seed, offset = 0.3, 0xFEDCBA9876543210, 0x8000000180000003
    k = F.kept(5, 21, p, seed, offset)
    for t in range(5):
        for j in range(21):
            w = F.philox((j // 8, t, offset & F.M, offset >> 32), (seed & F.M, seed >> 32))[j % 8 // 2]
            assert k[t, j] == ((w >> (16 * (j % 2)) & 0xFFFF) >= round(65536 * p))


def test_threshold_and_scale():
    assert F.threshold(0.0) == 0 and F.threshold(1.0) == 65536 and F.threshold(0.1) == 6554
    f = F.factor(64, 64, (0.1, 1, 2))
    assert set(np.unique(f)) == {0.0, 65536 / (65536 - 6554)}
    assert (F.factor(9, 9, (1.0, 1, 2)) == 0).all() and (F.factor(9, 9, (0.0, 1, 2)) == 1).all()
    # 4096 draws kept with probability 0.9: 5 standard deviations are 96
    assert abs((f > 0).sum() - 4096 * 0.9) < 100


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh", "relu", "sigmoid"])
def test_derivatives(kind):
    z = np.linspace(-6, 6, 240) + 1e-3
    e = 1e-5
    d = (F.act(z + e, kind)[0] - F.act(z - e, kind)[0]) / (2 * e)
    assert np.abs(F.act(z, kind)[1] - d).max() < 1e-8


def test_gradients_against_differences():
    g = np.random.default_rng(5)
    x, wg, wu, dh = (g.standard_normal(s) for s in ((4, 6), (9, 6), (9, 6), (4, 9)))
    f = F.factor(4, 9, (0.25, 3, 4))
    for kind in ("silu", "gelu", "gelu_tanh", "sigmoid"):
        _, z, u = F.glu_forward(x, wg, wu, kind, f)
        dz, du = F.glu_gradients(dh, z, u, kind, f)
        v = g.standard_normal(x.shape)
        loss = lambda y: (dh * F.glu_forward(y, wg, wu, kind, f)[0]).sum()   # noqa: E731
        num = (loss(x + 1e-6 * v) - loss(x - 1e-6 * v)) / 2e-6
        assert abs(((dz @ wg + du @ wu) * v).sum() - num) < 1e-7 * (1 + abs(num))
        vg, vu = g.standard_normal(wg.shape), g.standard_normal(wu.shape)
        loss = lambda s: (dh * F.glu_forward(x, wg + s * vg, wu + s * vu, kind, f)[0]).sum()   # noqa: E731
        num = (loss(1e-6) - loss(-1e-6)) / 2e-6
        assert abs((dz.T @ x * vg).sum() + (du.T @ x * vu).sum() - num) < 1e-7 * (1 + abs(num))
