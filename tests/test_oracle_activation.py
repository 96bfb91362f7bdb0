"""The activation operators' oracle: the checkpoint format against its
definition, and the norm's gradients against central differences."""
import numpy as np
import pytest

from oracle import activation as A
from oracle import fp8


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_checkpoint_scale_is_the_smallest_that_does_not_saturate(fmt):
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((50, 70)) * 10.0 ** rng.uniform(-6, 6, (50, 1))).astype(np.float32)
    x[3] = 0
    x[4, :32] = 448.0
    x[5, :32] = np.nextafter(np.float32(448), np.float32(500))
    codes, e = A.ckpt_save(x, fmt)
    v = A.ckpt_values(codes, e, 70, fmt)
    pad = np.zeros((50, 96))
    pad[:, :70] = x
    amax = np.abs(pad).reshape(50, 3, 32).max(2)
    assert (amax <= fp8.FMAX[fmt] * 2.0 ** (e - 127)).all()
    assert ((e == 32) | (amax > fp8.FMAX[fmt] * 2.0 ** (e - 128))).all()
    step = 2.0 ** -4 if fmt == "e4m3" else 2.0 ** -3
    small = np.repeat(2.0 ** (e - 127.0), 32, axis=1)[:, :70] * fp8.value_table(fmt)[1] / 2
    assert (np.abs(v - x) <= np.maximum(step * np.abs(x), small)).all()
    assert (codes[:, 70:] == 0).all()


def test_checkpoint_marks_nonfinite_blocks():
    x = np.ones((2, 64), np.float32)
    x[0, 5], x[1, 40] = np.inf, np.nan
    codes, e = A.ckpt_save(x, "e4m3")
    assert e[0, 0] == 255 and e[1, 1] == 255 and e[0, 1] == e[1, 0] != 255
    assert (codes[0, :32] == 0x7F).all() and (codes[1, 32:] == 0x7F).all()
    assert np.isnan(A.ckpt_values(codes, e, 64, "e4m3")[0, :32]).all()


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_gradients_against_differences(kind):
    rng = np.random.default_rng(1)
    T, d, eps, h = 3, 7, 1e-3, 1e-6
    x, dy = rng.standard_normal((T, d)), rng.standard_normal((T, d))
    w, b = 1 + 0.2 * rng.standard_normal(d), rng.standard_normal(d)

    def loss(x, w, b):
        return (A.norm_forward(x, w, b, eps, kind)[0] * dy).sum()

    _, mean, rstd = A.norm_forward(x, w, b, eps, kind)
    dx, dw, db = A.norm_backward(dy, x, mean, rstd, w, kind)
    for arr, grad, f in ((x, dx, lambda v: loss(v, w, b)), (w, dw, lambda v: loss(x, v, b)),
                         (b, db, lambda v: loss(x, w, v))):
        for i in np.ndindex(arr.shape):
            p, q = arr.copy(), arr.copy()
            p[i] += h
            q[i] -= h
            assert abs((f(p) - f(q)) / (2 * h) - grad[i]) < 1e-7 * max(1, abs(grad[i])) + 1e-8
