"""Activation operators: forms that the sizes of the other tests do not reach."""
import numpy as np
import pytest
import torch

from tests.test_gpu_activation import DEV, DT, _params, draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fw():
    import fac_whitening_amd as fw
    return fw


@pytest.mark.parametrize("T,d", [(40, 264), (1500, 264), (40, 2056)])
def test_norm_rows_side_by_side(fw, T, d):
    """Inputs and outputs as column ranges of one buffer share no element: the
    same bits as from buffers of their own."""
    x, dy = draw(T, d, torch.bfloat16, 1), draw(T, d, torch.bfloat16, 2)
    w, b = _params(d, "bf16", "layer", "same", 3)
    y, mean, rstd = fw.norm_forward(x, w, b)
    dx, dw, db = fw.norm_backward(dy, x, mean, rstd, w)
    buf = torch.zeros(T, 4 * d + 8, dtype=torch.bfloat16, device=DEV)
    vx, vdy, vy, vdx = (buf[:, i * d:(i + 1) * d] for i in range(4))
    vx.copy_(x)
    vdy.copy_(dy)
    y2, mean2, rstd2 = fw.norm_forward(vx, w, b, out=vy)
    dx2, dw2, db2 = fw.norm_backward(vdy, vx, mean2, rstd2, w, dx=vdx)
    assert torch.equal(y2, y) and torch.equal(dx2, dx) and torch.equal(rstd2, rstd)
    # (rows that meet in memory take the columns in a launch of their own: the same sums)
    assert torch.equal(dw2, dw) and torch.equal(db2, db)
    assert torch.equal(vx, x) and torch.equal(vdy, dy) and (buf[:, 4 * d:] == 0).all()
    with pytest.raises(fw.GiftError):
        fw.norm_forward(vx, w, b, out=buf[:, 8:8 + d])
