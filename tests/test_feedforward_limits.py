"""Sizes at which the gated block and the weight gradient from a whole
activation are refused, and just below them (no GPU is needed: the calls that
are not refused for their size end at a workspace that is too small or have no
rows, so the pointers are never followed)."""
import pytest

from test_feedforward_abi import FAR, INVALID, OK, P, UNSUPPORTED, WORKSPACE, _backward, _drop

# workgroups that lay out one operand: 256 chunks of eight columns each
MOST = ((1 << 23) - 1) // 4


@pytest.fixture(scope="module")
def fw():
    import fac_whitening_amd as fw
    return fw


def _grad(fw, T, m, d, dtype, x=P + FAR, ldx=None, nbytes=0):
    return fw._lib.gift_weight_grad_x(P, dtype, m, m, x, ldx or d, T, d, 1.0, 0, P + 3 * FAR, d, P + 4 * FAR, nbytes, None)


def test_large_operands_read_in_place_are_taken(fw):
    """16-bit rows that the products read as they are need no launch that lays them out."""
    n = 2048
    for T in (2_000_000, 2_200_000, 1 << 28):
        assert fw._lib.gift_weight_grad_x_workspace_bytes(T, n, n, fw.BF16, 1) > 0
        assert _grad(fw, T, n, n, fw.BF16) == WORKSPACE
        assert _grad(fw, T, n, n, fw.FP16, x=P + FAR + 2) == WORKSPACE      # (any alignment)
    # few tokens, weights of 2^33 elements: every form reads them in place
    f, d = 1 << 21, 1 << 12
    for dt in (fw.BF16, fw.FP32):
        assert fw._lib.gift_glu_backward_workspace_bytes(4, d, f, dt, 1) > 0
        assert _backward(fw, T=4, d=d, f=f, dtype=dt, bytes=0) == WORKSPACE
        assert fw._lib.gift_glu_forward(0, None, dt, d, 0, d, P, d, P + FAR, d, f, None, None, f, None, 0, None, 0, None, None, 0,
                                        None) == OK
    # and tiles of more tokens, aligned
    assert fw._lib.gift_glu_backward_workspace_bytes(100, d, f, fw.BF16, 1) > 0
    assert _backward(fw, T=100, d=d, f=f, bytes=0) == WORKSPACE


def test_operands_too_large_to_lay_out_are_refused(fw):
    """fp32 operands, and rows that the products cannot read as they are, on both sides of the limit."""
    n = 2048                                       # one workgroup a row
    for dt, d in ((fw.FP32, n), (fw.BF16, n - 1)):
        assert _grad(fw, MOST, n, d, dt) == WORKSPACE
        assert _grad(fw, MOST + 1, n, d, dt) == UNSUPPORTED
    far = (1 << 21) + 8                             # rows more than 4 MB apart
    assert _grad(fw, MOST, 64, n, fw.BF16, ldx=far) == WORKSPACE
    assert _grad(fw, MOST + 1, 64, n, fw.BF16, ldx=far) == UNSUPPORTED
    assert _backward(fw, T=100, d=n, f=MOST, bytes=0) == WORKSPACE
    f, d = 1 << 21, 1 << 12
    assert _backward(fw, T=100, d=d, f=f, dtype=fw.FP32, bytes=1 << 60) == UNSUPPORTED
    assert _backward(fw, T=100, d=d, f=f, ldg=d + 8, bytes=1 << 60) == UNSUPPORTED
    # the query counts what can be laid out
    assert fw._lib.gift_weight_grad_x_workspace_bytes(MOST, n, n, fw.FP32, 0) >= 6 * MOST * n
    assert fw._lib.gift_weight_grad_x_workspace_bytes(MOST + 1, n, n, fw.FP32, 0) < 6 * MOST * n


def test_rows_past_dropouts_counter_are_refused(fw):
    T = (1 << 32) + 1
    one = dict(T=T, f=1, lddh=1, ldz=1, ldup=1, lddz=1, lddup=1, dx=None)
    assert _backward(fw, **one, drop=_drop(fw)) == UNSUPPORTED
    assert _backward(fw, **dict(one, lddh=0), drop=_drop(fw)) == INVALID
