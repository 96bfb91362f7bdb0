"""Outputs of the norms that share memory with an input in another way than
element for element: rows would be read after others are written over them.
Refused before anything is enqueued (the pointers are never followed; no GPU
is needed).  Rows side by side in one buffer are not an overlap."""
import pytest

P = 1 << 20
INVALID = 1

# x's leading dimension, output's leading dimension, output's offset in elements, for 5 rows of 1000
OVERLAPS = [(1000, 1008, 0), (1008, 1000, 0), (1000, 1000, 8), (1000, 1000, 1000), (2000, 2000, 992), (2000, 2000, 1008),
            (2000, 2000, -8), (1000, 1000, -4000), (2000, 1000, 0), (2000, 3000, 1000), (2000, 2000, 3008)]


@pytest.fixture(scope="module")
def fw():
    import fac_whitening_amd as fw
    return fw


@pytest.mark.parametrize("ldx,ldo,off", OVERLAPS)
@pytest.mark.parametrize("dtype,size", [(0, 2), (1, 4), (2, 2)])
def test_outputs_that_overlap_an_input(fw, ldx, ldo, off, dtype, size):
    L, O, Q, T, d = fw._lib, P + off * size, 1 << 28, 5, 1000
    assert L.gift_norm_forward(0, P, dtype, ldx, T, d, Q, Q, dtype, 1e-5, O, ldo, Q, Q, None, None) == INVALID
    wb = L.gift_norm_workspace_bytes(T, d)
    for dy, x in ((P, Q), (Q, P)):
        assert L.gift_norm_backward(0, dy, dtype, ldx, x, ldx, None, T, d, Q, dtype, Q, Q, O, ldo, Q, Q, 0, Q, wb,
                                    None) == INVALID


def test_one_row(fw):
    L, Q = fw._lib, 1 << 28
    for off in (2, -1998):
        assert L.gift_norm_forward(1, P, 0, 1000, 1, 1000, Q, Q, 0, 1e-5, P + off, 1000, None, Q, None, None) == INVALID
