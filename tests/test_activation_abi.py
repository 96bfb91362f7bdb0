"""Refusals of the activation operators: every bad argument is an error
before anything is enqueued (no GPU is needed: the pointers are never
followed)."""
import ctypes

import pytest

P = 1 << 20          # a well-aligned address that is never followed
OK, INVALID, WORKSPACE, UNSUPPORTED = 0, 1, 2, 5


@pytest.fixture(scope="module")
def fw():
    import fac_whitening_amd as fw
    return fw


def _ck(fw, **kw):
    c = dict(d_codes=P, ldc=1024, d_bscales=P, fmt=fw.E4M3)
    c.update(kw)
    return ctypes.byref(fw.ActCkpt(c["d_codes"], c["ldc"], c["d_bscales"], c["fmt"]))


def test_scale_bytes(fw):
    f = fw._lib.gift_act_scale_bytes
    assert f(0, 100) == 0 and f(1, 1) == 8 and f(8, 32) == 8 and f(9, 33) == 2 * 2 * 8
    assert f(-1, 8) == 0 and f(8, 0) == 0
    assert f(1 << 33, 4096) == (1 << 30) * 128 * 8      # past 32 bits


BAD_CKPT = [dict(d_codes=None), dict(d_codes=P + 8), dict(d_bscales=None), dict(d_bscales=P + 8), dict(ldc=992),
            dict(ldc=1008), dict(fmt=2), dict(fmt=-1)]


@pytest.mark.parametrize("bad", BAD_CKPT + [None])
def test_bad_checkpoints(fw, bad):
    L = fw._lib
    ck = None if bad is None else _ck(fw, **bad)
    assert L.gift_act_save(P, fw.BF16, 1000, 5, 1000, ck, None) == INVALID
    assert L.gift_act_restore(ck, 5, 1000, P, fw.BF16, 1000, None) == INVALID
    assert L.gift_weight_grad(P, fw.BF16, 64, 64, ck, 5, 1000, 1.0, 0, P, 1000, P, 1 << 40, None) == INVALID
    if bad is not None:
        assert L.gift_norm_forward(0, P, fw.BF16, 1000, 5, 1000, P, P, fw.BF16, 1e-5, P, 1000, P, P, ck,
                                   None) == INVALID
        assert L.gift_norm_backward(0, P, fw.BF16, 1000, None, 0, ck, 5, 1000, P, fw.BF16, P, P, P, 1000, P, P, 0, P,
                                    1 << 40, None) == INVALID


def test_save_and_restore_arguments(fw):
    L, ck = fw._lib, _ck(fw)
    good = [P, fw.BF16, 1000, 5, 1000, ck, None]
    for i, v in [(0, None), (0, P + 1), (1, 3), (1, -1), (2, 999), (2, -1000), (3, -1), (4, 0), (4, -5)]:
        a = list(good)
        a[i] = v
        assert L.gift_act_save(*a) == INVALID, (i, v)
    assert L.gift_act_save(P + 2, fw.FP32, 1000, 5, 1000, ck, None) == INVALID      # fp32 needs 4 bytes
    for i, v in [(1, -1), (2, 0), (3, None), (3, P + 1), (4, 7), (5, 999)]:
        a = [ck, 5, 1000, P, fw.FP16, 1000, None]
        a[i] = v
        assert L.gift_act_restore(*a) == INVALID, (i, v)
    # nothing to do
    assert L.gift_act_save(None, fw.BF16, 0, 0, 1000, ck, None) == OK
    assert L.gift_act_restore(ck, 0, 1000, None, fw.BF16, 0, None) == OK
    # more workgroups than a launch takes
    assert L.gift_act_save(P, fw.BF16, 1000, 1 << 38, 1000, ck, None) == UNSUPPORTED


def test_norm_forward_arguments(fw):
    L = fw._lib
    good = [0, P, fw.BF16, 1000, 5, 1000, P, P, fw.BF16, 1e-5, P, 1000, P, P, None, None]
    for i, v in [(0, 2), (0, -1), (1, None), (1, P + 1), (2, 3), (3, 999), (4, -1), (5, 0), (6, P + 1), (7, P + 1),
                 (8, fw.FP16), (9, -1.0), (9, float("nan")), (9, float("inf")), (10, None), (11, 999), (12, P + 2),
                 (13, P + 1)]:
        a = list(good)
        a[i] = v
        assert L.gift_norm_forward(*a) == INVALID, (i, v)
    wide = list(good)
    wide[3] = wide[5] = wide[11] = 16385
    assert L.gift_norm_forward(*wide) == UNSUPPORTED
    empty = list(good)
    empty[4] = 0
    assert L.gift_norm_forward(*empty) == OK


def test_norm_backward_arguments(fw):
    L = fw._lib
    wb = L.gift_norm_workspace_bytes(5, 1000)
    assert wb >= 2 * 1000 * 4 and L.gift_norm_workspace_bytes(-1, 8) == 0 and L.gift_norm_workspace_bytes(5, 16385) == 0
    #       kind dy  dtype    ld    x  ldx   ck   T   d    gamma wtype  mean rstd dx ld   dg db acc work bytes
    good = [0, P, fw.BF16, 1000, P, 1000, None, 5, 1000, P, fw.BF16, P, P, P, 1000, P, P, 0, P, wb, None]
    for i, v in [(0, 5), (1, None), (1, P + 1), (2, 9), (3, 999), (4, None), (4, P + 1), (5, 10), (7, -1), (8, 0),
                 (9, P + 1), (10, fw.FP16), (11, None), (11, P + 2), (12, None), (13, None), (14, 1), (15, P + 1),
                 (16, P + 2), (18, None), (18, P + 4)]:
        a = list(good)
        a[i] = v
        assert L.gift_norm_backward(*a) == INVALID, (i, v)
    both = list(good)
    both[6] = _ck(fw)                                    # an input and a checkpoint
    assert L.gift_norm_backward(*both) == INVALID
    small = list(good)
    small[19] = wb - 1
    assert L.gift_norm_backward(*small) == WORKSPACE
    # no rows and no parameter gradient: nothing to do
    none = list(good)
    none[7], none[15], none[16], none[18], none[19] = 0, None, None, None, 0
    assert L.gift_norm_backward(*none) == OK


def test_weight_grad_arguments(fw):
    L, ck = fw._lib, _ck(fw)
    wb = L.gift_weight_grad_workspace_bytes(5, 64, 1000, fw.BF16)
    assert L.gift_weight_grad_workspace_bytes(5, 0, 1000, fw.BF16) == 0
    good = [P, fw.BF16, 64, 64, ck, 5, 1000, 1.0, 0, P, 1000, P, wb, None]
    for i, v in [(0, None), (0, P + 1), (1, 4), (2, 63), (3, 0), (3, -2), (5, -1), (6, 0), (9, None), (9, P + 2),
                 (10, 999)]:
        a = list(good)
        a[i] = v
        assert L.gift_weight_grad(*a) == INVALID, (i, v)
    # an accumulating call over no tokens leaves W as it is
    assert L.gift_weight_grad(None, fw.BF16, 0, 64, ck, 0, 1000, 1.0, 1, P, 1000, P, wb, None) == OK


def test_wrapper_refuses_what_it_cannot_describe(fw):
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        fw.norm_forward(x)                               # not on the GPU
    with pytest.raises(ValueError):
        fw.norm_forward(torch.zeros(4, 8, dtype=torch.float64))
    with pytest.raises(ValueError):
        fw.norm_forward(torch.zeros(8))
    with pytest.raises(ValueError):
        fw.ActCheckpoint(4, 0)
    with pytest.raises(ValueError):
        fw.ActCheckpoint(4, 8, fmt=fw.E2M1)
    with pytest.raises(ValueError):
        fw.ActCheckpoint(4, 8, codes=torch.zeros(4, 8, dtype=torch.uint8))
