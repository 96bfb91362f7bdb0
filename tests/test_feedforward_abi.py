"""Refusals of the gated feed-forward, dropout and whole-activation
weight-gradient operators: every bad argument is an error before anything is
enqueued (no GPU is needed: the pointers are never followed)."""
import ctypes
import types

import pytest
import torch

from test_activation_operands import BF16, D0, D1, F32, Library, Operand

P = 1 << 20          # well-aligned addresses, far apart, that are never followed
FAR = 1 << 50
OK, INVALID, WORKSPACE, UNSUPPORTED = 0, 1, 2, 5


@pytest.fixture(scope="module")
def lib():
    import fac_whitening_amd as fw
    return fw


def _drop(fw, p=0.1, d_offset=None):
    return ctypes.byref(fw.DropoutDesc(p, 1, 2, d_offset))


def _refused(call, good, bad):
    for i, v in bad:
        a = list(good)
        a[i] = v
        assert call(*a) == INVALID, (i, v)


def test_dropout_arguments(lib):
    fw, L = lib, lib._lib
    y = P + FAR
    #       drop        x  dtype    ld    T  d     r       ld    y  ld
    good = [_drop(fw), P, fw.BF16, 1000, 5, 1000, P + 2 * FAR, 1000, y, 1000, None]
    _refused(L.gift_dropout_apply, good, [
        (0, None), (0, _drop(fw, -0.1)), (0, _drop(fw, 1.1)), (0, _drop(fw, float("nan"))), (0, _drop(fw, 0.1, P + 4)),
        (1, None), (1, P + 1), (2, 3), (2, -1), (3, 999), (4, -1), (5, 0), (5, (1 << 24) + 1), (6, P + 1), (7, 999), (8, None),
        (8, y + 1), (9, 999),
        (8, P + 16), (8, P + 2 * FAR + 8000), (1, y - 2)])     # an output that shares memory with an input
    # side by side in one buffer is no overlap, but one column too many is
    a = list(good)
    a[1], a[3], a[8], a[9], a[6] = P, 2000, P + 2000, 2000, None
    a[4] = 0
    assert L.gift_dropout_apply(*a) == OK
    a[4], a[8] = 5, P + 1998
    assert L.gift_dropout_apply(*a) == INVALID
    big = list(good)
    big[4] = (1 << 32) + 1
    big[1], big[6], big[8] = P, None, P
    assert L.gift_dropout_apply(*big) == UNSUPPORTED
    none = [_drop(fw), None, fw.FP32, 8, 0, 8, None, 0, None, 8, None]
    assert L.gift_dropout_apply(*none) == OK


def _forward(fw, T=5, d=64, f=96, dtype=None, **kw):
    dtype = fw.BF16 if dtype is None else dtype
    a = dict(act=0, x=P, dtype=dtype, ldx=d, T=T, d=d, wg=P + FAR, ldg=d, wu=P + 2 * FAR, ldu=d, f=f, drop=None,
             h=P + 3 * FAR, ldh=f, gate=P + 4 * FAR, ldz=f, up=P + 5 * FAR, ldup=f, ckpt=None, work=P + 6 * FAR, bytes=1 << 40,
             stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return fw._lib.gift_glu_forward(*a.values())


def test_glu_forward_arguments(lib):
    fw = lib
    for kw in (dict(act=5), dict(act=-1), dict(x=None), dict(x=P + 1), dict(dtype=3), dict(ldx=63), dict(T=-1), dict(d=0),
               dict(d=(1 << 24) + 1), dict(wg=None), dict(wg=P + FAR + 1), dict(ldg=63), dict(wu=None), dict(ldu=0), dict(f=0),
               dict(drop=_drop(fw, 2.0)), dict(drop=_drop(fw, 0.1, P + 1)), dict(h=None), dict(h=P + 1), dict(ldh=95),
               dict(gate=None), dict(up=None), dict(ldz=95), dict(ldup=95), dict(gate=P + 4 * FAR + 1),
               dict(h=P), dict(h=P + FAR + 100), dict(gate=P + 2 * FAR), dict(up=P + 64),          # outputs over inputs
               dict(gate=P + 3 * FAR), dict(up=P + 3 * FAR + 2), dict(up=P + 4 * FAR),            # outputs over outputs
               dict(gate=P + 4 * FAR, up=P + 4 * FAR + 2 * 95, ldz=192, ldup=192),
               dict(ckpt=ctypes.byref(fw.ActCkpt(P + 7 * FAR, 64, P + 8 * FAR, 0))),
               dict(ckpt=ctypes.byref(fw.ActCkpt(P + 7 * FAR, 96, P + 8 * FAR, 2))),
               dict(ckpt=ctypes.byref(fw.ActCkpt(P + 7 * FAR + 8, 96, P + 8 * FAR, 0))),
               dict(ckpt=ctypes.byref(fw.ActCkpt(P + 7 * FAR, 96, None, 0))),
               dict(ckpt=ctypes.byref(fw.ActCkpt(P, 96, P + 8 * FAR, 0))),
               dict(ckpt=ctypes.byref(fw.ActCkpt(P + 7 * FAR, 96, P + 3 * FAR + 16, 0)))):
        assert _forward(fw, **kw) == INVALID, kw
    assert _forward(fw, T=0, x=None, h=None, gate=None, up=None) == OK
    # gate and up side by side in one matrix, the weights as halves of one
    assert _forward(fw, T=0, gate=P + 4 * FAR, up=P + 4 * FAR + 192, ldz=192, ldup=192) == OK
    assert _forward(fw, T=1 << 36) == UNSUPPORTED
    assert _forward(fw, T=(1 << 32) + 1, drop=_drop(fw)) == UNSUPPORTED


def _backward(fw, T=5, d=64, f=96, **kw):
    a = dict(act=0, dh=P, dtype=fw.BF16, lddh=f, T=T, f=f, gate=P + FAR, ldz=f, up=P + 2 * FAR, ldup=f, drop=None,
             dgate=P + 3 * FAR, lddz=f, dup=P + 4 * FAR, lddup=f, wg=P + 5 * FAR, ldg=d, wu=P + 6 * FAR, ldu=d, d=d,
             dx=P + 7 * FAR, lddx=d, work=P + 8 * FAR, bytes=1 << 40, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return fw._lib.gift_glu_backward(*a.values())


def test_glu_backward_arguments(lib):
    fw = lib
    for kw in (dict(act=5), dict(dh=None), dict(dh=P + 1), dict(dtype=7), dict(lddh=95), dict(T=-1), dict(f=0), dict(gate=None),
               dict(ldz=95), dict(up=None), dict(ldup=95), dict(drop=_drop(fw, -1.0)), dict(dgate=None), dict(lddz=95),
               dict(dup=None), dict(dup=P + 4 * FAR + 1), dict(lddup=0), dict(wg=None), dict(ldg=63), dict(wu=None), dict(ldu=63),
               dict(d=0), dict(lddx=63), dict(dx=P + 7 * FAR + 1),
               dict(dgate=P + FAR + 2), dict(dup=P + FAR + 192), dict(dgate=P + FAR, lddz=100), dict(dup=P + 3 * FAR),
               dict(dx=P + 3 * FAR), dict(dx=P + 5 * FAR), dict(dgate=P + 6 * FAR), dict(dup=P + FAR, dgate=P + FAR)):
        assert _backward(fw, **kw) == INVALID, kw
    none = dict(T=0, dh=None, gate=None, up=None, dgate=None, dup=None)
    assert _backward(fw, **none, dx=None) == OK
    assert _backward(fw, **none, dx=None, wg=None, wu=None, d=0, work=None, bytes=0) == OK
    assert _backward(fw, T=1 << 36) == UNSUPPORTED
    assert _backward(fw, T=(1 << 32) + 1, f=1, lddh=1, ldz=1, ldup=1, lddz=1, lddup=1, drop=_drop(fw), dx=None) in (
        INVALID, UNSUPPORTED)


def test_weight_grad_x_arguments(lib):
    fw, L = lib, lib._lib
    W = P + 3 * FAR
    good = [P, fw.BF16, 64, 64, P + FAR, 1000, 5, 1000, 1.0, 0, W, 1000, P + 4 * FAR, 1 << 40, None]
    _refused(L.gift_weight_grad_x, good, [
        (0, None), (0, P + 1), (1, 4), (2, 63), (3, 0), (3, -2), (4, None), (4, P + FAR + 1), (5, 999), (6, -1), (7, 0), (10, None),
        (10, W + 2), (11, 999), (10, P + 4), (10, P + FAR)])
    big = list(good)
    big[2] = big[3] = big[5] = big[7] = big[11] = 1 << 24
    big[10], big[6] = P + 4 * FAR, 1
    assert L.gift_weight_grad_x(*big) == UNSUPPORTED
    # an accumulating call over no tokens leaves W as it is
    assert L.gift_weight_grad_x(None, fw.BF16, 0, 64, None, 0, 0, 1000, 1.0, 1, W, 1000, None, 0, None) == OK


# -- the wrappers, with stand-ins for device tensors and for the library ---------

@pytest.fixture
def fw(monkeypatch):
    import fac_whitening_amd as fw
    monkeypatch.setattr(fw, "_lib", Library(fw._lib))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    monkeypatch.setattr(fw, "_empty", lambda stream, shape, dtype, device: Operand(*shape, dtype=dtype, device=device))
    monkeypatch.setattr(fw, "_empty_like", lambda stream, t: Operand(*t.shape, dtype=t.dtype, device=t.device))
    return fw


T, DIM, HID = 16, 64, 96


def _counter(dev=D0, n=1, dtype=torch.int64):
    return Operand(n, dtype=dtype, device=dev)


def _calls(fw):
    """Each wrapper with every tensor that it takes, by name."""
    def mat(r, c, dt=BF16):
        return lambda dev=D0: Operand(r, c, dtype=dt, device=dev)
    work = lambda dev=D0: Operand(1 << 30, dtype=torch.uint8, device=dev)   # noqa: E731
    drop = lambda dev=D0: fw.Dropout(0.1, 1, counter=_counter(dev))         # noqa: E731
    ck = lambda dev=D0: fw.ActCheckpoint(T, HID, codes=Operand(T, HID, dtype=torch.uint8, device=dev),   # noqa: E731
                                         bscales=Operand(2, 3, 8, dtype=torch.uint8, device=dev))
    x, w, h = mat(T, DIM), mat(HID, DIM), mat(T, HID)
    return {
        "dropout_forward": (fw.dropout_forward, dict(x=x, drop=drop, residual=x, out=x)),
        "dropout_backward": (fw.dropout_backward, dict(dy=x, drop=drop, dx=x)),
        "glu_forward": (fw.glu_forward, dict(x=x, w_gate=w, w_up=w, drop=drop, ckpt=ck, out=h, gate=h, up=h, work=work)),
        "glu_backward": (fw.glu_backward, dict(dh=h, gate=h, up=h, w_gate=w, w_up=w, drop=drop, dx=x, dgate=h, dup=h,
                                               work=work)),
        "weight_grad": (fw.weight_grad, dict(delta=h, ckpt=x, out=mat(HID, DIM, F32), work=work)),
    }


NAMES = ["dropout_forward", "dropout_backward", "glu_forward", "glu_backward", "weight_grad"]


@pytest.mark.parametrize("name", NAMES)
def test_operands_of_one_device(fw, name):
    call, args = _calls(fw)[name]
    call(**{k: v() for k, v in args.items()})
    assert len(fw._lib.calls) == 1
    for k, v in args.items():
        with pytest.raises(ValueError):
            call(**{q: (v(D1) if q == k else w()) for q, w in args.items()})
    with pytest.raises(ValueError):      # all on a device that is not the current one
        call(**{k: v(D1) for k, v in args.items()})
    with pytest.raises(ValueError):      # a stream of another device
        call(**{k: v() for k, v in args.items()}, stream=types.SimpleNamespace(device=D1, cuda_stream=0))
    assert len(fw._lib.calls) == 1


@pytest.mark.parametrize("name", NAMES)
def test_shapes_and_types(fw, name):
    call, args = _calls(fw)[name]
    for k in args:
        if k in ("drop", "work", "ckpt") and name != "weight_grad":
            continue
        good = args[k]()
        if good.dtype == torch.uint8:
            continue
        r, c = good.shape
        bad = [Operand(r, c, dtype=torch.float64), Operand(r, c, dtype=torch.float16), Operand(r * c)]
        if (name, k) not in (("dropout_backward", "dy"), ("dropout_forward", "x"), ("weight_grad", "delta")):
            bad += [Operand(r + 1, c)] if k not in ("w_gate",) or name == "glu_backward" else []
        if r > 1:
            bad.append(Operand(r, c, dtype=good.dtype, stride=(1, r)))
        for b in bad:
            with pytest.raises(ValueError):
                call(**{q: (b if q == k else w()) for q, w in args.items()})
    assert not fw._lib.calls


def test_arguments_that_belong_together(fw):
    x, w, h = Operand(T, DIM), Operand(HID, DIM), Operand(T, HID)
    for kw in (dict(gate=h), dict(up=h), dict(act="swish"), dict(act=9),
               dict(ckpt=fw.ActCheckpoint(T, 32, codes=Operand(T, 32, dtype=torch.uint8), bscales=Operand(2, 1, 8, dtype=torch.uint8)))):
        with pytest.raises(ValueError):
            fw.glu_forward(x, w, w, **kw)
    for kw in (dict(w_gate=w), dict(w_up=w), dict(dx=x)):
        with pytest.raises(ValueError):
            fw.glu_backward(h, h, h, **kw)
    with pytest.raises(ValueError):
        fw.weight_grad(h, x, accumulate=True)
    with pytest.raises(ValueError):      # a sparse workspace
        fw.glu_forward(x, w, w, work=Operand(1 << 20, dtype=torch.uint8, stride=(2,)))
    assert not fw._lib.calls


def test_dropout_arguments_of_the_wrapper(fw):
    for bad in (dict(p=-0.1), dict(p=1.5), dict(p=float("nan")), dict(seed=-1), dict(seed=1 << 64), dict(offset=-1),
                dict(offset=1 << 64), dict(counter=_counter(n=2)), dict(counter=_counter(dtype=torch.int32)),
                dict(counter=torch.zeros(1, dtype=torch.int64))):
        with pytest.raises(ValueError):
            fw.Dropout(**{"p": 0.1, "seed": 3, **bad})
    d = fw.Dropout(0.1, 3)
    for k in ("p", "seed", "offset", "counter"):
        with pytest.raises(AttributeError):
            setattr(d, k, 0)
