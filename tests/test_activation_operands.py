"""Operands that the activation operators' wrappers have to refuse before
anything is enqueued, with stand-ins for device tensors and for the library
(no GPU is needed)."""
import types

import pytest
import torch

D0, D1 = torch.device("cuda:0"), torch.device("cuda:1")
BF16, F32 = torch.bfloat16, torch.float32


class Operand:
    """What the wrappers see of a dense device tensor."""

    def __init__(self, *shape, dtype=BF16, device=D0, stride=None):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, device
        self._stride = torch.empty(shape, device="meta").stride() if stride is None else stride
        self.is_cuda = device.type == "cuda"

    def stride(self, i=None):
        return self._stride if i is None else self._stride[i]

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def is_contiguous(self):
        return self._stride == torch.empty(self.shape, device="meta").stride()

    def data_ptr(self):
        return 1 << 20


class Library:
    """The real library's sizes; every other call is noted and not made."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.real, name)

        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def fw(monkeypatch):
    import fac_whitening_amd as fw
    monkeypatch.setattr(fw, "_lib", Library(fw._lib))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    monkeypatch.setattr(fw, "_empty", lambda stream, shape, dtype, device: Operand(*shape, dtype=dtype, device=device))
    monkeypatch.setattr(fw, "_empty_like", lambda stream, t: Operand(*t.shape, dtype=t.dtype, device=t.device))
    return fw


T, DIM, M = 16, 64, 32


def _ckpt(fw, device=D0):
    return fw.ActCheckpoint(T, DIM, codes=Operand(T, DIM, dtype=torch.uint8, device=device),
                            bscales=Operand(2, 2, 8, dtype=torch.uint8, device=device))


def _calls(fw):
    """Each wrapper with every tensor that it takes, by name."""
    rows, vec = (lambda dev=D0, dt=BF16: Operand(T, DIM, dtype=dt, device=dev)), (lambda n, dev=D0: Operand(n, dtype=F32, device=dev))
    work = lambda dev=D0: Operand(1 << 24, dtype=torch.uint8, device=dev)   # noqa: E731
    return {
        "save": (lambda ck, x, **k: ck.save(x, **k), dict(ck=lambda dev=D0: _ckpt(fw, dev), x=rows)),
        "restore": (lambda ck, out, **k: ck.restore(out=out, **k), dict(ck=lambda dev=D0: _ckpt(fw, dev), out=rows)),
        "norm_forward": (fw.norm_forward, dict(x=rows, weight=lambda dev=D0: vec(DIM, dev), bias=lambda dev=D0: vec(DIM, dev),
                                               ckpt=lambda dev=D0: _ckpt(fw, dev), out=rows)),
        "norm_backward": (fw.norm_backward, dict(dy=rows, x=rows, mean=lambda dev=D0: vec(T, dev), rstd=lambda dev=D0: vec(T, dev),
                                                 weight=lambda dev=D0: vec(DIM, dev), dx=rows,
                                                 dweight=lambda dev=D0: vec(DIM, dev), dbias=lambda dev=D0: vec(DIM, dev),
                                                 work=work)),
        "norm_backward_ckpt": (fw.norm_backward, dict(dy=rows, x=lambda dev=D0: _ckpt(fw, dev), mean=lambda dev=D0: vec(T, dev),
                                                      rstd=lambda dev=D0: vec(T, dev), dx=rows, work=work)),
        "weight_grad": (fw.weight_grad, dict(delta=lambda dev=D0: Operand(T, M, device=dev), ckpt=lambda dev=D0: _ckpt(fw, dev),
                                             out=lambda dev=D0: Operand(M, DIM, dtype=F32, device=dev), work=work)),
    }


NAMES = ["save", "restore", "norm_forward", "norm_backward", "norm_backward_ckpt", "weight_grad"]


@pytest.mark.parametrize("name", NAMES)
def test_operands_of_one_call_are_on_one_device(fw, name):
    call, makers = _calls(fw)[name]
    call(**{k: f() for k, f in makers.items()})
    assert len(fw._lib.calls) == 1
    for other in makers:
        for dev in (D1, torch.device("cpu")):
            if dev.type == "cpu" and other in ("ck", "ckpt") or (other == "x" and "ckpt" in name and dev.type == "cpu"):
                continue                                     # a checkpoint refuses the host itself
            with pytest.raises(ValueError):
                call(**{k: f(dev) if k == other else f() for k, f in makers.items()})
    assert len(fw._lib.calls) == 1


@pytest.mark.parametrize("name", NAMES)
def test_a_call_runs_on_its_operands_device(fw, name, monkeypatch):
    call, makers = _calls(fw)[name]
    # all operands on a device that is not the current one
    with pytest.raises(ValueError):
        call(**{k: f(D1) for k, f in makers.items()})
    # a stream of another device
    with pytest.raises(ValueError):
        call(**{k: f() for k, f in makers.items()}, stream=types.SimpleNamespace(cuda_stream=7, device=D1))
    assert not fw._lib.calls
    call(**{k: f() for k, f in makers.items()}, stream=types.SimpleNamespace(cuda_stream=7, device=D0))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    call(**{k: f(D1) for k, f in makers.items()})
    assert len(fw._lib.calls) == 2 and fw._lib.calls[0][1][-1] == 7


@pytest.mark.parametrize("name", ["norm_backward", "weight_grad"])
def test_workspace_is_what_it_says_it_is(fw, name):
    """The library writes as many bytes as it is told: they have to be there."""
    call, makers = _calls(fw)[name]
    need = 1 << 24

    def with_work(work):
        fw._lib.calls.clear()
        call(**{**{k: f() for k, f in makers.items()}, "work": work})
        ((_, args),) = fw._lib.calls
        return args[-2]

    assert with_work(Operand(need, dtype=torch.uint8)) == need
    assert with_work(Operand(need // 4, dtype=F32)) == need
    for bad in (Operand(need, dtype=torch.uint8, stride=(0,)), Operand(need, dtype=torch.uint8, stride=(2,)),
                Operand(64, need // 64, dtype=torch.uint8, stride=(0, 1))):
        with pytest.raises(ValueError):
            with_work(bad)
        assert not fw._lib.calls


def test_wrong_types_and_kinds_are_value_errors(fw):
    x, ck = Operand(T, DIM), _ckpt(fw)
    v = lambda dt: Operand(DIM, dtype=dt)                    # noqa: E731
    stats = Operand(T, dtype=F32)
    calls = [
        lambda: ck.restore(torch.float64), lambda: ck.restore(torch.uint8),
        lambda: fw.norm_forward(x, None, v(torch.float64)), lambda: fw.norm_forward(x, None, v(torch.float16)),
        lambda: fw.norm_forward(x, v(F32), v(BF16)), lambda: fw.norm_forward(x, v(torch.float16)),
        lambda: fw.norm_forward(x, kind="batch"), lambda: fw.norm_forward(x, kind=None),
        lambda: fw.norm_backward(x, x, stats, stats, kind="batch"),
        lambda: fw.norm_backward(x, x, stats, stats, v(torch.float64)),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            print("accepted", i)
    assert not fw._lib.calls
    fw.norm_forward(x, None, v(F32))
    fw.norm_forward(x, None, v(BF16), kind=fw.NORM_LAYER)
    assert [a[1][8] for a in fw._lib.calls] == [fw.FP32, fw.BF16]      # the bias alone gives the type


def test_a_checkpoint_keeps_the_buffers_it_was_made_with(fw):
    """The library is given the addresses taken when it was made."""
    ck = _ckpt(fw)
    codes, bscales = ck.codes, ck.bscales
    for name, v in (("codes", Operand(T, DIM, dtype=torch.uint8)), ("bscales", Operand(2, 2, 8, dtype=torch.uint8)),
                    ("T", T + 1), ("d", DIM + 1), ("fmt", fw.E5M2), ("device", D1)):
        with pytest.raises(AttributeError):
            setattr(ck, name, v)
    assert ck.codes is codes and ck.bscales is bscales and (ck.T, ck.d, ck.fmt) == (T, DIM, fw.E4M3)
    ck.name = "fc1"                                          # a user's own attribute
