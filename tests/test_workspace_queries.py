"""A wrapper that is given its workspace does not ask how large one would have
to be: the query plans the product, 1 to 2 us of a call that takes about 10."""
import pytest
import torch

from test_activation_operands import F32, Library, Operand
from test_feedforward_abi import DIM, HID, T, _calls, fw  # noqa: F401  (a fixture)


class Counting(Library):
    def __init__(self, real):
        super().__init__(real)
        self.queries = []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            self.queries.append(name)
        return super().__getattr__(name)


@pytest.mark.parametrize("name", ["glu_forward", "glu_backward", "weight_grad", "weight_grad of a checkpoint"])
def test_given_workspace_is_not_asked_for(fw, name):
    call, args = _calls(fw)[name.split()[0]]
    kw = {k: v() for k, v in args.items()}
    if name.endswith("checkpoint"):
        kw["ckpt"] = fw.ActCheckpoint(T, DIM, codes=Operand(T, DIM, dtype=torch.uint8),
                                      bscales=Operand(2, DIM // 32, 8, dtype=torch.uint8))
        kw["out"] = Operand(HID, DIM, dtype=F32)
    fw._lib = Counting(fw._lib.real)
    call(**kw)
    assert len(fw._lib.calls) == 1 and not fw._lib.queries
    kw["work"] = None
    call(**kw)
    assert len(fw._lib.calls) == 2 and len(fw._lib.queries) == 1
