"""Checks that the Python binding makes before a call, on stand-ins for device tensors."""

import pytest
import torch


@pytest.fixture(scope="module")
def ict():
    from integer_only_nn_02_b200 import ict as _ict

    return _ict


class Fake:
    """What DevCE and the calls ask of a tensor, on a device of any index (-1: the host)."""

    dtype = torch.int8

    def __init__(self, index, *shape):
        self.shape, self.index = shape, index
        self.is_cuda, self.device = index >= 0, torch.device("cuda", index) if index >= 0 else torch.device("cpu")

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 1 << 20

    def dim(self):
        return len(self.shape)

    def stride(self, k):
        return (self.shape[1], 1)[k]


@pytest.mark.parametrize("exp_on", [-1, 1])
def test_exponents_elsewhere_are_refused(ict, exp_on, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    mant, exp = Fake(0, 4, 32), Fake(exp_on, 4, 1)
    with pytest.raises(ValueError):
        ict.DevCE(mant, exp, 1, 32)
    t = ict.DevCE(mant, Fake(0, 4, 1), 1, 32)
    assert ict._refs(t, None)[1] is None
    t.exp = exp
    with pytest.raises(ValueError):
        ict._refs(t)
