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
        self.device = torch.device("cuda", index) if index >= 0 else torch.device("cpu")

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 1 << 20

    def stride(self):
        return self.shape[1], 1

    def is_contiguous(self):
        return True


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


def test_strided_exponents_are_refused(ict):
    """A view of some columns of a wider tensor: its exponents do not lie one after the other."""

    class On(torch.Tensor):  # host tensors that say they are on a device
        def get_device(self):
            return 0

    on = lambda *shape: torch.zeros(shape, dtype=torch.int8).as_subclass(On)  # noqa: E731
    mant, exp = on(4, 128), on(4, 4)
    assert ict.DevCE(mant[:, 32:64], exp[:, 1:2].contiguous(), 1, 32).ld == 128
    for bad in ((mant[:, 32:64], exp[:, 1:2]), (on(32, 4).t(), on(4, 1)), (mant[:, ::2], exp[:, :2].contiguous())):
        with pytest.raises(ValueError):
            ict.DevCE(*bad, 1, 32)
    ict.DevCE(mant[:1], exp[:1], 1, 32)
    ict.DevCE(mant[1:3], exp[1:3], 1, 32)
    ict.DevCE(torch.empty_strided((0, 128), (0, 0), dtype=torch.int8).as_subclass(On), exp[:0], 1, 32)


def tensor(ict, rows, cols, mant, exp, g_cols=32, ld=None):
    """A description only: the checks read no memory."""
    return ict.ict_tensor(mant, exp, rows, cols, ld or cols, 1, g_cols)


def brute(a, ca, wa, b, cb, wb):
    """The bytes that the columns stand on, one by one."""

    def bytes_of(t, c, w):
        ng = -(-t.cols // t.g_cols)
        return ({t.mant + r * t.ld + k for r in range(t.rows) for k in range(c, c + w)}
                | {t.exp + r * ng + k for r in range(t.rows) for k in range(c // t.g_cols, -(-(c + w) // t.g_cols))})

    return bool(bytes_of(a, ca, wa) & bytes_of(b, cb, wb))


# descriptions that pass the checks end at the missing device; with one they would be launched
no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses of no memory")


@no_device
def test_shared_rows_of_gradients_are_refused(ict):
    """dQ and dK shifted against each other by bytes and rows, in tensors of one ld (where the check is exact) and with
    exponents of their own or shared."""
    M, E = 1 << 20, 1 << 24
    d = dict(batch=1, heads_q=2, heads_kv=1, len_q=5, len_k=4, head_dim=32, scale=(1, 3))
    o = tensor(ict, 5, 64, 1 << 28, 1 << 29)
    k = tensor(ict, 4, 160, 1 << 27, 1 << 26)
    q = tensor(ict, 5, 160, 1 << 27, 1 << 26)
    dv = tensor(ict, 4, 160, 1 << 22, 1 << 23)
    seen = set()
    for shift in [16 * n for n in range(-60, 61)] + [0]:
        for qc, kc in ((0, 64), (96, 0), (32, 128)):
            for own in (True, False):
                dq = tensor(ict, 5, 160, M, E)
                dk = tensor(ict, 4, 160, M + shift, E + 4096 if own else E)
                c = ict.attn_desc(dict(d, q_col=qc, k_col=kc, v_col=0))
                code = ict.lib.ict_attention_bwd(c, q, k, k, None, None, o, o, 1 << 20, dq, dk, dv, 1 << 20, 1 << 30, None)
                want = brute(dq, qc, 64, dk, kc, 32)
                seen.add(want)
                assert (code == 1) == want, (shift, qc, kc, own, code)
    assert seen == {True, False}


@no_device
def test_shared_layer_norm_gradients_are_refused(ict):
    M, E = 1 << 20, 1 << 24
    x, dy, dx = (tensor(ict, 8, 192, M * k, E + 4096 * k) for k in (1, 2, 3))
    g, dg, db = (tensor(ict, 1, 192, M * k, E + 4096 * k) for k in (4, 5, 6))

    def refused(dx=dx, dg=dg, db=db):
        return ict.lib.ict_layernorm_bwd(x, g, dy, 1, 20, dx, dg, db, 1 << 20, 1 << 30, None) == 1

    assert not refused() and not refused(db=None)
    for t in (x, dy):
        for rows in (-7, -1, 0, 1, 7):                       # rows of the other tensor
            assert refused(dx=tensor(ict, 8, 192, t.mant + 192 * rows, E + 8192 * 7))
        assert not refused(dx=tensor(ict, 8, 192, t.mant + 192 * 8, E + 8192 * 7))
        assert refused(dx=tensor(ict, 8, 192, M * 9, t.exp))  # exponents alone
        assert refused(dx=tensor(ict, 8, 192, M * 9, t.exp + 47)) and not refused(dx=tensor(ict, 8, 192, M * 9, t.exp + 48))
        assert refused(dx=tensor(ict, 8, 192, t.mant, E + 8192 * 7, ld=208))
    assert refused(dg=tensor(ict, 1, 192, dx.mant + 192 * 3, E + 8192 * 7))
    assert refused(db=tensor(ict, 1, 192, dg.mant + 176, E + 8192 * 7)) and refused(db=tensor(ict, 1, 192, M * 9, dg.exp + 5))
    assert not refused(db=tensor(ict, 1, 192, dg.mant + 192, dg.exp + 6))
