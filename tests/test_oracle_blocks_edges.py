"""The oracle of layer norm and attention at the edges of their ranges, against 64-bit floating point."""
import numpy as np
import pytest

from integer_only_nn_02_b200.workloads import CE, E_ZERO
from oracle import blocks
from tests.test_oracle_blocks import quantise, values


def layernorm_gradient(x, g, dy, eps):
    """dX in 64 bits, with 1 / sqrt(var + eps) and the normalised rows."""
    inv = 1 / np.sqrt(x.var(1, keepdims=True) + eps)
    xh, gd = (x - x.mean(1, keepdims=True)) * inv, dy * g
    return (gd - gd.mean(1, keepdims=True) - xh * (gd * xh).mean(1, keepdims=True)) * inv, xh, gd, inv


@pytest.mark.parametrize("N", [16, 768, 4096])
@pytest.mark.parametrize("eps", [(1, 20), (1, 0), (512, 0), (1, 64), (300, 17)])
def test_layernorm_gradient_of_small_rows(N, eps):
    """Rows of every size down to 2^-127, of one group each, whose variance vanishes beside eps: the gradient tends to
    (g - mean g) / sqrt(eps) and no further.  The bound is that of rows of ordinary size: FIT rounds dX within half a
    step of its largest value / 64; t is off by at most 1 (m1 and z by half a unit each), a quarter of g's unit, within
    the half below; and h's error of 2^-9 enters through m2 and through z."""
    rng = np.random.default_rng(N)
    down = [0, 4, 10, 20, 24, 27, 31, 34, 40, 50, 64, 90, 120]
    v = rng.standard_normal((len(down), N)) * 2.0
    X = quantise(v, N)
    X.exp[:] = np.maximum(X.exp.astype(int) - np.array(down)[:, None], -127)
    gamma, dY = quantise(1 + 0.2 * rng.standard_normal((1, N)), N), quantise(rng.standard_normal((len(down), N)) * 1e-3, N)
    x, g, dy = values(X), values(gamma)[0], values(dY)
    ref, xh, gd, inv = layernorm_gradient(x, g, dy, eps[0] * 2.0 ** -eps[1])
    dX = values(blocks.layernorm_bwd(X, gamma, dY, eps, N)[0])
    unit = np.exp2(blocks.exps(dY).astype(float) + blocks.exps(gamma).astype(float))
    slack = unit * (0.5 + 2.0 ** -8 * np.abs((gd * xh).mean(1, keepdims=True) / unit) * np.abs(xh).max() +
                    2.0 ** -9 * np.abs(gd / unit).max() * np.abs(xh).max()) * inv
    tol = np.abs(ref).max(1, keepdims=True) / 128 * 1.01 + slack
    assert (np.abs(dX - ref) <= tol).all(), (np.abs(dX - ref) / tol).max(1)
    assert (np.linalg.norm(dX, axis=1) < 1.1 * np.linalg.norm(ref, axis=1)).all()


@pytest.mark.parametrize("eps", [(1, 20), (512, 0), (1, 64)])
def test_layernorm_gradient_of_zero_rows(eps):
    """A row of zeros is the limit of small rows: (g - mean g) / sqrt(eps).  t is off by at most half a unit (m1), an
    eighth of g's; R by three roundings to 24 bits; FIT by half a step."""
    rng = np.random.default_rng(3)
    N = 192
    X = CE(np.zeros((4, N), np.int8), np.full((4, N // 32), E_ZERO, np.int8), 1, 32)
    gamma, dY = quantise(1 + 0.2 * rng.standard_normal((1, N)), N), quantise(rng.standard_normal((4, N)) * 1e-3, N)
    dY.mant[3], dY.exp[3] = 0, E_ZERO
    dX, dg, db = (values(t) for t in blocks.layernorm_bwd(X, gamma, dY, eps, 32))
    ref, _, _, inv = layernorm_gradient(values(X), values(gamma)[0], values(dY), eps[0] * 2.0 ** -eps[1])
    unit = np.exp2(blocks.exps(dY)[:3].astype(float) + blocks.exps(gamma).astype(float))
    tol = np.abs(ref[:3]).max(1, keepdims=True) / 128 * 1.01 + unit / 8 * 1.01 * inv[:3]
    assert (np.abs(dX[:3] - ref[:3]) <= tol).all() and not dX[3].any()
    assert not dg.any() and db.any()
    assert not values(blocks.layernorm_bwd(X, gamma, dY, (0, 0), 32)[0]).any()
