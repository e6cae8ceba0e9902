"""The oracle of layer norm and attention at the edges of their ranges, against 64-bit floating point."""
import numpy as np
import pytest

from integer_only_nn_02_b200.workloads import CE, E_ZERO
from oracle import blocks
from tests.test_oracle_blocks import quantise, rel, smooth_case, softmax_attention, values


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


def aligned_attention(d, Q, K, V, O, dO):
    """O, dQ, dK and dV of one head in 64 bits, from the operands as they are aligned."""
    H = blocks._Head(d, Q, K, V, 0, 0, d["len_q"], d["len_k"], dO)
    q, k, v, do = (a.astype(np.float64) * 2.0 ** e for a, e in ((H.q[0], H.eq), (H.k, H.ek), (H.v, H.ev), (H.d[0], H.ed)))
    scale = d["scale"][0] * 2.0 ** -d["scale"][1]
    s = q @ k.T * scale
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    dP = do @ v.T
    dS = p * (dP - (p * dP).sum(1, keepdims=True))
    return p @ v, dS @ k * scale, dS.T @ q * scale, p.T @ do


@pytest.mark.parametrize("m", [300, 4096, 8192])
def test_gradients_beside_a_peaked_query_without_one(m):
    """64 queries over m keys, one of which puts all its weight on one key and has no gradient: it does not choose the
    others' digits.  A weight is off by at most 2^(1/128) - 1 = 0.54 percent (its exponent's rounding) and 2^-12 (E's
    and P's, at logits within +-2 of the mean), a normalised one by twice that; dP's correction and U's 14 bits add
    less than 1 percent, and FIT half a step of a group's largest value / 64, 0.5 percent of the norm: 3 percent of
    the gradients' norms in all."""
    rng = np.random.default_rng(m)
    D, n = 32, 64
    q, k = rng.standard_normal((n, D)), rng.standard_normal((m, D))
    q *= 0.3
    k[5] = 4 * np.sign(rng.standard_normal(D))
    q[:, :] -= (q @ k[5])[:, None] * k[5] / (k[5] @ k[5])     # the others do not see that key apart
    q[9] = k[5]
    v, do = rng.standard_normal((m, D)), rng.standard_normal((n, D)) * 1e-3
    do[9] = 0
    d = dict(batch=1, heads_q=1, heads_kv=1, len_q=n, len_k=m, head_dim=D, scale=(181, 10))
    Q, K, V, dO = (quantise(t, D) for t in (q, k, v, do))
    O, stats = blocks.attention_fwd(d, Q, K, V, g_cols=32)
    assert stats[9, 1] < 2 ** 14 + 2 ** 8 and np.delete(stats[:, 1], 9).min() > 0.1 * m * 2 ** 14
    _, _, dK, dV = aligned_attention(d, Q, K, V, O, dO)
    _, gk, gv = (values(t) for t in blocks.attention_bwd(d, Q, K, V, O, dO, g_cols=32))
    for got, want in ((gk, dK), (gv, dV)):
        assert np.linalg.norm(got - want) < 0.03 * np.linalg.norm(want)


@pytest.mark.parametrize("n,m,causal,D", [(200, 700, False, 64), (300, 300, True, 64), (40, 1500, False, 32)])
def test_attention_follows_the_formula_at_length(n, m, causal, D):
    """Attention and its gradients of the operands' own values.  An aligned element is off by at most half a step of a
    grid on which the largest of all rows, below 5 (of up to 10^5 normal draws), is at least 64 steps: 5 / 128 / sqrt(3)
    = 2.3 percent of a standard deviation.  A score, scaled by 1 / sqrt(D), sums D products with such an error in either
    factor: 2.3 sqrt(2) = 3.2 percent, and a weight with it.  V adds 2.3 percent and FIT 0.5: 6 percent of the norm,
    twice that as the bound; the gradients pass through two such products."""
    d, q, k, v, do, vis = smooth_case(n + m, n, m, D, causal)
    d["scale"] = {64: (1, 3), 32: (181, 10)}[D]
    scale = d["scale"][0] * 2.0 ** -d["scale"][1]
    o, _ = blocks.attention_fwd(d, q, k, v, g_cols=32)
    Q, K, V, dO = (values(t) for t in (q, k, v, do))
    p, ref = softmax_attention(Q, K, V, vis, scale)
    assert rel(values(o), ref) < 0.12
    dP = dO @ V.T
    dS = p * (dP - (p * dP).sum(1, keepdims=True))
    dQ, dK, dV = blocks.attention_bwd(d, q, k, v, o, do, g_cols=32)
    for got, want in ((dQ, dS @ K * scale), (dK, dS.T @ Q * scale), (dV, p.T @ dO)):
        assert rel(values(got), want) < 0.24


@pytest.mark.parametrize("m", [300, 2048])
def test_attention_of_the_aligned_operands(m):
    """Beside the alignment, what is rounded moves outputs and gradients by 3 percent at any length (the sum of
    test_gradients_beside_a_peaked_query_without_one)."""
    rng = np.random.default_rng(m)
    D, n = 64, 48
    d = dict(batch=1, heads_q=1, heads_kv=1, len_q=n, len_k=m, head_dim=D, scale=(1, 3))
    Q, K, V = (quantise(rng.standard_normal((r, D)), 32) for r in (n, m, m))
    dO = quantise(rng.standard_normal((n, D)) * 1e-3, 32)
    O, _ = blocks.attention_fwd(d, Q, K, V, g_cols=32)
    want = aligned_attention(d, Q, K, V, O, dO)
    for got, ref in zip((O, *blocks.attention_bwd(d, Q, K, V, O, dO, g_cols=32)), want):
        assert rel(values(got), ref) < 0.03
