"""The oracle of layer norm and attention against the formulas in 64-bit floating point,
against differences, and in closed form; refusals of the library's entry points (their
checks run on the host before any device is asked for)."""
import ctypes

import numpy as np
import pytest

from integer_only_nn_02_b200.workloads import CE, E_ZERO
from oracle import blocks
from tests.brute import fit_brute
from tests.test_oracle_pins import rand_ce


def values(t):
    return t.mant * np.exp2(blocks.exps(t).astype(np.float64)) * (blocks.exps(t) != E_ZERO)


def quantise(v, G):
    out = CE(np.zeros(v.shape, np.int8), np.zeros((v.shape[0], -(-v.shape[1] // G)), np.int8), 1, G)
    for i in range(v.shape[0]):
        for g in range(0, v.shape[1], G):
            from fractions import Fraction

            m, e = fit_brute([Fraction(float(x)) for x in v[i, g: g + G]])
            out.mant[i, g: g + G], out.exp[i, g // G] = m, e
    return out


def rel(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


def softmax_attention(q, k, v, vis, scale):
    s = np.where(vis, q @ k.T * scale, -np.inf)
    s = s - np.where(vis.any(1), s.max(1), 0)[:, None]
    p = np.where(vis, np.exp(s), 0)
    p /= np.maximum(p.sum(1, keepdims=True), 1e-300)
    return p, p @ v


def smooth_case(seed, n, m, D, causal):
    """Operands whose rows share one size, as the int8 grids resolve them best."""
    rng = np.random.default_rng(seed)
    d = dict(batch=1, heads_q=1, heads_kv=1, len_q=n, len_k=m, head_dim=D, causal=causal, scale=(1, 3))
    q, k, v = (quantise(rng.standard_normal((x, D)), D) for x in (n, m, m))
    do = quantise(rng.standard_normal((n, D)) * 1e-3, D)
    vis = np.arange(m)[None] <= np.arange(n)[:, None] + m - n if causal else np.ones((n, m), bool)
    return d, q, k, v, do, vis


@pytest.mark.parametrize("n,m,causal", [(9, 9, False), (24, 40, True), (33, 20, False)])
def test_attention_follows_the_formula(n, m, causal):
    """Bounds: an aligned operand's element is off by at most half a step of a grid on which the largest
    element is at least 64 steps, so by 2^-7 of it; a score of D = 64 products of values below c = 4.5 (the
    largest of a few thousand normal draws) is then off by at most 8 (2^-7 c) c + ... < 3 in the worst case, but
    its typical error is sqrt(64) * 4.5 / 128 / sqrt(3) / 8 * sqrt(2) = 0.03 (one standard deviation of a sum
    of 64 independent errors times normal values, scaled by 1/8), which moves a weight by 3 percent; O adds
    V's own 2^-7 c / sqrt(3) = 2 percent and its own rounding.  The gradients pass through two such products.
    Relative to the norms: 0.1 forward (twice the sum), 0.2 backward."""
    d, q, k, v, do, vis = smooth_case(n + m, n, m, 64, causal)
    o, _ = blocks.attention_fwd(d, q, k, v, g_cols=32)
    Q, K, V, dO = (values(t) for t in (q, k, v, do))
    p, ref = softmax_attention(Q, K, V, vis, 0.125)
    assert rel(values(o), ref) < 0.1
    dP = dO @ V.T
    dS = p * (dP - (p * dP).sum(1, keepdims=True))
    dQ, dK, dV = blocks.attention_bwd(d, q, k, v, o, do, g_cols=32)
    for got, want in ((dQ, dS @ K / 8), (dK, dS.T @ Q / 8), (dV, p.T @ dO)):
        assert rel(values(got), want) < 0.2


def test_attention_gradient_against_differences():
    """The formula that the test above holds the gradients to is itself the derivative: central differences of
    sum(O dO) in 64 bits (step h: error h^2 |f'''| / 6 + 2^-52 |f| / h, about 1e-9 here)."""
    rng = np.random.default_rng(0)
    q, k, v, do = (rng.standard_normal((s, 8)) for s in (5, 7, 7, 5))
    vis = np.arange(7)[None] <= np.arange(5)[:, None] + 2
    f = lambda q, k, v: float((softmax_attention(q, k, v, vis, 0.3)[1] * do).sum())  # noqa: E731
    p, _ = softmax_attention(q, k, v, vis, 0.3)
    dP = do @ v.T
    dS = p * (dP - (p * dP).sum(1, keepdims=True))
    for at, grad in ((0, dS @ k * 0.3), (1, dS.T @ q * 0.3), (2, p.T @ do)):
        x = [q, k, v]
        for i, j in ((0, 0), (3, 5), (4, 7)):
            h = 1e-5
            up, dn = [t.copy() for t in x], [t.copy() for t in x]
            up[at][i, j] += h
            dn[at][i, j] -= h
            assert abs((f(*up) - f(*dn)) / (2 * h) - grad[i, j]) < 1e-7


def test_attention_closed_forms():
    rng = np.random.default_rng(1)
    D = 16
    d = dict(batch=1, heads_q=1, heads_kv=1, len_q=3, len_k=4, head_dim=D, causal=False, scale=(1, 2))
    zero = CE(np.zeros((3, D), np.int8), np.full((3, 1), E_ZERO, np.int8), 1, D)
    k, v = rand_ce(rng, 4, D, 1, D, elo=-3, ehi=-3), rand_ce(rng, 4, D, 1, D, elo=-5, ehi=-5)
    o, stats = blocks.attention_fwd(d, zero, k, v, g_cols=D)
    # equal scores: the mean of the values, every weight 2^14
    assert (stats == [0, 4 * 2 ** 14]).all()
    from fractions import Fraction

    for i in range(3):
        m, e = fit_brute([Fraction(int(v.mant[:, j].sum()), 4) * Fraction(1, 32) for j in range(D)])
        assert list(o.mant[i]) == m and o.exp[i, 0] == e
    # one visible key: its value; no visible key: zeros
    d = dict(d, len_q=6, causal=True)
    q = rand_ce(rng, 6, D, 1, D, elo=-4, ehi=-2)
    o, stats = blocks.attention_fwd(d, q, k, v, g_cols=D)
    assert (o.mant[:2] == 0).all() and (o.exp[:2] == E_ZERO).all() and (stats[:2] == 0).all()
    m, e = fit_brute([Fraction(int(x), 32) for x in v.mant[0]])
    assert list(o.mant[2]) == m and o.exp[2, 0] == e and stats[2, 1] == 2 ** 14


@pytest.mark.parametrize("N", [16, 192])
def test_layernorm_follows_the_formula(N):
    """One group per row, so that nothing is lost in aligning: h is within half of 2^-8 (and 3 2^-24 of itself),
    and FIT rounds y within half a step of at most |y|max / 64.  dX repeats this with gamma and dy exact: t is
    within one quarter and the final rounding half a step; dgamma and dbeta align dy's rows by column."""
    rng = np.random.default_rng(N)
    X = quantise(rng.standard_normal((6, N)) * 3 + 1, N)
    gamma, beta = quantise(1 + 0.2 * rng.standard_normal((1, N)), N), quantise(rng.standard_normal((1, N)) * 0.1, N)
    x, g, b = values(X), values(gamma)[0], values(beta)[0]
    mu, sd = x.mean(1, keepdims=True), np.sqrt(x.var(1, keepdims=True) + 2.0 ** -20)
    xh = (x - mu) / sd
    Y = values(blocks.layernorm_fwd(X, gamma, beta, (1, 20), N))
    ref = xh * g + b
    assert (np.abs(Y - ref) <= np.abs(ref).max(1, keepdims=True) / 128 * 1.01 + np.abs(g) * 2.0 ** -9 * 1.01).all()
    dY = quantise(rng.standard_normal((6, N)) * 1e-3, N)
    dy = values(dY)
    dX, dg, db = (values(t) for t in blocks.layernorm_bwd(X, gamma, dY, (1, 20), N))
    gd = dy * g
    ref = (gd - gd.mean(1, keepdims=True) - xh * (gd * xh).mean(1, keepdims=True)) / sd
    unit = np.exp2(blocks.exps(dY).astype(float) + blocks.exps(gamma).astype(float))  # g's unit
    # h's error of 2^-9 enters z through m2 and sum(g h): 2 |m2| 2^-9 sqrt(N) and the quarter units of t
    slack = unit * (0.5 + 2.0 ** -8 * np.abs((gd * xh).mean(1, keepdims=True) / unit) * np.abs(xh).max() +
                    2.0 ** -9 * np.abs(gd / unit).max() * np.abs(xh).max()) / sd
    assert (np.abs(dX - ref) <= np.abs(ref).max(1, keepdims=True) / 128 * 1.01 + slack).all()
    for got, want, terms in ((dg, (dy * xh).sum(0), np.abs(xh)), (db, dy.sum(0), np.ones_like(xh))):
        step = np.exp2(float(blocks.exps(dY).max()))
        tol = np.abs(want).max() / 128 * 1.01 + (0.5 * step * terms).sum(0) + np.abs(dy).sum(0) * 2.0 ** -9 * 1.01
        assert (np.abs(got[0] - want) <= tol).all()


def test_layernorm_gradient_against_differences():
    rng = np.random.default_rng(2)
    x, g, dy = rng.standard_normal((1, 12)), rng.standard_normal(12), rng.standard_normal((1, 12))
    norm = lambda x: (x - x.mean()) / np.sqrt(x.var() + 2.0 ** -20)  # noqa: E731
    gd, xh, sd = dy * g, norm(x), np.sqrt(x.var() + 2.0 ** -20)
    grad = (gd - gd.mean() - xh * (gd * xh).mean()) / sd
    for j in (0, 5, 11):
        h = 1e-5
        e = np.eye(12)[j: j + 1] * h
        assert abs(((norm(x + e) - norm(x - e)) * gd).sum() / (2 * h) - grad[0, j]) < 1e-7


def test_layernorm_constant_and_zero_rows():
    X = CE(np.array([[5] * 16, [0] * 16], np.int8), np.array([[3], [E_ZERO]], np.int8), 1, 16)
    gamma = CE(np.full((1, 16), 64, np.int8), np.array([[-6]], np.int8), 1, 16)
    beta = CE(np.arange(16, dtype=np.int8)[None] * 8, np.array([[-4]], np.int8), 1, 16)
    Y = values(blocks.layernorm_fwd(X, gamma, beta, (1, 20), 16))
    assert (Y == values(beta)).all()
    assert (values(blocks.layernorm_fwd(X, gamma, None, (0, 0), 16)) == 0).all()


# ------------------------------------------------------------------ refusals

OK, INVALID, LAYOUT, ALIGN, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def ict():
    from integer_only_nn_02_b200 import ict as _ict

    return _ict


def tensor(ict, rows, cols, g_cols=32, g_rows=1, ld=None, mant=1 << 20, exp=1 << 20):
    """A description only: the checks read no memory."""
    return ict.ict_tensor(mant, exp, rows, cols, ld or -(-cols // 16) * 16, g_rows, g_cols)


def desc(ict, **kw):
    d = dict(batch=2, heads_q=4, heads_kv=2, len_q=8, len_k=12, head_dim=64, causal=False, scale=(1, 3), q_col=0, k_col=0,
             v_col=0)
    d.update(kw)
    return d


def attn_call(ict, d, q=None, k=None, o=None, stats=1 << 20, ws=1 << 20, ws_bytes=1 << 30, back=False, dq=None):
    q = q or tensor(ict, 16, 256)
    k = k or tensor(ict, 24, 128)
    o = o or tensor(ict, 16, 256)
    c = ict.attn_desc(d)
    if back:
        dq = dq or tensor(ict, 16, 256)
        return ict.lib.ict_attention_bwd(c, q, k, k, None, None, o, o, stats, dq, k, k, ws, ws_bytes, None)
    return ict.lib.ict_attention_fwd(c, q, k, k, None, None, o, stats, ws, ws_bytes, None)


BAD_DESC = [(dict(batch=-1), INVALID), (dict(heads_q=0), INVALID), (dict(heads_q=3), INVALID), (dict(len_k=-1), INVALID),
            (dict(head_dim=0), INVALID), (dict(scale=(0, 3)), INVALID), (dict(scale=(513, 3)), INVALID),
            (dict(scale=(1, 65)), INVALID), (dict(head_dim=24), LAYOUT), (dict(head_dim=144), LAYOUT),
            (dict(len_q=65537), LAYOUT), (dict(len_k=65537), LAYOUT), (dict(batch=65535), LAYOUT)]


@pytest.mark.parametrize("kw,code", BAD_DESC)
@pytest.mark.parametrize("back", [False, True])
def test_attention_refuses_descriptions(ict, kw, code, back):
    assert attn_call(ict, desc(ict, **kw), back=back) == code
    assert ict.ict_attention_workspace(back, desc(ict, **kw)) == 0


def test_attention_refuses_tensors(ict):
    d = desc(ict)
    T = lambda *a, **k: tensor(ict, *a, **k)  # noqa: E731
    for back in (False, True):
        call = lambda back=back, **kw: attn_call(ict, kw.pop("d", d), back=back, **kw)  # noqa: E731
        assert call(q=T(15, 256)) == INVALID                     # rows
        assert call(q=T(16, 240)) == INVALID                     # too few columns
        assert call(d=desc(ict, q_col=16)) == INVALID            # heads beyond the last column
        assert call(d=desc(ict, q_col=-16)) == INVALID
        assert call(q=T(16, 512), d=desc(ict, q_col=8)) == LAYOUT
        assert call(q=T(16, 256, g_rows=2)) == LAYOUT
        assert call(q=T(16, 256, g_cols=24)) == LAYOUT
        assert call(q=T(16, 256, ld=264)) == ALIGN
        assert call(q=T(16, 256, mant=(1 << 20) + 8)) == ALIGN
        assert call(q=T(16, 256, mant=0)) == INVALID
        assert call(stats=None) == INVALID
        assert call(stats=(1 << 20) + 4) == ALIGN
        assert call(ws=None) == WORKSPACE
        assert call(ws=(1 << 20) + 128) == WORKSPACE
        assert call(ws_bytes=ict.ict_attention_workspace(back, d) - 1) == WORKSPACE
    assert attn_call(ict, d, o=T(16, 256, g_cols=128)) == LAYOUT   # a group across two heads
    assert attn_call(ict, d, o=T(16, 256, g_cols=256)) == LAYOUT
    assert attn_call(ict, d, back=True, dq=T(16, 256, g_cols=128)) == LAYOUT
    # 32-bit sums over the queries that share a key head
    d = desc(ict, batch=1, heads_q=64, heads_kv=1, len_q=2048, len_k=16)
    assert ict.ict_attention_workspace(False, d) > 0 and ict.ict_attention_workspace(True, d) == 0


def test_layernorm_and_values_refuse(ict):
    T = lambda *a, **k: tensor(ict, *a, **k)  # noqa: E731
    L = ict.lib
    x, v = T(8, 192), T(1, 192)
    fwd = lambda x=x, g=v, b=v, y=x, e=(1, 20): L.ict_layernorm_fwd(x, g, b, *e, y, None)  # noqa: E731
    assert fwd(x=T(8, 200)) == LAYOUT and fwd(x=T(8, 8208)) == LAYOUT
    assert fwd(x=T(8, 0)) == INVALID and fwd(g=T(1, 176)) == INVALID and fwd(g=T(2, 192)) == INVALID
    assert fwd(b=T(1, 208)) == INVALID and fwd(y=T(7, 192)) == INVALID and fwd(y=T(8, 192, g_rows=8)) == LAYOUT
    assert fwd(e=(-1, 20)) == INVALID and fwd(e=(513, 20)) == INVALID and fwd(e=(1, 65)) == INVALID
    assert fwd(x=T(8, 192, g_cols=24)) == LAYOUT and fwd(x=T(8, 192, ld=200)) == ALIGN
    bwd = lambda dy=x, dx=x, dg=v, db=v, ws=1 << 20, n=1 << 30: L.ict_layernorm_bwd(  # noqa: E731
        x, v, dy, 1, 20, dx, dg, db, ws, n, None)
    assert bwd(dy=T(8, 208)) == INVALID and bwd(dg=T(1, 208)) == INVALID and bwd(db=T(3, 192)) == INVALID
    assert bwd(ws=None) == WORKSPACE and bwd(n=L.ict_layernorm_bwd_workspace(x) - 1) == WORKSPACE
    assert L.ict_layernorm_bwd_workspace(None) == 0
    vals = lambda t=x, bf=1, out=1 << 20, ld=192: L.ict_values(t, bf, out, ld, None)  # noqa: E731
    assert vals(bf=2) == INVALID and vals(out=None) == INVALID and vals(ld=191) == INVALID
    assert vals(out=(1 << 20) + 1) == ALIGN and vals(bf=0, out=(1 << 20) + 2) == ALIGN


def test_gradients_that_share_memory_are_refused(ict):
    T = lambda mant, rows=16, cols=256, **k: tensor(ict, rows, cols, mant=mant << 20, **k)  # noqa: E731
    d = desc(ict, len_k=8)
    o = T(3)

    def back(dq, dk, dv, **kw):
        c = ict.attn_desc(dict(d, **kw))
        return ict.lib.ict_attention_bwd(c, T(1, cols=512), T(2, cols=512), T(2, cols=512), None, None, o, o, 1 << 20, dq, dk, dv,
                                         1 << 20, 1 << 30, None)

    w = T(7, cols=512)
    assert back(T(4), T(5, cols=128), T(5, cols=128)) == INVALID
    assert back(w, w, w) == INVALID and back(w, w, w, k_col=256, v_col=256) == INVALID
    assert back(w, w, w, k_col=224, v_col=384) == INVALID
    # a view that begins inside a row of the other tensor
    inside = tensor(ict, 16, 128, mant=(7 << 20) + 128, ld=512)
    assert back(w, inside, T(5, cols=128)) == INVALID and back(T(4), inside, w, v_col=128) == INVALID
    L, v = ict.lib, tensor(ict, 1, 192, mant=9 << 20)
    x, dy, dx, g = (T(m, 8, 192) for m in (1, 2, 3, 4))
    db = tensor(ict, 1, 192, mant=10 << 20)
    bwd = lambda dx, dg, db: L.ict_layernorm_bwd(x, v, dy, 1, 20, dx, dg, db, 1 << 20, 1 << 30, None)  # noqa: E731
    assert bwd(x, v, db) == INVALID and bwd(dy, v, db) == INVALID and bwd(dx, db, db) == INVALID


def test_other_mantissa_widths_are_refused(ict):
    ict.ict_set_mantissa_bits(6)
    try:
        assert attn_call(ict, desc(ict)) == LAYOUT and attn_call(ict, desc(ict), back=True) == LAYOUT
        x, v = tensor(ict, 8, 192), tensor(ict, 1, 192)
        assert ict.lib.ict_layernorm_fwd(x, v, v, 1, 20, x, None) == LAYOUT
    finally:
        ict.ict_set_mantissa_bits(8)
