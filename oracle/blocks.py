"""Oracle of layer norm and attention on (C,e) tensors (test infrastructure only).

Plain numpy on whole numbers (int64), written from the definitions in include/ict.h one
sequence and one head at a time.  Rounding is half to even throughout.  A number that the
definition rounds to 24 significant bits is a numpy float32, whose conversion, division and
square root round correctly, or a Fraction where its exponent has no bound; everything else is
an int64 with a power of two beside it.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

from integer_only_nn_02_b200.workloads import CE, E_ZERO, empty_ce

LOG2E = 12102203  # log2(e) 2^23


def rne_shift(x, s):
    """RNE(x 2^-s) of int64 x (s may be negative: an exact left shift)."""
    x = np.asarray(x, np.int64)
    if s <= 0:
        return x << -s
    if s > 62:
        return np.zeros_like(x)
    q = x >> s
    rem = x - (q << s)
    half = np.int64(1) << (s - 1)
    return q + ((rem > half) | ((rem == half) & ((q & 1) == 1)))


def bitlen(x) -> int:
    return int(x).bit_length()


def parts(x: np.float32):
    """x = m 2^k, m a whole number below 2^24."""
    m, k = np.frexp(np.float64(x))
    return int(m * 2 ** 24), int(k) - 24


def exps(t: CE):
    return np.repeat(np.repeat(t.exp.astype(np.int64), t.g_rows, 0), t.g_cols, 1)[: t.rows, : t.cols]


def align(C, e):
    """ALIGN_MAX of a block: RNE(C 2^(e - e*)) and e*, the largest exponent of a group that is not zero (else 0)."""
    C, out = np.asarray(C, np.int64), np.zeros(np.shape(C), np.int64)
    live = e != E_ZERO
    if not live.any():
        return out, None
    top = int(e[live].max())
    for v in np.unique(e[live]):
        out[e == v] = rne_shift(C[e == v], top - int(v))
    return out, top


def _mant(num: int, den: int, k: int) -> int:
    """RNE(num 2^k / den)."""
    n, d = (num << k, den) if k >= 0 else (num, den << -k)
    q, r = divmod(n, d)
    return q + (1 if 2 * r > d or (2 * r == d and q & 1) else 0)


def fit_group(nums, den, r):
    """FIT of the exact values nums / den 2^r (Python ints): mantissas and the group exponent."""
    big = max((abs(int(n)) for n in nums), default=0)
    if big == 0:
        return [0] * len(nums), E_ZERO
    e = bitlen(big) - bitlen(den) - 9  # the quotient is above 2^7 here
    while _mant(big, den, -e) > 127:
        e += 1
    if e + r < -127:
        e = -127 - r
    assert e + r <= 127
    return [_mant(int(n), den, -e) for n in nums], e + r


def store(out: CE, row, col, nums, den, r):
    """FIT of one row's values into the row-local groups of out that start at col."""
    G = out.g_cols
    for g in range(0, len(nums), G):
        m, e = fit_group([int(v) for v in nums[g: g + G]], int(den), int(r))
        out.mant[row, col + g: col + g + len(m)] = m
        out.exp[row, (col + g) // G] = e


# ------------------------------------------------------------------ layer norm

def _rn24(x: Fraction) -> Fraction:
    if x == 0:
        return x
    k = bitlen(abs(x.numerator)) - bitlen(x.denominator) - 25
    while abs(x) / Fraction(2) ** k >= 2 ** 24:
        k += 1
    return round(x / Fraction(2) ** k) * Fraction(2) ** k


def _rn24_sqrt(d: Fraction) -> Fraction:
    """rn24 of the root of a number of 24 bits and any exponent: the whole root of it times 2^60, with a half behind
    where digits follow."""
    k = bitlen(d.numerator) - bitlen(d.denominator) & ~1
    m = d / Fraction(2) ** k * 2 ** 60
    assert m.denominator == 1
    r = math.isqrt(int(m))
    return _rn24(Fraction(2 * r + (r * r != m), 2 ** 31)) * Fraction(2) ** (k // 2)


def _row_norm(C, e, eps):
    """h (at 2^-8), R and the row's exponent (E_ZERO for a row of zeros)."""
    a, top = align(C, e)
    top = E_ZERO if top is None else top
    N = len(a)
    s1, s2 = int(a.sum()), int((a * a).sum())
    D = N * s2 - s1 * s1
    k = -eps[1] - 2 * top
    add = eps[0] * N * N
    D += add << k if k >= 0 else add >> -k
    R = _rn24(1 / _rn24_sqrt(_rn24(Fraction(D)))) if D > 0 else Fraction(0)
    k = bitlen(R.denominator) - 1
    return rne_shift((N * a - s1) * R.numerator, k - 8), R, top


def _vector(t: CE, base):
    e = exps(t)[0]
    keep = (e != E_ZERO) & (e >= base - 100)
    return np.where(keep, t.mant[0].astype(np.int64), 0), np.where(keep, e, base)


def _fit_fractions(out: CE, row, vals, r):
    G = out.g_cols
    for g in range(0, len(vals), G):
        v = vals[g: g + G]
        den = max(x.denominator for x in v)
        m, e = fit_group([x.numerator * (den // x.denominator) for x in v], den, r)
        out.mant[row, g: g + len(v)] = m
        out.exp[row, g // G] = e


def layernorm_fwd(X: CE, gamma: CE, beta: CE | None, eps=(1, 20), g_cols=32) -> CE:
    out = empty_ce(X.rows, X.cols, 1, g_cols)
    ex = exps(X)
    live = [int(t.exp[t.exp != E_ZERO].max()) for t in (gamma, beta) if t is not None and (t.exp != E_ZERO).any()]
    base = max(live, default=0)
    g, eg = _vector(gamma, base)
    b, eb = _vector(beta, base) if beta is not None else (np.zeros_like(g), np.full_like(g, base))
    two = Fraction(2)
    gf = [int(v) * two ** int(k - base - 8) for v, k in zip(g, eg)]
    bf = [int(v) * two ** int(k - base) for v, k in zip(b, eb)]
    for i in range(X.rows):
        h, _, _ = _row_norm(X.mant[i], ex[i], eps)
        _fit_fractions(out, i, [_rn24(gf[j] * int(h[j]) + bf[j]) for j in range(X.cols)], base)
    return out


def layernorm_bwd(X: CE, gamma: CE, dY: CE, eps=(1, 20), g_cols=32):
    rows, N = X.rows, X.cols
    dX, dg, db = empty_ce(rows, N, 1, g_cols), empty_ce(1, N, 1, g_cols), empty_ce(1, N, 1, g_cols)
    ex, ed = exps(X), exps(dY)
    ga, top_g = align(gamma.mant[0], exps(gamma)[0])
    H = np.zeros((rows, N), np.int64)
    for i in range(rows):
        h, R, top = _row_norm(X.mant[i], ex[i], eps)
        H[i] = h
        dy, top_d = align(dY.mant[i], ed[i])
        g = ga * dy
        s3, s4 = int(g.sum()), int((g * h).sum())
        m1 = _mant(4 * s3, N, 0)
        m2, k2 = parts(np.float32(np.float64(s4) / np.float64(N)))
        t = 4 * g - m1 - rne_shift(h * m2, 14 - k2)
        RN = _rn24(R * N)
        _fit_fractions(dX, i, [_rn24(int(v) * RN) for v in t], (top_g or 0) + (top_d or 0) - top - 2)
    sums, bsum, r = np.zeros(N, object), np.zeros(N, object), np.zeros(N, np.int64)
    for j in range(0, N, dY.g_cols):
        dy, top = align(dY.mant[:, j: j + dY.g_cols], ed[:, j: j + dY.g_cols])
        sums[j: j + dY.g_cols] = (dy * H[:, j: j + dY.g_cols]).sum(0)
        bsum[j: j + dY.g_cols] = dy.sum(0)
        r[j: j + dY.g_cols] = top or 0
    two = Fraction(2)
    _fit_fractions(dg, 0, [Fraction(int(v)) * two ** int(k) for v, k in zip(sums, r)], -8)
    _fit_fractions(db, 0, [Fraction(int(v)) * two ** int(k) for v, k in zip(bsum, r)], 0)
    return dX, dg, db


# ------------------------------------------------------------------ attention

def weight_table():
    """RNE(2^14 2^(-k / 64)) for k = 0 .. 1023."""
    return np.rint(np.exp2(np.longdouble(-1) * np.arange(1024) / 64) * 2 ** 14).astype(np.int64)


class _Head:
    """One sequence and key/value head: aligned operands, weights, visible pairs."""

    def __init__(self, d, Q, K, V, b, g, n, m, dO=None):
        rep, D = d["heads_q"] // d["heads_kv"], d["head_dim"]
        self.rep, self.D, self.n, self.m = rep, D, n, m

        def operand(t, col, heads, L, count):
            e = exps(t)
            rows = slice(b * L, b * L + count)
            C = np.concatenate([t.mant[rows, col + h * D: col + (h + 1) * D] for h in heads])
            E = np.concatenate([e[rows, col + h * D: col + (h + 1) * D] for h in heads])
            a, top = align(C, E)
            return a.reshape(len(heads), count, D), top or 0

        hq = range(g * rep, (g + 1) * rep)
        self.q, self.eq = operand(Q, d.get("q_col", 0), hq, d["len_q"], n)
        self.k, self.ek = operand(K, d.get("k_col", 0), [g], d["len_k"], m)
        self.v, self.ev = operand(V, d.get("v_col", 0), [g], d["len_k"], m)
        if dO is not None:
            self.d, self.ed = operand(dO, 0, hq, d["len_q"], n)
        self.k, self.v = self.k[0], self.v[0]
        self.vis = np.ones((n, m), bool)
        if d.get("causal"):
            self.vis = np.arange(m)[None] <= np.arange(n)[:, None] + m - n
        mul, shift = d["scale"]
        fm, fk = parts(np.float32(mul * LOG2E))
        self.fm, self.fk = fm, fk - 23 - shift + self.eq + self.ek + 6
        self.mul, self.shift = mul, shift

    def weights(self, r):
        s = self.q[r] @ self.k.T
        seen = self.vis.any(1) if self.m else np.zeros(self.n, bool)
        top = np.where(self.vis, s, np.iinfo(np.int64).min).max(1, initial=np.iinfo(np.int64).min)
        top = np.where(seen, top, 0)
        k = rne_shift(np.where(self.vis, top[:, None] - s, 0) * self.fm, -self.fk) if self.fk < 10 else \
            np.where(self.vis & (s < top[:, None]), 1 << 20, 0)
        E = np.where(self.vis & (k < 1024), weight_table()[np.minimum(k, 1023)], 0)
        return E, top, E.sum(1)


def _lengths(lens, b, L):
    return L if lens is None else min(max(int(lens[b]), 0), L)


def attention_fwd(d, Q: CE, K: CE, V: CE, lens_q=None, lens_k=None, g_cols=32):
    B, Hq, Hkv, D = d["batch"], d["heads_q"], d["heads_kv"], d["head_dim"]
    out = empty_ce(B * d["len_q"], Hq * D, 1, g_cols)
    stats = np.zeros((B, Hq, d["len_q"], 2), np.int32)
    for b in range(B):
        n, m = _lengths(lens_q, b, d["len_q"]), _lengths(lens_k, b, d["len_k"])
        for g in range(Hkv):
            H = _Head(d, Q, K, V, b, g, n, m)
            for r in range(H.rep):
                h = g * H.rep + r
                E, top, S = H.weights(r)
                num = E @ H.v
                stats[b, h, :n, 0], stats[b, h, :n, 1] = top, S
                for i in range(n):
                    store(out, b * d["len_q"] + i, h * D, num[i], max(int(S[i]), 1), H.ev)
    return out, stats.reshape(-1, 2)


def attention_bwd(d, Q: CE, K: CE, V: CE, O: CE, dO: CE, lens_q=None, lens_k=None, g_cols=32):
    """(dQ, dK, dV), each of its own tensor's shape; columns of no head stay zero."""
    B, Hkv, D, Lq, Lk = d["batch"], d["heads_kv"], d["head_dim"], d["len_q"], d["len_k"]
    dQ, dK, dV = (empty_ce(t.rows, t.cols, 1, g_cols) for t in (Q, K, V))
    eo = exps(O)
    lim = (1 << 22) - 1
    for b in range(B):
        n, m = _lengths(lens_q, b, Lq), _lengths(lens_k, b, Lk)
        for g in range(Hkv):
            H = _Head(d, Q, K, V, b, g, n, m, dO)
            base = H.ed + H.ev
            per = []  # per query head: E, S, x, X, max |T| and t of every row
            for r in range(H.rep):
                h = g * H.rep + r
                E, _, S = H.weights(r)
                delta = np.zeros(n, np.int64)
                for i in range(n):
                    row, cols = b * Lq + i, slice(h * D, (h + 1) * D)
                    ao, top = align(O.mant[row, cols], eo[row, cols])
                    w = int((H.d[r, i] * ao).sum())
                    k = 0 if top is None else top - H.ev
                    w = w << k if k >= 0 else int(rne_shift(w, -k))
                    delta[i] = min(max(w, -lim), lim)
                X = 127 * np.abs(H.d[r]).sum(1) + np.abs(delta)
                x = H.d[r] @ H.v.T - delta[:, None]
                tm = np.zeros(n, np.int64)
                for i in range(n):
                    t = bitlen(X[i])
                    T = rne_shift(E[i] * x[i], t)
                    tm[i] = np.abs(T).max(initial=0)
                    store(dQ, b * Lq + i, d.get("q_col", 0) + h * D, (T @ H.k) * H.mul, max(int(S[i]), 1),
                          t + base + H.ek - H.shift)
                per.append((E, S, x, X, tm))
            for j in range(0, m, 128):
                js = slice(j, min(m, j + 128))
                rows = H.vis[:, js].any(1)
                if not rows.any():
                    continue
                # queries without a gradient add nothing and choose no exponent
                sums = [int(s) for _, S, _, X, _ in per for s in S[rows & (X > 0)]]
                if not sums:
                    continue
                p = bitlen(min(sums)) - 1
                rho = [np.float32(2.0 ** p) / np.maximum(S, 1).astype(np.float32) for _, S, _, _, _ in per]
                bound = 0
                for (E, S, x, X, tm), rr in zip(per, rho):
                    for i in np.flatnonzero(rows & (X > 0)):
                        mm, kk = parts(rr[i])
                        v = mm * (int(tm[i]) + 1)
                        k = kk + bitlen(X[i])
                        bound = max(bound, (v << k if k >= 0 else v >> -k) + int(X[i]))
                c = max(0, bitlen(bound) - 14)
                sv, sk = np.zeros((js.stop - j, D), np.int64), np.zeros((js.stop - j, D), np.int64)
                for r, ((E, S, x, X, tm), rr) in enumerate(zip(per, rho)):
                    for i in np.flatnonzero(rows & (X > 0)):
                        mm, kk = parts(rr[i])
                        P = rne_shift(E[i, js] * mm, -kk)
                        U = rne_shift(P * x[i, js], c)
                        sv += P[:, None] * H.d[r, i]
                        sk += U[:, None] * H.q[r, i]
                for t in range(js.stop - j):
                    row = b * Lk + j + t
                    store(dV, row, d.get("v_col", 0) + g * D, sv[t], 1, H.ed - p)
                    store(dK, row, d.get("k_col", 0) + g * D, sk[t] * H.mul, 1, c - p - H.shift + base + H.eq)
    return dQ, dK, dV
