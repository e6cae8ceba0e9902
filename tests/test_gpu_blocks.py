"""GPU parity of layer norm and attention (forward, backward) against the oracle, bit for
bit: the whole numbers they are defined on leave no tolerance."""
import importlib.util
import os
import random

import numpy as np
import pytest
import torch

from integer_only_nn_02_b200.workloads import CE, E_ZERO
from oracle import blocks
from tests.test_oracle_pins import rand_ce

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ict():
    from integer_only_nn_02_b200 import ict as _ict

    return _ict


def same(got: CE, ref: CE, what="", cols=None):
    cols = cols or slice(0, ref.cols)
    gc = slice(cols.start // ref.g_cols, -(-cols.stop // ref.g_cols))
    bad = np.argwhere(got.exp[:, gc] != ref.exp[:, gc])
    assert bad.size == 0, f"{what}: {len(bad)} of {ref.exp[:, gc].size} exponents differ, first {bad[:5].tolist()}"
    bad = np.argwhere(got.mant[:, cols] != ref.mant[:, cols])
    assert bad.size == 0, f"{what}: {len(bad)} of {ref.mant[:, cols].size} mantissas differ, first {bad[:5].tolist()}"


def status_ok(ict):
    code, raw = ict.ict_get_device_status()
    assert code == 0, (code, raw)


SCALE = {16: (1, 2), 32: (181, 10), 48: (148, 10), 64: (1, 3), 80: (229, 11), 96: (209, 11), 112: (193, 11), 128: (181, 11)}


class Case:
    def __init__(self, seed, B, Hq, Hkv, Lq, Lk, D, causal=False, lens_q=None, lens_k=None, packed=False, G=16, extra=0,
                 elo=-6, ehi=-4, zero=0.02):
        rng = np.random.default_rng(seed)
        self.B, self.D, self.G = B, D, G
        off = 16 * extra
        if packed:
            self.Q = self.K = self.V = rand_ce(rng, B * Lq, off + (Hq + 2 * Hkv) * D, 1, G, elo=elo, ehi=ehi, zero_groups=zero)
            cols = (off, off + Hq * D, off + (Hq + Hkv) * D)
        else:
            self.Q, self.K, self.V = (rand_ce(rng, B * L, off + H * D, 1, G, elo=elo, ehi=ehi, zero_groups=zero)
                                      for L, H in ((Lq, Hq), (Lk, Hkv), (Lk, Hkv)))
            cols = (off,) * 3
        self.dO = rand_ce(rng, B * Lq, Hq * D, 1, G, elo=elo - 10, ehi=ehi - 10, zero_groups=zero)
        self.d = dict(batch=B, heads_q=Hq, heads_kv=Hkv, len_q=Lq, len_k=Lk, head_dim=D, causal=causal, scale=SCALE[D],
                      q_col=cols[0], k_col=cols[1], v_col=cols[2])
        self.lens = [None if t is None else np.asarray(t, np.int32) for t in (lens_q, lens_k)]

    def gpu(self, ict, g_out, back=True):
        up = {id(t): ict.DevCE.from_host(t) for t in (self.Q, self.K, self.V, self.dO)}
        q, k, v = up[id(self.Q)], up[id(self.K)], up[id(self.V)]
        lens = [None if t is None else torch.from_numpy(t).cuda() for t in self.lens]
        o, stats = ict.attention_fwd(self.d, q, k, v, g_out, *lens)
        if not back:
            return o, stats
        return (o, stats) + ict.attention_bwd(self.d, q, k, v, o, up[id(self.dO)], stats, g_out, *lens)

    def check(self, ict, g_out, back=True):
        o, stats = blocks.attention_fwd(self.d, self.Q, self.K, self.V, *self.lens, g_out)
        got = self.gpu(ict, g_out, back)
        assert np.array_equal(got[1].cpu().numpy(), stats), "stats"
        same(got[0].to_host(), o, "O")
        if back:
            ref = blocks.attention_bwd(self.d, self.Q, self.K, self.V, o, self.dO, *self.lens, g_out)
            for name, t, r, col, H in (("dQ", got[2], ref[0], "q_col", "heads_q"), ("dK", got[3], ref[1], "k_col", "heads_kv"),
                                       ("dV", got[4], ref[2], "v_col", "heads_kv")):
                at = self.d[col]
                same(t.to_host(), r, name, slice(at, at + self.d[H] * self.D))
        status_ok(ict)


@pytest.mark.parametrize("B,Hq,Hkv,Lq,Lk,D,causal,packed,G,g_out", [
    (1, 1, 1, 1, 1, 16, False, False, 16, 16),         # one token
    (2, 3, 3, 17, 17, 64, False, True, 32, 32),
    (1, 3, 3, 197, 197, 64, False, True, 32, 32),      # ViT-Ti
    (2, 2, 2, 128, 128, 32, True, True, 16, 32),       # exactly one tile
    (1, 2, 1, 129, 129, 64, True, True, 64, 64),       # one row beyond it
    (2, 4, 2, 60, 130, 48, True, False, 16, 48),       # keys before the first query
    (1, 4, 1, 130, 60, 80, True, False, 16, 16),       # queries that see no key
    (1, 2, 2, 100, 257, 96, False, False, 48, 32),
    (1, 2, 1, 200, 200, 128, True, True, 128, 64),
    (2, 6, 2, 31, 300, 112, False, False, 16, 16),
    (1, 1, 1, 300, 1, 64, False, False, 64, 16),       # one key
    (3, 2, 1, 1, 290, 64, True, False, 64, 64),        # a single query
    (2, 4, 1, 3, 77, 64, True, False, 32, 32),         # a few queries, shared keys
    (1, 8, 1, 40, 40, 64, True, True, 32, 32),         # eight query heads on one key head
])
def test_attention(ict, B, Hq, Hkv, Lq, Lk, D, causal, packed, G, g_out):
    Case(Lq * 7 + Lk + D, B, Hq, Hkv, Lq, Lk, D, causal, packed=packed, G=G).check(ict, g_out)


@pytest.mark.parametrize("lens_q,lens_k,causal", [
    ([40, 1, 0, 25], [40, 1, 0, 25], True),      # a sequence of no tokens, one of one
    ([40, 40, 13, 7], [0, 50, 5, 1], False),     # no key at all; fewer keys than queries
    ([40, 40, 13, 7], [0, 50, 5, 1], True),
    ([99, -3, 40, 40], [50, 50, 99, -1], True),  # lengths out of range are clamped
])
def test_attention_lengths(ict, lens_q, lens_k, causal):
    Case(5, 4, 2, 1, 40, 50, 64, causal, lens_q, lens_k, G=32).check(ict, 32)


@pytest.mark.parametrize("elo,ehi,zero", [
    (-127, -120, 0.0), (60, 70, 0.0), (-30, 30, 0.1), (-3, 3, 0.0), (-6, -4, 0.9), (-5, -5, 1.0)])
def test_attention_exponents(ict, elo, ehi, zero):
    """Tiny and huge scores, spread exponents, mostly or only zero groups.  Products of exponents beyond the int8
    range raise the status on both sides, so the gradients are checked where they stay inside."""
    Case(11, 2, 2, 1, 33, 45, 32, False, G=16, elo=elo, ehi=ehi, zero=zero).check(ict, 16, back=-40 < elo and ehi < 40)


def test_attention_strided_heads(ict):
    """Heads that start inside a wider tensor, and outputs that leave its other columns alone."""
    c = Case(3, 2, 2, 2, 33, 33, 64, True, packed=True, G=32, extra=4)
    c.check(ict, 32)
    q = ict.DevCE.from_host(c.Q)
    o, stats = ict.attention_fwd(c.d, q, q, q, 32)
    dq = ict.DevCE.empty(c.Q.rows, c.Q.cols, 1, 32)
    dq.mant.fill_(77)
    dq.exp.fill_(55)
    ws = torch.empty(ict.ict_attention_workspace(True, c.d), dtype=torch.uint8, device="cuda")
    ict.ict_attention_bwd(c.d, q, q, q, None, None, o, ict.DevCE.from_host(c.dO), stats, dq, dq, dq, ws)
    assert (dq.mant[:, :64] == 77).all() and (dq.exp[:, :2] == 55).all()


def test_attention_weights_at_every_argument(ict):
    """E = RNE(2^14 2^(k / 64)) for every k with a result above zero: a query of ones against keys whose scores
    descend one by one, on a scale that makes f exactly 1 (f = rn24(mul log2(e) 2^23) 2^x is never a power of two,
    so the scores are chosen from the k that they give)."""
    f = 64 * 12102203 / 2 ** 23  # unit scores: k = RNE(n f) skips most values, so sweep scales by shifts
    D, seen = 128, set()
    table = blocks.weight_table()
    for shift in range(0, 12):
        fs = f * 2.0 ** -shift
        n = np.arange(0, min(4000, int(1100 / fs) + 2))
        k = np.rint(n * fs).astype(int)
        keep = k < 1024
        n, k = n[keep], k[keep]
        # score -n as a dot product with 1: -n spread over D columns of at most 127
        m = np.zeros((len(n), D), np.int8)
        for c in range(D):
            m[:, c] = -np.clip(n - 127 * c, 0, 127)
        K = CE(m, np.zeros((len(n), 1), np.int8), 1, D)
        Q = CE(np.ones((1, D), np.int8), np.zeros((1, 1), np.int8), 1, D)
        # one sequence per key: the sum of its weights and the key of score 0 gives E
        rows = np.zeros((2 * len(n), D), np.int8)
        rows[1::2] = m
        K = CE(rows, np.zeros((2 * len(n), 1), np.int8), 1, D)
        rows = np.zeros((2 * len(n), D), np.int8)
        rows[::2, 0] = 127  # the operand's exponent stays 0
        V = CE(rows, np.zeros((2 * len(n), 1), np.int8), 1, D)
        Q = CE(np.ones((len(n), D), np.int8), np.zeros((len(n), 1), np.int8), 1, D)
        d = dict(batch=len(n), heads_q=1, heads_kv=1, len_q=1, len_k=2, head_dim=D, scale=(1, shift))
        # f = rn24(mul * 12102203) 2^(-23 - shift + 6): in units of 2^-6
        _, stats = ict.attention_fwd(d, ict.DevCE.from_host(Q), ict.DevCE.from_host(K), ict.DevCE.from_host(V), 128)
        E = stats[:, 1].cpu().numpy() - 2 ** 14
        assert np.array_equal(E, table[k]), shift
        seen |= set(k.tolist())
    assert seen >= set(range(0, 960)), sorted(set(range(960)) - seen)[:10]


@pytest.mark.parametrize("rows,N,G,g_out", [
    (1, 16, 16, 16), (7, 64, 32, 16), (197, 192, 32, 32), (33, 768, 64, 64), (9, 1024, 128, 32), (5, 208, 16, 48),
    (3, 2064, 48, 2064), (4, 4096, 64, 128), (2, 8192, 8192, 16), (3, 8192, 64, 8192), (65, 80, 80, 80), (40, 768, 768, 32)])
def test_layernorm(ict, rows, N, G, g_out):
    rng = np.random.default_rng(rows + N)
    X, dY = (rand_ce(rng, rows, N, 1, G, elo=e, ehi=e + 3, zero_groups=0.05) for e in (-6, -16))
    gamma, beta = rand_ce(rng, 1, N, 1, min(G, 64) if N % min(G, 64) == 0 else 16, elo=-7, ehi=-6), rand_ce(rng, 1, N, 1, 16, elo=-9, ehi=-6)
    if rows > 2:
        X.mant[1], X.exp[1] = 0, E_ZERO                # a row of zeros
        X.mant[2], X.exp[2] = 9, -4                    # a constant row
        dY.mant[0], dY.exp[0] = 0, E_ZERO
    dX_, dY_, dg_, db_ = (ict.DevCE.from_host(t) for t in (X, dY, gamma, beta))
    for b, b_, eps in ((beta, db_, (1, 20)), (None, None, (0, 0)), (beta, db_, (512, 3))):
        same(ict.layernorm_fwd(dX_, dg_, b_, eps, g_out).to_host(), blocks.layernorm_fwd(X, gamma, b, eps, g_out), "Y")
    for eps in ((1, 20), (300, 9)):
        ref = blocks.layernorm_bwd(X, gamma, dY, eps, g_out)
        for name, t, r in zip(("dX", "dgamma", "dbeta"), ict.layernorm_bwd(dX_, dg_, dY_, eps, g_out), ref):
            same(t.to_host(), r, name)
    status_ok(ict)


@pytest.mark.parametrize("xe,ge,be", [((-127, -120), (-6, -6), (-6, -6)), ((-40, 40), (-6, -6), (-6, -6)),
                                      ((100, 110), (-40, -20), (-6, -6)), ((-5, -3), (-120, -20), (-127, 90))])
def test_layernorm_exponents(ict, xe, ge, be):
    rng = np.random.default_rng(1000 + xe[0] + be[1])
    X = rand_ce(rng, 20, 96, 1, 16, elo=xe[0], ehi=xe[1], zero_groups=0.2)
    gamma, beta = rand_ce(rng, 1, 96, 1, 16, elo=ge[0], ehi=ge[1]), rand_ce(rng, 1, 96, 1, 16, elo=be[0], ehi=be[1])
    dX_, dg_, db_ = (ict.DevCE.from_host(t) for t in (X, gamma, beta))
    for eps in ((0, 0), (1, 20), (512, 0), (512, 64)):
        same(ict.layernorm_fwd(dX_, dg_, db_, eps, 32).to_host(), blocks.layernorm_fwd(X, gamma, beta, eps, 32), f"Y {eps}")
    status_ok(ict)


def test_layernorm_strided_rows(ict):
    rng = np.random.default_rng(8)
    X, gamma = rand_ce(rng, 50, 96, 1, 32, elo=-6, ehi=-4), rand_ce(rng, 1, 96, 1, 32, elo=-7, ehi=-6)
    wide = torch.full((50, 160), 99, dtype=torch.int8, device="cuda")
    wide[:, :96] = torch.from_numpy(X.mant).cuda()
    x = ict.DevCE(wide, torch.from_numpy(X.exp).cuda(), 1, 32, cols=96)
    out = torch.full((50, 112), 99, dtype=torch.int8, device="cuda")
    y = ict.DevCE(out, torch.empty((50, 3), dtype=torch.int8, device="cuda"), 1, 32, cols=96)
    ict.ict_layernorm_fwd(x, ict.DevCE.from_host(gamma), None, (1, 20), y)
    same(y.to_host(), blocks.layernorm_fwd(X, gamma, None, (1, 20), 32))
    assert (out[:, 96:] == 99).all()


@pytest.mark.parametrize("rows,cols,g_rows,g_cols", [(1, 1, 1, 1), (5, 37, 1, 10), (64, 96, 1, 32), (30, 48, 7, 16), (8, 16, 8, 16)])
def test_values(ict, rows, cols, g_rows, g_cols):
    rng = np.random.default_rng(cols)
    t = rand_ce(rng, rows, cols, g_rows, g_cols, elo=-127, ehi=110, zero_groups=0.2)
    want = np.where(blocks.exps(t) == E_ZERO, 0.0, np.ldexp(t.mant.astype(np.float64), blocks.exps(t)))
    for dt in (torch.float32, torch.bfloat16):
        got = ict.values(ict.DevCE.from_host(t), dt)
        assert torch.equal(got.cpu().double(), torch.from_numpy(want).to(dt).double())


def _operators():
    spec = importlib.util.spec_from_file_location("perf_operators", os.path.join(ROOT, "perf", "operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _compare(m, case, seed):
    if case["op"].startswith("ln"):
        # torch's division by a number and its square root are not correctly rounded everywhere, as layer norm's
        # statistics are defined to be; numpy's are
        case = dict(case, rows=min(case["rows"], 4_000_000 // case["cols"]))
    st = m.prepare(case, seed)
    m.own = False
    ref = m.exact(case, seed) if case["op"].startswith("ln") else m.run(st)
    ref = [t if isinstance(t, torch.Tensor) else torch.from_numpy(t).to("cuda", torch.bfloat16) for t in ref]
    m.own = True
    got = m.run(st)
    for k, (x, y) in enumerate(zip(got, ref)):
        assert x.shape == y.shape and torch.equal(x, y), (case, k, (x != y).float().mean().item())


@pytest.mark.parametrize("k", range(24))
def test_long_and_odd_sizes(ict, k):
    """Sizes beyond the oracle's reach against the plain torch form in 64 bits, which has the same whole numbers."""
    m = _operators()
    _compare(m, m.draw(random.Random(1000 + k)), 7 + k)
    status_ok(ict)


@pytest.mark.parametrize("case", [
    dict(op="attn_fwd", B=1, Hq=2, Hkv=1, Lq=1, Lk=65536, D=64, causal=False, ragged=False, packed=False, G=32),
    dict(op="attn_fwd", B=1, Hq=1, Hkv=1, Lq=20000, Lk=700, D=128, causal=False, ragged=False, packed=False, G=128),
    dict(op="attn_bwd", B=1, Hq=2, Hkv=1, Lq=8000, Lk=300, D=64, causal=True, ragged=False, packed=False, G=32),
    dict(op="ln_bwd", rows=62000, cols=64, G=64),
    dict(op="ln_bwd", rows=5000, cols=784, G=16),
])
def test_extreme_lengths(ict, case):
    _compare(_operators(), case, 3)
    status_ok(ict)


@pytest.mark.parametrize("lens_q,lens_k,causal,D", [
    ([140, 3, 0, 129], [150, 150, 150, 0], False, 64), ([140, 70, 1, 129], [150, 20, 129, 64], True, 64),
    ([140, 3, 0, 129], [150, 150, 150, 0], True, 128), ([140, 70, 1, 129], [150, 20, 129, 64], False, 112)])
def test_few_key_blocks(ict, lens_q, lens_k, causal, D):
    """Key blocks whose queries (eight heads of up to two tiles each) are shared by several thread blocks."""
    Case(D + causal, 4, 8, 1, 140, 150, D, causal, lens_q, lens_k, G=16).check(ict, 16)
    status_ok(ict)


@pytest.mark.parametrize("case", [
    dict(op="attn_bwd", B=2, Hq=6, Hkv=2, Lq=700, Lk=520, D=128, causal=True, ragged=True, packed=False, G=64),
    dict(op="attn_bwd", B=1, Hq=1, Hkv=1, Lq=3000, Lk=3000, D=64, causal=True, ragged=False, packed=True, G=32),
    dict(op="attn_bwd", B=1, Hq=4, Hkv=4, Lq=2500, Lk=130, D=80, causal=False, ragged=False, packed=False, G=80),
])
def test_few_long_key_blocks(ict, case):
    _compare(_operators(), case, 4)
    status_ok(ict)


def test_few_long_key_blocks_replayed(ict):
    """Two captured graphs of shared key blocks, replayed in turn with an eager call between: the counters and sums
    that the parts meet in are cleared by every call."""
    m = _operators()
    st = [m.prepare(dict(op="attn_bwd", B=1, Hq=4, Hkv=2, Lq=600, Lk=L, D=64, causal=True, ragged=False, packed=False, G=32), 5)
          for L in (600, 300)]
    m.own = True
    want = [[t.clone() for t in m.run(k)] for k in st]
    outs = [{}, {}]
    graphs = [ict.StepGraph(lambda k=k: outs[k].update(r=m.run(st[k]))) for k in (0, 1)]
    for _ in range(3):
        for k in (0, 1):
            for t in outs[k]["r"]:
                t.zero_()
            graphs[k].replay()
            eager = m.run(st[1 - k])
            torch.cuda.synchronize()
            for x, y, z in zip(outs[k]["r"], want[k], range(9)):
                assert torch.equal(x, y), (k, z)
            for x, y in zip(eager, want[1 - k]):
                assert torch.equal(x, y)
    status_ok(ict)


def test_one_tensor_for_everything(ict):
    """Q, K and V the same columns of one tensor: each has a gradient of its own."""
    c = Case(2, 2, 2, 2, 33, 33, 64, G=32)
    c.K = c.V = c.Q
    got = c.gpu(ict, 32)
    assert len({t.mant.data_ptr() for t in got[2:]}) == 3
    c.check(ict, 32)


@pytest.mark.parametrize("B,Lq,Lk", [(0, 5, 5), (2, 0, 7), (2, 7, 0), (1, 0, 0)])
def test_nothing_to_attend(ict, B, Lq, Lk):
    """No sequence, no query, no key: empty outputs, or zeros."""
    D, H = 64, 2
    make = lambda rows: ict.DevCE(torch.ones((rows, H * D), dtype=torch.int8, device="cuda"),  # noqa: E731
                                  torch.zeros((rows, H * D // 32), dtype=torch.int8, device="cuda"), 1, 32)
    d = dict(batch=B, heads_q=H, heads_kv=H, len_q=Lq, len_k=Lk, head_dim=D, causal=False, scale=SCALE[D])
    q, k = make(B * Lq), make(B * Lk)
    o, stats = ict.attention_fwd(d, q, k, k, 32)
    dq, dk, dv = ict.attention_bwd(d, q, k, k, o, make(B * Lq), stats, 32)
    torch.cuda.synchronize()
    assert not stats.any()
    for t, rows in ((o, B * Lq), (dq, B * Lq), (dk, B * Lk), (dv, B * Lk)):
        assert t.mant.shape[0] == rows and not t.mant.any() and (t.exp == E_ZERO).all()
    status_ok(ict)


def test_lengths_outside_the_range(ict):
    """Lengths are clamped to [0, len]."""
    c = Case(6, 3, 2, 2, 40, 50, 64, True, [40, 1000, -3], [-1, 50, 2000])
    a, lens = c.gpu(ict, 16), c.lens
    c.lens = [np.clip(t, 0, n).astype(np.int32) for t, n in zip(lens, (40, 50))]
    c.check(ict, 16)
    for x, y in zip(a, c.gpu(ict, 16)):
        for p, q in ((x, y),) if isinstance(x, torch.Tensor) else ((x.mant, y.mant), (x.exp, y.exp)):
            assert torch.equal(p, q)


def test_tensors_elsewhere_are_refused(ict):
    """Plain tensors that a kernel would read or write at an address of another device."""
    c = Case(1, 1, 1, 1, 8, 8, 16)
    q = ict.DevCE.from_host(c.Q)
    o, stats = ict.attention_fwd(c.d, q, q, q, 16)
    host = torch.tensor([8], dtype=torch.int32)
    for lens in ((host, None), (None, host)):
        with pytest.raises(ValueError):
            ict.attention_fwd(c.d, q, q, q, 16, *lens)
    ws = torch.empty(ict.ict_attention_workspace(False, c.d), dtype=torch.uint8)
    with pytest.raises(ValueError):
        ict.ict_attention_fwd(c.d, q, q, q, None, None, o, stats, ws)
    with pytest.raises(ValueError):
        ict.ict_attention_fwd(c.d, q, q, q, None, None, o, stats.cpu(), ws.cuda())
    with pytest.raises(ValueError):
        ict.attention_bwd(c.d, q, q, q, o, o, stats.cpu(), 16)
    with pytest.raises(ValueError):
        ict.ict_values(o, torch.empty((8, 16), dtype=torch.bfloat16))
    status_ok(ict)


def test_streams_and_graph(ict):
    """The same calls on two streams at once and as one replayed graph: a transformer layer's norm, attention and
    both backward passes, each with its own workspace."""
    m = _operators()
    st = [m.prepare(dict(op="attn_bwd", B=2, Hq=3, Hkv=3, Lq=197, Lk=197, D=64, causal=False, ragged=False, packed=True,
                         G=32), s) for s in (1, 2)]
    ln = [m.prepare(dict(op="ln_bwd", rows=394, cols=192, G=32), s) for s in (1, 2)]
    m.own = True

    def layer(k):
        c = dict(st[k], case=dict(st[k]["case"], op="attn_fwd"))
        n = dict(ln[k], case=dict(ln[k]["case"], op="ln_fwd"))
        return m.run(n) + m.run(c) + m.run(st[k]) + m.run(ln[k])

    want = [[t.clone() for t in layer(k)] for k in (0, 1)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for _ in range(3):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                got[k] = layer(k)
    torch.cuda.synchronize()
    for k in (0, 1):
        for x, y in zip(got[k], want[k]):
            assert torch.equal(x, y)
    outs = {}
    g = ict.StepGraph(lambda: outs.update(a=layer(0), b=layer(1)))
    for _ in range(2):
        for t in outs["a"] + outs["b"]:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for k, key in ((0, "a"), (1, "b")):
            for x, y in zip(outs[key], want[k]):
                assert torch.equal(x, y)
    status_ok(ict)


def test_vit_layer_runs_together(ict):
    """One attention half of a ViT-Ti layer as a training step uses it: norm, packed QKV product, attention, output
    product, residual sum, and back, every step bit for bit against the oracle."""
    import oracle

    rng = np.random.default_rng(4)
    B, L, C, H, D, G = 2, 50, 192, 3, 64, 32
    X = rand_ce(rng, B * L, C, 1, G, elo=-6, ehi=-4)
    Wqkv, Wo = rand_ce(rng, 3 * C, C, 1, G, elo=-11, ehi=-10), rand_ce(rng, C, C, 1, G, elo=-11, ehi=-10)
    gamma, beta = rand_ce(rng, 1, C, 1, G, elo=-6, ehi=-6), rand_ce(rng, 1, C, 1, G, elo=-9, ehi=-9)
    dZ = rand_ce(rng, B * L, C, 1, G, elo=-16, ehi=-14)
    d = dict(batch=B, heads_q=H, heads_kv=H, len_q=L, len_k=L, head_dim=D, scale=(1, 3), q_col=0, k_col=C, v_col=2 * C)
    up = ict.DevCE.from_host
    x, wqkv, wo, ga, be, dz = (up(t) for t in (X, Wqkv, Wo, gamma, beta, dZ))
    n = ict.layernorm_fwd(x, ga, be, (1, 20), G)
    qkv = ict.linear_fwd(n, wqkv, G)
    o, stats = ict.attention_fwd(d, qkv, qkv, qkv, G)
    y = ict.linear_fwd(o, wo, G)
    z = ict.sum_(x, y)
    do = ict.linear_bwd_data(dz, wo, G)
    dqkv, _, _ = ict.attention_bwd(d, qkv, qkv, qkv, o, do, stats, G)
    dn = ict.linear_bwd_data(dqkv, wqkv, G)
    dx, dg, db = ict.layernorm_bwd(x, ga, dn, (1, 20), G)
    dw = ict.linear_bwd_weight(dqkv, n)
    N = blocks.layernorm_fwd(X, gamma, beta, (1, 20), G)
    same(n.to_host(), N, "norm")
    QKV = oracle.linear_fwd(N, Wqkv, 1, G)
    O, S = blocks.attention_fwd(d, QKV, QKV, QKV, g_cols=G)
    same(o.to_host(), O, "attention")
    Y = oracle.linear_fwd(O, Wo, 1, G)
    same(z.to_host(), oracle.sum_(X, Y, 1, G), "residual")
    DO = oracle.linear_bwd_data(dZ, Wo, 1, G)
    a, b, c = blocks.attention_bwd(d, QKV, QKV, QKV, O, DO, g_cols=G)
    exp = np.concatenate([a.exp[:, :6], b.exp[:, 6:12], c.exp[:, 12:]], 1)
    DQKV = CE((a.mant + b.mant + c.mant).astype(np.int8), exp, 1, G)
    same(dqkv.to_host(), DQKV, "dQKV")
    DN = oracle.linear_bwd_data(DQKV, Wqkv, 1, G)
    for name, t, r in zip(("dX", "dgamma", "dbeta"), (dx, dg, db), blocks.layernorm_bwd(X, gamma, DN, (1, 20), G)):
        same(t.to_host(), r, name)
    same(dw.to_host(), oracle.linear_bwd_weight(DQKV, N, 1, C), "dW")
    status_ok(ict)
