"""Attention and layer norm at the edges of their ranges: persistent blocks with many items, exponents at the ends,
rows of almost nothing, tensors that hold more than the heads."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from integer_only_nn_02_b200.workloads import CE, E_ZERO
from oracle import blocks
from tests.test_gpu_blocks import Case, _operators, same, status_ok
from tests.test_oracle_pins import rand_ce

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ict():
    from integer_only_nn_02_b200 import ict as _ict

    return _ict


@pytest.mark.parametrize("D,L,causal,ragged", [(64, 129, False, False), (64, 200, True, True), (64, 320, False, True),
                                               (64, 500, True, False), (128, 129, False, True), (128, 300, True, False),
                                               (96, 512, False, False)])
def test_many_items_of_several_steps(ict, D, L, causal, ragged):
    """Up to 512 keys a block walks through many items, the next one's scores in the columns of the last one's
    weights: every item's output, call after call, is the plain form's."""
    m = _operators()
    st = m.prepare(dict(op="attn_fwd", B=30, Hq=12, Hkv=12, Lq=L, Lk=L, D=D, causal=causal, ragged=ragged, packed=True, G=32), L)
    m.own = False
    ref = m.run(st)
    m.own = True
    for _ in range(8):
        for x, y in zip(m.run(st), ref):
            assert torch.equal(x, y)
    status_ok(ict)


@pytest.mark.parametrize("D,G", [(64, 32), (64, 16), (128, 128)])
def test_backward_items_of_one_and_two_steps(ict, D, G):
    """Sequences of 1 to 128 keys: pairs of warpgroups run ahead of each other by whole items."""
    m = _operators()
    lens = torch.tensor([1, 128, 64, 65, 3, 90, 128, 20, 0, 70] * 4, dtype=torch.int32, device="cuda")
    m._lens = lambda g, B, L, ragged: lens
    st = m.prepare(dict(op="attn_bwd", B=40, Hq=12, Hkv=12, Lq=128, Lk=128, D=D, causal=False, ragged=True, packed=True, G=G), D)
    m.own = False
    ref = m.run(st)
    m.own = True
    for _ in range(8):
        for x, y in zip(m.run(st), ref):
            assert torch.equal(x, y)
    status_ok(ict)


@pytest.mark.parametrize("D,G,Lq", [(64, 64, 1500), (128, 128, 1200), (96, 96, 900)])
def test_joined_parts_with_wide_groups(ict, D, G, Lq):
    """More than 1024 queries on a key block, shared by several thread blocks, in groups as wide as a head: the last
    part's sums are written to and read from the accumulators by different warpgroups."""
    m = _operators()
    st = m.prepare(dict(op="attn_bwd", B=1, Hq=4, Hkv=2, Lq=Lq, Lk=300, D=D, causal=False, ragged=False, packed=False, G=G), D)
    m.own = False
    ref = m.run(st)
    m.own = True
    for _ in range(4):
        for x, y in zip(m.run(st), ref):
            assert torch.equal(x, y)
    status_ok(ict)


@pytest.mark.parametrize("N,g_out", [(6112, 16), (6128, 6128), (6144, 64), (6144, 48), (6016, 32), (6160, 16)])
def test_layernorm_rows_near_48_kb(ict, N, g_out):
    """Rows whose weight and bias as floats take almost the 48 KB of shared memory that a kernel has without asking."""
    rng = np.random.default_rng(N + g_out)
    X, dY = (rand_ce(rng, 3, N, 1, 16, elo=e, ehi=e + 2) for e in (-6, -16))
    gamma, beta = rand_ce(rng, 1, N, 1, 16, elo=-7, ehi=-6), rand_ce(rng, 1, N, 1, 16, elo=-9, ehi=-6)
    x, dy, g, b = (ict.DevCE.from_host(t) for t in (X, dY, gamma, beta))
    same(ict.layernorm_fwd(x, g, b, (1, 20), g_out).to_host(), blocks.layernorm_fwd(X, gamma, beta, (1, 20), g_out), "Y")
    for t, r in zip(ict.layernorm_bwd(x, g, dy, (1, 20), g_out), blocks.layernorm_bwd(X, gamma, dY, (1, 20), g_out)):
        same(t.to_host(), r)
    status_ok(ict)


THREADS = """
import sys, threading
import numpy as np, torch
from integer_only_nn_02_b200 import ict
from integer_only_nn_02_b200.workloads import CE
torch.cuda.init()
widths = [8192, 6208, 7168, 8000, 6400, 8192, 6800, 7600]
xs = []
for k, n in enumerate(widths):
    rng = np.random.default_rng(k)
    make = lambda rows: ict.DevCE.from_host(CE(rng.integers(-127, 128, (rows, n), dtype=np.int8), np.zeros((rows, n // 16), np.int8), 1, 16))
    xs.append((make(2), make(1), torch.cuda.Stream()))
torch.cuda.synchronize()
start, failed = threading.Barrier(len(widths)), []
def work(x, g, s):
    torch.cuda.set_device(0)
    start.wait()
    try:
        for _ in range(20):
            ict.layernorm_fwd(x, g, None, (1, 20), 32, stream=s)
    except Exception as e:
        failed.append(repr(e))
ts = [threading.Thread(target=work, args=t) for t in xs]
[t.start() for t in ts]; [t.join() for t in ts]
torch.cuda.synchronize()
sys.exit(f"{failed}" if failed else 0)
"""


def test_first_calls_of_several_threads(ict):
    """The first calls of a process, from eight threads at once, with rows that need different amounts of shared memory."""
    r = subprocess.run([sys.executable, "-c", THREADS], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("Lq,Lk,D,G,g_out", [(40, 150, 64, 32, 32), (3, 1100, 64, 64, 64), (1, 2000, 128, 32, 16), (140, 40, 128, 128, 128),
                                             (5, 1500, 64, 16, 64), (2, 3, 16, 16, 16)])
def test_attention_of_the_largest_values(ict, Lq, Lk, D, G, g_out):
    """Values whose exponents are 126 and 127: the outputs need at most 127, and are rounded as any others, by the
    kernels for tiles and for a few queries alike."""
    c = Case(Lk + D, 2, 2, 1, Lq, Lk, D, G=G)
    c.V = rand_ce(np.random.default_rng(D), 2 * Lk, D, 1, G, elo=126, ehi=127)
    o, stats = blocks.attention_fwd(c.d, c.Q, c.K, c.V, *c.lens, g_out)
    got = c.gpu(ict, g_out, back=False)
    same(got[0].to_host(), o, "O")
    if D == 16 or Lk == 40:
        assert (o.exp == 127).any()
    status_ok(ict)


def test_attention_of_a_tie_at_the_largest_exponent(ict):
    """The mean of 101 2^127 and 102 2^127 rounds to 102."""
    D = 16
    zero = CE(np.zeros((2, D), np.int8), np.full((2, 1), E_ZERO, np.int8), 1, D)
    V = CE(np.repeat(np.array([[101], [102]], np.int8), D, 1), np.full((2, 1), 127, np.int8), 1, D)
    V.mant[:, 1] = [-102, -101]
    q, v = ict.DevCE.from_host(zero), ict.DevCE.from_host(V)
    o, _ = ict.attention_fwd(dict(batch=1, heads_q=1, heads_kv=1, len_q=2, len_k=2, head_dim=D, scale=(1, 2)), q, q, v, D)
    m = o.to_host().mant
    assert (m[:, 0] == 102).all() and (m[:, 1] == -102).all() and (m[:, 2:] == 102).all() and (o.to_host().exp == 127).all()
    status_ok(ict)


@pytest.mark.parametrize("D,G,Lq,Lk", [(64, 32, 40, 150), (64, 64, 40, 150), (128, 32, 40, 150), (128, 128, 150, 40),
                                       (64, 16, 1100, 30)])
def test_attention_gradients_at_the_largest_exponent(ict, D, G, Lq, Lk):
    """dO times 2^s makes every gradient times 2^s, rounded alike up to an exponent of 127 and saturated, with the
    status raised, beyond it."""
    c = Case(D + G, 1, 2, 1, Lq, Lk, D, G=G)
    ref = [t.to_host() for t in c.gpu(ict, G)[2:]]
    tops = [int(t.exp[t.exp != E_ZERO].max()) for t in ref]
    base, hit = c.dO.exp.astype(int), 0
    for s in [127 - t for t in tops] + [min(127 - int(base.max()), 140 - min(tops))]:
        c.dO.exp = np.where(base == E_ZERO, base, base + s).astype(np.int8)
        for name, t, r in zip(("dQ", "dK", "dV"), [t.to_host() for t in c.gpu(ict, G)[2:]], ref):
            zero = r.exp == E_ZERO
            k = np.where(zero, 0, r.exp.astype(int) + s - 127)  # how far the exponent passes 127
            assert np.array_equal(t.exp, np.where(zero, E_ZERO, np.minimum(r.exp.astype(int) + s, 127))), (name, s)
            kk = np.repeat(k, G, 1)
            fits = kk <= 0
            assert np.array_equal(t.mant[fits], r.mant[fits]), (name, s)
            over = (np.abs(r.mant) - 0.5) * np.exp2(np.maximum(kk, 0)) >= 127.5
            over &= ~fits
            assert np.array_equal(t.mant[over], 127 * np.sign(r.mant[over])), (name, s)
            hit += int((k == 0).any())
        code, _ = ict.ict_get_device_status()
        assert (code != 0) == (max(tops) + s > 127)
    assert hit >= 3


@pytest.mark.parametrize("G,g_out", [(32, 32), (16, 48), (96, 96)])
def test_layernorm_gradients_beyond_the_largest_exponent(ict, G, g_out):
    """dX scales with weight and dY: rounded alike up to an exponent of 127, and saturated with its sign beyond."""
    rng = np.random.default_rng(G)
    X, gamma, dY = (rand_ce(rng, r, 96, 1, G, elo=e, ehi=e) for r, e in ((6, -100), (1, -20), (6, -120)))
    ref = blocks.layernorm_bwd(X, gamma, dY, (0, 0), g_out)[0]
    top = int(ref.exp[ref.exp != E_ZERO].max())
    x = ict.DevCE.from_host(X)
    for s in [127 - top + k for k in (0, 1, 2, 7, 20, 100, 127, 128, 129, 130, 160, 200)]:
        up = min(147, s)  # of the weight, the rest of dY
        if s - up > 247:
            continue
        g, dy = (ict.DevCE.from_host(CE(t.mant, (t.exp.astype(int) + k).astype(np.int8), 1, G)) for t, k in ((gamma, up), (dY, s - up)))
        got = ict.layernorm_bwd(x, g, dy, (0, 0), g_out)[0].to_host()
        k = np.where(ref.exp == E_ZERO, 0, ref.exp.astype(int) + s - 127)
        assert np.array_equal(got.exp, np.where(ref.exp == E_ZERO, E_ZERO, np.minimum(ref.exp.astype(int) + s, 127))), s
        kk = np.repeat(k, g_out, 1)
        assert np.array_equal(got.mant[kk <= 0], ref.mant[kk <= 0]), s
        over = (kk > 0) & ((np.abs(ref.mant) - 0.5) * np.exp2(np.clip(kk, 0, 60)) >= 127.5)
        assert over.any() == (s > 127 - top) and np.array_equal(got.mant[over], 127 * np.sign(ref.mant[over])), s
        code, _ = ict.ict_get_device_status()
        assert (code != 0) == (s > 127 - top)


@pytest.mark.parametrize("N,G,g_out", [(16, 16, 16), (64, 32, 32), (208, 16, 48), (768, 64, 32), (2064, 48, 16), (8192, 64, 128)])
def test_layernorm_of_small_rows(ict, N, G, g_out):
    """Rows of every exponent down to -127, where the eps term in the row's units grows from nothing to 2^290."""
    rng = np.random.default_rng(N)
    es = list(range(-127, -18)) if N < 1000 else [-127, -126, -90, -60, -51, -50, -41, -40, -33, -32, -31, -30, -29, -28, -27, -26, -20]
    X, dY = rand_ce(rng, len(es), N, 1, G, elo=0, ehi=0, zero_groups=0.1), rand_ce(rng, len(es), N, 1, G, elo=-17, ehi=-15)
    X.exp = np.where(X.exp == E_ZERO, E_ZERO, np.array(es)[:, None]).astype(np.int8)
    gamma = rand_ce(rng, 1, N, 1, 16, elo=-7, ehi=-6)
    x, dy, g = (ict.DevCE.from_host(t) for t in (X, dY, gamma))
    for eps in ((1, 20), (512, 0), (7, 64)):
        same(ict.layernorm_fwd(x, g, None, eps, g_out).to_host(), blocks.layernorm_fwd(X, gamma, None, eps, g_out), f"Y {eps}")
        ref = blocks.layernorm_bwd(X, gamma, dY, eps, g_out)
        for name, t, r in zip(("dX", "dgamma", "dbeta"), ict.layernorm_bwd(x, g, dy, eps, g_out), ref):
            same(t.to_host(), r, f"{name} {eps}")
    status_ok(ict)


@pytest.mark.parametrize("rows,N,G,g_out", [(1, 16, 16, 16), (9, 192, 32, 32), (5, 80, 16, 80), (3, 1600, 64, 32), (2, 8192, 64, 64)])
def test_layernorm_of_zero_rows(ict, rows, N, G, g_out):
    """Rows of zeros alone, and among others."""
    rng = np.random.default_rng(rows)
    X, dY, gamma = (rand_ce(rng, r, N, 1, G, elo=e, ehi=e + 2) for r, e in ((rows, -6), (rows, -17), (1, -7)))
    for zero in (slice(0, 1), slice(rows - 1, rows), slice(0, rows)):
        X.mant[zero], X.exp[zero] = 0, E_ZERO
        for eps in ((1, 20), (0, 0), (512, 64)):
            ref = blocks.layernorm_bwd(X, gamma, dY, eps, g_out)
            got = ict.layernorm_bwd(*(ict.DevCE.from_host(t) for t in (X, gamma, dY)), eps, g_out)
            for name, t, r in zip(("dX", "dgamma", "dbeta"), got, ref):
                same(t.to_host(), r, f"{name} {eps}")
    status_ok(ict)


@pytest.mark.parametrize("Hq,Hkv,Lq,Lk,D,G,causal", [(1, 1, 64, 3000, 32, 32, False), (4, 2, 40, 300, 64, 64, True),
                                                     (2, 1, 30, 700, 128, 32, False), (8, 1, 150, 260, 64, 16, True)])
def test_attention_backward_of_queries_without_a_gradient(ict, Hq, Hkv, Lq, Lk, D, G, causal):
    """Peaked queries whose dO is zero, among flat ones: the others' digits are their own.  And a key head of which no
    query has a gradient."""
    c = Case(Lk, 2, Hq, Hkv, Lq, Lk, D, causal, G=G, elo=-8, ehi=-8, zero=0.0)
    c.Q.mant = (c.Q.mant // 8).astype(np.int8)
    for i in (3, 17):
        for b in range(2):
            c.Q.mant[b * Lq + i] = np.sign(c.Q.mant[b * Lq + i]) * 127
            c.K.mant[b * Lk + 2, : Hkv * D] = np.tile(np.sign(c.Q.mant[b * Lq + 3, :D]) * 127, Hkv)
            c.dO.mant[b * Lq + i], c.dO.exp[b * Lq + i] = 0, E_ZERO
    c.Q.exp[:] = c.K.exp[:] = -5
    c.check(ict, G)
    if Hkv > 1:
        half = Hq // Hkv * D
        c.dO.mant[:, :half], c.dO.exp[:, : half // G] = 0, E_ZERO
        c.check(ict, G)
    c.dO.mant[:], c.dO.exp[:] = 0, E_ZERO
    c.check(ict, G)


@pytest.mark.parametrize("packed,extra,Hq,Hkv", [(True, 4, 2, 2), (False, 2, 2, 2), (False, 0, 4, 2), (True, 0, 2, 1)])
def test_columns_of_no_head_are_zero(ict, monkeypatch, packed, extra, Hq, Hkv):
    """A gradient as wide as its operand is whole: what belongs to no head is zero, ready for the next product."""
    near = ict.DevCE.near

    def dirty(*a):
        t = near(*a)
        t.mant.fill_(77)
        t.exp.fill_(55)
        return t

    c = Case(9, 2, Hq, Hkv, 33, 33, 32, True, packed=packed, G=16, extra=extra)
    if not extra:
        c.K = c.V = c.Q  # the heads of K and V are some of Q's columns
        c.d.update(q_col=0, k_col=0, v_col=0)
    o, _ = blocks.attention_fwd(c.d, c.Q, c.K, c.V, g_cols=16)
    ref = blocks.attention_bwd(c.d, c.Q, c.K, c.V, o, c.dO, g_cols=16)
    monkeypatch.setattr(ict.DevCE, "near", staticmethod(dirty))
    got = c.gpu(ict, 16)[2:]
    for k, t in enumerate(got):
        want = ref[k]
        if packed and extra:  # one tensor; 4 groups each of Q, K and V behind the further columns
            at = extra + 4
            want = CE(sum(r.mant for r in ref), np.concatenate([ref[0].exp[:, :at], ref[1].exp[:, at: at + 4], ref[2].exp[:, at + 4:]], 1),
                      1, 16)
        same(t.to_host(), want, "dQ dK dV".split()[k])
    status_ok(ict)


CAPTURED = """
import torch
from integer_only_nn_02_b200 import ict
torch.manual_seed(0)

def rnd(rows, cols, e=-6):
    return ict.DevCE(torch.randint(-127, 128, (rows, cols), device="cuda", dtype=torch.int8),
                     torch.full((rows, cols // 32), e, device="cuda", dtype=torch.int8), 1, 32)

x, g, dy, q, do = rnd(50, 192), rnd(1, 192), rnd(50, 192, -16), rnd(260, 192), rnd(260, 64, -16)
d = dict(batch=2, heads_q=1, heads_kv=1, len_q=130, len_k=130, head_dim=64, scale=(1, 3), q_col=0, k_col=64, v_col=128)

def step():
    o, st = ict.attention_fwd(d, q, q, q, 32)
    r = ict.attention_bwd(d, q, q, q, o, do, st, 32)
    y = ict.layernorm_fwd(x, g)
    z = ict.layernorm_bwd(x, g, dy)
    return [st, ict.values(y)] + [t for c in (o, r[0], y, *z) for t in (c.mant, c.exp)]

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step()))
"""


def test_first_calls_are_captured(ict):
    """A process whose first calls of all are captured into a graph."""
    r = subprocess.run([sys.executable, "-c", CAPTURED], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("D,scale,causal", [(64, (1, 3), False), (64, (1, 3), True), (128, (181, 11), True)])
def test_longest_sequences(ict, D, scale, causal):
    """65536 queries over 65536 keys, of which the last 64 have a gradient: what a call with those 64 alone gives
    (every exponent the same, so that their alignment is)."""
    gen = torch.Generator(device="cuda").manual_seed(D)
    L, n = 65536, 64

    def rnd(top, e):
        return ict.DevCE(torch.randint(-top, top + 1, (L, D), generator=gen, device="cuda", dtype=torch.int8),
                         torch.full((L, D // 32), e, device="cuda", dtype=torch.int8), 1, 32)

    last = lambda t: ict.DevCE(t.mant[L - n:].contiguous(), t.exp[L - n:].contiguous(), 1, 32)  # noqa: E731
    q, k, v, do = rnd(20, -6), rnd(20, -6), rnd(127, -6), rnd(127, -16)
    do.mant[: L - n], do.exp[: L - n] = 0, E_ZERO
    d = dict(batch=1, heads_q=1, heads_kv=1, len_q=L, len_k=L, head_dim=D, scale=scale, causal=causal)
    o, stats = ict.attention_fwd(d, q, k, v, 32)
    dq, dk, dv = ict.attention_bwd(d, q, k, v, o, do, stats, 32)
    d["len_q"] = n
    o1, stats1 = ict.attention_fwd(d, last(q), k, v, 32)
    dq1, dk1, dv1 = ict.attention_bwd(d, last(q), k, v, o1, last(do), stats1, 32)
    assert torch.equal(stats1, stats[L - n:])
    for t, t1 in ((last(o), o1), (last(dq), dq1), (dk, dk1), (dv, dv1)):
        assert torch.equal(t.mant, t1.mant) and torch.equal(t.exp, t1.exp)
    assert not dq.mant[: L - n].any() and (dq.exp[: L - n] == E_ZERO).all() and dk1.mant.any() and dv1.mant.any()
    status_ok(ict)


def rnd(gen, rows, cols, e=-6, top=127):
    return torch.randint(-top, top + 1, (rows, cols), generator=gen, device="cuda", dtype=torch.int8), \
        torch.full((rows, cols // 32), e, device="cuda", dtype=torch.int8)


def test_offsets_beyond_32_bits(ict):
    """40 sequences of 65536 keys with 16 heads of 64 columns (2.7 GB each of K and V): the last sequence's outputs and
    gradients are those of a call with it alone, by the kernels for a few queries and for tiles."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    B, L, H, D = 40, 65536, 16, 64
    ce = lambda t, rows=None: ict.DevCE(*(x if rows is None else x[-rows:].contiguous() for x in t), 1, 32)  # noqa: E731
    k, v = rnd(gen, B * L, H * D), rnd(gen, B * L, H * D)
    for n in (1, 20):
        q, do = rnd(gen, B * n, H * D, top=20), rnd(gen, B * n, H * D, e=-16)
        d = dict(batch=B, heads_q=H, heads_kv=H, len_q=n, len_k=L, head_dim=D, scale=(1, 3))
        o, stats = ict.attention_fwd(d, ce(q), ce(k), ce(v), 32)
        d1 = dict(d, batch=1)
        o1, stats1 = ict.attention_fwd(d1, ce(q, n), ce(k, L), ce(v, L), 32)
        assert torch.equal(o.mant[-n:], o1.mant) and torch.equal(o.exp[-n:], o1.exp) and torch.equal(stats[-n * H:], stats1)
        assert o1.mant.any()
    got = ict.attention_bwd(d, ce(q), ce(k), ce(v), o, ce(do), stats, 32)
    want = ict.attention_bwd(d1, ce(q, n), ce(k, L), ce(v, L), o1, ce(do, n), stats1, 32)
    for t, t1 in zip(got, want):
        rows = t1.mant.shape[0]
        assert torch.equal(t.mant[-rows:], t1.mant) and torch.equal(t.exp[-rows:], t1.exp) and t1.mant.any()
    status_ok(ict)


def test_layernorm_offsets_beyond_32_bits(ict):
    """2.8 million rows of 768 values, of which the last 1000 have a gradient."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    rows, N, n = 2_800_000, 768, 1000
    x, dy, g = rnd(gen, rows, N), rnd(gen, rows, N, e=-16), rnd(gen, 1, N)
    dy[0][:-n], dy[1][:-n] = 0, E_ZERO
    ce = lambda t, rows=None: ict.DevCE(*(a if rows is None else a[-rows:].contiguous() for a in t), 1, 32)  # noqa: E731
    y, y1 = ict.layernorm_fwd(ce(x), ce(g), ce(g)), ict.layernorm_fwd(ce(x, n), ce(g), ce(g))
    assert torch.equal(y.mant[-n:], y1.mant) and torch.equal(y.exp[-n:], y1.exp)
    dx, dg, db = ict.layernorm_bwd(ce(x), ce(g), ce(dy))
    for t, t1 in zip((dx, dg, db), ict.layernorm_bwd(ce(x, n), ce(g), ce(dy, n))):
        r = t1.mant.shape[0]
        assert torch.equal(t.mant[-r:], t1.mant) and torch.equal(t.exp[-r:], t1.exp) and t1.mant.any()
    assert not dx.mant[:-n].any()
    for dt in (torch.float32, torch.bfloat16):
        assert torch.equal(ict.values(y, dt)[-n:], ict.values(y1, dt))
    status_ok(ict)
