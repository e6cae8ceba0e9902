"""Attention and layer norm on (C,e) tensors: cases, plain forms and exact values.

A (C,e) tensor holds int8 mantissas C [rows, cols] and one int8 exponent per row and group
of G columns; its values are C 2^e, and e = -128 marks a group of zeros.  Results are
returned as the values they stand for (bfloat16 holds C 2^e exactly).

attention   per sequence b and key/value head g (rep query heads share it): every operand
            is aligned to one exponent per (b, g); s = AQ AK^T exactly;
            k = RNE((s - max s) f), f = scale log2(e) 2^(eQ + eK + 6);  E = RNE(2^14 2^(k / 64));
            O = FIT(E AV / sum E), the quotient exact.  The backward pass recomputes E.
layer norm  rows aligned to one exponent; mean and variance from exact integer sums; the
            normalised value is an integer multiple of 2^-8.
FIT(group)  the smallest exponent at which every member rounds (half to even) into +-127.

``run`` computes this with elementary torch operations where ``own`` is false and with the
library's entry points where it is true.
"""
import math

import numpy as np
import torch

own = False

E_ZERO = -128
LOG2E = 12102203  # log2(e) 2^23
_DEV = "cuda" if torch.cuda.is_available() else "cpu"
SCALES = {32: (181, 10), 64: (1, 3), 80: (229, 11), 96: (209, 11), 128: (181, 11), 48: (148, 10), 16: (1, 2)}  # 1 / sqrt(D) as mul 2^-shift


# ------------------------------------------------------------------ cases

def _attn(op, B, Hq, Hkv, Lq, Lk, D, causal=False, ragged=False, packed=True, G=32):
    return {"op": op, "B": B, "Hq": Hq, "Hkv": Hkv, "Lq": Lq, "Lk": Lk, "D": D, "causal": causal, "ragged": ragged,
            "packed": packed, "G": G}


def _norm(op, rows, cols, G=32):
    return {"op": op, "rows": rows, "cols": cols, "G": G}


def listed():
    return [
        # one image through one attention layer of ViT-Ti (3 heads of 64, 14 x 14 patches + class token): latency
        dict(_attn("attn_fwd", 1, 3, 3, 197, 197, 64), name="attn fwd vit-ti 1 image"),
        # a training batch of ViT-B: 64 images, 12 heads, the 12608 tokens of the linear layers' configuration
        dict(_attn("attn_fwd", 64, 12, 12, 197, 197, 64), name="attn fwd vit-b batch 64"),
        # long causal sequences, the largest contraction
        dict(_attn("attn_fwd", 2, 12, 12, 4096, 4096, 64, causal=True), name="attn fwd causal 4096"),
        # shared key/value heads of 128, padded batch of odd lengths, 16-wide groups
        dict(_attn("attn_fwd", 4, 8, 2, 1000, 1000, 128, causal=True, ragged=True, G=16), name="attn fwd shared ragged d128"),
        # a single new token (or class-token query) per sequence over long keys: reads K and V once
        dict(_attn("attn_fwd", 16, 12, 4, 1, 16384, 64, ragged=True, packed=False), name="attn fwd one query 16k"),
        # backward of the same layers
        dict(_attn("attn_bwd", 1, 3, 3, 197, 197, 64), name="attn bwd vit-ti 1 image"),
        dict(_attn("attn_bwd", 64, 12, 12, 197, 197, 64), name="attn bwd vit-b batch 64"),
        dict(_attn("attn_bwd", 3, 8, 2, 2048, 2048, 64, causal=True, ragged=True), name="attn bwd shared causal 2048"),
        # layer norm of one ViT-Ti image's tokens (latency) and of ViT-B batches
        dict(_norm("ln_fwd", 197, 192), name="ln fwd vit-ti 1 image"),
        dict(_norm("ln_fwd", 50432, 768), name="ln fwd vit-b batch 256"),
        dict(_norm("ln_bwd", 12608, 192), name="ln bwd vit-ti batch 64"),
        dict(_norm("ln_bwd", 50432, 768, G=64), name="ln bwd vit-b batch 256"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "ln_fwd", "ln_bwd"])
    if op.startswith("ln"):
        cols = 16 * _log_int(rng, 4, 256)
        rows = _log_int(rng, 16, max(16, min(60000, 38_000_000 // cols)))
        return _norm(op, rows, cols, rng.choice([16, 32, 64, 128]))
    D = rng.choice([32, 48, 64, 64, 96, 128])
    Hkv = rng.choice([1, 2, 3, 4, 6])
    Hq = Hkv * rng.choice([1, 1, 2, 4])
    single = op == "attn_fwd" and rng.random() < 0.3
    cap = 60_000_000 if op == "attn_bwd" else 150_000_000
    if single:
        Lk = _log_int(rng, 64, 16384)
        B = _log_int(rng, 1, max(1, min(32, cap // (Hq * Lk * 8))))
        return _attn(op, B, Hq, Hkv, rng.choice([1, 1, 3]), Lk, D, rng.random() < 0.5, rng.random() < 0.5, False,
                     rng.choice([16, D]))
    L = _log_int(rng, 17, 3000)
    B = _log_int(rng, 1, max(1, min(64, cap // (Hq * L * L))))
    packed = rng.random() < 0.5
    Lk = L if packed else max(1, int(L * rng.uniform(0.3, 1.5)))
    return _attn(op, B, Hq, Hkv, L, Lk, D, rng.random() < 0.5, rng.random() < 0.5, packed, rng.choice([16, D]))


# ------------------------------------------------------------------ inputs

def _fit_groups(v, G):
    """float64 [rows, cols] -> mantissas int8, exponents int8 in (1, G) groups."""
    rows, cols = v.shape
    ng = -(-cols // G)
    pad = torch.zeros(rows, ng * G, dtype=v.dtype, device=v.device)
    pad[:, :cols] = v
    g = pad.view(rows, ng, G)
    m = g.abs().amax(-1)
    e = torch.frexp(m)[1] - 7
    e = e + (torch.ldexp(m, -e) >= 127.5).to(e.dtype)
    e = e.clamp(min=-127)
    c = torch.ldexp(g, -e[..., None]).round()
    zero = m == 0
    return (torch.where(zero[..., None], 0, c).reshape(rows, ng * G)[:, :cols].to(torch.int8).contiguous(),
            torch.where(zero, E_ZERO, e).to(torch.int8).contiguous())


def _gen(seed):
    return torch.Generator(device=_DEV).manual_seed(int(seed))


def _rand_ce(g, rows, cols, G, spread=0.5, scale=1.0):
    """Activations and gradients: normal values, rows of unequal size, some larger channels."""
    v = torch.randn(rows, cols, generator=g, device=_DEV, dtype=torch.float32)
    v *= torch.exp(spread * torch.randn(rows, 1, generator=g, device=_DEV)) * scale
    v *= torch.exp(0.3 * torch.randn(1, cols, generator=g, device=_DEV))
    return _fit_groups(v.double(), G)


def _lens(g, B, L, ragged):
    if not ragged:
        return None
    n = torch.randint(max(1, L // 3), L + 1, (B,), generator=g, device=_DEV, dtype=torch.int32)
    n[-1] = L
    return n


def _attn_state(case, seed):
    g, c = _gen(seed), case
    B, Hq, Hkv, Lq, Lk, D, G = (c[k] for k in ("B", "Hq", "Hkv", "Lq", "Lk", "D", "G"))
    st = dict(case=c)
    # projections of normalised tokens: rows of nearly equal size
    if c["packed"]:  # the output of one linear layer: Q, K and V side by side
        st["q"] = st["k"] = st["v"] = _rand_ce(g, B * Lq, (Hq + 2 * Hkv) * D, G, 0.15)
        st["cols"] = (0, Hq * D, (Hq + Hkv) * D)
    else:
        st["q"] = _rand_ce(g, B * Lq, Hq * D, G, 0.15)
        st["k"] = st["v"] = _rand_ce(g, B * Lk, 2 * Hkv * D, G, 0.15)
        st["cols"] = (0, 0, Hkv * D)
    st["lens_k"] = _lens(g, B, Lk, c["ragged"])
    st["lens_q"] = st["lens_k"] if c["packed"] else None
    if c["op"] == "attn_bwd":
        st["do"] = _rand_ce(g, B * Lq, Hq * D, G, scale=1e-3)
        o, mx, sm = _attn_plain_fwd(st)  # the forward's output, which a training step keeps
        st["o"] = _fit_groups(o, G)
        st["stats"] = torch.stack([mx, sm], -1).to(torch.int32).reshape(B * Hq * Lq, 2).contiguous()
    return st


def _norm_state(case, seed):
    g, c = _gen(seed), case
    rows, cols, G = c["rows"], c["cols"], c["G"]
    st = dict(case=c, x=_rand_ce(g, rows, cols, G, scale=2.0))
    st["gamma"] = _fit_groups(1 + 0.2 * torch.randn(1, cols, generator=g, device=_DEV, dtype=torch.float64), G)
    st["beta"] = _fit_groups(0.1 * torch.randn(1, cols, generator=g, device=_DEV, dtype=torch.float64), G)
    if c["op"] == "ln_bwd":
        st["dy"] = _rand_ce(g, rows, cols, G, scale=1e-3)
    return st


def prepare(case, seed):
    return _attn_state(case, seed) if case["op"].startswith("attn") else _norm_state(case, seed)


EPS = (1, 20)  # 2^-20


# ------------------------------------------------------------------ plain forms

def _groups(e, G, cols):
    return e.repeat_interleave(G, -1)[..., :cols]


def _fit_values(v, G):
    """The values that FIT gives v (float64, exact or within 2^-45) in groups of G columns."""
    shape = v.shape
    ng = -(-shape[-1] // G)
    if ng * G != shape[-1]:
        v = torch.nn.functional.pad(v, (0, ng * G - shape[-1]))
    g = v.reshape(*shape[:-1], ng, G)
    m = g.abs().amax(-1, keepdim=True)
    e = torch.frexp(m)[1] - 7
    e = (e + (torch.ldexp(m, -e) >= 127.5).to(e.dtype)).clamp(min=-127)
    out = torch.ldexp(torch.ldexp(g, -e).round(), e)
    return out.reshape(*shape[:-1], ng * G)[..., : shape[-1]]


def _heads(t, B, L, H, D, G, col):
    """Mantissas and exponents of one operand as [B, H, L, D] float32 and int32."""
    C, e = t
    ng = e.shape[1]
    ex = e.to(torch.int32).repeat_interleave(G, 1)[:, : C.shape[1]] if ng * G >= C.shape[1] else e
    view = lambda x: x[:, col: col + H * D].reshape(B, L, H, D).transpose(1, 2)  # noqa: E731
    return view(C).to(torch.float32), view(ex)


def _align(C, e, over):
    """RNE(C 2^(e - e*)), e* the largest exponent over the dimensions `over` (no group of zeros counts)."""
    es = torch.where(e == E_ZERO, -1000, e).amax(over, keepdim=True)
    es = torch.where(es == -1000, torch.zeros_like(es), es)
    return torch.ldexp(C, torch.where(e == E_ZERO, torch.zeros_like(e), e - es)).round(), es


def _attn_parts(st):
    """Aligned operands [B, Hkv, rep, L, D], their exponents, the visible pairs."""
    c = st["case"]
    B, Hq, Hkv, Lq, Lk, D, G = (c[k] for k in ("B", "Hq", "Hkv", "Lq", "Lk", "D", "G"))
    rep = Hq // Hkv
    dev = st["q"][0].device
    nq = st["lens_q"] if st["lens_q"] is not None else torch.full((B,), Lq, device=dev)
    nk = st["lens_k"] if st["lens_k"] is not None else torch.full((B,), Lk, device=dev)
    nq, nk = nq.to(torch.int64), nk.to(torch.int64)
    okq = (torch.arange(Lq, device=dev) < nq[:, None])[:, None, None, :, None]
    okk = (torch.arange(Lk, device=dev) < nk[:, None])[:, None, None, :, None]

    def side(t, L, H, col, ok):
        C, e = _heads(t, B, L, H, D, G, col)
        C, e = C.reshape(B, Hkv, H // Hkv, L, D), e.reshape(B, Hkv, H // Hkv, L, D)
        C, e = torch.where(ok, C, 0), torch.where(ok, e, E_ZERO)
        a, es = _align(C, e, (2, 3, 4))
        return a, es.to(torch.float64)

    q = side(st["q"], Lq, Hq, st["cols"][0], okq)
    k = side(st["k"], Lk, Hkv, st["cols"][1], okk)
    v = side(st["v"], Lk, Hkv, st["cols"][2], okk)
    vis = okq & okk.transpose(-1, -2)
    if c["causal"]:
        i, j = torch.arange(Lq, device=dev)[:, None], torch.arange(Lk, device=dev)
        vis = vis & (j <= i + (nk - nq)[:, None, None, None, None])
    return q, k, v, vis, okq, rep


def _attn_weights(q, k, vis, scale):
    s = torch.matmul(q[0], k[0].transpose(-1, -2))  # whole numbers below 2^24: exact
    s = torch.where(vis, s, torch.full_like(s, -1e9))
    mx = s.amax(-1, keepdim=True)
    f = torch.exp2(q[1] + k[1] + 6 - 23 - scale[1]) * float(np.float32(scale[0] * LOG2E))
    n = ((s - mx).double() * f).round_().clamp_(min=-1024)
    E = n.div_(64).exp2_().mul_(2 ** 14).round_()
    E = torch.where(vis, E, 0)
    return E, mx[..., 0], E.sum(-1)


def _attn_plain_fwd(st):
    c = st["case"]
    q, k, v, vis, okq, rep = _attn_parts(st)
    E, mx, S = _attn_weights(q, k, vis, SCALES[c["D"]])
    N = torch.matmul(E, v[0].double())
    O = _fit_values(N / S.clamp(min=1)[..., None] * torch.exp2(v[1]), c["G"])
    empty = S == 0
    O = torch.where(empty[..., None], 0, O)
    return (O.reshape(c["B"], c["Hq"], c["Lq"], c["D"]).transpose(1, 2).reshape(c["B"] * c["Lq"], -1),
            torch.where(empty, 0, mx), S)


def _bitlen(x):
    return torch.frexp(x)[1]  # x a whole number in float64


def _attn_plain_bwd(st):
    c = st["case"]
    B, Hq, Hkv, Lq, Lk, D, G = (c[k] for k in ("B", "Hq", "Hkv", "Lq", "Lk", "D", "G"))
    q, k, v, vis, okq, rep = _attn_parts(st)
    mul, shift = SCALES[D]
    E, _, S = _attn_weights(q, k, vis, (mul, shift))
    head = lambda t: [x.reshape(B, Hkv, rep, Lq, D) for x in _heads(t, B, Lq, Hq, D, G, 0)]  # noqa: E731
    Cd, ed = head(st["do"])
    Cd, ed = torch.where(okq, Cd, 0), torch.where(okq, ed, E_ZERO)
    ado, edo = _align(Cd, ed, (2, 3, 4))
    edo = edo.to(torch.float64)
    ao, eo = _align(*head(st["o"]), (4,))
    ev = v[1]
    delta = ((ado * ao).double().sum(-1, keepdim=True) * torch.exp2(eo.double() - ev)).round()
    delta = delta.clamp(-(2 ** 22 - 1), 2 ** 22 - 1)
    X = 127 * ado.abs().double().sum(-1, keepdim=True) + delta.abs()
    x = torch.matmul(ado, v[0].transpose(-1, -2)).double() - delta
    # gradient of Q: products of 15 bits, one exponent per row
    tau = _bitlen(X).double()
    T = (E * x * torch.exp2(-tau)).round_()
    ds = S.clamp(min=1)[..., None]
    dQ = torch.matmul(T, k[0].double()) * mul / ds * torch.exp2(tau + edo + ev + k[1] - shift)
    dQ = _fit_values(torch.where(S[..., None] > 0, dQ, 0), G)
    M = T.abs().amax(-1, keepdim=True)
    del T
    # gradients of K and V: probabilities of 15 bits, one exponent per block of 128 keys
    nb = -(-Lk // 128)
    pad = nb * 128 - Lk
    sees = torch.nn.functional.pad(vis.expand(B, Hkv, rep, Lq, Lk), (0, pad)).reshape(B, Hkv, rep, Lq, nb, 128).any(-1)
    Sb = torch.where(sees, S[..., None], float("inf"))
    pi = _bitlen(torch.where(torch.isinf(m := Sb.amin((2, 3), keepdim=True)), 1.0, m)).double() - 1  # [B, Hkv, 1, 1, nb]
    rho = (torch.exp2(pi) / ds.float().double()).float().double() * (S[..., None] > 0)
    W = torch.where(sees, (rho * (M + 1) * torch.exp2(tau)).floor() + X, 0)  # no |P x| is larger
    cj = (_bitlen(W.amax((2, 3), keepdim=True)) - 14).clamp(min=0).double()
    cols = lambda t: t.repeat_interleave(128, -1)[..., :Lk]  # noqa: E731
    P = E.mul_(cols(rho)).round_()
    keys = lambda t: cols(t).reshape(B, Hkv, 1, Lk, 1)  # noqa: E731
    dV = torch.matmul(P.transpose(-1, -2), ado.double()).sum(2, keepdim=True) * torch.exp2(edo - keys(pi))
    dS = P.mul_(x).mul_(cols(torch.exp2(-cj))).round_()
    dK = torch.matmul(dS.transpose(-1, -2), q[0].double()).sum(2, keepdim=True)
    dK = dK * mul * torch.exp2(keys(cj - pi) - shift + edo + ev + q[1])
    flat = lambda t, H, L: t.reshape(B, H, L, D).transpose(1, 2).reshape(B * L, H * D)  # noqa: E731
    dQ, dK, dV = flat(dQ, Hq, Lq), flat(_fit_values(dK, G), Hkv, Lk), flat(_fit_values(dV, G), Hkv, Lk)
    if c["packed"]:
        return [torch.cat([dQ, dK, dV], 1).to(torch.bfloat16)]
    return [dQ.to(torch.bfloat16), torch.cat([dK, dV], 1).to(torch.bfloat16)]


def _norm_rows(st):
    c = st["case"]
    N, G = c["cols"], c["G"]
    a, e = _align(st["x"][0].float(), _groups(st["x"][1].to(torch.int32), G, N), (1,))
    a, e = a.double(), e.double()
    s1, s2 = a.sum(1, keepdim=True), (a * a).sum(1, keepdim=True)
    eps = torch.floor(EPS[0] * N * N * torch.exp2(-EPS[1] - 2 * e))
    zero = (st["x"][1] == E_ZERO).all(1, keepdim=True)
    D = (N * s2 - s1 * s1 + torch.where(zero, 0, eps)).float()
    R = torch.where(D > 0, 1 / D.sqrt(), 0)
    u = N * a - s1
    return u, R, (u * (R.double() * 256)).round(), e


def _vector(t, G, N):
    return t[0].double(), _groups(t[1].to(torch.int32), G, N).double()


def _norm_plain_fwd(st):
    c = st["case"]
    N, G = c["cols"], c["G"]
    _, _, h, _ = _norm_rows(st)
    (g, eg), (b, eb) = _vector(st["gamma"], G, N), _vector(st["beta"], G, N)
    y = (g * torch.exp2(eg - 8) * h + b * torch.exp2(eb)).float()
    return [_fit_values(y.double(), G).to(torch.bfloat16)]


def _norm_plain_bwd(st):
    c = st["case"]
    N, G = c["cols"], c["G"]
    _, R, h, e = _norm_rows(st)
    ga, eg = _align(st["gamma"][0].float(), _groups(st["gamma"][1].to(torch.int32), G, N), (1,))
    Cd, ed = st["dy"][0].float(), _groups(st["dy"][1].to(torch.int32), G, N)
    dy, edr = _align(Cd, ed, (1,))
    g = (ga * dy).double()
    m1 = (4 * g.sum(1, keepdim=True) / N).round()
    m2 = ((g * h).sum(1, keepdim=True) / N).float().double()
    t = 4 * g - m1 - (h * m2 * 2.0 ** -14).round()
    v = t.float() * (R * N)
    dX = _fit_values(v.double() * torch.exp2(eg.double() + edr.double() - e - 2), G)
    dc, ec = _align(Cd, ed, (0,))
    dg = (dc.double() * h).sum(0, keepdim=True) * torch.exp2(ec.double() - 8)
    db = dc.double().sum(0, keepdim=True) * torch.exp2(ec.double())
    return [x.to(torch.bfloat16) for x in (dX, _fit_values(dg, G), _fit_values(db, G))]


# ------------------------------------------------------------------ the library's calls

def _run_own(st):
    from integer_only_nn_02_b200 import ict

    c = st["case"]
    G = c["G"]
    ce = lambda t: ict.DevCE(t[0], t[1], 1, G)  # noqa: E731
    if c["op"].startswith("ln"):
        x, gamma = ce(st["x"]), ce(st["gamma"])
        if c["op"] == "ln_fwd":
            return [ict.values(ict.layernorm_fwd(x, gamma, ce(st["beta"]), EPS, G))]
        return [ict.values(t) for t in ict.layernorm_bwd(x, gamma, ce(st["dy"]), EPS, G)]
    d = {"batch": c["B"], "heads_q": c["Hq"], "heads_kv": c["Hkv"], "len_q": c["Lq"], "len_k": c["Lk"],
         "head_dim": c["D"], "causal": c["causal"], "scale": SCALES[c["D"]],
         "q_col": st["cols"][0], "k_col": st["cols"][1], "v_col": st["cols"][2]}
    q = ce(st["q"])
    k = q if c["packed"] else ce(st["k"])
    lens = (st["lens_q"], st["lens_k"])
    if c["op"] == "attn_fwd":
        o, stats = ict.attention_fwd(d, q, k, k, G, *lens)
        return [ict.values(o), stats]
    dq, dk, _ = ict.attention_bwd(d, q, k, k, ce(st["o"]), ce(st["do"]), st["stats"], G, *lens)
    return [ict.values(dq)] if c["packed"] else [ict.values(dq), ict.values(dk)]


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "attn_fwd":
        o, mx, sm = _attn_plain_fwd(state)
        return [o.to(torch.bfloat16), torch.stack([mx, sm], -1).to(torch.int32).reshape(-1, 2)]
    return {"attn_bwd": _attn_plain_bwd, "ln_fwd": _norm_plain_fwd, "ln_bwd": _norm_plain_bwd}[op](state)


# ------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"].startswith("ln"):
        n, back = c["rows"] * c["cols"], c["op"] == "ln_bwd"
        # mantissas and exponents in (x, and dy), out as bf16 values, about 8 (16) operations a value
        return {"bytes": n * (1 + 1 / c["G"]) * (2 if back else 1) + 2 * n + 8 * c["cols"], "flops": (16 if back else 8) * n}
    B, Hq, Hkv, Lq, Lk, D = (c[k] for k in ("B", "Hq", "Hkv", "Lq", "Lk", "D"))
    pairs = Lq * Lk
    if c["causal"] and Lq <= Lk:
        pairs -= Lq * (Lq - 1) // 2
    elif c["causal"]:
        pairs = Lk * (Lk + 1) // 2
    if c["ragged"]:
        pairs = pairs // 2  # lengths between a third and all of the longest
    q, kv = B * Lq * Hq * D, 2 * B * Lk * Hkv * D
    one = 1 + 1 / c["G"]
    if c["op"] == "attn_fwd":
        return {"bytes": (q + kv) * one + 2 * q + 8 * B * Lq * Hq, "flops": 4 * B * Hq * D * pairs}
    return {"bytes": (3 * q + kv) * one + 2 * (q + kv) + 8 * B * Lq * Hq, "flops": 10 * B * Hq * D * pairs}


# ------------------------------------------------------------------ exact values

def _np_values(C, e, G):
    return C, np.repeat(e.astype(np.int64), G, 1)[:, : C.shape[1]]


def _np_align(C, e):
    live = e != E_ZERO
    top = int(e[live].max()) if live.any() else 0
    return np.rint(np.ldexp(C.astype(np.float64), np.where(live, e - top, 0))), top


def _np_fit(v, G):
    out = np.zeros(v.shape)
    for g in range(0, v.shape[1], G):
        w = v[:, g: g + G]
        m = np.abs(w).max(1)
        e = np.frexp(m)[1] - 7
        e = np.maximum(np.where(np.ldexp(m, -e) >= 127.5, e + 1, e), -127)[:, None]
        out[:, g: g + G] = np.ldexp(np.rint(np.ldexp(w, -e)), e)
    return out


def _np_bits(x):
    return int(x).bit_length()


def _exact_attn(case, seed):
    c = case
    B, Hq, Hkv, Lq, Lk, D, G = (c[k] for k in ("B", "Hq", "Hkv", "Lq", "Lk", "D", "G"))
    back = c["op"] == "attn_bwd"
    if B * Hq * Lq * Lk * (3 if back else 1) > 60_000_000 or B * Lk * Hkv * D > 20_000_000:
        return None
    st = _attn_state(case, seed)
    host = lambda t: _np_values(t[0].cpu().numpy(), t[1].cpu().numpy(), G)  # noqa: E731
    q, k = host(st["q"]), host(st["k"])
    o, do = (host(st["o"]), host(st["do"])) if back else (None, None)
    nq = [Lq] * B if st["lens_q"] is None else st["lens_q"].tolist()
    nk = [Lk] * B if st["lens_k"] is None else st["lens_k"].tolist()
    rep, (mul, shift) = Hq // Hkv, SCALES[D]
    table = np.rint(2 ** 14 * np.exp2(np.arange(1024) / -64.0))
    log2e = float(np.float32(mul * LOG2E)) / 2 ** 23
    O, stats = np.zeros((B * Lq, Hq * D)), np.zeros((B, Hq, Lq, 2), np.int64)
    dQ, dK, dV = np.zeros((B * Lq, Hq * D)), np.zeros((B * Lk, Hkv * D)), np.zeros((B * Lk, Hkv * D))

    def block(t, b, L, n, col, heads):  # the heads' valid rows one below the other
        C, e = t
        pick = lambda x: np.concatenate([x[b * L: b * L + n, col + h * D: col + (h + 1) * D] for h in heads])  # noqa: E731
        return pick(C), pick(e)

    for b in range(B):
        n, m = nq[b], nk[b]
        if n == 0 or m == 0:
            continue
        vis = np.ones((n, m), bool)
        if c["causal"]:
            vis = np.arange(m)[None, :] <= np.arange(n)[:, None] + (m - n)
        for g in range(Hkv):
            heads = range(g * rep, (g + 1) * rep)
            aq, eq = _np_align(*block(q, b, Lq, n, st["cols"][0], heads))
            ak, ek = _np_align(*block(k, b, Lk, m, st["cols"][1], [g]))
            av, ev = _np_align(*block(k, b, Lk, m, st["cols"][2], [g]))
            f = log2e * 2.0 ** (-shift + eq + ek + 6)
            Es, Ss = [], []
            for r, h in enumerate(heads):
                s = aq[r * n: (r + 1) * n] @ ak.T
                top = np.where(vis, s, -np.inf).max(1)
                seen = np.isfinite(top)
                top = np.where(seen, top, 0)
                kk = np.minimum(np.rint((top[:, None] - s) * f), 1023)
                E = np.where(vis, table[np.where(vis, kk, 0).astype(np.int64)], 0)
                S = E.sum(1)
                stats[b, h, :n, 0], stats[b, h, :n, 1] = top, S
                O[b * Lq: b * Lq + n, h * D: (h + 1) * D] = _np_fit((E @ av) / np.maximum(S, 1)[:, None] * 2.0 ** ev, G)
                Es.append(E)
                Ss.append(S)
            if not back:
                continue
            ad, ed = _np_align(*block(do, b, Lq, n, 0, heads))
            xs, Xs, Ms = [], [], []
            for r, h in enumerate(heads):
                a = ad[r * n: (r + 1) * n]
                Co, eo = block(o, b, Lq, n, 0, [h])
                delta = np.zeros(n)
                for i in range(n):
                    ao, e1 = _np_align(Co[i: i + 1], eo[i: i + 1])
                    delta[i] = np.clip(np.rint(float(a[i] @ ao[0]) * 2.0 ** (e1 - ev)), -(2 ** 22 - 1), 2 ** 22 - 1)
                X = 127 * np.abs(a).sum(1) + np.abs(delta)
                x = a @ av.T - delta[:, None]
                tau = np.array([_np_bits(v) for v in X])[:, None]
                T = np.rint(Es[r] * x * 2.0 ** -tau)
                acc = (T @ ak) * mul / np.maximum(Ss[r], 1)[:, None]
                dQ[b * Lq: b * Lq + n, h * D: (h + 1) * D] = _np_fit(acc * 2.0 ** (tau + ed + ev + ek - shift), G)
                xs.append(x)
                Xs.append(X)
                Ms.append((np.abs(T).max(1) + 1) * 2.0 ** tau[:, 0])
            E, S, x, X, M = (np.concatenate(t) for t in (Es, Ss, xs, Xs, Ms))
            see = np.concatenate([vis] * rep)
            for j in range(0, m, 128):
                rows = see[:, j: j + 128].any(1)
                if not rows.any():
                    continue
                pi = _np_bits(S[rows].min()) - 1
                rho = (2.0 ** pi / S[rows].astype(np.float32).astype(np.float64)).astype(np.float32).astype(np.float64)
                cj = max(0, _np_bits((np.floor(rho * M[rows]) + X[rows]).max()) - 14)
                P = np.rint(E[rows, j: j + 128] * rho[:, None])
                U = np.rint(P * x[rows, j: j + 128] * 2.0 ** -cj)
                at = slice(b * Lk + j, b * Lk + min(m, j + 128)), slice(g * D, (g + 1) * D)
                dV[at] = _np_fit(P.T @ ad[rows] * 2.0 ** (ed - pi), G)
                dK[at] = _np_fit(U.T @ aq[rows] * mul * 2.0 ** (cj - pi - shift + ed + ev + eq), G)
    if not back:
        return [O, stats.reshape(-1, 2)]
    return [np.concatenate([dQ, dK, dV], 1)] if c["packed"] else [dQ, np.concatenate([dK, dV], 1)]


def _exact_norm(case, seed):
    c = case
    rows, N, G = c["rows"], c["cols"], c["G"]
    back = c["op"] == "ln_bwd"
    if rows * N > 4_000_000:
        return None
    st = _norm_state(case, seed)
    host = lambda t: _np_values(t[0].cpu().numpy(), t[1].cpu().numpy(), G)  # noqa: E731
    (C, e), (Cg, eg), (Cb, eb) = host(st["x"]), host(st["gamma"]), host(st["beta"])
    f32 = np.float32
    out, H, Dy = np.zeros((rows, N)), np.zeros((rows, N)), None
    gv = np.ldexp(Cg[0].astype(np.float64), eg[0])
    bv = np.ldexp(Cb[0].astype(np.float64), eb[0])
    if back:
        Cd, ed = host(st["dy"])
        ga, top = _np_align(Cg, eg)
    for i in range(rows):
        a, e1 = _np_align(C[i: i + 1], e[i: i + 1])
        a = a[0].astype(np.int64)
        s1 = int(a.sum())
        D = N * int((a * a).sum()) - s1 * s1
        if (e[i] != E_ZERO).any():
            D += int(math.floor(EPS[0] * N * N * 2.0 ** (-EPS[1] - 2 * e1)))
        R = f32(1) / np.sqrt(f32(D)) if D else f32(0)
        h = np.rint((N * a - s1) * (float(R) * 256))
        H[i] = h
        if not back:
            out[i] = (gv * h / 256 + bv).astype(f32)
            continue
        dy, e2 = _np_align(Cd[i: i + 1], ed[i: i + 1])
        g = (ga[0] * dy[0]).astype(np.int64)
        m1 = np.rint(4 * int(g.sum()) / N)
        m2 = float(f32(int((g * h.astype(np.int64)).sum()) / N))
        t = 4 * g - m1 - np.rint(h * m2 / 16384)
        out[i] = (t.astype(f32) * (R * f32(N))).astype(np.float64) * 2.0 ** (top + e2 - e1 - 2)
    if not back:
        return [_np_fit(out, G)]
    dg, db = np.zeros((1, N)), np.zeros((1, N))
    for j in range(0, N, G):
        dy, e2 = _np_align(Cd[:, j: j + G], ed[:, j: j + G])
        dg[0, j: j + G] = (dy * H[:, j: j + G]).sum(0) * 2.0 ** (e2 - 8)
        db[0, j: j + G] = dy.sum(0) * 2.0 ** e2
    return [_np_fit(out, G), _np_fit(dg, G), _np_fit(db, G)]


def exact(case, seed):
    return _exact_attn(case, seed) if case["op"].startswith("attn") else _exact_norm(case, seed)
