// ict_attention.cu -- attention on (C,e) tensors, forward and backward (include/ict.h).
#include <string.h>

#include <algorithm>
#include <cmath>

#include "ict_attention.cuh"
#include "ict_attention_fwd.cuh"
#include "ict_host.h"

namespace ict {
namespace {

// ------------------------------------------------------------------ aligned operands

constexpr int kTopRows = 64;

// Largest group exponent of every operand's valid rows, per sequence and key/value head.
__global__ void __launch_bounds__(256) attn_top_kernel(const __grid_constant__ AttnArgs a) {
    __shared__ int m[256];
    const AttnOperand &o = a.op[blockIdx.z];
    const int b = blockIdx.y, n = clamp_len(o.lens, b, o.L), l0 = blockIdx.x * kTopRows;
    if (l0 >= n) return;
    const int rows = min(kTopRows, n - l0), vecs = o.heads * (a.D / 16), per = vecs / a.Hkv;
    for (int g = threadIdx.x; g < a.Hkv; g += 256) m[g] = kNoExp;
    __syncthreads();
    for (int t = threadIdx.x; t < rows * vecs; t += 256) {
        const int l = t / vecs, v = t - l * vecs;
        const int e = o.exp[((int64_t)b * o.L + l0 + l) * o.ngc + (o.col / 16 + v) / o.gv];
        if (e != kEZero) atomicMax(&m[v / per], e);
    }
    __syncthreads();
    for (int g = threadIdx.x; g < a.Hkv; g += 256)
        if (m[g] > kNoExp) atomicMax(&a.top[(blockIdx.z * a.B + b) * a.Hkv + g], m[g]);
}

// Aligned copies [B][heads][L][Dp]: RNE(C 2^(e - e*)), zeros beyond the sequence's length
// and the head's width.
__global__ void __launch_bounds__(256) attn_copy_kernel(const __grid_constant__ AttnArgs a) {
    const AttnOperand &o = a.op[blockIdx.y];
    const int nv = a.Dp / 16;
    const int64_t n = (int64_t)a.B * o.heads * o.L * nv;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < n; t += (int64_t)gridDim.x * 256) {
        const int v = (int)(t % nv);
        const int64_t r = t / nv;
        const int l = (int)(r % o.L);
        const int bh = (int)(r / o.L), h = bh % o.heads, b = bh / o.heads;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (v < a.D / 16 && l < clamp_len(o.lens, b, o.L)) {
            const int64_t row = (int64_t)b * o.L + l;
            const int col = o.col + h * a.D + v * 16;
            const int e = o.exp[row * o.ngc + (col / 16) / o.gv];
            const int es = a.top[(blockIdx.y * a.B + b) * a.Hkv + h / (o.heads / a.Hkv)];
            w = *reinterpret_cast<const uint4 *>(o.mant + row * o.ld + col);
            w = rne_shift16(w, rne_index(es, e));
        }
        *reinterpret_cast<uint4 *>(o.copy + t * 16) = w;
    }
}

__device__ __forceinline__ int dot_row(const uint4 *x, const uint4 *y, int nv) {
    int s = 0;
    for (int v = 0; v < nv; ++v) {
        const uint4 p = x[v], q = y[v];
        s = __dp4a((int)p.x, (int)q.x, s);
        s = __dp4a((int)p.y, (int)q.y, s);
        s = __dp4a((int)p.z, (int)q.z, s);
        s = __dp4a((int)p.w, (int)q.w, s);
    }
    return s;
}
__device__ __forceinline__ const uint4 *copy_row(const AttnArgs &a, int op, int b, int h, int l) {
    const AttnOperand &o = a.op[op];
    return reinterpret_cast<const uint4 *>(o.copy + (((int64_t)b * o.heads + h) * o.L + l) * a.Dp);
}

// A row of D quotients acc / den at exponent r (lane holds columns lane, lane + 32, ...),
// FIT into groups of out.G columns.  One warp.
__device__ __forceinline__ void store_row(const AttnArgs &a, const AttnOut &out, int64_t row, int h,
                                          const int64_t (&acc)[4], double den, int r) {
    const int lane = threadIdx.x & 31;
    const int col = out.col + h * a.D;
    for (int g = 0; g < a.D / out.G; ++g) {
        double mx = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int d = k * 32 + lane;
            if (d < a.D && d / out.G == g) mx = fmax(mx, fabs((double)acc[k] / den));
        }
        for (int o = 16; o > 0; o >>= 1) mx = fmax(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const int e = mx > 0 ? finalize_exp(need_quot(mx) + r) : kEZero;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int d = k * 32 + lane;
            if (d < a.D && d / out.G == g)
                out.mant[row * out.ld + col + d] = mx > 0 ? (int8_t)quot_mant((double)acc[k] / den, e - r) : (int8_t)0;
        }
        if (lane == 0) out.exp[row * out.ngc + col / out.G + g] = (int8_t)e;
    }
}

// ------------------------------------------------------------------ backward

// delta' = clamp(RNE(sum_d dO O 2^(eO - eV))), X = 127 sum |dO| + |delta'|; one warp per row
__global__ void __launch_bounds__(256) attn_row_kernel(const __grid_constant__ AttnArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (r >= (int64_t)a.B * a.Hq * a.Lq) return;
    const int i = (int)(r % a.Lq), bh = (int)(r / a.Lq), h = bh % a.Hq, b = bh / a.Hq;
    const bool valid = i < clamp_len(a.op[OPQ].lens, b, a.Lq);
    const int64_t row = (int64_t)b * a.Lq + i;
    const int v = lane, vec = (h * a.D) / 16 + v;
    const bool on = v < a.D / 16 && valid;
    const int e = on ? a.o_exp[row * a.o_ngc + vec / a.o_gv] : kEZero;
    const int es = warp_max(e == kEZero ? kNoExp : e);
    int dot = 0, sum = 0;
    if (on) {
        const uint4 w = rne_shift16(*reinterpret_cast<const uint4 *>(a.o_mant + row * a.o_ld + vec * 16), rne_index(es, e));
        const uint4 d = copy_row(a, OPD, b, h, i)[v];
        const uint32_t o4[4] = {w.x, w.y, w.z, w.w}, d4[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            dot = __dp4a((int)o4[q], (int)d4[q], dot);
            sum = __dp4a((int)__vabs4(d4[q]), 0x01010101, sum);
        }
    }
    for (int o = 16; o > 0; o >>= 1) {
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane == 0) {
        const int k = es <= kNoExp ? 0 : es - attn_top(a, OPV, b * a.Hkv + h / a.rep);
        int delta;
        if (k >= 0) {
            const int64_t w = (int64_t)dot << min(k, 24);  // |dot| < 2^22: beyond 24 only the bound remains
            delta = (int)max((int64_t)-kDeltaMax, min((int64_t)kDeltaMax, w));
        } else {
            delta = rne_shr32(dot, -k);
        }
        a.row[r] = make_int2(delta, 127 * sum + abs(delta));
    }
}

__device__ __forceinline__ int bitlen32(int x) { return 32 - __clz(x); }

// dQ, one warp per query row
__global__ void __launch_bounds__(128) attn_dq_simple(const __grid_constant__ AttnArgs a) {
    __shared__ int sw[4][32];
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const int64_t r = (int64_t)blockIdx.x * 4 + wp;
    if (r >= (int64_t)a.B * a.Hq * a.Lq) return;
    const int i = (int)(r % a.Lq), bh = (int)(r / a.Lq), h = bh % a.Hq, b = bh / a.Hq, g = h / a.rep;
    const int nq = clamp_len(a.op[OPQ].lens, b, a.Lq), nk = clamp_len(a.op[OPK].lens, b, a.Lk);
    const int see = i >= nq ? 0 : (a.causal ? min(nk, max(0, i + nk - nq + 1)) : nk);
    const int nv = a.Dp / 16;
    const uint4 *q = copy_row(a, OPQ, b, h, i), *dd = copy_row(a, OPD, b, h, i);
    const int2 st = a.stats[r], rw = a.row[r];
    const int tau = bitlen32(rw.y);
    const float f = attn_factor(a, b * a.Hkv + g), sc = pow2f(-tau);
    int64_t acc[4] = {0, 0, 0, 0};
    int tm = 0;
    for (int j0 = 0; j0 < see; j0 += 32) {
        int T = 0;
        if (j0 + lane < see) {
            const int s = dot_row(q, copy_row(a, OPK, b, g, j0 + lane), nv);
            const float E = attn_weight((float)(s - st.x), f) - kAttnMagic;
            const int x = dot_row(dd, copy_row(a, OPV, b, g, j0 + lane), nv) - rw.x;
            T = __float_as_int(__fmaf_rn(E * sc, (float)x, kAttnMagic)) - 0x4B400000;
        }
        tm = max(tm, abs(T));
        sw[wp][lane] = T;
        __syncwarp();
        for (int j = 0; j < 32 && j0 + j < see; ++j) {
            const int8_t *v = reinterpret_cast<const int8_t *>(copy_row(a, OPK, b, g, j0 + j));
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k * 32 + lane < a.Dp) acc[k] += (int64_t)sw[wp][j] * v[k * 32 + lane];
        }
        __syncwarp();
    }
    tm = warp_max(tm);
    if (lane == 0) a.tmax[r] = tm;
    const int bg = b * a.Hkv + g;
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] *= a.mul;
    store_row(a, a.o, (int64_t)b * a.Lq + i, h, acc, st.y ? (double)st.y : 1.0,
              tau + attn_top(a, OPD, bg) + attn_top(a, OPV, bg) + attn_top(a, OPK, bg) - a.shift);
}

// rn24(2^pi / rn24(S)) of a row; 0 for a row that sees no key
__device__ __forceinline__ float attn_rho(int S, int pi) { return S > 0 ? __fdiv_rn(pow2f(pi), (float)S) : 0.0f; }
// no |P x| of the row is larger
__device__ __forceinline__ int64_t attn_bound(float rho, int tmax, int X) {
    return (int64_t)floor((double)rho * (double)(tmax + 1) * pow2d(bitlen32(X))) + X;
}

// pi and c of every block of 128 keys: the smallest sum of weights, then the largest bound,
// over the rows of all the head's queries that see the block.  One block per (b, g, J).
__global__ void __launch_bounds__(256) attn_block_kernel(const __grid_constant__ AttnArgs a) {
    __shared__ int smin;
    __shared__ unsigned long long wmax;
    const int J = blockIdx.x, bg = blockIdx.y, b = bg / a.Hkv, g = bg % a.Hkv;
    const int nq = clamp_len(a.op[OPQ].lens, b, a.Lq), nk = clamp_len(a.op[OPK].lens, b, a.Lk);
    const int j0 = J * kKeyBlock;
    const int i0 = a.causal ? max(0, j0 - (nk - nq)) : 0;
    if (threadIdx.x == 0) smin = INT_MAX, wmax = 0;
    __syncthreads();
    const int n = j0 < nk ? max(0, nq - i0) : 0, total = n * a.rep;
    auto index = [&](int t) { return ((int64_t)b * a.Hq + g * a.rep + t / n) * a.Lq + i0 + t % n; };
    int m = INT_MAX;
    for (int t = threadIdx.x; t < total; t += 256) {
        const int S = a.stats[index(t)].y;
        if (S > 0) m = min(m, S);
    }
    m = -warp_max(-m);
    if ((threadIdx.x & 31) == 0) atomicMin(&smin, m);
    __syncthreads();
    const int pi = smin == INT_MAX ? 0 : bitlen32(smin) - 1;
    int64_t w = 0;
    for (int t = threadIdx.x; t < total; t += 256) {
        const int64_t at = index(t);
        const int S = a.stats[at].y;
        if (S > 0) w = max(w, attn_bound(attn_rho(S, pi), a.tmax[at], a.row[at].y));
    }
    atomicMax(&wmax, (unsigned long long)w);
    __syncthreads();
    if (threadIdx.x == 0) a.blk[(int64_t)bg * gridDim.x + J] = make_int2(pi, max(0, 64 - __clzll((long long)wmax) - 14));
}

// dK and dV, one warp per key
__global__ void __launch_bounds__(128) attn_dkv_simple(const __grid_constant__ AttnArgs a) {
    __shared__ int sp[4][32], ss[4][32];
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const int64_t r = (int64_t)blockIdx.x * 4 + wp;
    if (r >= (int64_t)a.B * a.Hkv * a.Lk) return;
    const int j = (int)(r % a.Lk), bg = (int)(r / a.Lk), g = bg % a.Hkv, b = bg / a.Hkv;
    const int nq = clamp_len(a.op[OPQ].lens, b, a.Lq), nk = clamp_len(a.op[OPK].lens, b, a.Lk);
    const int i0 = a.causal ? max(0, j - (nk - nq)) : 0;
    const int nv = a.Dp / 16;
    const uint4 *kr = copy_row(a, OPK, b, g, j), *vr = copy_row(a, OPV, b, g, j);
    const int2 pc = a.blk[(int64_t)bg * ((a.Lk + kKeyBlock - 1) / kKeyBlock) + j / kKeyBlock];
    const float f = attn_factor(a, bg), sc = pow2f(-pc.y);
    int64_t ak[4] = {0, 0, 0, 0}, av[4] = {0, 0, 0, 0};
    for (int h = g * a.rep; h < (g + 1) * a.rep && j < nk; ++h)
        for (int t0 = i0; t0 < nq; t0 += 32) {
            const int i = t0 + lane;
            int P = 0, U = 0;
            if (i < nq) {
                const int64_t at = ((int64_t)b * a.Hq + h) * a.Lq + i;
                const int2 st = a.stats[at];
                const int s = dot_row(copy_row(a, OPQ, b, h, i), kr, nv);
                const float E = attn_weight((float)(s - st.x), f) - kAttnMagic;
                const float p = __fmaf_rn(E, attn_rho(st.y, pc.x), kAttnMagic);
                const int x = dot_row(copy_row(a, OPD, b, h, i), vr, nv) - a.row[at].x;
                P = __float_as_int(p) - 0x4B400000;
                U = __float_as_int(__fmaf_rn((p - kAttnMagic) * sc, (float)x, kAttnMagic)) - 0x4B400000;
            }
            sp[wp][lane] = P;
            ss[wp][lane] = U;
            __syncwarp();
            for (int k = 0; k < 32 && t0 + k < nq; ++k) {
                const int8_t *qd = reinterpret_cast<const int8_t *>(copy_row(a, OPQ, b, h, t0 + k));
                const int8_t *dd = reinterpret_cast<const int8_t *>(copy_row(a, OPD, b, h, t0 + k));
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (c * 32 + lane < a.Dp) {
                        av[c] += (int64_t)sp[wp][k] * dd[c * 32 + lane];
                        ak[c] += (int64_t)ss[wp][k] * qd[c * 32 + lane];
                    }
            }
            __syncwarp();
        }
    const int64_t row = (int64_t)b * a.Lk + j;
    const int ed = attn_top(a, OPD, bg), ev = attn_top(a, OPV, bg), eq = attn_top(a, OPQ, bg);
    store_row(a, a.dv, row, g, av, 1.0, ed - pc.x);
#pragma unroll
    for (int c = 0; c < 4; ++c) ak[c] *= a.mul;
    store_row(a, a.dk, row, g, ak, 1.0, pc.y - pc.x - a.shift + ed + ev + eq);
}

// ------------------------------------------------------------------ host

int vec_per_group(const ict_tensor *t) {
    return t->g_cols >= t->cols ? (int)host::cdiv(t->cols, 16) : t->g_cols / 16;
}
int groups_per_row(const ict_tensor *t) { return (int)host::cdiv(t->cols, t->g_cols); }

// an operand (or output): heads of D columns from `col` on, row-local groups of whole vectors
int check_heads(const ict_tensor *t, int64_t rows, int col, int64_t width) {
    int st;
    if ((st = host::check_tensor(t))) return st;
    if (t->rows != rows || col < 0 || col + width > t->cols) return ICT_ERR_INVALID_ARG;
    if ((col & 15) || (t->g_rows != 1 && rows > 1)) return ICT_ERR_LAYOUT;
    return host::check_vec(t);
}
int check_out(const ict_tensor *t, int64_t rows, int col, int64_t width, int D) {
    int st;
    if ((st = check_heads(t, rows, col, width))) return st;
    // groups inside one head
    const int64_t G = std::min<int64_t>(t->g_cols, t->cols);
    if (D % G || col % G) return ICT_ERR_LAYOUT;
    return ICT_OK;
}

int plan(AttnArgs &a, const ict_attn_desc *d, bool back) {
    if (!d) return ICT_ERR_INVALID_ARG;
    if (d->batch < 0 || d->heads_q < 1 || d->heads_kv < 1 || d->len_q < 0 || d->len_k < 0 || d->head_dim < 1 ||
        d->heads_q % d->heads_kv || (d->causal != 0 && d->causal != 1) || d->scale_mul < 1 || d->scale_mul > 512 ||
        d->scale_shift < 0 || d->scale_shift > 64)
        return ICT_ERR_INVALID_ARG;
    if (d->head_dim % 16 || d->head_dim > 128 || d->heads_q > 256 || (int64_t)d->batch * d->heads_kv > 65535 ||
        d->len_k > 65536 || d->len_q > 65536)
        return ICT_ERR_LAYOUT;
    // 32-bit sums over all the queries of a key/value head
    if (back && (int64_t)d->len_q * (d->heads_q / d->heads_kv) > 65536) return ICT_ERR_LAYOUT;
    memset(&a, 0, sizeof(a));
    a.B = d->batch, a.Hq = d->heads_q, a.Hkv = d->heads_kv, a.rep = a.Hq / a.Hkv, a.Lq = d->len_q, a.Lk = d->len_k;
    a.D = d->head_dim, a.Dp = a.D <= 64 ? 64 : 128, a.causal = d->causal, a.mul = d->scale_mul, a.shift = d->scale_shift;
    a.fmul = (float)((double)d->scale_mul * 12102203.0);  // log2(e) 2^23
    a.n_op = back ? 4 : 3;
    return ICT_OK;
}

struct Scratch {
    size_t top, copy[OPN], row, tmax, blk, total;
};
Scratch scratch(const AttnArgs &a, bool back) {
    Scratch s;
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t p = at;
        at += (size_t)host::round_up(std::max<int64_t>(bytes, 1), 1024);
        return p;
    };
    const int64_t q = (int64_t)a.B * a.Hq * a.Lq, k = (int64_t)a.B * a.Hkv * a.Lk;
    s.top = take((int64_t)OPN * a.B * a.Hkv * 4);
    s.copy[OPQ] = take(q * a.Dp);
    s.copy[OPK] = take(k * a.Dp);
    s.copy[OPV] = take(k * a.Dp);
    s.copy[OPD] = take(back ? q * a.Dp : 0);
    s.row = take(back ? q * 8 : 0);
    s.tmax = take(back ? q * 4 : 0);
    s.blk = take(back ? (int64_t)a.B * a.Hkv * host::cdiv(std::max(a.Lk, 1), kKeyBlock) * 8 : 0);
    s.total = at;
    return s;
}

void operand(AttnOperand &o, const ict_tensor *t, int col, int heads, int L, const int32_t *lens, int8_t *copy) {
    o.mant = t->mant, o.exp = t->exp, o.ld = t->ld, o.ngc = groups_per_row(t), o.gv = vec_per_group(t);
    o.col = col, o.heads = heads, o.L = L, o.lens = lens, o.copy = copy;
}
void output(AttnOut &o, const ict_tensor *t, int col) {
    o.mant = t->mant, o.exp = t->exp, o.ld = t->ld, o.ngc = groups_per_row(t);
    o.G = (int)std::min<int64_t>(t->g_cols, t->cols), o.col = col;
}

// Common to both directions: checks, workspace, operands.
int setup(AttnArgs &a, Scratch &w, const ict_attn_desc *d, bool back, const ict_tensor *Q, const ict_tensor *K,
          const ict_tensor *V, const int32_t *lens_q, const int32_t *lens_k, int32_t *stats, void *ws, size_t ws_bytes) {
    int st;
    if ((st = host::int8_only()) || (st = plan(a, d, back))) return st;
    const int64_t rq = (int64_t)a.B * a.Lq, rk = (int64_t)a.B * a.Lk;
    if ((st = check_heads(Q, rq, d->q_col, (int64_t)a.Hq * a.D)) || (st = check_heads(K, rk, d->k_col, (int64_t)a.Hkv * a.D)) ||
        (st = check_heads(V, rk, d->v_col, (int64_t)a.Hkv * a.D)))
        return st;
    if (rq > 0 && !stats) return ICT_ERR_INVALID_ARG;
    if ((uintptr_t)stats & 7) return ICT_ERR_ALIGNMENT;
    w = scratch(a, back);
    if (!ws || ((uintptr_t)ws & 255) || ws_bytes < w.total) return ICT_ERR_WORKSPACE;
    uint8_t *base = (uint8_t *)ws;
    a.top = (int32_t *)(base + w.top);
    operand(a.op[OPQ], Q, d->q_col, a.Hq, a.Lq, lens_q, (int8_t *)(base + w.copy[OPQ]));
    operand(a.op[OPK], K, d->k_col, a.Hkv, a.Lk, lens_k, (int8_t *)(base + w.copy[OPK]));
    operand(a.op[OPV], V, d->v_col, a.Hkv, a.Lk, lens_k, (int8_t *)(base + w.copy[OPV]));
    a.stats = (int2 *)stats;
    return ICT_OK;
}

int align_operands(const AttnArgs &a, cudaStream_t s) {
    if (cudaMemsetAsync(a.top, 0x80, (size_t)OPN * a.B * a.Hkv * 4, s) != cudaSuccess) return ICT_ERR_CUDA;
    const int L = std::max(a.Lq, a.Lk);
    attn_top_kernel<<<dim3((unsigned)host::cdiv(L, kTopRows), (unsigned)a.B, (unsigned)a.n_op), 256, 0, s>>>(a);
    const int64_t n = std::max((int64_t)a.Hq * a.Lq, (int64_t)a.Hkv * a.Lk) * a.B * (a.Dp / 16);
    attn_copy_kernel<<<dim3((unsigned)std::min<int64_t>(host::cdiv(n, 256), 148 * 16), (unsigned)a.n_op), 256, 0, s>>>(a);
    host::counted(2);
    return host::launch_status();
}

// [rows][Dp] aligned copy of an operand as boxes of 128 rows and 64 columns
int copy_map(CUtensorMap *m, const AttnArgs &a, int op) {
    const AttnOperand &o = a.op[op];
    return host::tmap_2d(m, o.copy, (uint64_t)a.Dp, (uint64_t)std::max<int64_t>((int64_t)a.B * o.heads * o.L, 1), (uint64_t)a.Dp,
                         64, 128, CU_TENSOR_MAP_SWIZZLE_64B);
}

template <int DP>
int launch_fwd(const AttnArgs &a, cudaStream_t s) {
    using L = FwdCfg<DP>;
    CUtensorMap q, k, v;
    int st;
    if ((st = copy_map(&q, a, OPQ)) || (st = copy_map(&k, a, OPK)) || (st = copy_map(&v, a, OPV))) return st;
    if (cudaFuncSetAttribute(attn_fwd_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) != cudaSuccess)
        return ICT_ERR_CUDA;
    AttnLimits lim;
    host::wait_limits(&lim.wait_ns, &lim.drain_ns);
    const int64_t blocks = host::cdiv(a.Lq, kQTile) * a.B * a.Hq;
    attn_fwd_kernel<DP><<<(unsigned)blocks, L::kThreads, L::kBytes, s>>>(q, k, v, a, lim);
    host::counted(1);
    return host::launch_status();
}

}  // namespace

namespace host {
int take_status_attention(int32_t *v) {
    int32_t w = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&w, g_status, sizeof(w)) != cudaSuccess) return ICT_ERR_CUDA;
    if (w && cudaMemcpyToSymbol(g_status, &zero, sizeof(zero)) != cudaSuccess) return ICT_ERR_CUDA;
    *v |= w;
    return ICT_OK;
}
}  // namespace host
}  // namespace ict

using namespace ict;

extern "C" {

size_t ict_attention_workspace(int32_t backward, const ict_attn_desc *d) {
    AttnArgs a;
    if (plan(a, d, backward != 0) != ICT_OK) return 0;
    return scratch(a, backward != 0).total;
}

int32_t ict_attention_fwd(const ict_attn_desc *d, const ict_tensor *Q, const ict_tensor *K, const ict_tensor *V,
                          const int32_t *lens_q, const int32_t *lens_k, ict_tensor *O, int32_t *stats, void *ws,
                          size_t ws_bytes, void *stream) {
    int st;
    AttnArgs a;
    Scratch w;
    if ((st = setup(a, w, d, false, Q, K, V, lens_q, lens_k, stats, ws, ws_bytes))) return st;
    if ((st = check_out(O, (int64_t)a.B * a.Lq, 0, (int64_t)a.Hq * a.D, a.D))) return st;
    if ((st = host::device_info(nullptr))) return st;
    output(a.o, O, 0);
    const int64_t rows = (int64_t)a.B * a.Hq * a.Lq;
    if (rows == 0) return ICT_OK;
    cudaStream_t s = (cudaStream_t)stream;
    host::Timer kt(s, ICT_KC_GEMM, 4.0 * (double)rows * a.Lk * a.D);
    if ((st = align_operands(a, s))) return st;
    return a.Dp == 64 ? launch_fwd<64>(a, s) : launch_fwd<128>(a, s);
}

int32_t ict_attention_bwd(const ict_attn_desc *d, const ict_tensor *Q, const ict_tensor *K, const ict_tensor *V,
                          const int32_t *lens_q, const int32_t *lens_k, const ict_tensor *O, const ict_tensor *dO,
                          const int32_t *stats, ict_tensor *dQ, ict_tensor *dK, ict_tensor *dV, void *ws,
                          size_t ws_bytes, void *stream) {
    int st;
    AttnArgs a;
    Scratch w;
    if ((st = setup(a, w, d, true, Q, K, V, lens_q, lens_k, const_cast<int32_t *>(stats), ws, ws_bytes))) return st;
    const int64_t rq = (int64_t)a.B * a.Lq, rk = (int64_t)a.B * a.Lk;
    const int64_t wq = (int64_t)a.Hq * a.D, wk = (int64_t)a.Hkv * a.D;
    if ((st = check_heads(O, rq, 0, wq)) || (st = check_heads(dO, rq, 0, wq)) ||
        (st = check_out(dQ, rq, d->q_col, wq, a.D)) || (st = check_out(dK, rk, d->k_col, wk, a.D)) ||
        (st = check_out(dV, rk, d->v_col, wk, a.D)))
        return st;
    if ((st = host::device_info(nullptr))) return st;
    uint8_t *base = (uint8_t *)ws;
    operand(a.op[OPD], dO, 0, a.Hq, a.Lq, lens_q, (int8_t *)(base + w.copy[OPD]));
    a.o_mant = O->mant, a.o_exp = O->exp, a.o_ld = O->ld, a.o_ngc = groups_per_row(O), a.o_gv = vec_per_group(O);
    output(a.o, dQ, d->q_col);
    output(a.dk, dK, d->k_col);
    output(a.dv, dV, d->v_col);
    a.row = (int2 *)(base + w.row);
    a.tmax = (int32_t *)(base + w.tmax);
    a.blk = (int2 *)(base + w.blk);
    if (rq == 0 && rk == 0) return ICT_OK;
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t rows = rq * a.Hq;
    host::Timer kt(s, ICT_KC_GEMM, 10.0 * (double)rows * a.Lk * a.D);
    if ((st = align_operands(a, s))) return st;
    if (rows > 0) {
        attn_row_kernel<<<(unsigned)host::cdiv(rows, 8), 256, 0, s>>>(a);
        attn_dq_simple<<<(unsigned)host::cdiv(rows, 4), 128, 0, s>>>(a);
        host::counted(2);
    }
    if (rk > 0) {
        attn_block_kernel<<<dim3((unsigned)host::cdiv(a.Lk, kKeyBlock), (unsigned)(a.B * a.Hkv)), 256, 0, s>>>(a);
        attn_dkv_simple<<<(unsigned)host::cdiv(rk * a.Hkv, 4), 128, 0, s>>>(a);
        host::counted(2);
    }
    return host::launch_status();
}

}  // extern "C"
