// ict_attention_few.cuh -- the attention forward for a few queries over many keys (a new token, a
// class token): every key and value is read once, from the operands themselves.
//
// A tile of 128 queries would leave the tensor cores and the softmax warps almost empty, and
// aligned copies would move three times the bytes.  Here the keys are split into chunks of
// kFewKeys over the blocks:
//   few_top_kernel     the exponents e* of K and V (1 / G of the bytes)
//   few_scores_kernel  s = AQ AK^T (dp4a, K aligned on the way), the queries' maxima
//   few_values_kernel  E from the true maximum, sum E, sum E AV (dp2a on pairs of keys)
//   few_out_kernel     FIT of the quotients
// Partial sums and maxima are whole numbers joined by integer atomics, so the split changes
// nothing.  Bound by memory: one byte per element of K and V, 4 bytes per score written and read.
#pragma once

#include "ict_attention.cuh"

namespace ict {

constexpr int kFewKeys = 1024;  // keys of a chunk: sums of 2^14 * 127 * 1024 fit 32 bits
constexpr int kFewQ = 4;        // queries of one key/value head that a block takes

struct FewArgs {
    AttnArgs a;
    int R;                    // rep * Lq: queries of a key/value head
    int32_t *scores;          // [B Hkv][R][Lk]
    int32_t *top;             // [2][B Hkv]: largest exponent of K, V + 256 (0: all zero)
    int32_t *mx;              // [B Hkv][R]: largest score + 2^22 (0: none)
    int32_t *sum;             // [B Hkv][R]
    unsigned long long *acc;  // [B Hkv][R][Dp]
};

__device__ __forceinline__ int few_top(const FewArgs &p, int op, int bg) {  // exponent, 0 when all zero
    const int t = p.top[op * p.a.B * p.a.Hkv + bg];
    return t ? t - 256 : 0;
}

// Rows are split over blockIdx.y; thread = row, heads one after the other.
__global__ void __launch_bounds__(256) few_top_kernel(const __grid_constant__ FewArgs p) {
    const AttnOperand &o = p.a.op[OPK + blockIdx.z];
    const int b = blockIdx.x, n = clamp_len(o.lens, b, o.L), lane = threadIdx.x & 31;
    const int l0 = blockIdx.y * kFewKeys;
    if (l0 >= n) return;
    __shared__ int m[256];
    for (int g = threadIdx.x; g < p.a.Hkv; g += 256) m[g] = 0;
    __syncthreads();
    const int nvd = p.a.D / 16;
    for (int g = 0; g < p.a.Hkv; ++g) {
        const int v0 = o.col / 16 + g * nvd, g0 = v0 / o.gv, g1 = (v0 + nvd - 1) / o.gv;
        int t = 0;
#pragma unroll 4
        for (int l = l0 + threadIdx.x; l < min(n, l0 + kFewKeys); l += 256) {
            const int8_t *e = o.exp + ((int64_t)b * o.L + l) * o.ngc;
            for (int k = g0; k <= g1; ++k) t = max(t, e[k] == kEZero ? 0 : e[k] + 256);
        }
        t = warp_max(t);
        if (lane == 0 && t) atomicMax(&m[g], t);
    }
    __syncthreads();
    for (int g = threadIdx.x; g < p.a.Hkv; g += 256)
        if (m[g]) atomicMax(&p.top[(blockIdx.z * p.a.B + b) * p.a.Hkv + g], m[g]);
}

// The queries r0 ... of key/value head g, aligned to the head group's exponent (returned), in
// shared memory as [kFewQ][Dp].
template <int NV>
__device__ __forceinline__ int few_queries(const FewArgs &p, int b, int g, int r0, uint4 (&q)[kFewQ][NV], int *scratch) {
    const AttnArgs &a = p.a;
    const AttnOperand &o = a.op[OPQ];
    const int nvd = a.D / 16, nq = clamp_len(o.lens, b, a.Lq);
    auto expo = [&](int r, int v) {
        const int k = r / a.Lq, i = r - k * a.Lq;
        if (i >= nq || v >= nvd) return kEZero;
        return (int)o.exp[((int64_t)b * a.Lq + i) * o.ngc + (o.col / 16 + (g * a.rep + k) * nvd + v) / o.gv];
    };
    if (threadIdx.x == 0) *scratch = kNoExp;
    __syncthreads();
    for (int t = threadIdx.x; t < p.R * NV; t += blockDim.x) {
        const int e = expo(t / NV, t % NV);
        if (e != kEZero) atomicMax(scratch, e);
    }
    __syncthreads();
    const int es = *scratch;
    for (int t = threadIdx.x; t < kFewQ * NV; t += blockDim.x) {
        const int r = r0 + t / NV, v = t % NV;
        uint4 w = make_uint4(0, 0, 0, 0);
        const int e = r < p.R ? expo(r, v) : kEZero;
        if (e != kEZero) {
            const int k = r / a.Lq, i = r - k * a.Lq;
            w = *reinterpret_cast<const uint4 *>(o.mant + ((int64_t)b * a.Lq + i) * o.ld + o.col + (g * a.rep + k) * a.D + v * 16);
            w = rne_shift16(w, rne_index(es, e));
        }
        q[t / NV][v] = w;
    }
    __syncthreads();
    return es <= kNoExp ? 0 : es;
}

__device__ __forceinline__ int few_see(const AttnArgs &a, int r, int nq, int nk) {  // keys that query r sees
    const int i = r % a.Lq;
    return i >= nq ? 0 : (a.causal ? max(0, min(nk, i + nk - nq + 1)) : nk);
}

// NV lanes per key; a warp takes 32 / NV neighbouring keys of one head at a time.
template <int NV>
__global__ void __launch_bounds__(256) few_scores_kernel(const __grid_constant__ FewArgs p) {
    __shared__ uint4 q[kFewQ][NV];
    __shared__ int scratch;
    __shared__ RneK rk[9];
    const AttnArgs &a = p.a;
    const AttnOperand &o = a.op[OPK];
    const int bg = blockIdx.x, b = bg / a.Hkv, g = bg - b * a.Hkv, r0 = blockIdx.z * kFewQ;
    const int nk = clamp_len(o.lens, b, a.Lk), nq = clamp_len(a.op[OPQ].lens, b, a.Lq);
    const int j0 = blockIdx.y * kFewKeys, j1 = min(nk, j0 + kFewKeys);
    if (j0 >= nk) return;
    rne_table_init(rk);
    few_queries<NV>(p, b, g, r0, q, &scratch);
    const int lane = threadIdx.x & 31, sub = lane % NV, nvd = a.D / 16, es = few_top(p, 0, bg);
    uint4 qv[kFewQ];
    int mx[kFewQ], see[kFewQ];
#pragma unroll
    for (int r = 0; r < kFewQ; ++r) {
        qv[r] = q[r][sub];
        mx[r] = 0;
        see[r] = r0 + r < p.R ? few_see(a, r0 + r, nq, nk) : 0;
    }
    const int vec = o.col / 16 + g * nvd + sub, grp = vec / o.gv;
    constexpr int KW = 256 / NV, U = 4;  // keys of a pass of the block
    for (int j = j0 + threadIdx.x / NV; j - (int)(threadIdx.x / NV) < j1; j += U * KW) {
        uint4 w[U];
        int e[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int ju = j + u * KW;
            w[u] = make_uint4(0, 0, 0, 0);
            e[u] = kEZero;
            if (ju < j1 && sub < nvd) {
                const int64_t row = (int64_t)b * a.Lk + ju;
                w[u] = *reinterpret_cast<const uint4 *>(o.mant + row * o.ld + (int64_t)vec * 16);
                e[u] = o.exp[row * o.ngc + grp];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int ju = j + u * KW;
            w[u] = rne_shift16_k(w[u], rk[rne_index(es, e[u])]);
            int s[kFewQ];
#pragma unroll
            for (int r = 0; r < kFewQ; ++r) {
                s[r] = __dp4a((int)w[u].x, (int)qv[r].x, __dp4a((int)w[u].y, (int)qv[r].y,
                       __dp4a((int)w[u].z, (int)qv[r].z, __dp4a((int)w[u].w, (int)qv[r].w, 0))));
#pragma unroll
                for (int x = 1; x < NV; x <<= 1) s[r] += __shfl_xor_sync(0xffffffffu, s[r], x);
                if (ju < see[r]) mx[r] = max(mx[r], s[r] + (1 << 22));
            }
#pragma unroll
            for (int r = 0; r < kFewQ; ++r)
                if (sub == r % NV && ju < j1 && r0 + r < p.R) p.scores[((int64_t)bg * p.R + r0 + r) * a.Lk + ju] = s[r];
        }
    }
#pragma unroll
    for (int r = 0; r < kFewQ; ++r) {
        const int m = warp_max(mx[r]);
        if (lane == 0 && m) atomicMax(&p.mx[bg * p.R + r0 + r], m);
    }
}

__device__ __forceinline__ int dp2a_lo(int a, int b, int c) {
    int d;
    asm("dp2a.lo.s32.s32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ int dp2a_hi(int a, int b, int c) {
    int d;
    asm("dp2a.hi.s32.s32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// NV lanes per pair of keys (j, j + 1): their bytes of a column side by side, times the pair's two
// weights in one dp2a.
template <int NV>
__global__ void __launch_bounds__(128) few_values_kernel(const __grid_constant__ FewArgs p) {
    __shared__ uint32_t E[kFewQ][kFewKeys / 2];  // weights of keys 2 t and 2 t + 1
    __shared__ int out[kFewQ][NV * 16];
    __shared__ RneK rk[9];
    const AttnArgs &a = p.a;
    const AttnOperand &o = a.op[OPV];
    const int bg = blockIdx.x, b = bg / a.Hkv, g = bg - b * a.Hkv, r0 = blockIdx.z * kFewQ;
    const int nk = clamp_len(o.lens, b, a.Lk), nq = clamp_len(a.op[OPQ].lens, b, a.Lq);
    const int j0 = blockIdx.y * kFewKeys, j1 = min(nk, j0 + kFewKeys);
    if (j0 >= nk) return;
    rne_table_init(rk);
    const int lane = threadIdx.x & 31, sub = lane % NV, nvd = a.D / 16, es = few_top(p, 1, bg);
    // the query operand's exponent: the queries' groups again (a few bytes)
    __shared__ int qtop;
    if (threadIdx.x == 0) qtop = kNoExp;
    __syncthreads();
    for (int t = threadIdx.x; t < p.R * nvd; t += 128) {
        const int r = t / nvd, v = t - r * nvd, k = r / a.Lq, i = r - k * a.Lq;
        if (i < nq) {
            const AttnOperand &oq = a.op[OPQ];
            const int e = oq.exp[((int64_t)b * a.Lq + i) * oq.ngc + (oq.col / 16 + (g * a.rep + k) * nvd + v) / oq.gv];
            if (e != kEZero) atomicMax(&qtop, e);
        }
    }
    for (int t = threadIdx.x; t < kFewQ * NV * 16; t += 128) out[t / (NV * 16)][t % (NV * 16)] = 0;
    __syncthreads();
    const int x = (qtop <= kNoExp ? 0 : qtop) + few_top(p, 0, bg) - a.shift - 23;
    const f2 f = pk(a.fmul * pow2f(min(max(x, -120), 60)));
    for (int r = 0; r < kFewQ; ++r) {
        const bool on = r0 + r < p.R;
        const int see = on ? min(j1, few_see(a, r0 + r, nq, nk)) : 0;
        const int m = on ? p.mx[bg * p.R + r0 + r] - (1 << 22) : 0;
        const f2 nm = pk(-(kAttnMagic + (float)m));
        const int32_t *s = p.scores + ((int64_t)bg * p.R + r0 + r) * a.Lk;
        int sum = 0;
        for (int t = threadIdx.x; t < kFewKeys / 2; t += 128) {
            const int j = j0 + 2 * t;
            float w0, w1;
            unpk(attn_weight2f(j < see ? (uint32_t)s[j] : 0u, j + 1 < see ? (uint32_t)s[j + 1] : 0u, nm, f), w0, w1);
            const uint32_t e0 = j < see ? __float_as_uint(w0) & 0xffffu : 0u, e1 = j + 1 < see ? __float_as_uint(w1) & 0xffffu : 0u;
            E[r][t] = e0 | e1 << 16;
            sum += (int)(e0 + e1);
        }
        for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        if (lane == 0 && sum) atomicAdd(&p.sum[bg * p.R + r0 + r], sum);
    }
    __syncthreads();
    int acc[kFewQ][16];
#pragma unroll
    for (int r = 0; r < kFewQ; ++r)
#pragma unroll
        for (int d = 0; d < 16; ++d) acc[r][d] = 0;
    const int vec = o.col / 16 + g * nvd + sub, grp = vec / o.gv;
    constexpr int PW = 128 / NV;  // pairs of a pass of the block
    for (int t = threadIdx.x / NV; 2 * (t - (int)(threadIdx.x / NV)) < j1 - j0; t += 2 * PW) {
        uint4 w[4];
        int e[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {  // two pairs of keys
            const int j = j0 + 2 * (t + (u >> 1) * PW) + (u & 1);
            w[u] = make_uint4(0, 0, 0, 0);
            e[u] = kEZero;
            if (j < j1 && sub < nvd) {
                const int64_t row = (int64_t)b * a.Lk + j;
                w[u] = *reinterpret_cast<const uint4 *>(o.mant + row * o.ld + (int64_t)vec * 16);
                e[u] = o.exp[row * o.ngc + grp];
            }
        }
#pragma unroll
        for (int u = 0; u < 4; u += 2) {
            const int tt = t + (u >> 1) * PW;
            const uint4 w0 = rne_shift16_k(w[u], rk[rne_index(es, e[u])]), w1 = rne_shift16_k(w[u + 1], rk[rne_index(es, e[u + 1])]);
            const uint32_t a4[4] = {w0.x, w0.y, w0.z, w0.w}, b4[4] = {w1.x, w1.y, w1.z, w1.w};
            int ee[kFewQ];
#pragma unroll
            for (int r = 0; r < kFewQ; ++r) ee[r] = tt < kFewKeys / 2 ? (int)E[r][tt] : 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int c01 = (int)__byte_perm(a4[k], b4[k], 0x5140), c23 = (int)__byte_perm(a4[k], b4[k], 0x7362);
#pragma unroll
                for (int r = 0; r < kFewQ; ++r) {
                    acc[r][4 * k] = dp2a_lo(ee[r], c01, acc[r][4 * k]);
                    acc[r][4 * k + 1] = dp2a_hi(ee[r], c01, acc[r][4 * k + 1]);
                    acc[r][4 * k + 2] = dp2a_lo(ee[r], c23, acc[r][4 * k + 2]);
                    acc[r][4 * k + 3] = dp2a_hi(ee[r], c23, acc[r][4 * k + 3]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kFewQ; ++r) {
        if (r0 + r >= p.R) break;
#pragma unroll
        for (int d = 0; d < 16; ++d) {
            int v = acc[r][d];
#pragma unroll
            for (int k = NV; k < 32; k <<= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
            if (lane < NV) atomicAdd(&out[r][lane * 16 + d], v);
        }
    }
    __syncthreads();
    for (int t = threadIdx.x; t < kFewQ * NV * 16; t += 128) {
        const int r = t / (NV * 16), d = t % (NV * 16);
        if (r0 + r < p.R && d < a.D)
            atomicAdd(&p.acc[((int64_t)bg * p.R + r0 + r) * (NV * 16) + d], (unsigned long long)(int64_t)out[r][d]);
    }
}

// One warp per query: stats and the FIT of its quotients (lane holds columns lane, lane + 32, ...).
__global__ void __launch_bounds__(256) few_out_kernel(const __grid_constant__ FewArgs p) {
    const AttnArgs &a = p.a;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (w >= (int64_t)a.B * a.Hkv * p.R) return;
    const int bg = (int)(w / p.R), r = (int)(w - (int64_t)bg * p.R), k = r / a.Lq, i = r - k * a.Lq;
    const int b = bg / a.Hkv, h = (bg - b * a.Hkv) * a.rep + k;
    const int m = p.mx[w], S = p.sum[w];
    if (lane == 0) a.stats[((int64_t)b * a.Hq + h) * a.Lq + i] = make_int2(m ? m - (1 << 22) : 0, S);
    const double den = S ? (double)S : 1.0;
    const int base = few_top(p, 1, bg), col = a.o.col + h * a.D;
    const int64_t row = (int64_t)b * a.Lq + i;
    double q[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int d = c * 32 + lane;
        q[c] = d < a.D ? (double)(int64_t)p.acc[w * a.Dp + d] / den : 0.0;
    }
    for (int g = 0; g < a.D / a.o.G; ++g) {
        double mx = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int d = c * 32 + lane;
            if (d < a.D && d / a.o.G == g) mx = fmax(mx, fabs(q[c]));
        }
        for (int o = 16; o > 0; o >>= 1) mx = fmax(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const int e = mx > 0 ? finalize_exp(need_quot(mx) + base) : kEZero;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int d = c * 32 + lane;
            if (d < a.D && d / a.o.G == g) {
                const double v = mx > 0 ? fmin(fmax(rint(q[c] * pow2d(base - e)), -127.0), 127.0) : 0.0;
                a.o.mant[row * a.o.ld + col + d] = (int8_t)(int)v;
            }
        }
        if (lane == 0) a.o.exp[row * a.o.ngc + col / a.o.G + g] = (int8_t)e;
    }
}

}  // namespace ict
