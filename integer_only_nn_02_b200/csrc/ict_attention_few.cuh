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
// nothing.  Needed of memory: one byte per element of K and V, 4 bytes per score written and read
// (21 us at the copy's rate for 16 sequences of up to 16384 keys, 4 heads of 64, 3 queries each).
// Measured there: exponents 8 us, scores 22 us, values 32 us, quotients 5 us; bound by the
// alignment of every vector to e* and the dp4a / dp2a (half of the issue slots), not by memory.
#pragma once

#include "ict_attention.cuh"

namespace ict {

constexpr int kFewKeys = 1024;  // keys of a chunk: sums of 2^14 * 127 * 1024 fit 32 bits
constexpr int kFewQ = 4;        // queries of one key/value head that a block takes

struct FewArgs {
    AttnArgs a;
    int R;                    // rep * Lq: queries of a key/value head
    int32_t *scores;          // [B Hkv][R][ldk]
    int64_t ldk;              // Lk rounded up to a multiple of 4
    int32_t *top;             // [3][B Hkv]: largest exponent of K, V, Q + 256 (0: all zero)
    int32_t *mx;              // [B Hkv][R]: largest score + 2^22 (0: none)
    int32_t *sum;             // [B Hkv][R]
    unsigned long long *acc;  // [B Hkv][R][Dp]
};

__device__ __forceinline__ int few_top(const FewArgs &p, int op, int bg) {  // exponent, 0 when all zero
    const int t = p.top[op * p.a.B * p.a.Hkv + bg];
    return t ? t - 256 : 0;
}

// Rows are split over blockIdx.y; a thread keeps one head and walks down the rows.
__global__ void __launch_bounds__(256) few_top_kernel(const __grid_constant__ FewArgs p) {
    const AttnOperand &o = p.a.op[OPK + blockIdx.z];
    const int b = blockIdx.x, n = clamp_len(o.lens, b, o.L), H = p.a.Hkv, l0 = blockIdx.y * kFewKeys;
    if (l0 >= n) return;
    __shared__ int m[256];
    for (int g = threadIdx.x; g < H; g += 256) m[g] = 0;
    __syncthreads();
    const int nvd = p.a.D / 16, slots = max(1, 256 / H), slot = (int)threadIdx.x / H, l1 = min(n, l0 + kFewKeys);
    if (slot < slots) {
        const int g = threadIdx.x - slot * H, v0 = o.col / 16 + g * nvd, g0 = v0 / o.gv, g1 = (v0 + nvd - 1) / o.gv;
        const int8_t *e = o.exp + ((int64_t)b * o.L) * o.ngc;
        int t = -128;
        for (int k = g0; k <= g1; ++k)
#pragma unroll 8
            for (int l = l0 + slot; l < l1; l += slots) t = max(t, (int)e[(int64_t)l * o.ngc + k]);
        if (t != kEZero) atomicMax(&m[g], t + 256);
    }
    __syncthreads();
    for (int g = threadIdx.x; g < H; g += 256)
        if (m[g]) atomicMax(&p.top[(blockIdx.z * p.a.B + b) * H + g], m[g]);
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
    const int qe = few_queries<NV>(p, b, g, r0, q, &scratch);
    if (threadIdx.x == 0 && blockIdx.y == 0 && r0 == 0) p.top[2 * a.B * a.Hkv + bg] = qe + 256;
    const int lane = threadIdx.x & 31, sub = lane % NV, nvd = a.D / 16, es = few_top(p, 0, bg);
    uint4 qv[kFewQ];
#pragma unroll
    for (int r = 0; r < kFewQ; ++r) qv[r] = q[r][sub];
    // after the reduction lane sub holds the sum of query sub % kFewQ
    const int mine = r0 + (sub & (kFewQ - 1)), see = mine < p.R ? few_see(a, mine, nq, nk) : 0;
    const bool writes = sub < kFewQ && mine < p.R;
    int32_t *dst = p.scores + ((int64_t)bg * p.R + min(mine, p.R - 1)) * p.ldk;
    int mx = 0;
    const int vec = o.col / 16 + g * nvd + sub, grp = vec / o.gv;
    const int8_t *src = o.mant + (int64_t)b * a.Lk * o.ld + (int64_t)vec * 16, *ex = o.exp + (int64_t)b * a.Lk * o.ngc + grp;
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
                w[u] = *reinterpret_cast<const uint4 *>(src + ju * o.ld);
                e[u] = ex[(int64_t)ju * o.ngc];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int ju = j + u * KW;
            w[u] = rne_shift16_k(w[u], rk[rne_index(es, e[u])]);
            int s[kFewQ];
#pragma unroll
            for (int r = 0; r < kFewQ; ++r)
                s[r] = __dp4a((int)w[u].x, (int)qv[r].x, __dp4a((int)w[u].y, (int)qv[r].y,
                       __dp4a((int)w[u].z, (int)qv[r].z, __dp4a((int)w[u].w, (int)qv[r].w, 0))));
            // four sums over NV lanes, one left per lane: each step halves the sums a lane keeps
            if (NV == 8) {
#pragma unroll
                for (int r = 0; r < kFewQ; ++r) s[r] += __shfl_xor_sync(0xffffffffu, s[r], 4);
            }
            const bool b1 = sub & 2, b0 = sub & 1;
            const int k0 = b1 ? s[2] : s[0], k1 = b1 ? s[3] : s[1];
            const int t0 = k0 + __shfl_xor_sync(0xffffffffu, b1 ? s[0] : s[2], 2);
            const int t1 = k1 + __shfl_xor_sync(0xffffffffu, b1 ? s[1] : s[3], 2);
            const int sum = (b0 ? t1 : t0) + __shfl_xor_sync(0xffffffffu, b0 ? t0 : t1, 1);
            if (ju < see) mx = max(mx, sum + (1 << 22));
            if (writes && ju < j1) dst[ju] = sum;
        }
    }
    // lanes of one query: every NV-th (and both halves of eight lanes)
#pragma unroll
    for (int k = kFewQ; k < 32; k <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    if (lane < kFewQ && mine < p.R && mx) atomicMax(&p.mx[bg * p.R + mine], mx);
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
template <int NV, int RQ>  // RQ: queries of a block
__global__ void __launch_bounds__(128, RQ <= 2 ? 5 : 4) few_values_kernel(const __grid_constant__ FewArgs p) {
    __shared__ __align__(16) uint32_t E[RQ][kFewKeys / 2];  // weights of keys 2 t and 2 t + 1
    __shared__ int out[RQ][NV * 16];
    __shared__ RneK rk[9];
    const AttnArgs &a = p.a;
    const AttnOperand &o = a.op[OPV];
    const int bg = blockIdx.x, b = bg / a.Hkv, g = bg - b * a.Hkv, r0 = blockIdx.z * RQ;
    const int nk = clamp_len(o.lens, b, a.Lk), nq = clamp_len(a.op[OPQ].lens, b, a.Lq);
    const int j0 = blockIdx.y * kFewKeys, j1 = min(nk, j0 + kFewKeys);
    if (j0 >= nk) return;
    rne_table_init(rk);
    const int lane = threadIdx.x & 31, sub = lane % NV, nvd = a.D / 16, es = few_top(p, 1, bg);
    const int vec = o.col / 16 + g * nvd + sub, grp = vec / o.gv, n = j1 - j0;
    const int8_t *src = o.mant + ((int64_t)b * a.Lk + j0) * o.ld + (int64_t)vec * 16;
    const int8_t *ex = o.exp + ((int64_t)b * a.Lk + j0) * o.ngc + grp;
    constexpr int PW = 128 / NV, U = 2;  // pairs of a pass of the block; pairs in flight per thread
    uint4 w[2 * U];
    int e[2 * U];
    auto fetch = [&](int t) {
#pragma unroll
        for (int u = 0; u < 2 * U; ++u) {
            const int j = 2 * (t + (u >> 1) * PW) + (u & 1);
            w[u] = make_uint4(0, 0, 0, 0);
            e[u] = kEZero;
            if (j < n && sub < nvd) {
                w[u] = *reinterpret_cast<const uint4 *>(src + j * o.ld);
                e[u] = ex[(int64_t)j * o.ngc];
            }
        }
    };
    fetch(threadIdx.x / NV);  // the first values arrive while the weights are made
    for (int t = threadIdx.x; t < RQ * NV * 16; t += 128) out[t / (NV * 16)][t % (NV * 16)] = 0;
    // four scores at a time, all loads first
    static_assert(kFewKeys == 1024, "two groups of four keys per thread");
    int4 sc[RQ][2];
#pragma unroll
    for (int r = 0; r < RQ; ++r)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int j = j0 + 4 * (threadIdx.x + 128 * k);
            sc[r][k] = make_int4(0, 0, 0, 0);
            if (r0 + r < p.R && j < j1) sc[r][k] = *reinterpret_cast<const int4 *>(p.scores + ((int64_t)bg * p.R + r0 + r) * p.ldk + j);
        }
    __syncthreads();
    const int x = few_top(p, 2, bg) + few_top(p, 0, bg) - a.shift - 23;
    const f2 f = pk(a.fmul * pow2f(min(max(x, -120), 60)));
#pragma unroll
    for (int r = 0; r < RQ; ++r) {
        const bool on = r0 + r < p.R;
        const int see = on ? min(j1, few_see(a, r0 + r, nq, nk)) : 0;
        const f2 nm = pk(-(kAttnMagic + (float)(on ? p.mx[bg * p.R + r0 + r] - (1 << 22) : 0)));
        int sum = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int j = j0 + 4 * (threadIdx.x + 128 * k);
            float w[4];
            unpk(attn_weight2f((uint32_t)sc[r][k].x, (uint32_t)sc[r][k].y, nm, f), w[0], w[1]);
            unpk(attn_weight2f((uint32_t)sc[r][k].z, (uint32_t)sc[r][k].w, nm, f), w[2], w[3]);
            uint32_t e[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) e[z] = j + z < see ? __float_as_uint(w[z]) & 0xffffu : 0u;
            sum += (int)(e[0] + e[1] + e[2] + e[3]);
            *reinterpret_cast<uint2 *>(&E[r][2 * (threadIdx.x + 128 * k)]) = make_uint2(e[0] | e[1] << 16, e[2] | e[3] << 16);
        }
        for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        if (lane == 0 && sum) atomicAdd(&p.sum[bg * p.R + r0 + r], sum);
    }
    __syncthreads();
    int acc[RQ][16];
#pragma unroll
    for (int r = 0; r < RQ; ++r)
#pragma unroll
        for (int d = 0; d < 16; ++d) acc[r][d] = 0;
    for (int t = threadIdx.x / NV; 2 * (t - (int)(threadIdx.x / NV)) < n; t += U * PW) {
        uint4 v[2 * U];
#pragma unroll
        for (int u = 0; u < 2 * U; ++u) v[u] = rne_shift16_k(w[u], rk[rne_index(es, e[u])]);
        fetch(t + U * PW);  // the next pass
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int tt = t + u * PW;
            const uint4 w0 = v[2 * u], w1 = v[2 * u + 1];
            const uint32_t a4[4] = {w0.x, w0.y, w0.z, w0.w}, b4[4] = {w1.x, w1.y, w1.z, w1.w};
            int ee[RQ];
#pragma unroll
            for (int r = 0; r < RQ; ++r) ee[r] = tt < kFewKeys / 2 ? (int)E[r][tt] : 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int c01 = (int)__byte_perm(a4[k], b4[k], 0x5140), c23 = (int)__byte_perm(a4[k], b4[k], 0x7362);
#pragma unroll
                for (int r = 0; r < RQ; ++r) {
                    acc[r][4 * k] = dp2a_lo(ee[r], c01, acc[r][4 * k]);
                    acc[r][4 * k + 1] = dp2a_hi(ee[r], c01, acc[r][4 * k + 1]);
                    acc[r][4 * k + 2] = dp2a_lo(ee[r], c23, acc[r][4 * k + 2]);
                    acc[r][4 * k + 3] = dp2a_hi(ee[r], c23, acc[r][4 * k + 3]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < RQ; ++r) {
#pragma unroll
        for (int d = 0; d < 16; ++d) {
            int v = acc[r][d];
#pragma unroll
            for (int k = NV; k < 32; k <<= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
            if (lane < NV) atomicAdd(&out[r][lane * 16 + d], v);
        }
    }
    __syncthreads();
    for (int t = threadIdx.x; t < RQ * NV * 16; t += 128) {
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
