// ict_norm.cu -- layer norm on (C,e) tensors (forward, backward) and the values of a
// (C,e) tensor as floating point numbers.
//
// "Memory-Efficient Integer-Only Training of Deep Neural Networks" trains vision
// transformers with integer normalisation layers but prints no formula for them; the
// reading built here (include/ict.h) works on one exponent per row and exact integer sums:
//   a = ALIGN_MAX(row), S1 = sum a, S2 = sum a^2, u = N a - S1, D = N S2 - S1^2 + eps
//   R = rn24(1 / rn24(sqrt(rn24(D)))),  h = RNE(u R 2^8)   (the normalised row at 2^-8)
//   forward   y = rn24(gamma h 2^-8 + beta), FIT
//   backward  g = A(gamma) A(dy), S3 = sum g, S4 = sum g h, m1 = RNE(4 S3 / N),
//             m2 = rn24(S4 / N), t = 4 g - m1 - RNE(h m2 2^-14), FIT of rn24(t rn24(R N))
//             dgamma = FIT(sum over rows of A_col(dy) h 2^-8), dbeta = FIT(sum A_col(dy))
// Every per-element step is one fp32 operation whose operands and rounding are exact by
// construction: |a| <= 127 and N <= 8192 keep N a and S1 below 2^21, so u is exact;
// |h| <= 2^8 sqrt(N) < 2^15; |g| < 2^14, |t| < 2^23; and RNE is one FMA onto 1.5 * 2^23.
#include <string.h>

#include <algorithm>

#include "ict_device.cuh"
#include "ict_host.h"

namespace ict {
namespace {

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
constexpr int kMaxCols = 8192;

// the bytes b and b + 1 of w (stored with 0x80 added to every byte) as floats C
__device__ __forceinline__ f2 bytes2(uint32_t w_biased, int b) {
    return add2(pk(__uint_as_float(__byte_perm(w_biased, 0x4B000000u, 0x7650 | b)),
                   __uint_as_float(__byte_perm(w_biased, 0x4B000000u, 0x7650 | (b + 1)))),
                pk(-8388736.0f));
}
__device__ __forceinline__ int dp2a_lo_s(int a, int b, int c) {
    int d;
    asm("dp2a.lo.s32.s32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ int dp2a_hi_s(int a, int b, int c) {
    int d;
    asm("dp2a.hi.s32.s32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ int dp2a_lo_u(int a, uint32_t b, int c) {
    int d;
    asm("dp2a.lo.s32.u32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ int dp2a_hi_u(int a, uint32_t b, int c) {
    int d;
    asm("dp2a.hi.s32.u32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ int dp4a_us(uint32_t a, int b, int c) {  // unsigned bytes of a, signed of b
    int d;
    asm("dp4a.u32.s32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

struct NormArgs {
    const int8_t *x, *x_exp;
    const int8_t *dy, *dy_exp;      // backward
    const int8_t *g, *g_exp;        // gamma [1][N]
    const int8_t *b, *b_exp;        // beta [1][N], or NULL
    int8_t *out, *out_exp;          // Y, or dX
    int64_t rows, ldx, lddy, ldo;
    int N, nvec;                    // columns, 16-column vectors of a row
    int gvx, gvd, gvg, gvb, gvo;    // vectors per group
    int ngx, ngd, ngg, ngb, ngo;    // groups per row
    int fast, gso;                  // an output group is a power of two of neighbouring lanes, its log2
    int eps_mul, eps_shift;
    float4 *stat;                   // backward: {S1, R 2^down, row exponent, 0} of every row
    int32_t *col_top;               // backward: largest exponent of dY's column groups + 256 (0: all zero)
};

// a row of zeros counts as the smallest there is: its gradient is that of small rows, (g - mean g) / sqrt(eps)
__device__ __forceinline__ int row_exponent(int e) { return e <= kNoExp ? kEZero : e; }

// R 2^down of a row: D is formed exactly, then rounded to 24 bits, its root and the reciprocal each
// again to 24 bits.  Rows of small values have an eps term of up to 2^292 in their units: from 2^62
// on it is brought down by an even power of two, 2^(2 down), to between 2^60 and 2^62, where the bits of
// the rest that fall off count as one (they lie far below the 24 bits).  There |u R 2^8| <=
// 2^21 2^-30 2^8 rounds to h = 0, so down matters to dX alone.
__device__ __forceinline__ float row_scale(const NormArgs &p, int s1, int s2, int e, int &down) {
    int64_t D = (int64_t)p.N * s2 - (int64_t)s1 * s1;  // below 2^41
    down = 0;
    if (p.eps_mul) {
        const int64_t m = (int64_t)p.eps_mul * p.N * p.N;  // 2^8 to 2^35
        const int k = -p.eps_shift - 2 * row_exponent(e);
        if (k >= 0) {
            down = max(0, 64 - __clzll(m) + k - 61) >> 1;
            const int j = 2 * down, jd = min(j, 62);
            const int64_t lost = D & ((1ll << jd) - 1);
            D = (m << (k - j)) + (D >> jd);
            D |= lost != 0;
        } else {
            D += k < -62 ? 0 : m >> -k;
        }
    }
    return D > 0 ? __frcp_rn(__fsqrt_rn(__ll2float_rn(D))) : 0.0f;
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Reductions over the L lanes of a row.  Rows of more than a warp meet in shared memory, every thread
// of the block at once; two buffers in turn, so that one barrier each is enough.
struct RowRed {
    long long *buf;  // [2][8 warps][2]
    int turn;
};
template <int L, int K, typename T, typename Op>
__device__ __forceinline__ void lanes_all(T (&v)[K], RowRed &red, const Op &op) {
#pragma unroll
    for (int o = (L < 32 ? L : 32) / 2; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = op(v[k], __shfl_xor_sync(0xffffffffu, v[k], o));
    if constexpr (L > 32) {
        T *s = reinterpret_cast<T *>(red.buf + red.turn * 16);
        red.turn ^= 1;
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) s[(threadIdx.x >> 5) * 2 + k] = v[k];
        }
        __syncthreads();
        const int w0 = (int)(threadIdx.x / L) * (L / 32);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            v[k] = s[w0 * 2 + k];
#pragma unroll
            for (int w = 1; w < L / 32; ++w) v[k] = op(v[k], s[(w0 + w) * 2 + k]);
        }
    }
}
struct Sum {
    template <typename T>
    __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};
struct Max {
    template <typename T>
    __device__ __forceinline__ T operator()(T a, T b) const { return max(a, b); }
};
template <int L>
__device__ __forceinline__ void row_sync() {
    if (L > 32) __syncthreads();
    else __syncwarp();
}

// One row's vectors, aligned to the row's largest group exponent (returned; kNoExp when
// every group is zero).  ex[v] is the group exponent of vector v.
template <int L, int V>
__device__ __forceinline__ int align_vectors(uint4 (&w)[V], const int (&ex)[V], const RneK *rk, RowRed &red) {
    int tops[1] = {kNoExp}, &top = tops[0];
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (ex[v] != kEZero) top = max(top, ex[v]);
    lanes_all<L>(tops, red, Max());
    bool shift = false;
#pragma unroll
    for (int v = 0; v < V; ++v) shift |= ex[v] != kEZero && ex[v] != top;
    if (__any_sync(0xffffffffu, shift)) {
#pragma unroll
        for (int v = 0; v < V; ++v) w[v] = rne_shift16_k(w[v], rk[rne_index(top, ex[v])]);
    }
    return top;
}

// FIT of 16 fp32 values y at base exponent `base`, the group's largest magnitude (as a bit
// pattern) in top: group exponent and packed mantissas.
__device__ __forceinline__ uint4 fit16(const f2 (&y)[8], uint32_t top, int base, int &e) {
    if (top == 0) {
        e = kEZero;
        return make_uint4(0, 0, 0, 0);
    }
    const int need = need_rel_f32(top, 8) + base;
    e = finalize_exp(need);
    // a capped exponent lies up to 250 below base; every y is 0 or at least 2^-27, so 2^127 saturates as well
    const f2 sc = pk(pow2f(min(base - e, 127))), mg = pk(kMagic);
    uint32_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float a, b, c, d;
        if (need > 127) {  // capped exponent: saturate
            unpk(mul2(y[2 * q], sc), a, b);
            unpk(mul2(y[2 * q + 1], sc), c, d);
            auto s = [](float v) { return fminf(fmaxf(v, -127.0f), 127.0f) + kMagic; };
            o[q] = low_bytes4(s(a), s(b), s(c), s(d));
        } else {
            unpk(fma2(y[2 * q], sc, mg), a, b);
            unpk(fma2(y[2 * q + 1], sc, mg), c, d);
            o[q] = low_bytes4(a, b, c, d);
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint32_t max16(const f2 (&y)[8]) {
    float m0 = 0, m1 = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        float a, b;
        unpk(y[q], a, b);
        m0 = fmaxf(m0, fabsf(a));
        m1 = fmaxf(m1, fabsf(b));
    }
    return __float_as_uint(fmaxf(m0, m1));
}

// Tables of per-column floats in shared memory: 4 floats of vector q's chunk k at
// [k][q], so that lanes holding neighbouring vectors read neighbouring 16-byte words.
__device__ __forceinline__ void table16(const float4 *t, int nvec, int q, f2 (&g)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float4 v = t[k * nvec + q];
        g[2 * k] = pk(v.x, v.y);
        g[2 * k + 1] = pk(v.z, v.w);
    }
}

// largest exponent (no zero group counts) of a vector of group exponents, by one block
__device__ __forceinline__ int block_top(const int8_t *e, int n, int *scratch) {
    int m = kNoExp;
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        if (e[i] != kEZero) m = max(m, (int)e[i]);
    m = warp_max(m);
    __syncthreads();
    if (threadIdx.x == 0) *scratch = kNoExp;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) atomicMax(scratch, m);
    __syncthreads();
    return *scratch;
}

// The output groups of one row, when a group is a power of two of neighbouring lanes
// (fast) or else through shared maxima (two evaluations of the row).  eval(v, y) gives the
// 16 values of the lane's vector v.
template <int L, int V, typename Eval>
__device__ __forceinline__ void fit_row(const NormArgs &p, int64_t row, bool live, int lane_in_row, int base,
                                        uint32_t *gmax, const Eval &eval) {
    int8_t *out = p.out + row * p.ldo;
    int8_t *oe = p.out_exp + row * p.ngo;
    if (p.fast) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int q = v * L + lane_in_row;
            f2 y[8];
            eval(v, y);
            uint32_t m = max16(y);
            if (q >= p.nvec) m = 0;
#pragma unroll
            for (int o = 1; o < (L < 32 ? L : 32); o <<= 1)
                if (o < p.gvo) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            int e;
            const uint4 w = fit16(y, m, base, e);
            if (live && q < p.nvec) {
                *reinterpret_cast<uint4 *>(out + q * 16) = w;
                if ((q & (p.gvo - 1)) == 0) oe[q >> p.gso] = (int8_t)e;
            }
        }
        return;
    }
    for (int g = lane_in_row; g < p.ngo; g += L) gmax[g] = 0;
    row_sync<L>();
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int q = v * L + lane_in_row;
            f2 y[8];
            eval(v, y);
            if (q >= p.nvec) continue;
            const int g = q / p.gvo;
            if (pass == 0) {
                atomicMax(&gmax[g], max16(y));
            } else {
                int e;
                const uint4 w = fit16(y, gmax[g], base, e);
                if (live) {
                    *reinterpret_cast<uint4 *>(out + q * 16) = w;
                    if (q % p.gvo == 0) oe[g] = (int8_t)e;
                }
            }
        }
        row_sync<L>();
    }
}

// Forward.  L lanes per row, V 16-byte vectors per lane, persistent blocks over the rows.
// Needs 2 bytes a value of memory; the row stays packed in registers between the sums and the
// output, gamma and beta stay in shared memory as floats.  50432 x 768: 36 us, where memory alone
// would take 12 us; bound by about 18 instructions a value (alignment, centring, scale, maximum,
// rounding: the ALU pipe 41 % busy, half of the issue slots) and their latencies.
template <int L, int V>
__global__ void __launch_bounds__(256, 3) norm_fwd_kernel(const __grid_constant__ NormArgs p) {
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ int top;
    __shared__ RneK rk[9];
    __shared__ long long rbuf[32];
    RowRed red{rbuf, 0};
    float4 *tg = reinterpret_cast<float4 *>(sm), *tb = tg + 4 * p.nvec;
    uint32_t *gm = reinterpret_cast<uint32_t *>(tb + 4 * p.nvec) + (threadIdx.x / L) * p.ngo;
    rne_table_init(rk);
    const int eg = block_top(p.g_exp, p.ngg, &top), ebt = p.b ? block_top(p.b_exp, p.ngb, &top) : kNoExp;
    int eb = max(eg, ebt);
    if (eb <= kNoExp) eb = 0;
    for (int c = threadIdx.x; c < p.N; c += blockDim.x) {
        const int q = c >> 4, at = ((c >> 2) & 3) * (4 * p.nvec) + q * 4 + (c & 3);
        const int e1 = p.g_exp[q / p.gvg];
        auto val = [&](int C, int e) { return (e == kEZero || e < eb - 100) ? 0.0f : (float)C * pow2f(e - eb); };
        reinterpret_cast<float *>(tg)[at] = val(p.g[c], e1) * 0.00390625f;  // h is at 2^-8
        reinterpret_cast<float *>(tb)[at] = p.b ? val(p.b[c], p.b_exp[q / p.gvb]) : 0.0f;
    }
    __syncthreads();
    const int lr = threadIdx.x % L;
    int gi[V];
#pragma unroll
    for (int v = 0; v < V; ++v) gi[v] = min(v * L + lr, p.nvec - 1) / p.gvx;
    const int64_t per = 256 / L;
    for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < p.rows; r0 += (int64_t)gridDim.x * per) {
        const int64_t row = r0 + threadIdx.x / L;
        const bool live = row < p.rows;
        const int64_t rr = live ? row : p.rows - 1;
        uint4 w[V];
        int ex[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int q = v * L + lr;
            w[v] = make_uint4(0, 0, 0, 0);
            ex[v] = kEZero;
            if (q < p.nvec) {
                w[v] = *reinterpret_cast<const uint4 *>(p.x + rr * p.ldx + q * 16);
                ex[v] = p.x_exp[rr * p.ngx + gi[v]];
            }
        }
        const int64_t nx = row + (int64_t)gridDim.x * per;
        if (nx < p.rows) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v * L + lr < p.nvec) prefetch_l2(p.x + nx * p.ldx + (v * L + lr) * 16);
            if (lr == 0) prefetch_l2(p.x_exp + nx * p.ngx);
        }
        const int e = align_vectors<L, V>(w, ex, rk, red);
        int s12[2] = {0, 0}, &s1 = s12[0], &s2 = s12[1];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t u[4] = {w[v].x, w[v].y, w[v].z, w[v].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                s1 = __dp4a((int)u[k], 0x01010101, s1);
                s2 = __dp4a((int)u[k], (int)u[k], s2);
            }
        }
        lanes_all<L>(s12, red, Sum());
        int down;
        const f2 N2 = pk((float)p.N), m1 = pk(-(float)s1), R2 = pk(row_scale(p, s1, s2, e, down) * 256.0f);
        const f2 mg = pk(kMagic), nmg = pk(-kMagic);
        fit_row<L, V>(p, row, live, lr, eb, gm, [&](int v, f2(&y)[8]) {
            const uint32_t u[4] = {w[v].x ^ 0x80808080u, w[v].y ^ 0x80808080u, w[v].z ^ 0x80808080u,
                                   w[v].w ^ 0x80808080u};
            const int q = min(v * L + lr, p.nvec - 1);
            f2 g[8], b[8];
            table16(tg, p.nvec, q, g);
            table16(tb, p.nvec, q, b);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const f2 uu = fma2(N2, bytes2(u[k >> 1], 2 * (k & 1)), m1);
                y[k] = fma2(g[k], add2(fma2(uu, R2, mg), nmg), b[k]);
            }
        });
    }
}

// Backward with respect to the row: dX, each row's statistics for the parameter gradients,
// and the largest exponent of every column group of dY.  50432 x 768: 62 us (18 us of memory),
// bound like the forward; h and g are formed twice, which costs less than keeping them.
template <int L, int V>
__global__ void __launch_bounds__(256, 2) norm_bwd_kernel(const __grid_constant__ NormArgs p) {
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ int top;
    __shared__ int cm[kMaxCols / 16];  // the block's largest exponent of every column group of dY
    __shared__ RneK rk[9];
    __shared__ long long rbuf[32];
    RowRed red{rbuf, 0};
    for (int g = threadIdx.x; g < p.ngd; g += blockDim.x) cm[g] = kNoExp;
    float4 *tg = reinterpret_cast<float4 *>(sm);
    uint32_t *gm = reinterpret_cast<uint32_t *>(tg + 4 * p.nvec) + (threadIdx.x / L) * p.ngo;
    rne_table_init(rk);
    int eg = block_top(p.g_exp, p.ngg, &top);
    if (eg <= kNoExp) eg = 0;
    for (int c = threadIdx.x; c < p.N; c += blockDim.x) {  // gamma aligned to one exponent
        const int q = c >> 4, at = ((c >> 2) & 3) * (4 * p.nvec) + q * 4 + (c & 3);
        const int e1 = p.g_exp[q / p.gvg];
        reinterpret_cast<float *>(tg)[at] =
            e1 == kEZero || e1 < eg - 100 ? 0.0f : __fadd_rn(__fmaf_rn((float)p.g[c], pow2f(e1 - eg), kMagic), -kMagic);
    }
    __syncthreads();
    const int lr = threadIdx.x % L;
    int gi[V], gd[V], ctop[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        gi[v] = min(v * L + lr, p.nvec - 1) / p.gvx;
        gd[v] = min(v * L + lr, p.nvec - 1) / p.gvd;
        ctop[v] = kNoExp;
    }
    const double invN = 1.0 / (double)p.N;
    auto mean = [&](double x) {  // x / N correctly rounded (one Newton step on the quotient)
        const double q = x * invN;
        return __fma_rn(__fma_rn(-q, (double)p.N, x), invN, q);
    };
    const int64_t per = 256 / L;
    for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < p.rows; r0 += (int64_t)gridDim.x * per) {
        const int64_t row = r0 + threadIdx.x / L;
        const bool live = row < p.rows;
        const int64_t rr = live ? row : p.rows - 1;
        uint4 w[V], d[V];
        int ex[V], ed[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int q = v * L + lr;
            w[v] = d[v] = make_uint4(0, 0, 0, 0);
            ex[v] = ed[v] = kEZero;
            if (q < p.nvec) {
                w[v] = *reinterpret_cast<const uint4 *>(p.x + rr * p.ldx + q * 16);
                d[v] = *reinterpret_cast<const uint4 *>(p.dy + rr * p.lddy + q * 16);
                ex[v] = p.x_exp[rr * p.ngx + gi[v]];
                ed[v] = p.dy_exp[rr * p.ngd + gd[v]];
            }
        }
        const int64_t nx = row + (int64_t)gridDim.x * per;
        if (nx < p.rows) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v * L + lr < p.nvec) {
                    prefetch_l2(p.x + nx * p.ldx + (v * L + lr) * 16);
                    prefetch_l2(p.dy + nx * p.lddy + (v * L + lr) * 16);
                }
            if (lr == 0) prefetch_l2(p.x_exp + nx * p.ngx);
            if (lr == 1) prefetch_l2(p.dy_exp + nx * p.ngd);
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (ed[v] != kEZero) ctop[v] = max(ctop[v], ed[v]);
        const int e = align_vectors<L, V>(w, ex, rk, red), e2 = align_vectors<L, V>(d, ed, rk, red);
        int s12[2] = {0, 0}, &s1 = s12[0], &s2 = s12[1];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t u[4] = {w[v].x, w[v].y, w[v].z, w[v].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                s1 = __dp4a((int)u[k], 0x01010101, s1);
                s2 = __dp4a((int)u[k], (int)u[k], s2);
            }
        }
        lanes_all<L>(s12, red, Sum());
        int down;
        const float R = row_scale(p, s1, s2, e, down);
        if (live && lr == 0) p.stat[row] = make_float4((float)s1, R, __int_as_float(e), 0.0f);
        const f2 N2 = pk((float)p.N), ms = pk(-(float)s1), R2 = pk(R * 256.0f), mg = pk(kMagic), nmg = pk(-kMagic);
        // S3 = sum g and S4 = sum g h: g in 16-bit halves, h in its two bytes
        int s3s[1] = {0}, &s3 = s3s[0], s4l = 0, s4h = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int q = min(v * L + lr, p.nvec - 1);
            const uint32_t u[4] = {w[v].x ^ 0x80808080u, w[v].y ^ 0x80808080u, w[v].z ^ 0x80808080u,
                                   w[v].w ^ 0x80808080u};
            const uint32_t t[4] = {d[v].x ^ 0x80808080u, d[v].y ^ 0x80808080u, d[v].z ^ 0x80808080u,
                                   d[v].w ^ 0x80808080u};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 ga = tg[k * p.nvec + q];
                float h0, h1, h2, h3, g0, g1, g2, g3;
                unpk(fma2(fma2(N2, bytes2(u[k], 0), ms), R2, mg), h0, h1);
                unpk(fma2(fma2(N2, bytes2(u[k], 2), ms), R2, mg), h2, h3);
                unpk(fma2(pk(ga.x, ga.y), bytes2(t[k], 0), mg), g0, g1);
                unpk(fma2(pk(ga.z, ga.w), bytes2(t[k], 2), mg), g2, g3);
                const uint32_t ha = __byte_perm(__float_as_uint(h0), __float_as_uint(h1), 0x5140);
                const uint32_t hb = __byte_perm(__float_as_uint(h2), __float_as_uint(h3), 0x5140);
                const uint32_t hl = __byte_perm(ha, hb, 0x5410), hh = __byte_perm(ha, hb, 0x7632);
                const int ga01 = (int)__byte_perm(__float_as_uint(g0), __float_as_uint(g1), 0x5410);
                const int ga23 = (int)__byte_perm(__float_as_uint(g2), __float_as_uint(g3), 0x5410);
                s3 = dp2a_lo_s(ga01, 0x01010101, dp2a_lo_s(ga23, 0x01010101, s3));
                s4l = dp2a_lo_u(ga01, hl, dp2a_hi_u(ga23, hl, s4l));
                s4h = dp2a_lo_s(ga01, (int)hh, dp2a_hi_s(ga23, (int)hh, s4h));
            }
        }
        long long s4s[1] = {(long long)s4h * 256 + s4l}, &s4 = s4s[0];
        lanes_all<L>(s3s, red, Sum());
        lanes_all<L>(s4s, red, Sum());
        const f2 m1 = pk(-(float)rint(mean(4.0 * (double)s3)));
        const f2 m2 = pk((float)mean((double)s4) * 6.103515625e-05f);  // 2^-14
        const f2 RN = pk(R * (float)p.N), four = pk(4.0f), one = pk(-1.0f);
        const int base = eg + (e2 <= kNoExp ? 0 : e2) - row_exponent(e) - 2 - down;
        fit_row<L, V>(p, row, live, lr, base, gm, [&](int v, f2(&y)[8]) {
            const int q = min(v * L + lr, p.nvec - 1);
            const uint32_t u[4] = {w[v].x ^ 0x80808080u, w[v].y ^ 0x80808080u, w[v].z ^ 0x80808080u,
                                   w[v].w ^ 0x80808080u};
            const uint32_t t[4] = {d[v].x ^ 0x80808080u, d[v].y ^ 0x80808080u, d[v].z ^ 0x80808080u,
                                   d[v].w ^ 0x80808080u};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float4 ga4 = tg[(k >> 1) * p.nvec + q];
                const f2 ga = (k & 1) ? pk(ga4.z, ga4.w) : pk(ga4.x, ga4.y);
                const f2 h = add2(fma2(fma2(N2, bytes2(u[k >> 1], 2 * (k & 1)), ms), R2, mg), nmg);
                const f2 g = mul2(ga, bytes2(t[k >> 1], 2 * (k & 1)));
                const f2 z = add2(fma2(h, m2, mg), nmg);
                y[k] = mul2(fma2(z, one, fma2(g, four, m1)), RN);
            }
        });
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (v * L + lr < p.nvec && ctop[v] > kNoExp) atomicMax(&cm[gd[v]], ctop[v]);
    __syncthreads();
    for (int g = threadIdx.x; g < p.ngd; g += blockDim.x)
        if (cm[g] > kNoExp) atomicMax(&p.col_top[g], cm[g] + 256);
}

struct NormColArgs {
    const int8_t *x, *x_exp, *dy, *dy_exp;
    int64_t rows, ldx, lddy, rows_per_block;
    int N, nvec, vb, gvx, gvd, ngx, ngd;  // vb: vectors (16 columns) of a block
    const float4 *stat;
    const int32_t *col_top;
    int64_t *acc;  // [2][N]: sums of A_col(dy) h and of A_col(dy)
};

// Parameter gradients: a thread owns 16 columns and walks down the rows four at a time; the four
// rows' bytes of a column are brought into one word, so that a dp4a adds four rows.  h goes in as
// its low and high byte.  The sums are whole numbers, so their order does not matter; threads
// meet in shared memory and blocks by 64-bit atomics.  Wide columns per thread because of the
// rows' addresses, exponents and statistics: with four columns they were two thirds of 28
// instructions a value.  50432 x 768: 38 us (12 us of memory), bound by the ALU pipe.
__global__ void __launch_bounds__(256, 2) norm_cols_kernel(const __grid_constant__ NormColArgs p) {
    extern __shared__ int sums[];  // [3][vb * 16]
    __shared__ RneK rk[9];
    const int slots = 256 / p.vb, slot = threadIdx.x / p.vb, cols = p.vb * 16;
    const int q = blockIdx.x * p.vb + threadIdx.x % p.vb;
    for (int t = threadIdx.x; t < 3 * cols; t += 256) sums[t] = 0;
    rne_table_init(rk);
    __syncthreads();
    if (slot < slots && q < p.nvec) {
        const int gx = q / p.gvx, gd = q / p.gvd, et = p.col_top[gd] - 256;
        const f2 N2 = pk((float)p.N), mg = pk(kMagic);
        int lo[16], hi[16], sb[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) lo[c] = hi[c] = sb[c] = 0;
        const int64_t r1 = min(p.rows, (int64_t)(blockIdx.y + 1) * p.rows_per_block);
        for (int64_t r = (int64_t)blockIdx.y * p.rows_per_block + slot * 4; r < r1; r += slots * 4) {
            uint4 xw[4], dw[4];
            int ex[4], ed[4];
            float4 st[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t row = min(r + i, r1 - 1);
                st[i] = p.stat[row];
                xw[i] = *reinterpret_cast<const uint4 *>(p.x + row * p.ldx + q * 16);
                dw[i] = *reinterpret_cast<const uint4 *>(p.dy + row * p.lddy + q * 16);
                ex[i] = p.x_exp[row * p.ngx + gx];
                ed[i] = r + i < r1 ? (int)p.dy_exp[row * p.ngd + gd] : kEZero;
            }
            f2 ms[4], R2[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dw[i] = rne_shift16_k(dw[i], rk[rne_index(et, ed[i])]);  // to the column group's exponent (0 beyond the rows)
                xw[i] = rne_shift16_k(xw[i], rk[rne_index(__float_as_int(st[i].z), ex[i])]);  // to the row's
                ms[i] = pk(-st[i].x);
                R2[i] = pk(st[i].y * 256.0f);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // four columns
                const uint32_t xk[4] = {(&xw[0].x)[k] ^ 0x80808080u, (&xw[1].x)[k] ^ 0x80808080u, (&xw[2].x)[k] ^ 0x80808080u,
                                        (&xw[3].x)[k] ^ 0x80808080u};
                const uint32_t dk[4] = {(&dw[0].x)[k], (&dw[1].x)[k], (&dw[2].x)[k], (&dw[3].x)[k]};
                // rows 0..3 of column c as the bytes of one word
                const uint32_t d01a = __byte_perm(dk[0], dk[1], 0x5140), d23a = __byte_perm(dk[2], dk[3], 0x5140);
                const uint32_t d01b = __byte_perm(dk[0], dk[1], 0x7362), d23b = __byte_perm(dk[2], dk[3], 0x7362);
                const uint32_t dc[4] = {__byte_perm(d01a, d23a, 0x5410), __byte_perm(d01a, d23a, 0x7632),
                                        __byte_perm(d01b, d23b, 0x5410), __byte_perm(d01b, d23b, 0x7632)};
#pragma unroll
                for (int c = 0; c < 4; c += 2) {
                    float h[4][2];
#pragma unroll
                    for (int i = 0; i < 4; ++i) unpk(fma2(fma2(N2, bytes2(xk[i], c), ms[i]), R2[i], mg), h[i][0], h[i][1]);
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const uint32_t a = __byte_perm(__float_as_uint(h[0][z]), __float_as_uint(h[1][z]), 0x5140);
                        const uint32_t b = __byte_perm(__float_as_uint(h[2][z]), __float_as_uint(h[3][z]), 0x5140);
                        const int at = 4 * k + c + z;
                        lo[at] = dp4a_us(__byte_perm(a, b, 0x5410), (int)dc[c + z], lo[at]);
                        hi[at] = __dp4a((int)__byte_perm(a, b, 0x7632), (int)dc[c + z], hi[at]);
                        sb[at] = __dp4a(0x01010101, (int)dc[c + z], sb[at]);
                    }
                }
            }
        }
        const int at = (threadIdx.x % p.vb) * 16;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            atomicAdd(&sums[at + c], lo[c]);
            atomicAdd(&sums[cols + at + c], hi[c]);
            atomicAdd(&sums[2 * cols + at + c], sb[c]);
        }
    }
    __syncthreads();
    for (int t = threadIdx.x; t < cols; t += 256) {
        const int64_t col = (int64_t)blockIdx.x * cols + t;
        if (col >= p.N) break;
        atomicAdd(reinterpret_cast<unsigned long long *>(p.acc) + col, (unsigned long long)((int64_t)sums[cols + t] * 256 + sums[t]));
        atomicAdd(reinterpret_cast<unsigned long long *>(p.acc) + p.N + col, (unsigned long long)(int64_t)sums[2 * cols + t]);
    }
}

struct NormFitArgs {
    const int64_t *acc;
    const int32_t *col_top;
    int N, gvd;
    int8_t *out[2], *out_exp[2];
    int G[2];
};
// FIT of the summed gradients: one warp per output group of dgamma (blockIdx.y = 0, sums at
// exponent e_j - 8) and of dbeta (1, at e_j).
__global__ void __launch_bounds__(256) norm_fit_kernel(const __grid_constant__ NormFitArgs p) {
    const int z = blockIdx.y, lane = threadIdx.x & 31;
    if (!p.out[z]) return;
    const int G = p.G[z], g = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int j0 = g * G, j1 = min(p.N, j0 + G);
    if (j0 >= p.N) return;
    const int64_t *acc = p.acc + (int64_t)z * p.N;
    auto expo = [&](int j) { return p.col_top[(j >> 4) / p.gvd] - 256 - (z == 0 ? 8 : 0); };
    int top = kNoExp;
    for (int j = j0 + lane; j < j1; j += 32) {
        const int64_t v = acc[j];
        if (v) top = max(top, expo(j) + need_off64((uint64_t)(v < 0 ? -v : v)));
    }
    const int e = finalize_exp(warp_max(top));
    for (int j = j0 + lane; j < j1; j += 32) {
        const int64_t v = acc[j];
        p.out[z][j] = v ? (int8_t)requant64(v, expo(j), e) : (int8_t)0;
    }
    if (lane == 0) p.out_exp[z][g] = (int8_t)e;
}

// ------------------------------------------------------------------ values

struct ValuesArgs {
    const int8_t *m, *e;
    int64_t rows, cols, ld, ldo, ngc;
    int g_rows, g_cols, gsh;  // gsh: log2 of g_cols, or -1
    int wide;                 // out and its rows begin at multiples of 32 bytes
    void *out;
};
__device__ __forceinline__ float ce_value(int C, int e) {  // C 2^e, in two exact steps
    if (e == kEZero) return 0.0f;
    const int a = e / 2;
    return (float)C * pow2f(a) * pow2f(e - a);
}
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
// 32 bytes by one store where they are aligned (whole sectors: two halves of a sector by two stores
// of every lane cost 50432 x 768 values 25 us against 18 us)
__device__ __forceinline__ void store32(uint8_t *p, const uint32_t (&v)[8], int wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}
// VEC: 16 columns per thread and step, four steps' loads in flight.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(256) values_kernel(const __grid_constant__ ValuesArgs a) {
    constexpr int W = VEC ? 16 : 1, U = VEC ? 4 : 1;
    const uint32_t per = (uint32_t)(a.cols / W);
    const int64_t n = a.rows * (int64_t)per, step = (int64_t)gridDim.x * 256;
    for (int64_t t0 = (int64_t)blockIdx.x * 256 + threadIdx.x; t0 < n; t0 += U * step) {
        uint4 w[U];
        int e[U];
        int64_t at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = t0 + u * step;
            at[u] = -1;
            if (t >= n) continue;
            const int64_t i = n <= 0xffffffffll ? (int64_t)((uint32_t)t / per) : t / per;
            const int j = (int)(t - i * per) * W;
            const int64_t gr = a.g_rows == 1 ? i : i / a.g_rows;
            e[u] = a.e[gr * a.ngc + (a.gsh >= 0 ? j >> a.gsh : j / a.g_cols)];
            at[u] = i * a.ldo + j;
            const int8_t *m = a.m + i * a.ld + j;
            if constexpr (VEC) w[u] = *reinterpret_cast<const uint4 *>(m);
            else w[u].x = (uint32_t)(uint8_t)*m;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (at[u] < 0) continue;
            if constexpr (VEC) {
                // 2^e in two exact factors
                const int h = e[u] == kEZero ? 0 : e[u] / 2;
                const float s0 = e[u] == kEZero ? 0.0f : pow2f(h), s1 = e[u] == kEZero ? 0.0f : pow2f(e[u] - h);
                const uint32_t b[4] = {w[u].x ^ 0x80808080u, w[u].y ^ 0x80808080u, w[u].z ^ 0x80808080u, w[u].w ^ 0x80808080u};
#pragma unroll
                for (int q = 0; q < 4; q += BF16 ? 4 : 2) {  // 32 bytes
                    uint32_t v[8];
                    if constexpr (BF16) {
#pragma unroll
                        for (int k = 0; k < 16; k += 2)
                            v[k / 2] = bf16x2(sx8f(b[k >> 2], k & 3) * s0 * s1, sx8f(b[k >> 2], (k & 3) + 1) * s0 * s1);
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = __float_as_uint(sx8f(b[q + (k >> 2)], k & 3) * s0 * s1);
                    }
                    store32((uint8_t *)a.out + at[u] * (BF16 ? 2 : 4) + 8 * q * (BF16 ? 1 : 2), v, a.wide);
                }
            } else {
                const float v = ce_value((int)(int8_t)w[u].x, e[u]);
                if constexpr (BF16) ((uint16_t *)a.out)[at[u]] = (uint16_t)bf16x2(v, 0.0f);
                else ((float *)a.out)[at[u]] = v;
            }
        }
    }
}

// ------------------------------------------------------------------ host

int check_rows(const ict_tensor *t, int64_t rows, int64_t cols) {
    int st;
    if ((st = host::check_tensor(t))) return st;
    if (t->rows != rows || t->cols != cols) return ICT_ERR_INVALID_ARG;
    if (t->g_rows != 1 && rows > 1) return ICT_ERR_LAYOUT;
    return host::check_vec(t);
}

int fill(NormArgs &a, const ict_tensor *X, const ict_tensor *gamma, const ict_tensor *out, int32_t eps_mul,
         int32_t eps_shift) {
    int st;
    if ((st = host::int8_only())) return st;
    if ((st = host::check_tensor(X))) return st;
    if (X->cols < 1) return ICT_ERR_INVALID_ARG;
    if (X->cols > kMaxCols) return ICT_ERR_LAYOUT;
    if (eps_mul < 0 || eps_mul > 512 || eps_shift < 0 || eps_shift > 64) return ICT_ERR_INVALID_ARG;
    if ((st = check_rows(X, X->rows, X->cols)) || (st = check_rows(gamma, 1, X->cols)) ||
        (st = check_rows(out, X->rows, X->cols)))
        return st;
    memset(&a, 0, sizeof(a));
    a.x = X->mant, a.x_exp = X->exp, a.ldx = X->ld, a.rows = X->rows, a.N = (int)X->cols, a.nvec = a.N / 16;
    a.gvx = host::vec_per_group(X), a.ngx = host::groups_per_row(X);
    a.g = gamma->mant, a.g_exp = gamma->exp, a.gvg = host::vec_per_group(gamma), a.ngg = host::groups_per_row(gamma);
    a.out = out->mant, a.out_exp = out->exp, a.ldo = out->ld, a.gvo = host::vec_per_group(out), a.ngo = host::groups_per_row(out);
    a.eps_mul = eps_mul, a.eps_shift = eps_shift;
    return ICT_OK;
}

// Lanes per row: the fewest (a power of two from 4) whose lanes hold at most three vectors
// each, so that the per-row work (reductions, root) is shared by as many values as possible
// while a warp keeps enough loads in flight.  Rows above 1536 values take several warps: with
// 4, 8 and 16 vectors a lane of one warp, rows of 2560, 4096 and 8192 values (30.7, 36.9 and 38.5
// million) cost 47, 48 and 91 us forward and 105, 122 and 318 us backward, registers spilled,
// against 41, 48 and 59 us forward and 67, 71 and 84 us with several warps.
template <typename F>
void dispatch(int nvec, F &&f) {
    auto go = [&](auto lanes) {
        constexpr int L = decltype(lanes)::value;
        const int v = (nvec + L - 1) / L;
        if (v <= 1) f(lanes, std::integral_constant<int, 1>());
        else if (v == 2) f(lanes, std::integral_constant<int, 2>());
        else f(lanes, std::integral_constant<int, 3>());
    };
    if (nvec <= 12) go(std::integral_constant<int, 4>());
    else if (nvec <= 24) go(std::integral_constant<int, 8>());
    else if (nvec <= 48) go(std::integral_constant<int, 16>());
    else if (nvec <= 96) go(std::integral_constant<int, 32>());
    else if (nvec <= 192) go(std::integral_constant<int, 64>());
    else if (nvec <= 384) go(std::integral_constant<int, 128>());
    else go(std::integral_constant<int, 256>());
}

template <int L>
void finish_plan(NormArgs &a) {
    a.fast = (a.gvo & (a.gvo - 1)) == 0 && a.gvo <= (L < 32 ? L : 32) && a.nvec % a.gvo == 0;
    a.gso = a.fast ? __builtin_ctz((unsigned)a.gvo) : 0;
}

// Two floats a column, and the maxima of the output groups of a block's rows: 256 / L rows of at most 3 L groups.
constexpr int kMaxSmem = kMaxCols * 8 + 256 * 3 * 4;

template <auto Kernel>
int run_rows(const NormArgs &a, int lanes, size_t smem, cudaStream_t s) {
    static std::atomic<uint64_t> fits[64];  // per device: shared memory asked for last, and how many blocks fit
    int sms = 0, dev = 0;
    int st;
    if ((st = host::device_info(&sms))) return st;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return ICT_ERR_CUDA;
    uint64_t f = fits[dev].load(std::memory_order_relaxed);
    if (f >> 16 != smem || f == 0) {
        int per = 0;
        // (asked for at any size: the kernel's static memory counts towards the 48 KB that need no asking)
        if ((st = host::allow_smem<Kernel, kMaxSmem>())) return st;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, Kernel, 256, smem) != cudaSuccess || per < 1) return ICT_ERR_CUDA;
        f = (uint64_t)smem << 16 | (uint64_t)per;
        fits[dev].store(f, std::memory_order_relaxed);
    }
    const int per = (int)(f & 0xffff);
    const int64_t blocks = std::min<int64_t>(host::cdiv(a.rows, 256 / lanes), (int64_t)sms * per);
    Kernel<<<(unsigned)blocks, 256, smem, s>>>(a);
    host::counted(1);
    return host::launch_status();
}

}  // namespace

namespace host {
int take_status_norm(int32_t *v) {
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

int32_t ict_layernorm_fwd(const ict_tensor *X, const ict_tensor *gamma, const ict_tensor *beta, int32_t eps_mul,
                          int32_t eps_shift, ict_tensor *Y, void *stream) {
    int st;
    NormArgs a;
    if ((st = fill(a, X, gamma, Y, eps_mul, eps_shift))) return st;
    if (beta) {
        if ((st = check_rows(beta, 1, X->cols))) return st;
        a.b = beta->mant, a.b_exp = beta->exp, a.gvb = host::vec_per_group(beta), a.ngb = host::groups_per_row(beta);
    }
    if ((st = host::device_info(nullptr))) return st;
    if (a.rows == 0) return ICT_OK;
    cudaStream_t s = (cudaStream_t)stream;
    host::Timer kt(s, ICT_KC_POINTWISE, 2.0 * (double)a.rows * a.N + (double)a.rows * (a.ngx + a.ngo));
    dispatch(a.nvec, [&](auto lanes, auto vecs) {
        constexpr int L = decltype(lanes)::value, V = decltype(vecs)::value;
        finish_plan<L>(a);
        const size_t smem = (size_t)a.N * 8 + (a.fast ? 0 : (size_t)(256 / L) * a.ngo * 4);
        st = run_rows<norm_fwd_kernel<L, V>>(a, L, smem, s);
    });
    return st;
}

size_t ict_layernorm_bwd_workspace(const ict_tensor *X) {
    if (host::check_tensor(X) != ICT_OK || X->cols < 1 || X->cols > kMaxCols) return 0;
    return (size_t)(host::round_up(X->cols * 16, 256) + host::round_up(X->cols / 4 + 4, 256) +
                    host::round_up(X->rows * 16, 256));
}

int32_t ict_layernorm_bwd(const ict_tensor *X, const ict_tensor *gamma, const ict_tensor *dY, int32_t eps_mul,
                          int32_t eps_shift, ict_tensor *dX, ict_tensor *dgamma, ict_tensor *dbeta, void *ws,
                          size_t ws_bytes, void *stream) {
    int st;
    NormArgs a;
    if ((st = fill(a, X, gamma, dX, eps_mul, eps_shift))) return st;
    if ((st = check_rows(dY, X->rows, X->cols)) || (st = check_rows(dgamma, 1, X->cols))) return st;
    if (dbeta && (st = check_rows(dbeta, 1, X->cols))) return st;
    if (X->rows > (1 << 30)) return ICT_ERR_LAYOUT;
    if (!ws || ((uintptr_t)ws & 255) || ws_bytes < ict_layernorm_bwd_workspace(X)) return ICT_ERR_WORKSPACE;
    // X and dY are read again after dX is written
    auto share = [&](const ict_tensor *t, const ict_tensor *u) { return t && u && host::share_columns(t, 0, X->cols, u, 0, X->cols); };
    if (share(dX, X) || share(dX, dY) || share(dX, dgamma) || share(dX, dbeta) || share(dgamma, dbeta)) return ICT_ERR_INVALID_ARG;
    if ((st = host::device_info(nullptr))) return st;
    cudaStream_t s = (cudaStream_t)stream;
    int64_t *acc = (int64_t *)ws;
    a.dy = dY->mant, a.dy_exp = dY->exp, a.lddy = dY->ld, a.gvd = host::vec_per_group(dY), a.ngd = host::groups_per_row(dY);
    const int64_t acc_bytes = host::round_up((int64_t)a.N * 16, 256);
    const int64_t top_bytes = host::round_up(a.N / 4 + 4, 256);
    a.col_top = (int32_t *)((uint8_t *)ws + acc_bytes);
    a.stat = (float4 *)((uint8_t *)ws + acc_bytes + top_bytes);
    if (cudaMemsetAsync(acc, 0, (size_t)(acc_bytes + top_bytes), s) != cudaSuccess) return ICT_ERR_CUDA;
    host::Timer kt(s, ICT_KC_POINTWISE, 3.0 * (double)a.rows * a.N + (double)a.rows * (a.ngx + a.ngd + a.ngo));
    if (a.rows > 0) {
        dispatch(a.nvec, [&](auto lanes, auto vecs) {
            constexpr int L = decltype(lanes)::value, V = decltype(vecs)::value;
            finish_plan<L>(a);
            const size_t smem = (size_t)a.N * 4 + (a.fast ? 0 : (size_t)(256 / L) * a.ngo * 4);
            st = run_rows<norm_bwd_kernel<L, V>>(a, L, smem, s);
        });
        if (st) return st;
        int sms = 0;
        host::device_info(&sms);
        NormColArgs c;
        memset(&c, 0, sizeof(c));
        c.x = a.x, c.x_exp = a.x_exp, c.dy = a.dy, c.dy_exp = a.dy_exp, c.rows = a.rows, c.ldx = a.ldx, c.lddy = a.lddy;
        c.N = a.N, c.gvx = a.gvx, c.gvd = a.gvd, c.ngx = a.ngx, c.ngd = a.ngd;
        c.stat = a.stat, c.col_top = a.col_top, c.acc = acc;
        // two blocks per SM, at least eight rows per thread and at most 2^15 rows each (the 32-bit sums)
        c.nvec = a.nvec;
        c.vb = a.nvec <= 64 ? a.nvec : 32;
        const int64_t tiles = host::cdiv(a.nvec, c.vb);
        const int64_t want = std::max<int64_t>(1, (int64_t)sms * 2 / tiles);
        c.rows_per_block = std::min<int64_t>(1 << 15, host::round_up(std::max<int64_t>(1, host::cdiv(a.rows, want)), 8 * (256 / c.vb)));
        norm_cols_kernel<<<dim3((unsigned)tiles, (unsigned)host::cdiv(a.rows, c.rows_per_block)), 256, (size_t)c.vb * 16 * 12, s>>>(c);
        host::counted(1);
    }
    NormFitArgs f;
    memset(&f, 0, sizeof(f));
    f.acc = acc, f.col_top = a.col_top, f.N = a.N, f.gvd = a.gvd;
    f.out[0] = dgamma->mant, f.out_exp[0] = dgamma->exp, f.G[0] = (int)std::min<int64_t>(dgamma->g_cols, a.N);
    f.G[1] = 1 << 30;
    if (dbeta) f.out[1] = dbeta->mant, f.out_exp[1] = dbeta->exp, f.G[1] = (int)std::min<int64_t>(dbeta->g_cols, a.N);
    const int most = (int)std::max(host::cdiv(a.N, f.G[0]), host::cdiv(a.N, f.G[1]));
    norm_fit_kernel<<<dim3((unsigned)host::cdiv(most, 8), 2), 256, 0, s>>>(f);
    host::counted(1);
    return host::launch_status();
}

int32_t ict_values(const ict_tensor *t, int32_t bf16, void *out, int64_t ld_out, void *stream) {
    int st;
    if ((st = host::check_tensor(t))) return st;
    if (bf16 != 0 && bf16 != 1) return ICT_ERR_INVALID_ARG;
    if (t->rows > 0 && t->cols > 0 && (!out || ld_out < t->cols)) return ICT_ERR_INVALID_ARG;
    if ((uintptr_t)out % (bf16 ? 2 : 4)) return ICT_ERR_ALIGNMENT;
    int sms = 0;
    if ((st = host::device_info(&sms))) return st;
    if (t->rows == 0 || t->cols == 0) return ICT_OK;
    ValuesArgs a;
    memset(&a, 0, sizeof(a));
    a.m = t->mant, a.e = t->exp, a.rows = t->rows, a.cols = t->cols, a.ld = t->ld, a.ldo = ld_out;
    a.g_rows = (int)std::min<int64_t>(t->g_rows, t->rows), a.g_cols = (int)std::min<int64_t>(t->g_cols, t->cols);
    a.gsh = (a.g_cols & (a.g_cols - 1)) == 0 ? __builtin_ctz((unsigned)a.g_cols) : -1;
    a.ngc = host::groups_per_row(t);
    a.out = out;
    const bool vec = host::check_vec(t) == ICT_OK && (uintptr_t)out % 16 == 0 && ld_out % 8 == 0;
    a.wide = (uintptr_t)out % 32 == 0 && ld_out % (bf16 ? 16 : 8) == 0;
    const int64_t n = t->rows * t->cols / (vec ? 16 : 1);
    const unsigned grid = (unsigned)std::min<int64_t>(host::cdiv(n, 256), (int64_t)sms * 8);
    cudaStream_t s = (cudaStream_t)stream;
    host::Timer kt(s, ICT_KC_OTHER, (double)t->rows * t->cols * (bf16 ? 3 : 5));
    if (vec && bf16) values_kernel<true, true><<<grid, 256, 0, s>>>(a);
    else if (vec) values_kernel<false, true><<<grid, 256, 0, s>>>(a);
    else if (bf16) values_kernel<true, false><<<grid, 256, 0, s>>>(a);
    else values_kernel<false, false><<<grid, 256, 0, s>>>(a);
    host::counted(1);
    return host::launch_status();
}

}  // extern "C"
