// ict_attention.cuh -- what the attention kernels share: arguments, the arithmetic of one
// weight, and the kernels around the contractions (exponents, aligned copies, row terms).
#pragma once

#include "ict_device.cuh"

namespace ict {

constexpr float kAttnMagic = 12582912.0f;  // 1.5 * 2^23: unit spacing
constexpr float kGridMagic = 196608.0f;    // 1.5 * 2^17: spacing 2^-6
constexpr int kKeyBlock = 128;             // keys that share the exponents of P and dS
constexpr int kDeltaMax = (1 << 22) - 1;

enum { OPQ = 0, OPK = 1, OPV = 2, OPD = 3, OPN = 4 };  // operands: Q, K, V, dO

// One operand: head h of row l of sequence b starts at column col + h D of row b L + l.
struct AttnOperand {
    const int8_t *mant, *exp;
    int64_t ld;
    int ngc, gv, gsh; // groups per row, 16-column vectors per group, their shift (-1: not a power of two)
    int col, heads, L;
    const int32_t *lens;
    int8_t *copy;     // aligned copy [B][heads][L][Dp]
};
// n / d for 0 <= n < 2^31 by a multiplication (a division costs every warp some hundred cycles)
struct Div {
    uint32_t m;
    int s;
    __device__ __forceinline__ int operator()(int n) const { return (int)((__umulhi((uint32_t)n, m) + (uint32_t)n) >> s); }
};
struct AttnOut {
    int8_t *mant, *exp;
    int64_t ld;
    int ngc, G, col;
    int gcol, dg;        // groups before the first head, groups of a head
};

struct AttnArgs {
    AttnOperand op[OPN];
    int n_op;
    int B, Hq, Hkv, rep, Lq, Lk, D, Dp, causal;
    Div heads_q, hq, by_rep, heads_kv, hkv;  // divisions by B Hq, Hq, rep, B Hkv, Hkv
    int mul, shift;
    float fmul;          // rn24(mul * log2(e) * 2^23)
    int32_t *top;        // [n_op][B * Hkv]: exponent of the aligned operand, very negative when all zero
    int2 *stats;         // [B * Hq * Lq]: largest score, sum of the weights
    AttnOut o;           // O, and dQ in the backward pass
    // backward
    const int8_t *o_mant, *o_exp;  // the forward's output
    int64_t o_ld;
    int o_ngc, o_gv;
    int2 *row;           // [B * Hq * Lq]: delta', X
    int32_t *tmax;       // [B * Hq * Lq]: largest |T| of the row
    AttnOut dk, dv;
    int4 *exps;          // [key blocks * B * Hkv]: pi, c, exponents of the sums of dV and dK
    int parts, blocks;   // each key block's queries are shared by so many; key blocks * B * Hkv
    uint4 *join;         // with parts > 1: their sums
    int32_t *tickets;    // and how many have left theirs
};

__device__ __forceinline__ int clamp_len(const int32_t *lens, int b, int L) {
    return lens ? min(max(lens[b], 0), L) : L;
}
// exponent of an aligned operand (an all-zero operand counts as exponent 0)
__device__ __forceinline__ int attn_top(const AttnArgs &a, int op, int bg) {
    const int e = a.top[op * a.B * a.Hkv + bg];
    return e < -1000 ? 0 : e;
}
// f / 64: scores times f are the logits in units of 2^-6 of a factor of two
__device__ __forceinline__ float attn_factor(const AttnArgs &a, int bg) {
    const int x = attn_top(a, OPQ, bg) + attn_top(a, OPK, bg) - a.shift - 23;
    return a.fmul * pow2f(min(max(x, -120), 60));
}
// quotient n / d as a group member: q = n / d rounded to 53 bits decides every rounding to
// 8 bits as the exact quotient does, since n < 2^48 and d < 2^31 keep an inexact quotient
// at least 2^-48 away (relatively) from every border between two mantissas
__device__ __forceinline__ int need_quot(double q) {  // q > 0
    const uint64_t b = (uint64_t)__double_as_longlong(q);
    return (int)(b >> 52) - 1023 - 6 + ((b & 0xFFFFFFFFFFFFFull) >= 0xFE00000000000ull ? 1 : 0);
}
__device__ __forceinline__ double pow2d(int k) { return __longlong_as_double((int64_t)(k + 1023) << 52); }

// Two weights E = RNE(2^14 2^(k / 64)), k = RNE((s - smax) f), as the floats 1.5 2^23 + E.  The
// FMA onto 1.5 2^17 rounds the exact product once to a multiple of 2^-6; there are 960
// arguments with a result above zero, and ex2.approx rounds to the right whole number at all
// of them (the GPU tests run through every one).
//  s + 0x4B400000 is the bit pattern of 1.5 2^23 + s
// (|s| < 2^21), and adding nm = -(1.5 2^23 + smax) leaves s - smax, both exact.
__device__ __forceinline__ f2 attn_weight2f(uint32_t s0, uint32_t s1, f2 nm, f2 f64th) {
    const f2 n = add2(pk(__uint_as_float(s0 + 0x4B400000u), __uint_as_float(s1 + 0x4B400000u)), nm);
    const f2 y = add2(fma2(n, f64th, pk(kGridMagic)), pk(-kGridMagic));
    float a, b;
    unpk(y, a, b);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
    return fma2(pk(a, b), pk(16384.0f), pk(kAttnMagic));
}
// low and second bytes of four words
__device__ __forceinline__ void split_bytes(float a, float b, float c, float d, uint32_t &lo, uint32_t &hi) {
    const uint32_t ab = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5140);
    const uint32_t cd = __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x5140);
    lo = __byte_perm(ab, cd, 0x5410);
    hi = __byte_perm(ab, cd, 0x7632);
}
// 16-byte chunk c of row r of a [128][128-byte] tile in the 128-byte swizzle
__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// tcgen05.wait::ld after which the loaded registers may be used: the empty statements take
// them as operands, so that no use is scheduled before the wait
template <int N>
__device__ __forceinline__ void tmem_tie(uint32_t (&v)[N]) {
#pragma unroll
    for (int q = 0; q < N; ++q) asm volatile("" : "+r"(v[q]));
}
template <int N>
__device__ __forceinline__ void tmem_ld_done(uint32_t (&v)[N]) {
    tmem_ld_wait();
    tmem_tie(v);
}
template <int N>
__device__ __forceinline__ void tmem_ld_done(uint32_t (&v)[N], uint32_t (&w)[N]) {
    tmem_ld_wait();
    tmem_tie(v);
    tmem_tie(w);
}

// mbar_wait with its waiting loop out of line: these kernels wait at some 30 places, and inlined
// loops push the softmax code out of the instruction caches.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, uint64_t limit_ns, const volatile int *abort) {
    return mbar_wait(bar, parity, limit_ns, abort);
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, uint64_t limit_ns, const volatile int *abort) {
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, limit_ns, abort);
}

// One arrival per warp once all its lanes are here (their TMEM reads waited for): an arrival
// per thread costs a serial shared-memory atomic each.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// n 2^-S / den as a mantissa, rden = 2^-S / den rounded: the product is within 2^-45 of the
// quotient, and a quotient that is not half way between two whole numbers is at least 2^-41
// away from that (n < 2^47), so adding and taking away 1.5 2^9 (spacing 2^-43) restores
// exact ties and moves nothing else across one.
__device__ __forceinline__ int quot_mant_fast(double n, double rden) {
    const double q = (n * rden + 768.0) - 768.0;
    return __double2loint(q + 6755399441055744.0);
}
// The same at a group exponent of 127, which may be the one that the group needs or capped: there quotients
// above 127 saturate.
__device__ __forceinline__ int quot_mant_capped(double n, double rden) {
    const double q = fmin(fmax(n * rden, -128.0), 128.0);
    return min(max(quot_mant_fast(q, 1.0), -127), 127);
}

}  // namespace ict
