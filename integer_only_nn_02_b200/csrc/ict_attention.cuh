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
    int ngc, gv;      // groups per row, 16-column vectors per group
    int col, heads, L;
    const int32_t *lens;
    int8_t *copy;     // aligned copy [B][heads][L][Dp]
};
struct AttnOut {
    int8_t *mant, *exp;
    int64_t ld;
    int ngc, G, col;
};

struct AttnArgs {
    AttnOperand op[OPN];
    int n_op;
    int B, Hq, Hkv, rep, Lq, Lk, D, Dp, causal;
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
    int2 *blk;           // [B * Hkv][key blocks]: pi, c
    AttnOut dk, dv;
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
// E = RNE(2^14 2^(k / 64)), k = RNE((s - smax) f), as the float 1.5 2^23 + E.  The FMA onto
// 1.5 2^17 rounds the exact product once to a multiple of 2^-6.  There are 1024 arguments
// with a result above zero and ex2.approx rounds to the right whole number at all of them
// (the GPU tests run through every one).
__device__ __forceinline__ float attn_weight(float n_neg, float f64th) {
    const float y = __fmaf_rn(n_neg, f64th, kGridMagic) - kGridMagic;
    float z;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(z) : "f"(y));
    return __fmaf_rn(z, 16384.0f, kAttnMagic);
}

// quotient n / d as a group member: q = n / d rounded to 53 bits decides every rounding to
// 8 bits as the exact quotient does, since n < 2^48 and d < 2^31 keep an inexact quotient
// at least 2^-48 away (relatively) from every border between two mantissas
__device__ __forceinline__ int need_quot(double q) {  // q > 0
    const uint64_t b = (uint64_t)__double_as_longlong(q);
    return (int)(b >> 52) - 1023 - 6 + ((b & 0xFFFFFFFFFFFFFull) >= 0xFE00000000000ull ? 1 : 0);
}
__device__ __forceinline__ double pow2d(int k) { return __longlong_as_double((int64_t)(k + 1023) << 52); }
__device__ __forceinline__ int quot_mant(double q, int S) {  // RNE(q 2^-S), saturated
    const int v = __double2int_rn(q * pow2d(-S));
    return v > 127 ? 127 : (v < -127 ? -127 : v);
}

}  // namespace ict
