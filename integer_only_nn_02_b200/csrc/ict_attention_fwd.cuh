// ict_attention_fwd.cuh -- the attention forward on the 5th-generation tensor cores.
//
// One work item per (sequence, query head, 128 queries).  All operands are the aligned int8
// copies, staged as [128 rows][64 bytes] tiles (64-byte swizzle) by TMA:
//   pass 1   S = AQ AK^T for every tile of 128 keys (tcgen05 kind::i8 into TMEM), row maxima
//   pass 2   the same S again, E = RNE(2^14 2^(k / 64)) split into two byte planes that take
//            the place of the scores in TMEM, O_hi += E_hi AV, O_lo += E_lo AV (A operand from
//            TMEM); sum of E on the way
//   end      O = FIT((256 O_hi + O_lo) / S)
// The weights are whole numbers relative to the row's true maximum, so that the result does
// not depend on the order or the split of the work; that is why the maxima come first, and a
// second S costs less than keeping or rescaling anything: the int8 contraction of a tile takes
// 128 (64 columns) of the about 1300 cycles that its 16384 weights take on the other pipes.
// Bound by the issue slots (6 instructions a weight beside the maxima) and the exponential unit
// (16 a cycle and SM), and for short rows by an item's ends: 2 x 12 causal heads of 4096 tokens
// and 64 columns 115 us (448 TFLOP/s of the contractions that are needed), 64 x 12 heads of 197
// tokens 46 us (the rounding of the outputs and the items' starts count there).  Two blocks per SM
// for heads up to 64 columns (256 TMEM columns each), one for wider heads.
//   warps 0 .. 4 NWG - 1   softmax (thread = query row = TMEM lane; each warpgroup half the columns)
//   next warp              TMA producer;  last warp: TMEM allocation and MMA issue
// Every wait is bounded as in the Product kernels.
#pragma once

#include <type_traits>

#include "ict_attention.cuh"

namespace ict {

constexpr int kQTile = 128;
constexpr int kHalfTile = 128 * 64;  // bytes of [128 rows][64 columns]

template <int DP>
struct FwdCfg {
    static constexpr int H = DP / 64;          // 64-column halves of a head
    static constexpr int NWG = 2;
    static constexpr int TN = DP == 64 ? 64 : 128;  // keys of a pass 2 step (two score buffers of TN columns)
    static constexpr int QS = 2, KS = DP == 64 ? 3 : 2, VS = 2;  // stages of the tile rings
    static constexpr int kTile = H * kHalfTile;
    static constexpr int kOffK = QS * kTile, kOffV = kOffK + KS * kTile;
    static constexpr int kOffRed = kOffV + VS * kTile;          // [2][NWG][128] ints, [8][128] float2
    static constexpr int kOffBar = kOffRed + 2 * 2 * 128 * 4 + 8 * 128 * 8;
    static constexpr int kBars = 2 * (QS + KS + VS) + 6 + 4;
    static constexpr int kBytes = kOffBar + kBars * 8 + 16 + 1024;
    static constexpr int kTmem = DP == 64 ? 256 : 512;
    static constexpr int kO = DP == 64 ? 128 : 256;             // column of O_hi; O_lo DP columns on
    static constexpr int kThreads = 128 * NWG + 64;
};

struct AttnLimits {
    uint64_t wait_ns, drain_ns;
};

// A 31-bit or wider accumulator 256 hi + lo as a float and the error scale: |value - n| <= err 2^-22.
__device__ __forceinline__ float acc_f32(uint32_t hi, uint32_t lo, float &err) {
    const float h = (float)(int)hi, l = (float)(int)lo;
    err = fmaf(fabsf(h), 256.0f, fabsf(l));
    return fmaf(h, 256.0f, l);
}
__device__ __forceinline__ double acc_f64(uint32_t hi, uint32_t lo) {
    return (double)((int64_t)(int)hi * 256 + (int)lo);
}

// Where a row's accumulators lie: TMEM address of column 0's high plane (this warp's lanes), the
// low plane `lo` columns on; nothing there (all zero) where on = false.
struct AccCols {
    uint32_t hi;
    int lo;
    bool on;
    __device__ __forceinline__ void load16(int c, uint32_t (&h)[16], uint32_t (&l)[16]) const {
        if (on) {
            tmem_ld16(hi + c, h);
            tmem_ld16(hi + lo + c, l);
            tmem_ld_done(h, l);
        } else {
#pragma unroll
            for (int q = 0; q < 16; ++q) h[q] = l[q] = 0;
        }
    }
    __device__ __forceinline__ double exact(int c) const {  // column c as a whole number
        uint32_t h[1] = {0}, l[1] = {0};
        if (on) {
            h[0] = tmem_ld1(hi + c);
            l[0] = tmem_ld1(hi + lo + c);
            tmem_ld_done(h, l);
        }
        return acc_f64(h[0], l[0]);
    }
};

// One output group of a row: its exponent and what rounding its quotients needs.  m: the largest
// magnitude, w: the error scale (acc_f32) as floats; first: the group's first column.
struct GroupFit {
    int e;
    float sc, lim;  // 2^(r - e) mul / den; half a step less the error bound
};
__device__ __forceinline__ GroupFit group_fit(const AccCols &acc, int first, int G, float m, float w, bool some, float rd,
                                              int den, int mul, int r) {
    // the exponents that the bounds of the largest magnitude give
    const float q0 = m * rd, dq = fmaf(w, rd, q0) * 4.76837158203125e-07f;  // 2^-21
    const bool zero = !(some && w > 0);
    const int n0 = zero ? 0 : need_rel_f32(__float_as_uint(fmaxf(q0 - dq, 1.17549435e-38f)), 8);
    const int n1 = zero ? 0 : need_rel_f32(__float_as_uint(q0 + dq), 8);
    int need = n1;
    bool none = zero;
    if (__any_sync(0xffffffffu, n0 != n1)) {  // exact: the largest magnitude as a whole number
        double best = 0;
#pragma unroll 1
        for (int c = first; c < first + G; ++c) best = fmax(best, fabs(acc.exact(c)));
        none = zero || best == 0;
        if (!none) need = need_quot(best * (double)mul / (double)den);
    }
    GroupFit f;
    f.e = none ? kEZero : finalize_exp(need + r);
    f.sc = none ? 0.0f : rd * pow2f(min(max(r - f.e, -126), 100));
    // w sc 2^-20; nothing was rounded (ties included) where den is 1 and every value below 2^24
    f.lim = den == 1 && w < 16777216.0f ? 1.0f : fmaf(w * f.sc, -9.5367431640625e-07f, 0.4999999f);
    return f;
}

// 16 mantissas of a group from its accumulators as floats, stored to dst (live).
__device__ __forceinline__ void round16(const AccCols &acc, int col, const float (&n)[16], const GroupFit &f, bool some,
                                        int den, int mul, int r, bool live, int8_t *dst) {
    uint32_t v[16], near = 0;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
        const float w = fmaf(n[q], f.sc, kAttnMagic);
        const float d = fmaf(n[q], f.sc, kAttnMagic - w);  // what the rounding took away
        if (!(fabsf(d) < f.lim)) near |= 1u << q;
        v[q] = __float_as_uint(w);
    }
    uint32_t w0 = pack4b(v[0], v[1], v[2], v[3]), w1 = pack4b(v[4], v[5], v[6], v[7]);
    uint32_t w2 = pack4b(v[8], v[9], v[10], v[11]), w3 = pack4b(v[12], v[13], v[14], v[15]);
    const bool capped = f.e == 127;
    if (capped) near = 0xffff;
    uint32_t todo = __reduce_or_sync(0xffffffffu, near);
    if (todo) {
        const double rden = f.e == kEZero || !some ? 0.0 : pow2d(r - f.e) * (double)mul / (double)den;
        while (todo) {
            const int q = __ffs(todo) - 1;
            todo &= todo - 1;
            const double x = acc.exact(col + q);
            if (near >> q & 1) {
                const int y = capped ? quot_mant_capped(x, rden) : quot_mant_fast(x, rden);
                const uint32_t sh = 8 * (q & 3), keep = ~(0xffu << sh), put = (uint32_t)(y & 0xff) << sh;
                const int k = q >> 2;
                w0 = k == 0 ? (w0 & keep) | put : w0;
                w1 = k == 1 ? (w1 & keep) | put : w1;
                w2 = k == 2 ? (w2 & keep) | put : w2;
                w3 = k == 3 ? (w3 & keep) | put : w3;
            }
        }
    }
    if (live) *reinterpret_cast<uint4 *>(dst) = make_uint4(w0, w1, w2, w3);
}

// What fp32 cannot decide, out of line: the exponent of the largest magnitude; 16 mantissas of which
// some lie too close to a border.
__device__ __noinline__ int exact_need(int m, int mul, int den) { return need_quot((double)m * (double)mul / (double)den); }
__device__ __noinline__ uint4 exact_round16(const int *x, uint4 w, int e, float sc, float lim, int r, int mul, int den) {
    uint32_t near = e == 127 ? 0xffff : 0;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
        const float n = (float)x[q], k = fmaf(n, sc, kAttnMagic);
        if (!(fabsf(fmaf(n, sc, kAttnMagic - k)) < lim)) near |= 1u << q;
    }
    const double rden = pow2d(r - e) * (double)mul / (double)den;
#pragma unroll 1
    for (; near; near &= near - 1) {
        const int q = __ffs(near) - 1, k = q >> 2;
        const int y = e == 127 ? quot_mant_capped(x[q], rden) : quot_mant_fast(x[q], rden);
        const uint32_t sh = 8 * (q & 3), keep = ~(0xffu << sh), put = (uint32_t)(y & 0xff) << sh;
        w.x = k == 0 ? (w.x & keep) | put : w.x;
        w.y = k == 1 ? (w.y & keep) | put : w.y;
        w.z = k == 2 ? (w.z & keep) | put : w.z;
        w.w = k == 3 ? (w.w & keep) | put : w.w;
    }
    return w;
}

// 32 columns of a row as whole numbers (narrow accumulators), and the largest magnitude of each half.
__device__ __forceinline__ void load32(const AccCols &acc, int c, int (&x)[32], int (&m)[2]) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        uint32_t hi[16], lo[16];
        acc.load16(c + 16 * s, hi, lo);
        int top = 0, low = 0;
#pragma unroll
        for (int q = 0; q < 16; q += 2) {
            x[16 * s + q] = (int)hi[q] * 256 + (int)lo[q];
            x[16 * s + q + 1] = (int)hi[q + 1] * 256 + (int)lo[q + 1];
            top = __vimax3_s32(top, x[16 * s + q], x[16 * s + q + 1]);
            low = __vimin3_s32(low, x[16 * s + q], x[16 * s + q + 1]);
        }
        m[s] = max(top, -low);
    }
}
// Exponent, factor and border of a group whose largest magnitude is mi.
__device__ __forceinline__ GroupFit group_fit_narrow(int mi, bool some, float rd, int den, int mul, int r) {
    GroupFit f;
    // four roundings: the magnitude, the divisor, the factor, the product
    const float w = (float)mi, q0 = w * rd, dq = q0 * 4.76837158203125e-07f;  // 2^-21
    const bool zero = !some || mi == 0;
    const int n0 = zero ? 0 : need_rel_f32(__float_as_uint(fmaxf(q0 - dq, 1.17549435e-38f)), 8);
    int need = zero ? 0 : need_rel_f32(__float_as_uint(q0 + dq), 8);
    if (n0 != need) need = exact_need(mi, mul, den);
    f.e = zero ? kEZero : finalize_exp(need + r);
    f.sc = zero ? 0.0f : rd * pow2f(min(max(r - f.e, -126), 100));
    // three roundings: w sc 2^-22; none at all (ties included) where den is 1 and every value below 2^24
    f.lim = den == 1 && mi < (1 << 24) ? 1.0f : fmaf(w * f.sc, -2.38418579e-07f, 0.4999999f);
    return f;
}
// 16 mantissas x mul / den 2^(r - e).
__device__ __forceinline__ uint4 round16_narrow(const int *x, const GroupFit &f, int r, int mul, int den) {
    const f2 M = pk(kAttnMagic), scp = pk(f.sc);
    uint32_t v[16];
    float far = 0;  // from a whole number
#pragma unroll
    for (int q = 0; q < 16; q += 2) {
        const f2 n = pk((float)x[q], (float)x[q + 1]), w = fma2(n, scp, M);
        float w0, w1, d0, d1;
        unpk(w, w0, w1);
        unpk(fma2(n, scp, sub2(M, w)), d0, d1);  // what the rounding took away
        far = fmaxf(far, fmaxf(fabsf(d0), fabsf(d1)));
        v[q] = __float_as_uint(w0), v[q + 1] = __float_as_uint(w1);
    }
    uint4 w = make_uint4(pack4b(v[0], v[1], v[2], v[3]), pack4b(v[4], v[5], v[6], v[7]), pack4b(v[8], v[9], v[10], v[11]),
                         pack4b(v[12], v[13], v[14], v[15]));
    if (!(far < f.lim) || f.e == 127) {
        int y[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) y[q] = x[q];
        w = exact_round16(y, w, f.e, f.sc, f.lim, r, mul, den);
    }
    return w;
}

// FIT of 16 SEGS columns of narrow accumulators, 32 columns at a time in registers.  Groups of one or
// two segments lie inside them; the maxima of others meet in gi (shared memory, [segment][stride]),
// and with more than 32 columns the accumulators are read twice.  They are free for the next item
// once the last of them are read.
template <int SEGS>
__device__ __forceinline__ void fit_row_narrow(const AttnArgs &a, int8_t *dst, int8_t *oe, int c0, int gs, int den, int mul,
                                               int r, bool live, bool some, float rd, int *gi, int stride, int bar,
                                               int nthreads, const AccCols &acc, uint32_t release) {
    static_assert(SEGS % 2 == 0, "32 columns at a time");
    const bool meet = gs > 2;
    int x[32], m[2];
    if (meet) {
#pragma unroll 1
        for (int h = 0; h < SEGS; h += 2) {
            load32(acc, c0 + 16 * h, x, m);
            gi[(c0 / 16 + h) * stride] = m[0];
            gi[(c0 / 16 + h + 1) * stride] = m[1];
        }
        if (SEGS == 2 && release) warp_arrive(release);
        named_bar_sync(bar, nthreads);
    }
#pragma unroll 1
    for (int h = 0; h < SEGS; h += 2) {
        const int c = c0 + 16 * h;
        if (!meet || SEGS > 2) {
            load32(acc, c, x, m);
            if (release && h + 2 >= SEGS) warp_arrive(release);
        }
        GroupFit f{kEZero, 0.0f, 0.5f};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int seg = c / 16 + s;
            if (16 * seg >= a.D) break;
            int mi = gs == 1 ? m[s] : max(m[0], m[1]), g = seg >> (gs - 1);
            bool first = s == 0 || gs == 1, writes = first;
            if (meet) {
                g = seg / gs;
                writes = seg == g * gs;
                first = s == 0 || writes;
                if (first) {
                    mi = 0;
                    for (int k = g * gs; k < (g + 1) * gs; ++k) mi = max(mi, gi[k * stride]);
                }
            }
            if (first) {
                f = group_fit_narrow(mi, some, rd, den, mul, r);
                if (live && writes) oe[g] = (int8_t)f.e;
            }
            const uint4 w = round16_narrow(x + 16 * s, f, r, mul, den);
            if (live) *reinterpret_cast<uint4 *>(dst + 16 * seg) = w;
        }
    }
}

// FIT of one row's accumulators (this thread's TMEM lane): quotients (256 hi + lo) mul / den at
// exponent r, SEGS segments of 16 columns from column c0 of head h; then they are released.
// Magnitudes and mantissas are computed in fp32 with an error bound; what lies within the bound
// of a border between two results (a mantissa in some ten thousand) is decided in fp64, where
// the quotient's rounding to 53 bits cannot hide the border.  narrow: the accumulators
// 256 hi + lo fit 32 bits (gi: see above).  Otherwise the threads that share the row join their
// segments' maxima in gmax (shared memory, [segment][stride]) and read the accumulators twice.
struct RowOut {  // what is known of a row before its accumulators are complete
    int8_t *dst, *oe;
    float rd;
    int den, mul;
    bool live, some;
};
__device__ __forceinline__ RowOut row_out(const AttnArgs &a, const AttnOut &out, int64_t row, int h, int den, int mul, bool live) {
    RowOut o;
    o.dst = out.mant + row * out.ld + out.col + h * a.D;
    o.oe = out.exp + row * out.ngc + out.gcol + h * out.dg;
    o.den = den, o.mul = mul, o.live = live, o.some = live && den != 0;
    // relative error below 2^-22 (two roundings); a quotient's, accumulator included, below err 2^-21
    o.rd = o.some ? __fdiv_rn((float)mul, (float)den) : 0.0f;
    return o;
}
template <int SEGS>
__device__ __forceinline__ void fit_row_tmem(const AttnArgs &a, const AttnOut &out, const RowOut &o, int c0, int r, bool narrow,
                                             float2 *gmax, int *gi, int stride, int bar, int nthreads, const AccCols &acc,
                                             uint32_t release) {
    const int gs = out.G / 16;  // segments of a group
    const float rd = o.rd;
    const int den = o.den, mul = o.mul;
    const bool live = o.live, some = o.some;
    int8_t *dst = o.dst, *oe = o.oe;
    if (narrow) {
        fit_row_narrow<SEGS>(a, dst, oe, c0, gs, den, mul, r, live, some, rd, gi, stride, bar, nthreads, acc, release);
        return;
    }
#pragma unroll 1
    for (int s = 0; s < SEGS; ++s) {
        uint32_t hi[16], lo[16];
        acc.load16(c0 + 16 * s, hi, lo);
        float m = 0, w = 0;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            float e;
            m = fmaxf(m, fabsf(acc_f32(hi[q], lo[q], e)));
            w = fmaxf(w, e);
        }
        gmax[(c0 / 16 + s) * stride] = make_float2(m, w);
    }
    named_bar_sync(bar, nthreads);
    tc_fence_after();  // group_fit reads the other warpgroups' columns, which join_parts may have written
    GroupFit f{kEZero, 0.0f, 0.5f};
#pragma unroll 1
    for (int s = 0; s < SEGS; ++s) {
        const int seg = c0 / 16 + s;
        if (seg * 16 >= a.D) break;
        if (s == 0 || seg % gs == 0) {
            const int g = seg / gs;
            float m = 0, w = 0;
            for (int k = g * gs; k < (g + 1) * gs; ++k) {
                const float2 v = gmax[k * stride];
                m = fmaxf(m, v.x);
                w = fmaxf(w, v.y);
            }
            f = group_fit(acc, g * out.G, out.G, m, w, some, rd, den, mul, r);
            if (live && seg % gs == 0) oe[g] = (int8_t)f.e;
        }
        uint32_t hi[16], lo[16];
        float n[16];
        acc.load16(seg * 16, hi, lo);
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            float er;
            n[q] = acc_f32(hi[q], lo[q], er);
        }
        round16(acc, seg * 16, n, f, some, den, mul, r, live, dst + seg * 16);
    }
    if (release) warp_arrive(release);
}

// 32 scores of a row to the two byte planes of their weights; PART: only the first `vis`
// columns are visible.  sum collects the bit patterns (1.5 2^23 + E each, mod 2^32).
template <bool PART>
__device__ __forceinline__ void weights32(const uint32_t (&v)[32], f2 nm, f2 f, int vis, uint32_t &sum,
                                          uint32_t (&lo)[8], uint32_t (&hi)[8]) {
    uint32_t s0 = 0, s1 = 0;
#pragma unroll
    for (int q = 0; q < 32; q += 4) {
        float w[4];
        unpk(attn_weight2f(v[q], v[q + 1], nm, f), w[0], w[1]);
        unpk(attn_weight2f(v[q + 2], v[q + 3], nm, f), w[2], w[3]);
        if (PART) {
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = q + k < vis ? w[k] : kAttnMagic;
        }
        s0 += __float_as_uint(w[0]) + __float_as_uint(w[1]);
        s1 += __float_as_uint(w[2]) + __float_as_uint(w[3]);
        split_bytes(w[0], w[1], w[2], w[3], lo[q >> 2], hi[q >> 2]);
    }
    sum += s0 + s1;
}

// One work item: a tile of queries of one head.  Heavy causal tiles come first.
struct AttnItem {
    int b, h, g, bh, i0, nq, nk, most, nt;
};
__device__ __forceinline__ AttnItem attn_item(const AttnArgs &a, int item) {
    AttnItem w;
    const int t = a.heads_q(item), tile = (a.Lq + kQTile - 1) / kQTile - 1 - t;
    w.bh = item - t * a.B * a.Hq;
    w.b = a.hq(w.bh);
    w.h = w.bh - w.b * a.Hq;
    w.g = a.by_rep(w.h);
    w.i0 = tile * kQTile;
    w.nq = clamp_len(a.op[OPQ].lens, w.b, a.Lq);
    w.nk = clamp_len(a.op[OPK].lens, w.b, a.Lk);
    const int last = min(w.nq, w.i0 + kQTile) - 1;
    w.most = last < w.i0 ? 0 : (a.causal ? max(0, min(w.nk, last + w.nk - w.nq + 1)) : w.nk);  // keys any query sees
    w.nt = (w.most + 127) / 128;
    return w;
}

// Persistent blocks: the next item's tiles are loaded and its first scores issued while the
// softmax warps still write the last item's output.
template <int DP>
__global__ void __launch_bounds__(FwdCfg<DP>::kThreads, DP == 64 ? 2 : 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ AttnArgs a,
                    const __grid_constant__ AttnLimits lim, int items) {
    using L = FwdCfg<DP>;
    // CW2: a softmax thread's columns of a TN-key step
    constexpr int H = L::H, NWG = L::NWG, CW2 = L::TN / NWG, NS = 128 * NWG;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t sb = smem_u32(smem);
    const uint32_t bar_qf = sb + L::kOffBar, bar_qe = bar_qf + 8 * L::QS;  // Q tile full / empty
    const uint32_t bar_kf = bar_qe + 8 * L::QS, bar_ke = bar_kf + 8 * L::KS;
    const uint32_t bar_vf = bar_ke + 8 * L::KS, bar_ve = bar_vf + 8 * L::VS;
    const uint32_t bar_sf = bar_ve + 8 * L::VS, bar_se = bar_sf + 16;  // scores full / read
    // weights written (a barrier per score buffer: the softmax may be two steps ahead of the MMA
    // warp's wait), weights used
    const uint32_t bar_ef = bar_se + 16, bar_ee = bar_ef + 16;
    const uint32_t bar_of = bar_ee + 8, bar_oe = bar_of + 8, bar_dr = bar_oe + 8;  // output complete / read, drain
    volatile int *misc = (volatile int *)(smem + L::kOffBar + L::kBars * 8);
    volatile int *abort_flag = &misc[1];
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 128 * NWG) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        for (int s = 0; s < L::QS; ++s) mbar_init(bar_qf + 8 * s, 1), mbar_init(bar_qe + 8 * s, 1);
        for (int s = 0; s < L::KS; ++s) mbar_init(bar_kf + 8 * s, 1), mbar_init(bar_ke + 8 * s, 1);
        for (int s = 0; s < L::VS; ++s) mbar_init(bar_vf + 8 * s, 1), mbar_init(bar_ve + 8 * s, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar_sf + 8 * s, 1);
            mbar_init(bar_se + 8 * s, NS / 64);
            mbar_init(bar_ef + 8 * s, NS / 32);
        }
        mbar_init(bar_ee, 1);
        mbar_init(bar_of, 1);
        mbar_init(bar_oe, NS / 32);
        mbar_init(bar_dr, 1);
        misc[1] = 0;
        fence_barrier_init();
    }
    __syncthreads();
    auto fail = [&]() {
        *abort_flag = 1;
        raise_status(ICT_ERR_DEVICE_TIMEOUT);
    };

    if (warp == 4 * NWG) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            auto load_tile = [&](const CUtensorMap *m, uint32_t dst, uint32_t bar, int row) {
                mbar_expect_tx(bar, L::kTile);
                for (int x = 0; x < H; ++x) tma_load_2d(dst + x * kHalfTile, m, bar, 64 * x, row);
            };
            auto free = [&](uint32_t bar, int n, int stages) {  // the n-th use of a ring's stage
                return n < stages || wait_bar(bar + 8 * (n % stages), (n / stages - 1) & 1, lim.wait_ns, abort_flag);
            };
            bool ok = true;
            int qn = 0, kn = 0, vn = 0;  // tiles issued so far
            for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
                const AttnItem w = attn_item(a, item);
                if (w.nt == 0) continue;
                if (!(ok = free(bar_qe, qn, L::QS))) break;
                load_tile(&tmQ, sb + (qn % L::QS) * L::kTile, bar_qf + 8 * (qn % L::QS), w.bh * a.Lq + w.i0);
                ++qn;
                const int krow = (w.b * a.Hkv + w.g) * a.Lk;
                for (int u = 0; u < 2 * w.nt; ++u) {
                    const int t = u < w.nt ? u : u - w.nt;
                    if (!(ok = free(bar_ke, kn, L::KS))) break;
                    load_tile(&tmK, sb + L::kOffK + (kn % L::KS) * L::kTile, bar_kf + 8 * (kn % L::KS), krow + t * 128);
                    ++kn;
                    if (u < w.nt) continue;
                    if (!(ok = free(bar_ve, vn, L::VS))) break;
                    load_tile(&tmV, sb + L::kOffV + (vn % L::VS) * L::kTile, bar_vf + 8 * (vn % L::VS), krow + t * 128);
                    ++vn;
                }
            }
            if (!ok) fail();
            // every copy lands before the block may end
            for (int k = max(0, qn - L::QS); k < qn; ++k)
                wait_bar(bar_qf + 8 * (k % L::QS), (k / L::QS) & 1, lim.drain_ns, nullptr);
            for (int k = max(0, kn - L::KS); k < kn; ++k)
                wait_bar(bar_kf + 8 * (k % L::KS), (k / L::KS) & 1, lim.drain_ns, nullptr);
            for (int k = max(0, vn - L::VS); k < vn; ++k)
                wait_bar(bar_vf + 8 * (k % L::VS), (k / L::VS) & 1, lim.drain_ns, nullptr);
        }
    } else if (warp == 4 * NWG + 1) {
        // ------------------------------------------------------------ TMEM and MMA issue
        tmem_alloc(smem_u32((const void *)&misc[0]), L::kTmem);
        tmem_relinquish();
        tc_fence_before();
        named_bar_sync(2, NS + 32);
        tc_fence_after();
        const uint32_t tm = __shfl_sync(0xffffffffu, (uint32_t)misc[0], 0);
        // the whole warp runs this loop, one elected lane issues
        constexpr uint32_t kIdO = idesc_i8(128, DP, false, true) & ~(1u << 7);  // unsigned A
        constexpr int PER = 128 / L::TN;  // steps of a K or V tile
        auto wait = [&](uint32_t bar, int parity) {
            return (bool)__all_sync(0xffffffffu, wait_bar(bar, (uint32_t)(parity & 1), lim.wait_ns, abort_flag));
        };
        bool ok = true;
        // uses so far: Q, K and V tiles, weights, outputs; and as bits (one per score buffer) the
        // parities of the next phase of pass 1's reads and of the written weights
        int qn = 0, kn = 0, vn = 0, pn = 0, on = 0;
        uint32_t rd_par = 0, ef_par = 0;
        for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
            const AttnItem w = attn_item(a, item);
            if (w.nt == 0) continue;
            const uint32_t qt = sb + (qn % L::QS) * L::kTile;
            if (!(ok = wait(bar_qf + 8 * (qn % L::QS), qn / L::QS))) break;
            const int nu = (w.most + L::TN - 1) / L::TN;
            // S of N keys from row `half` * N of the next K tile into score buffer buf at column col
            auto scores = [&](auto n_keys, int buf, int col, int half, bool done, bool last) {
                constexpr int N = decltype(n_keys)::value;
                const int s = kn % L::KS;
                if (half == 0 && !wait(bar_kf + 8 * s, kn / L::KS)) return false;
                tc_fence_after();
                const uint32_t kb = sb + L::kOffK + s * L::kTile + half * N * 64;
                const uint64_t da = smem_desc_kmajor(qt, 64), db = smem_desc_kmajor(kb, 64);
                if (elect_one()) {
#pragma unroll
                    for (int x = 0; x < 2 * H; ++x)
                        umma_i8(tm + col, da + (x >> 1) * (kHalfTile >> 4) + 2 * (x & 1),
                                db + (x >> 1) * (kHalfTile >> 4) + 2 * (x & 1), idesc_i8(128, N), x ? 1u : 0u);
                    if (done) umma_commit(bar_ke + 8 * s);
                    if (last) umma_commit(bar_qe + 8 * (qn % L::QS));
                    umma_commit(bar_sf + 8 * buf);
                }
                __syncwarp();
                if (done) ++kn;
                return true;
            };
            constexpr auto n128 = std::integral_constant<int, 128>();
            constexpr auto nTN = std::integral_constant<int, L::TN>();
            // the last item's weights lie in both buffers' columns, its output in the second's (64 columns)
            if (pn > 0 && !(ok = wait(bar_ee, pn - 1))) break;
            for (int t = 0; t < w.nt && ok; ++t) {
                const int buf = t & 1;  // free once pass 1 has read its last scores
                if (t == 1 && DP == 64 && on > 0) ok = wait(bar_oe, on - 1);
                if (t >= 2) ok = ok && wait(bar_se + 8 * buf, (rd_par >> buf ^ 1) & 1);
                ok = ok && scores(n128, buf, buf * 128, 0, true, false);
                rd_par ^= 1u << buf;
            }
            // both of pass 2's 64-wide buffers lie in pass 1's first one
            if (ok) ok = wait(bar_se, (rd_par ^ 1) & 1) && scores(nTN, 0, 0, 0, PER == 1 || nu == 1, nu == 1);
            // the output's columns are free
            if (ok && on > 0 && !(DP == 64 && w.nt > 1)) ok = wait(bar_oe, on - 1);
            for (int u = 0; u < nu && ok; ++u) {
                // one product is open at a time, the last two of an item included: of two open phases a parity
                // cannot tell the first from the second, and the next item's scores would be issued into
                // weights that a product still reads
                if (u > 0 && !(ok = wait(bar_ee, pn - 1))) break;
                if (u + 1 < nu) {  // the next scores, in the buffer of the weights u - 1
                    // before its barrier completes another phase, every warp has seen pass 1's last
                    if (u == 0 && w.nt > 1) ok = wait(bar_se + 8, (rd_par >> 1 ^ 1) & 1);
                    const int half = (u + 1) % PER;
                    if (!ok || !(ok = scores(nTN, (u + 1) & 1, ((u + 1) & 1) * L::TN, half, half == PER - 1 || u + 2 == nu,
                                             u + 2 == nu)))
                        break;
                }
                const int v = vn % L::VS;
                ok = (u % PER != 0 || wait(bar_vf + 8 * v, vn / L::VS)) && wait(bar_ef + 8 * (u & 1), (ef_par >> (u & 1)) & 1);
                if (!ok) break;
                ef_par ^= 1u << (u & 1);
                tc_fence_after();
                const int ks = (min(L::TN, w.most - u * L::TN) + 31) / 32;
                const uint64_t dv = smem_desc_mnmajor64(sb + L::kOffV + v * L::kTile + (u % PER) * L::TN * 64, kHalfTile);
                const uint32_t e0 = tm + (u & 1) * L::TN, first = u ? 1u : 0u;
                const bool done = u % PER == PER - 1 || u + 1 == nu;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < L::TN / 32; ++kk)
                        if (kk < ks) {
                            const uint32_t e = e0 + kk * 32;
                            umma_i8_ta(tm + L::kO, e, dv + 128 * kk, kIdO, kk ? 1u : first);
                            umma_i8_ta(tm + L::kO + DP, e + 8, dv + 128 * kk, kIdO, kk ? 1u : first);
                        }
                    if (done) umma_commit(bar_ve + 8 * v);
                    umma_commit(bar_ee);
                    if (u + 1 == nu) umma_commit(bar_of);
                }
                __syncwarp();
                ++pn;
                if (done) ++vn;
            }
            ++qn;
            ++on;
        }
        if (!ok && lane == 0) fail();
        if (elect_one()) umma_commit(bar_dr);
        __syncwarp();
        wait_bar(bar_dr, 0, lim.drain_ns, nullptr);
    } else {
        // ------------------------------------------------------------ softmax
        named_bar_sync(2, NS + 32);
        tc_fence_after();
        const uint32_t tm = (uint32_t)misc[0];
        const int wg = warp >> 2, et = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        int *red = (int *)(smem + L::kOffRed);
        int on = 0;
        uint32_t sf_par = 0;  // parity of the next phase of each score buffer, as bits
        bool ok = true;
        auto full = [&](int buf) {
            ok = __all_sync(0xffffffffu, wait_bar(bar_sf + 8 * buf, (sf_par >> buf) & 1, lim.wait_ns, abort_flag));
            sf_par ^= 1u << buf;
            tc_fence_after();
            return ok;
        };
        for (int item = blockIdx.x; item < items; item += gridDim.x) {  // (outputs are written after a failure too)
            const AttnItem w = attn_item(a, item);
            const int i = w.i0 + et;
            const int see = i >= w.nq ? 0 : (a.causal ? max(0, min(w.nk, i + w.nk - w.nq + 1)) : w.nk);
            const int see_max = warp_max(see), see_min = -warp_max(-see);
            // pass 1: each warpgroup takes the tiles of one buffer
            int mx = INT_MIN;
            for (int t = wg; t < w.nt && ok; t += 2) {
                ok = __all_sync(0xffffffffu, wait_bar(bar_sf + 8 * wg, ((sf_par >> wg) + (t >> 1)) & 1, lim.wait_ns, abort_flag));
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < 128; c += 64) {
                    const int col = t * 128 + c;
                    if (col >= see_max) break;
                    uint32_t v[64];
                    tmem_ld64(tm + lanes + wg * 128 + c, v);
                    tmem_ld_wait(v);
                    if (col + 64 > see_min) {
#pragma unroll
                        for (int q = 0; q < 64; ++q) v[q] = col + q < see ? v[q] : 0x80000000u;
                    }
                    int m0 = mx, m1 = (int)v[0];
#pragma unroll
                    for (int q = 0; q < 64; q += 4) {
                        m0 = __vimax3_s32(m0, (int)v[q], (int)v[q + 1]);
                        m1 = __vimax3_s32(m1, (int)v[q + 2], (int)v[q + 3]);
                    }
                    mx = max(m0, m1);
                }
                warp_arrive(bar_se + 8 * wg);
            }
            sf_par ^= (uint32_t)(((w.nt + 1) >> 1 & 1) | (w.nt >> 1 & 1) << 1);
            red[wg * 128 + et] = mx;
            named_bar_sync(1, NS);
            mx = max(mx, red[(wg ^ 1) * 128 + et]);
            if (see == 0) mx = 0;
            const f2 nm = pk(-(kAttnMagic + (float)mx));
            const f2 f = pk(attn_factor(a, w.b * a.Hkv + w.g));
            uint32_t sum = 0;
            int n_sum = 0;
            const int nu = (w.most + L::TN - 1) / L::TN;
            for (int u = 0; u < nu && ok; ++u) {
                const int buf = u & 1;
                if (!full(buf)) break;
                const int end = min(L::TN, w.most - u * L::TN);  // columns that the MMAs read
                const uint32_t mine = tm + lanes + buf * L::TN + wg * CW2;
#pragma unroll 1
                for (int c = 0; c < CW2; c += 32) {
                    const int cc = wg * CW2 + c, col = u * L::TN + cc;
                    if (cc >= end) break;
                    uint32_t lo[8], hi[8];
                    if (col < see_max) {
                        uint32_t v[32];
                        tmem_ld32(mine + c, v);
                        tmem_ld_done(v);
                        if (col + 32 <= see_min) weights32<false>(v, nm, f, 0, sum, lo, hi);
                        else weights32<true>(v, nm, f, see - col, sum, lo, hi);
                        n_sum += 32;
                    } else {
#pragma unroll
                        for (int q = 0; q < 8; ++q) lo[q] = hi[q] = 0;
                    }
                    tmem_st8(mine + c, hi);  // in the place of the scores just read
                    tmem_st8(mine + c + 8, lo);
                }
                tmem_st_wait();
                warp_arrive(bar_ef + 8 * buf);
            }
            sum -= (uint32_t)n_sum * 0x4B400000u;
            red[256 + wg * 128 + et] = (int)sum;
            named_bar_sync(1, NS);
            sum += (uint32_t)red[256 + (wg ^ 1) * 128 + et];
            const bool live = i < a.Lq;
            const RowOut row = row_out(a, a.o, (int64_t)w.b * a.Lq + i, w.h, w.nt > 0 ? (int)sum : 0, 1, live);
            const int top_v = attn_top(a, OPV, w.b * a.Hkv + w.g);
            if (w.nt > 0 && ok) {
                ok = __all_sync(0xffffffffu, wait_bar(bar_of, on & 1, lim.wait_ns, abort_flag));
                tc_fence_after();
            }
            const bool read = w.nt > 0 && ok;
            if (live && wg == 0) a.stats[(int64_t)w.bh * a.Lq + i] = make_int2(mx, (int)sum);
            // outputs: columns [wg DP / NWG, ...) of the head; every thread takes part in the barriers
            const int c0 = wg * (DP / NWG);
            float2 *gm = (float2 *)(smem + L::kOffRed + 2048) + et;
            fit_row_tmem<DP / NWG / 16>(a, a.o, row, c0, top_v, w.nk <= 1024, gm, (int *)(gm - et) + et, 128, 1, NS,
                                        AccCols{tm + lanes + L::kO, DP, read}, w.nt > 0 ? bar_oe : 0);
            if (w.nt > 0) ++on;
        }
        if (!ok && lane == 0) fail();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4 * NWG + 1) tmem_dealloc(__shfl_sync(0xffffffffu, (uint32_t)misc[0], 0), L::kTmem);
}

}  // namespace ict
