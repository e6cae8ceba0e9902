// ict_attention_fwd.cuh -- the attention forward on the 5th-generation tensor cores.
//
// One block per (sequence, query head, 128 queries).  All operands are the aligned int8
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
// Bound by the exponential unit (16 a cycle and SM) and the issue slots (6 instructions a
// weight).  Two blocks per SM for heads up to 64 columns (256 TMEM columns each); one block with
// two softmax warpgroups, each half a tile's columns, for wider heads.
//   warps 0 .. 4 NWG - 1   softmax (thread = query row = TMEM lane)
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
    static constexpr int KS = DP == 64 ? 3 : 2, VS = 2;
    static constexpr int kTile = H * kHalfTile;
    static constexpr int kOffK = kTile, kOffV = kOffK + KS * kTile;
    static constexpr int kOffRed = kOffV + VS * kTile;          // [2][NWG][128] ints, [8][128] float2
    static constexpr int kOffBar = kOffRed + 2 * 2 * 128 * 4 + 8 * 128 * 8;
    static constexpr int kBars = 1 + 2 * KS + 2 * VS + 4 + 3 + 2;
    static constexpr int kBytes = kOffBar + kBars * 8 + 16 + 1024;
    static constexpr int kTmem = DP == 64 ? 256 : 512;
    static constexpr int kO = DP == 64 ? 128 : 256;             // column of O_hi; O_lo DP columns on
    static constexpr int kThreads = 128 * NWG + 64;
};

struct AttnLimits {
    uint64_t wait_ns, drain_ns;
};

// A 31-bit or wider accumulator 256 hi + lo as a float and the error scale: |value - n| <= err 2^-22.
__device__ __forceinline__ float acc_f32(uint32_t hi, uint32_t lo, bool narrow, float &err) {
    if (narrow) {
        const float n = (float)((int)hi * 256 + (int)lo);
        err = fabsf(n);
        return n;
    }
    const float h = (float)(int)hi, l = (float)(int)lo;
    err = fmaf(fabsf(h), 256.0f, fabsf(l));
    return fmaf(h, 256.0f, l);
}
__device__ __forceinline__ double acc_f64(uint32_t hi, uint32_t lo) {
    return (double)((int64_t)(int)hi * 256 + (int)lo);
}

// FIT of one row's accumulators (this thread's TMEM lane): quotients (256 hi + lo) mul / den at
// exponent r, SEGS segments of 16 columns from column c0 of head h.  Two threads share a row;
// gmax (shared memory, [segment][stride], two floats each) joins their segments' maxima.
// Magnitudes and mantissas are computed in fp32 with an error bound; a warp in which any
// group exponent or mantissa lies within the bound of a border between two results decides
// that segment in fp64, where the quotient's rounding to 53 bits cannot hide the border.
template <int SEGS, typename Load>
__device__ __forceinline__ void fit_row_tmem(const AttnArgs &a, const AttnOut &out, int64_t row, int h, int c0, int den,
                                             int mul, int r, bool live, bool narrow, float2 *gmax, int stride, int bar,
                                             int nthreads, const Load &load) {
    const int col = out.col + h * a.D;
#pragma unroll
    for (int s = 0; s < SEGS; ++s) {
        uint32_t hi[16], lo[16];
        load(s, hi, lo);
        float m = 0, w = 0;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            float e;
            m = fmaxf(m, fabsf(acc_f32(hi[q], lo[q], narrow, e)));
            w = fmaxf(w, e);
        }
        gmax[(c0 / 16 + s) * stride] = make_float2(m, w);
    }
    named_bar_sync(bar, nthreads);
    const int gs = out.G / 16;  // segments of a group
    const bool some = live && den != 0;
    // relative error below 2^-22 (two roundings); a quotient's, accumulator included, below err 2^-21
    const float rd = some ? __fdiv_rn((float)mul, (float)den) : 0.0f;
    int e = kEZero;
    float sc = 0;
#pragma unroll
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
            // the exponents that the bounds of the largest magnitude give
            const float q0 = m * rd, dq = fmaf(w, rd, q0) * 4.76837158203125e-07f;  // 2^-21
            const bool zero = !(some && w > 0);
            const int n0 = zero ? 0 : need_rel_f32(__float_as_uint(fmaxf(q0 - dq, 1.17549435e-38f)), 8);
            const int n1 = zero ? 0 : need_rel_f32(__float_as_uint(q0 + dq), 8);
            int need = n1;
            bool none = zero;
            if (__any_sync(0xffffffffu, n0 != n1)) {
                // exact: the largest magnitude as a whole number, from this thread's and the other's columns
                double best = 0;
                for (int k = g * gs; k < (g + 1) * gs; ++k) {
                    uint32_t hi[16], lo[16];
                    load(k - c0 / 16, hi, lo);
#pragma unroll
                    for (int q = 0; q < 16; ++q) best = fmax(best, fabs(acc_f64(hi[q], lo[q])));
                }
                none = zero || best == 0;
                if (!none) need = need_quot(best * (double)mul / (double)den);
            }
            e = none ? kEZero : finalize_exp(need + r);
            sc = none ? 0.0f : rd * pow2f(min(max(r - e, -126), 100));
            if (live && seg % gs == 0) out.exp[row * out.ngc + col / out.G + g] = (int8_t)e;
        }
        uint32_t hi[16], lo[16], v[16];
        load(s, hi, lo);
        bool near = false;
        const bool capped = e == 127;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            float er;
            const float n = acc_f32(hi[q], lo[q], narrow, er);
            const float w = fmaf(n, sc, kAttnMagic);
            const float d = fmaf(n, sc, kAttnMagic - w);  // what the rounding took away
            near |= fabsf(d) >= fmaf(er * sc, -9.5367431640625e-07f, 0.4999999f);  // 2^-20
            v[q] = __float_as_uint(w);
        }
        if (__any_sync(0xffffffffu, near || capped)) {
            const double rden = e == kEZero ? 0.0 : pow2d(r - e) * (double)mul / (double)den;
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                const double n = acc_f64(hi[q], lo[q]);
                v[q] = (uint32_t)(capped ? (int)fmin(fmax(n * rden, -127.0), 127.0) : quot_mant_fast(n, rden));
            }
        }
        if (live)
            *reinterpret_cast<uint4 *>(out.mant + row * out.ld + col + seg * 16) =
                make_uint4(pack4b(v[0], v[1], v[2], v[3]), pack4b(v[4], v[5], v[6], v[7]),
                           pack4b(v[8], v[9], v[10], v[11]), pack4b(v[12], v[13], v[14], v[15]));
    }
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

template <int DP>
__global__ void __launch_bounds__(FwdCfg<DP>::kThreads, DP == 64 ? 2 : 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ AttnArgs a,
                    const __grid_constant__ AttnLimits lim) {
    using L = FwdCfg<DP>;
    // a softmax thread's columns of a 128-key tile (pass 1) and of a TN-key step (pass 2)
    constexpr int H = L::H, NWG = L::NWG, CW = 128 / NWG, CW2 = L::TN / NWG, NS = 128 * NWG;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t sb = smem_u32(smem);
    const uint32_t bar_q = sb + L::kOffBar;
    const uint32_t bar_kf = bar_q + 8, bar_ke = bar_kf + 8 * L::KS;    // K tile full / empty
    const uint32_t bar_vf = bar_ke + 8 * L::KS, bar_ve = bar_vf + 8 * L::VS;
    const uint32_t bar_sf = bar_ve + 8 * L::VS, bar_se = bar_sf + 16;  // scores full / read
    // weights written (a barrier per score buffer: with two of them the softmax may be two tiles
    // ahead of the MMA thread's wait), weights used
    const uint32_t bar_ef = bar_se + 16, bar_ee = bar_ef + 16;
    const uint32_t bar_of = bar_ee + 8, bar_dr = bar_of + 8;           // output complete, drain
    volatile int *misc = (volatile int *)(smem + L::kOffBar + L::kBars * 8);
    volatile int *abort_flag = &misc[1];
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    // heavy causal tiles first
    const int ntq = (a.Lq + kQTile - 1) / kQTile, heads = a.B * a.Hq;
    const int tile = ntq - 1 - (int)blockIdx.x / heads, bh = (int)blockIdx.x % heads;
    const int b = bh / a.Hq, h = bh % a.Hq, g = h / a.rep, i0 = tile * kQTile;
    const int nq = clamp_len(a.op[OPQ].lens, b, a.Lq), nk = clamp_len(a.op[OPK].lens, b, a.Lk);
    const int last = min(nq, i0 + kQTile) - 1;
    const int most = last < i0 ? 0 : (a.causal ? max(0, min(nk, last + nk - nq + 1)) : nk);
    const int nt = (most + 127) / 128;  // key tiles

    const int qrow = bh * a.Lq + i0, krow = (b * a.Hkv + g) * a.Lk;
    auto load_tile = [&](const CUtensorMap *m, uint32_t dst, uint32_t bar, int row) {
        mbar_expect_tx(bar, L::kTile);
        for (int x = 0; x < H; ++x) tma_load_2d(dst + x * kHalfTile, m, bar, 64 * x, row);
    };
    if (threadIdx.x == 128 * NWG) {  // the producer starts loading before the block meets
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        mbar_init(bar_q, 1);
        for (int s = 0; s < L::KS; ++s) mbar_init(bar_kf + 8 * s, 1), mbar_init(bar_ke + 8 * s, 1);
        for (int s = 0; s < L::VS; ++s) mbar_init(bar_vf + 8 * s, 1), mbar_init(bar_ve + 8 * s, 1);
        for (int s = 0; s < 2; ++s) mbar_init(bar_sf + 8 * s, 1), mbar_init(bar_se + 8 * s, NS / 32);
        for (int s = 0; s < 2; ++s) mbar_init(bar_ef + 8 * s, NS / 32);
        mbar_init(bar_ee, 1);
        mbar_init(bar_of, 1);
        mbar_init(bar_dr, 1);
        misc[1] = 0;
        fence_barrier_init();
        if (nt > 0) load_tile(&tmQ, sb, bar_q, qrow);
        for (int k = 0; k < min(L::KS, 2 * nt); ++k)
            load_tile(&tmK, sb + L::kOffK + k * L::kTile, bar_kf + 8 * k, krow + (k % nt) * 128);
    }
    if (warp == 4 * NWG + 1) {
        tmem_alloc(smem_u32((const void *)&misc[0]), L::kTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, (uint32_t)misc[0], 0);
    auto fail = [&]() {
        *abort_flag = 1;
        raise_status(ICT_ERR_DEVICE_TIMEOUT);
    };

    if (warp == 4 * NWG) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0 && nt > 0) {
            bool ok = true;
            int kn = 0, vn = 0;  // tiles issued so far (the first KS of K before the block met)
            for (int u = 0; u < 2 * nt && ok; ++u) {
                const int t = u < nt ? u : u - nt, s = kn % L::KS;
                if (kn >= L::KS) {
                    if (!mbar_wait(bar_ke + 8 * s, (kn / L::KS - 1) & 1, lim.wait_ns, abort_flag)) {
                        ok = false;
                        break;
                    }
                    load_tile(&tmK, sb + L::kOffK + s * L::kTile, bar_kf + 8 * s, krow + t * 128);
                }
                ++kn;
                if (u >= nt) {
                    const int v = vn % L::VS;
                    if (vn >= L::VS && !mbar_wait(bar_ve + 8 * v, (vn / L::VS - 1) & 1, lim.wait_ns, abort_flag)) {
                        ok = false;
                        break;
                    }
                    load_tile(&tmV, sb + L::kOffV + v * L::kTile, bar_vf + 8 * v, krow + t * 128);
                    ++vn;
                }
            }
            kn = max(kn, min(L::KS, 2 * nt));
            if (!ok) fail();
            // every copy lands before the block may end
            mbar_wait(bar_q, 0, lim.drain_ns, nullptr);
            for (int k = max(0, kn - L::KS); k < kn; ++k)
                mbar_wait(bar_kf + 8 * (k % L::KS), (k / L::KS) & 1, lim.drain_ns, nullptr);
            for (int k = max(0, vn - L::VS); k < vn; ++k)
                mbar_wait(bar_vf + 8 * (k % L::VS), (k / L::VS) & 1, lim.drain_ns, nullptr);
        }
    } else if (warp == 4 * NWG + 1) {
        // ------------------------------------------------------------ MMA issuer
        // the whole warp runs this loop, one elected lane issues
        if (nt > 0) {
            constexpr uint32_t kIdO = idesc_i8(128, DP, false, true) & ~(1u << 7);  // unsigned A
            auto wait = [&](uint32_t bar, uint32_t parity) {
                return (bool)__all_sync(0xffffffffu, mbar_wait(bar, parity, lim.wait_ns, abort_flag));
            };
            bool ok = wait(bar_q, 0);
            int kn = 0, n1[2] = {0, 0};
            // S of N keys from row `half` * N of the next K tile into score buffer buf at column col
            auto scores = [&](auto n_keys, int buf, int col, int half, bool done) {
                constexpr int N = decltype(n_keys)::value;
                const int s = kn % L::KS;
                if (half == 0 && !wait(bar_kf + 8 * s, (kn / L::KS) & 1)) return false;
                tc_fence_after();
                const uint32_t kb = sb + L::kOffK + s * L::kTile + half * N * 64;
                const uint64_t da = smem_desc_kmajor(sb, 64), db = smem_desc_kmajor(kb, 64);
                if (elect_one()) {
#pragma unroll
                    for (int x = 0; x < 2 * H; ++x)
                        umma_i8(tm + col, da + (x >> 1) * (kHalfTile >> 4) + 2 * (x & 1),
                                db + (x >> 1) * (kHalfTile >> 4) + 2 * (x & 1), idesc_i8(128, N), x ? 1u : 0u);
                    if (done) umma_commit(bar_ke + 8 * s);
                    umma_commit(bar_sf + 8 * buf);
                }
                __syncwarp();
                if (done) ++kn;
                return true;
            };
            constexpr auto n128 = std::integral_constant<int, 128>();
            constexpr auto nTN = std::integral_constant<int, L::TN>();
            for (int t = 0; t < nt && ok; ++t) {
                const int buf = t & 1;  // free once pass 1 has read its last scores
                ok = (n1[buf] == 0 || wait(bar_se + 8 * buf, (n1[buf] - 1) & 1)) && scores(n128, buf, buf * 128, 0, true);
                ++n1[buf];
            }
            constexpr int PER = 128 / L::TN;  // steps of a K or V tile
            const int nu = (most + L::TN - 1) / L::TN;
            // both of pass 2's 64-wide buffers lie in pass 1's first one
            if (ok) ok = wait(bar_se, (n1[0] - 1) & 1) && scores(nTN, 0, 0, 0, PER == 1 || nu == 1);
            for (int u = 0; u < nu && ok; ++u) {
                if (u + 1 < nu) {  // the next scores, in the buffer of the weights u - 1
                    if (u > 0) ok = wait(bar_ee, (u - 1) & 1);
                    // before its barrier completes another phase, every warp has seen pass 1's last
                    else if (n1[1] > 0) ok = wait(bar_se + 8, (n1[1] - 1) & 1);
                    const int half = (u + 1) % PER;
                    if (!ok || !(ok = scores(nTN, (u + 1) & 1, ((u + 1) & 1) * L::TN, half, half == PER - 1 || u + 2 == nu))) break;
                }
                const int v = (u / PER) % L::VS;
                ok = (u % PER != 0 || wait(bar_vf + 8 * v, (u / PER / L::VS) & 1)) && wait(bar_ef + 8 * (u & 1), (u >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                const int ks = (min(L::TN, most - u * L::TN) + 31) / 32;
                const uint64_t dv = smem_desc_mnmajor64(sb + L::kOffV + v * L::kTile + (u % PER) * L::TN * 64, kHalfTile);
                const uint32_t e0 = tm + (u & 1) * L::TN, first = u ? 1u : 0u;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < L::TN / 32; ++kk)
                        if (kk < ks) {
                            const uint32_t e = e0 + kk / (CW2 / 32) * CW2 + kk % (CW2 / 32) * 8;
                            umma_i8_ta(tm + L::kO, e, dv + 128 * kk, kIdO, kk ? 1u : first);
                            umma_i8_ta(tm + L::kO + DP, e + CW2 / 4, dv + 128 * kk, kIdO, kk ? 1u : first);
                        }
                    if (u % PER == PER - 1 || u + 1 == nu) umma_commit(bar_ve + 8 * v);
                    umma_commit(bar_ee);
                }
                __syncwarp();
            }
            if (!ok && lane == 0) fail();
            if (elect_one()) {
                umma_commit(bar_of);
                umma_commit(bar_dr);
            }
            __syncwarp();
            mbar_wait(bar_dr, 0, lim.drain_ns, nullptr);
        }
    } else {
        // ------------------------------------------------------------ softmax
        const int wg = warp >> 2, et = threadIdx.x & 127, i = i0 + et;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const int see = i >= nq ? 0 : (a.causal ? max(0, min(nk, i + nk - nq + 1)) : nk);
        const int see_max = warp_max(see), see_min = -warp_max(-see);
        int sn[2] = {0, 0};
        bool ok = true;
        int mx = INT_MIN;
        for (int t = 0; t < nt && ok; ++t) {
            const int buf = t & 1;
            ok = __all_sync(0xffffffffu, mbar_wait(bar_sf + 8 * buf, sn[buf] & 1, lim.wait_ns, abort_flag));
            if (!ok) break;
            ++sn[buf];
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < CW; c += 32) {
                const int col = t * 128 + wg * CW + c;
                if (col >= see_max) break;
                uint32_t v[32];
                tmem_ld32(tm + lanes + buf * 128 + wg * CW + c, v);
                tmem_ld_done(v);
                if (col + 32 <= see_min) {
#pragma unroll
                    for (int q = 0; q < 32; q += 2) mx = max(mx, max((int)v[q], (int)v[q + 1]));
                } else {
#pragma unroll
                    for (int q = 0; q < 32; ++q) mx = max(mx, col + q < see ? (int)v[q] : INT_MIN);
                }
            }
            warp_arrive(bar_se + 8 * buf);
        }
        int *red = (int *)(smem + L::kOffRed);
        if (NWG == 2) {
            red[wg * 128 + et] = mx;
            named_bar_sync(1, NS);
            mx = max(mx, red[(wg ^ 1) * 128 + et]);
        }
        if (see == 0) mx = 0;
        const f2 nm = pk(-(kAttnMagic + (float)mx));
        const f2 f = pk(attn_factor(a, b * a.Hkv + g));
        uint32_t sum = 0;
        int n_sum = 0;
        const int nu = (most + L::TN - 1) / L::TN;
        for (int u = 0; u < nu && ok; ++u) {
            const int buf = u & 1;
            ok = __all_sync(0xffffffffu, mbar_wait(bar_sf + 8 * buf, sn[buf] & 1, lim.wait_ns, abort_flag));
            if (!ok) break;
            ++sn[buf];
            tc_fence_after();
            const int end = min(L::TN, most - u * L::TN);  // columns that the MMAs read
            // the weights' two byte planes take the first half of this thread's own score columns
            const uint32_t mine = tm + lanes + buf * L::TN + wg * CW2;
#pragma unroll
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
                tmem_st8(mine + c / 4, hi);
                tmem_st8(mine + CW2 / 4 + c / 4, lo);
            }
            tmem_st_wait();
            warp_arrive(bar_ef + 8 * buf);
        }
        sum -= (uint32_t)n_sum * 0x4B400000u;
        if (NWG == 2) {
            red[256 + wg * 128 + et] = (int)sum;
            named_bar_sync(1, NS);
            sum += (uint32_t)red[256 + (wg ^ 1) * 128 + et];
        }
        if (nt > 0 && ok) {
            ok = __all_sync(0xffffffffu, mbar_wait(bar_of, 0, lim.wait_ns, abort_flag));
            tc_fence_after();
        }
        if (!ok && lane == 0) fail();
        const bool live = i < a.Lq;
        if (live && wg == 0) a.stats[(int64_t)bh * a.Lq + i] = make_int2(mx, (int)sum);
        // outputs: columns [wg DP / NWG, ...) of the head; every thread takes part in the barriers
        const int c0 = wg * (DP / NWG);
        const bool read = nt > 0 && ok;
        float2 *gm = (float2 *)(smem + L::kOffRed + 2048) + et;
        fit_row_tmem<DP / NWG / 16>(
            a, a.o, (int64_t)b * a.Lq + i, h, c0, read ? (int)sum : 0, 1, attn_top(a, OPV, b * a.Hkv + g), live,
            nk <= 1024, gm, 128, 1, NS, [&](int s, uint32_t(&hi)[16], uint32_t(&lo)[16]) {
                if (read) {
                    tmem_ld16(tm + lanes + L::kO + c0 + s * 16, hi);
                    tmem_ld16(tm + lanes + L::kO + DP + c0 + s * 16, lo);
                    tmem_ld_done(hi, lo);
                } else {
#pragma unroll
                    for (int q = 0; q < 16; ++q) hi[q] = lo[q] = 0;
                }
            });
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4 * NWG + 1) tmem_dealloc(tm, L::kTmem);
}

}  // namespace ict
