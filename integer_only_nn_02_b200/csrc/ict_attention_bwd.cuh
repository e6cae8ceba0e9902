// ict_attention_bwd.cuh -- the attention backward pass on the 5th-generation tensor cores.
//
// Two kernels, each recomputing S and dP = AdO AV^T and the weights E from the forward's
// statistics, so that no gradient is joined by atomics and every accumulator stays in TMEM:
//   attn_dq_kernel   one block per 128 queries, walking over the keys:
//                      T = RNE(E x 2^-t) (two byte planes, in the scores' place in TMEM),
//                      dQ_hi += T_hi AK, dQ_lo += T_lo AK; the largest |T| of every row
//   attn_dkv_kernel  one block per 128 keys, walking over the queries of all the heads that
//                    share them; scores transposed (TMEM lane = key), so that P and U are A
//                    operands again: P = RNE(E r), U = RNE(P x 2^-c),
//                      dV += P^T AdO, dK += U^T AQ (two planes each)
// Steps of 64 columns, double-buffered; two pairs of softmax warpgroups take alternate steps,
// each warpgroup 32 columns.  One block per SM (512 TMEM columns: two buffers of 64 + 64 scores
// and 256 columns of accumulators).  For heads wider than 64 columns dV and dK do not fit side
// by side: one block computes dV, another dK.
// Bound by the elementwise work: per (query, key) about 9 instructions for dQ and 11 for dK and
// dV beside one exponential each; the contractions take 128 x 64 x 64 multiply-adds in 64
// cycles and there are six of them (eight with the recomputation) per step.
#pragma once

#include "ict_attention_fwd.cuh"

namespace ict {

constexpr int kStep = 64;           // columns of a step
constexpr int kAccCol = 256;        // first accumulator column
constexpr int kSoftWarps = 16;

// One step's 16 columns of T (two byte planes), the row's query in this thread.
template <bool PART>
__device__ __forceinline__ void dq16(const uint32_t (&vs)[16], const uint32_t (&vd)[16], f2 nm, f2 nd, f2 f, f2 sc, int vis,
                                     int &tmax, int &tmin, uint32_t (&lo)[4], uint32_t (&hi)[4]) {
    const f2 M = pk(kAttnMagic), nM = pk(-kAttnMagic);
#pragma unroll
    for (int q = 0; q < 16; q += 4) {
        float t[4];
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
            const f2 w = attn_weight2f(vs[q + k], vs[q + k + 1], nm, f);
            const f2 x = add2(pk(__uint_as_float(vd[q + k] + 0x4B400000u), __uint_as_float(vd[q + k + 1] + 0x4B400000u)), nd);
            unpk(fma2(mul2(add2(w, nM), sc), x, M), t[k], t[k + 1]);
        }
        if (PART) {
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] = q + k < vis ? t[k] : kAttnMagic;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            tmax = max(tmax, __float_as_int(t[k]));
            tmin = min(tmin, __float_as_int(t[k]));
        }
        split_bytes(t[0], t[1], t[2], t[3], lo[q >> 2], hi[q >> 2]);
    }
}

// 16 queries' P and U for the key in this thread; vec: the queries' -(M + smax), r, -(M + d)
// (64 floats each).  PART: queries before `first` do not see the key.  MODE bit 0: dV, bit 1: dK.
template <bool PART, int MODE>
__device__ __forceinline__ void dkv16(const uint32_t (&vs)[16], const uint32_t (&vd)[16], const float *vec, f2 f, f2 sc,
                                      int first, uint32_t (&plo)[4], uint32_t (&phi)[4], uint32_t (&ulo)[4],
                                      uint32_t (&uhi)[4]) {
    const f2 M = pk(kAttnMagic), nM = pk(-kAttnMagic);
#pragma unroll
    for (int q = 0; q < 16; q += 4) {
        const ulonglong2 nm = *reinterpret_cast<const ulonglong2 *>(vec + q);
        const ulonglong2 rho = *reinterpret_cast<const ulonglong2 *>(vec + kStep + q);
        float p[4];
        unpk(fma2(add2(attn_weight2f(vs[q], vs[q + 1], nm.x, f), nM), rho.x, M), p[0], p[1]);
        unpk(fma2(add2(attn_weight2f(vs[q + 2], vs[q + 3], nm.y, f), nM), rho.y, M), p[2], p[3]);
        if (PART) {
#pragma unroll
            for (int k = 0; k < 4; ++k) p[k] = q + k >= first ? p[k] : kAttnMagic;
        }
        if (MODE & 1) split_bytes(p[0], p[1], p[2], p[3], plo[q >> 2], phi[q >> 2]);
        if (MODE & 2) {
            const ulonglong2 nd = *reinterpret_cast<const ulonglong2 *>(vec + 2 * kStep + q);
            float u[4];
            const f2 x0 = add2(pk(__uint_as_float(vd[q] + 0x4B400000u), __uint_as_float(vd[q + 1] + 0x4B400000u)), nd.x);
            const f2 x1 = add2(pk(__uint_as_float(vd[q + 2] + 0x4B400000u), __uint_as_float(vd[q + 3] + 0x4B400000u)), nd.y);
            unpk(fma2(mul2(add2(pk(p[0], p[1]), nM), sc), x0, M), u[0], u[1]);
            unpk(fma2(mul2(add2(pk(p[2], p[3]), nM), sc), x1, M), u[2], u[3]);
            split_bytes(u[0], u[1], u[2], u[3], ulo[q >> 2], uhi[q >> 2]);
        }
    }
}

template <int DP>
struct DqCfg {
    static constexpr int H = DP / 64, kTile = H * kHalfTile, KS = 3, VS = 2;
    static constexpr int kOffD = kTile, kOffK = 2 * kTile, kOffV = kOffK + KS * kTile;
    static constexpr int kOffRed = kOffV + VS * kTile;  // [8][128] float2, [4][128] int
    static constexpr int kOffBar = kOffRed + 8 * 128 * 8 + 4 * 128 * 4;
    static constexpr int kBars = 1 + 2 * KS + 2 * VS + 2 + 2 + 3;
    static constexpr int kBytes = kOffBar + kBars * 8 + 16 + 1024;
    static constexpr int kThreads = 32 * kSoftWarps + 64;
};

template <int DP>
__global__ void __launch_bounds__(DqCfg<DP>::kThreads, 1)
    attn_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmD,
                   const __grid_constant__ AttnArgs a, const __grid_constant__ AttnLimits lim) {
    using L = DqCfg<DP>;
    constexpr int H = L::H;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t sb = smem_u32(smem);
    const uint32_t bar_q = sb + L::kOffBar;
    const uint32_t bar_kf = bar_q + 8, bar_ke = bar_kf + 8 * L::KS;
    const uint32_t bar_vf = bar_ke + 8 * L::KS, bar_ve = bar_vf + 8 * L::VS;
    const uint32_t bar_sf = bar_ve + 8 * L::VS, bar_ef = bar_sf + 16, bar_ee = bar_ef + 16;
    const uint32_t bar_of = bar_ee + 8, bar_dr = bar_of + 8;
    volatile int *misc = (volatile int *)(smem + L::kOffBar + L::kBars * 8);
    volatile int *abort_flag = &misc[1];
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    const int ntq = (a.Lq + kQTile - 1) / kQTile, heads = a.B * a.Hq;
    const int tile = ntq - 1 - (int)blockIdx.x / heads, bh = (int)blockIdx.x % heads;
    const int b = bh / a.Hq, h = bh % a.Hq, g = h / a.rep, i0 = tile * kQTile;
    const int nq = clamp_len(a.op[OPQ].lens, b, a.Lq), nk = clamp_len(a.op[OPK].lens, b, a.Lk);
    const int last = min(nq, i0 + kQTile) - 1;
    const int most = last < i0 ? 0 : (a.causal ? max(0, min(nk, last + nk - nq + 1)) : nk);
    const int nt = (most + 127) / 128, nu = (most + kStep - 1) / kStep;
    const int qrow = bh * a.Lq + i0, krow = (b * a.Hkv + g) * a.Lk;
    auto load_tile = [&](const CUtensorMap *m, uint32_t dst, uint32_t bar, int row) {
        for (int x = 0; x < H; ++x) tma_load_2d(dst + x * kHalfTile, m, bar, 64 * x, row);
    };
    if (threadIdx.x == 32 * kSoftWarps) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        prefetch_tmap(&tmD);
        mbar_init(bar_q, 1);
        for (int s = 0; s < L::KS; ++s) mbar_init(bar_kf + 8 * s, 1), mbar_init(bar_ke + 8 * s, 1);
        for (int s = 0; s < L::VS; ++s) mbar_init(bar_vf + 8 * s, 1), mbar_init(bar_ve + 8 * s, 1);
        for (int s = 0; s < 2; ++s) mbar_init(bar_sf + 8 * s, 1), mbar_init(bar_ef + 8 * s, kSoftWarps / 2);
        mbar_init(bar_ee, 1);
        mbar_init(bar_of, 1);
        mbar_init(bar_dr, 1);
        misc[1] = 0;
        fence_barrier_init();
        if (nt > 0) {
            mbar_expect_tx(bar_q, 2 * L::kTile);
            load_tile(&tmQ, sb, bar_q, qrow);
            load_tile(&tmD, sb + L::kOffD, bar_q, qrow);
        }
    }
    if (warp == kSoftWarps + 1) {
        tmem_alloc(smem_u32((const void *)&misc[0]), 512);
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

    if (warp == kSoftWarps) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0 && nt > 0) {
            bool ok = true;
            int n = 0;
            for (int t = 0; t < nt; ++t) {
                const int s = t % L::KS, v = t % L::VS;
                if (t >= L::KS && !wait_bar(bar_ke + 8 * s, (t / L::KS - 1) & 1, lim.wait_ns, abort_flag)) ok = false;
                if (ok && t >= L::VS && !wait_bar(bar_ve + 8 * v, (t / L::VS - 1) & 1, lim.wait_ns, abort_flag)) ok = false;
                if (!ok) break;
                mbar_expect_tx(bar_kf + 8 * s, L::kTile);
                load_tile(&tmK, sb + L::kOffK + s * L::kTile, bar_kf + 8 * s, krow + t * 128);
                mbar_expect_tx(bar_vf + 8 * v, L::kTile);
                load_tile(&tmV, sb + L::kOffV + v * L::kTile, bar_vf + 8 * v, krow + t * 128);
                ++n;
            }
            if (!ok) fail();
            wait_bar(bar_q, 0, lim.drain_ns, nullptr);
            for (int t = max(0, n - L::KS); t < n; ++t)
                wait_bar(bar_kf + 8 * (t % L::KS), (t / L::KS) & 1, lim.drain_ns, nullptr);
            for (int t = max(0, n - L::VS); t < n; ++t)
                wait_bar(bar_vf + 8 * (t % L::VS), (t / L::VS) & 1, lim.drain_ns, nullptr);
        }
    } else if (warp == kSoftWarps + 1) {
        // ------------------------------------------------------------ MMA issuer
        if (nt > 0) {
            constexpr uint32_t kIdS = idesc_i8(128, kStep);
            constexpr uint32_t kIdHi = idesc_i8(128, DP, false, true);              // signed high plane
            constexpr uint32_t kIdLo = idesc_i8(128, DP, false, true) & ~(1u << 7);  // unsigned low plane
            auto wait = [&](uint32_t bar, uint32_t parity) {
                return (bool)__all_sync(0xffffffffu, wait_bar(bar, parity, lim.wait_ns, abort_flag));
            };
            bool ok = wait(bar_q, 0);
            // S and dP of step u into buffer u & 1
            auto scores = [&](int u) {
                const int t = u >> 1, s = t % L::KS, v = t % L::VS, half = u & 1;
                if (half == 0 && (!wait(bar_kf + 8 * s, (t / L::KS) & 1) || !wait(bar_vf + 8 * v, (t / L::VS) & 1))) return false;
                tc_fence_after();
                const uint64_t dq = smem_desc_kmajor(sb, 64), dd = smem_desc_kmajor(sb + L::kOffD, 64);
                const uint64_t dk = smem_desc_kmajor(sb + L::kOffK + s * L::kTile + half * kStep * 64, 64);
                const uint64_t dv = smem_desc_kmajor(sb + L::kOffV + v * L::kTile + half * kStep * 64, 64);
                const uint32_t col = tm + (u & 1) * 128;
                if (elect_one()) {
#pragma unroll
                    for (int x = 0; x < 2 * H; ++x) {
                        const int o = (x >> 1) * (kHalfTile >> 4) + 2 * (x & 1);
                        umma_i8(col, dq + o, dk + o, kIdS, x ? 1u : 0u);
                    }
#pragma unroll
                    for (int x = 0; x < 2 * H; ++x) {
                        const int o = (x >> 1) * (kHalfTile >> 4) + 2 * (x & 1);
                        umma_i8(col + kStep, dd + o, dv + o, kIdS, x ? 1u : 0u);
                    }
                    if (half == 1 || u + 1 == nu) umma_commit(bar_ve + 8 * v);
                    umma_commit(bar_sf + 8 * (u & 1));
                }
                __syncwarp();
                return true;
            };
            if (ok) ok = scores(0);
            for (int u = 0; u < nu && ok; ++u) {
                if (u + 1 < nu) {
                    if (u > 0) ok = wait(bar_ee, (u - 1) & 1);
                    if (!ok || !(ok = scores(u + 1))) break;
                }
                if (!(ok = wait(bar_ef + 8 * (u & 1), (u >> 1) & 1))) break;
                tc_fence_after();
                const int s = (u >> 1) % L::KS, ks = (min(kStep, most - u * kStep) + 31) / 32;
                const uint64_t dk = smem_desc_mnmajor64(sb + L::kOffK + s * L::kTile + (u & 1) * kStep * 64, kHalfTile);
                const uint32_t e0 = tm + (u & 1) * 128, first = u ? 1u : 0u;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk)
                        if (kk < ks) {
                            umma_i8_ta(tm + kAccCol, e0 + kk * 32, dk + 128 * kk, kIdHi, kk ? 1u : first);
                            umma_i8_ta(tm + kAccCol + DP, e0 + kk * 32 + 8, dk + 128 * kk, kIdLo, kk ? 1u : first);
                        }
                    if ((u & 1) || u + 1 == nu) umma_commit(bar_ke + 8 * s);
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
            wait_bar(bar_dr, 0, lim.drain_ns, nullptr);
        }
    } else {
        // ------------------------------------------------------------ softmax
        const int wg = warp >> 2, et = threadIdx.x & 127, i = i0 + et, pair = wg >> 1, c0 = (wg & 1) * 32;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const int see = i >= nq ? 0 : (a.causal ? max(0, min(nk, i + nk - nq + 1)) : nk);
        const int see_max = warp_max(see), see_min = -warp_max(-see);
        const bool live = i < a.Lq;
        const int64_t at = (int64_t)bh * a.Lq + (live ? i : 0);
        int2 st = make_int2(0, 0), rw = make_int2(0, 0);
        if (live && nt > 0) st = a.stats[at], rw = a.row[at];
        const int tau = 32 - __clz(rw.y), bg = b * a.Hkv + g;
        const f2 nm = pk(-(kAttnMagic + (float)st.x)), nd = pk(-(kAttnMagic + (float)rw.x));
        const f2 f = pk(attn_factor(a, bg)), sc = pk(pow2f(-tau));
        int tmax = 0x4B400000, tmin = 0x4B400000;
        bool ok = true;
        for (int u = pair; u < nu && ok; u += 2) {
            ok = __all_sync(0xffffffffu, wait_bar(bar_sf + 8 * pair, (u >> 1) & 1, lim.wait_ns, abort_flag));
            if (!ok) break;
            tc_fence_after();
            const int col = u * kStep + c0;
            if (c0 < most - u * kStep) {
                const uint32_t mine = tm + lanes + pair * 128 + c0;
#pragma unroll 1
                for (int c = 0; c < 32; c += 16) {
                    uint32_t lo[4] = {0, 0, 0, 0}, hi[4] = {0, 0, 0, 0};
                    if (col + c < see_max) {
                        uint32_t vs[16], vd[16];
                        tmem_ld16(mine + c, vs);
                        tmem_ld16(mine + kStep + c, vd);
                        tmem_ld_done(vs, vd);
                        if (col + c + 16 <= see_min) dq16<false>(vs, vd, nm, nd, f, sc, 0, tmax, tmin, lo, hi);
                        else dq16<true>(vs, vd, nm, nd, f, sc, see - col - c, tmax, tmin, lo, hi);
                    }
                    tmem_st4(mine + c / 4, hi);  // in the place of scores already read
                    tmem_st4(mine + 8 + c / 4, lo);
                }
                tmem_st_wait();
            }
            warp_arrive(bar_ef + 8 * pair);
        }
        int *red = (int *)(smem + L::kOffRed + 8 * 128 * 8);
        red[wg * 128 + et] = max(tmax - 0x4B400000, 0x4B400000 - tmin);
        if (nt > 0 && ok) {
            ok = __all_sync(0xffffffffu, wait_bar(bar_of, 0, lim.wait_ns, abort_flag));
            tc_fence_after();
        }
        if (!ok && lane == 0) fail();
        const bool read = nt > 0 && ok;
        float2 *gm = (float2 *)(smem + L::kOffRed) + et;
        const int cc = wg * (DP / 4);
        fit_row_tmem<DP / 64>(a, a.o, (int64_t)b * a.Lq + i, h, cc, read ? st.y : 0, a.mul,
                              tau + attn_top(a, OPD, bg) + attn_top(a, OPV, bg) + attn_top(a, OPK, bg) - a.shift, live,
                              nk <= 1024, gm, 128, 1, 32 * kSoftWarps, AccCols{tm + lanes + kAccCol, DP, read});
        if (wg == 0 && live) a.tmax[at] = max(max(red[et], red[128 + et]), max(red[256 + et], red[384 + et]));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kSoftWarps + 1) tmem_dealloc(tm, 512);
}

// rn24(2^pi / rn24(S)) of a row; 0 for a row that sees no key
__device__ __forceinline__ float attn_rho(int S, int pi) { return S > 0 ? __fdiv_rn(pow2f(pi), (float)S) : 0.0f; }
// no |P x| of the row is larger
__device__ __forceinline__ int64_t attn_bound(float rho, int tmax, int X) {
    return (int64_t)floor((double)rho * (double)(tmax + 1) * pow2d(32 - __clz(X))) + X;
}

template <int DP>
struct DkvCfg {
    static constexpr int H = DP / 64, kTile = H * kHalfTile, QS = 2;
    static constexpr int kOffV = kTile, kOffQ = 2 * kTile;                 // stage: Q tile, dO tile
    static constexpr int kOffVec = kOffQ + QS * 2 * kTile;                 // [4][3][64] floats
    static constexpr int kOffRed = kOffVec + 4 * 3 * kStep * 4;            // [2][8][128] float2
    static constexpr int kOffBar = kOffRed + 2 * 8 * 128 * 8;
    static constexpr int kBars = 1 + 2 * QS + 2 + 2 + 4 + 4 + 3;
    static constexpr int kBytes = kOffBar + kBars * 8 + 48 + 1024;
    static constexpr int kThreads = 32 * kSoftWarps + 96;
};

// MODE: 3 computes dV and dK (heads of 64 columns), 1 only dV, 2 only dK.
template <int DP, int MODE>
__global__ void __launch_bounds__(DkvCfg<DP>::kThreads, 1)
    attn_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmD,
                    const __grid_constant__ AttnArgs a, const __grid_constant__ AttnLimits lim) {
    using L = DkvCfg<DP>;
    constexpr int H = L::H;
    static_assert(MODE != 3 || DP == 64, "both gradients: 256 accumulator columns");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t sb = smem_u32(smem);
    const uint32_t bar_k = sb + L::kOffBar;
    const uint32_t bar_qf = bar_k + 8, bar_qe = bar_qf + 8 * L::QS;
    const uint32_t bar_sf = bar_qe + 8 * L::QS, bar_ef = bar_sf + 16;
    const uint32_t bar_cf = bar_ef + 16, bar_ce = bar_cf + 32;  // the queries' vectors full / empty
    const uint32_t bar_ee = bar_ce + 32, bar_of = bar_ee + 8, bar_dr = bar_of + 8;
    volatile int *misc = (volatile int *)(smem + L::kOffBar + L::kBars * 8);  // tmem, abort, min S, -, bound (64 bits)
    volatile int *abort_flag = &misc[1];
    unsigned long long *wmax = (unsigned long long *)(smem + L::kOffBar + L::kBars * 8 + 16);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    const int bg = (int)blockIdx.x % (a.B * a.Hkv), J = (int)blockIdx.x / (a.B * a.Hkv);  // heavy causal blocks first
    const int b = bg / a.Hkv, g = bg % a.Hkv, j0 = J * kKeyBlock;
    const int nq = clamp_len(a.op[OPQ].lens, b, a.Lq), nk = clamp_len(a.op[OPK].lens, b, a.Lk);
    const int off = nk - nq;
    const int i0 = a.causal ? max(0, j0 - off) : 0;             // first query that sees the block
    const int n = j0 < nk ? max(0, nq - i0) : 0;                // such queries of one head
    const int base = i0 & ~(kStep - 1), tiles = n > 0 ? (nq - base + 127) / 128 : 0;
    const int per = n > 0 ? (nq - base + kStep - 1) / kStep : 0;  // steps of one head
    const int nw = tiles * a.rep, nu = per * a.rep;
    auto load_tile = [&](const CUtensorMap *m, uint32_t dst, uint32_t bar, int row) {
        for (int x = 0; x < H; ++x) tma_load_2d(dst + x * kHalfTile, m, bar, 64 * x, row);
    };
    if (threadIdx.x == 32 * kSoftWarps) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        prefetch_tmap(&tmD);
        mbar_init(bar_k, 1);
        for (int s = 0; s < L::QS; ++s) mbar_init(bar_qf + 8 * s, 1), mbar_init(bar_qe + 8 * s, 1);
        for (int s = 0; s < 2; ++s) mbar_init(bar_sf + 8 * s, 1), mbar_init(bar_ef + 8 * s, kSoftWarps / 2);
        for (int s = 0; s < 4; ++s) mbar_init(bar_cf + 8 * s, 1), mbar_init(bar_ce + 8 * s, kSoftWarps / 2);
        mbar_init(bar_ee, 1);
        mbar_init(bar_of, 1);
        mbar_init(bar_dr, 1);
        misc[1] = 0;
        misc[2] = INT_MAX;
        *wmax = 0;
        fence_barrier_init();
        if (nu > 0) {
            const int krow = bg * a.Lk + j0;
            mbar_expect_tx(bar_k, 2 * L::kTile);
            load_tile(&tmK, sb, bar_k, krow);
            load_tile(&tmV, sb + L::kOffV, bar_k, krow);
        }
    }
    if (warp == kSoftWarps + 1) {
        tmem_alloc(smem_u32((const void *)&misc[0]), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, (uint32_t)misc[0], 0);
    // the block's exponents: pi from the smallest sum of weights, c from the largest bound
    const int total = n * a.rep;
    auto index = [&](int t) { return ((int64_t)b * a.Hq + g * a.rep + t / n) * a.Lq + i0 + t % n; };
    {
        int m = INT_MAX;
        for (int t = threadIdx.x; t < total; t += L::kThreads) {
            const int S = a.stats[index(t)].y;
            if (S > 0) m = min(m, S);
        }
        m = -warp_max(-m);
        if (lane == 0) atomicMin((int *)&misc[2], m);
    }
    __syncthreads();
    const int pi = misc[2] == INT_MAX ? 0 : 31 - __clz(misc[2]);
    if (MODE & 2) {
        unsigned long long w = 0;
        for (int t = threadIdx.x; t < total; t += L::kThreads) {
            const int64_t at = index(t);
            const int S = a.stats[at].y;
            if (S > 0) w = max(w, (unsigned long long)attn_bound(attn_rho(S, pi), a.tmax[at], a.row[at].y));
        }
        for (int o = 16; o > 0; o >>= 1) w = max(w, __shfl_xor_sync(0xffffffffu, w, o));
        if (lane == 0) atomicMax(wmax, w);
    }
    __syncthreads();
    const int cexp = max(0, 64 - __clzll((long long)*wmax) - 14);
    auto fail = [&]() {
        *abort_flag = 1;
        raise_status(ICT_ERR_DEVICE_TIMEOUT);
    };
    // step u: query head g rep + u / per, queries base + (u % per) 64 ...
    if (warp == kSoftWarps) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0 && nu > 0) {
            bool ok = true;
            int w = 0;
            for (; w < nw; ++w) {
                const int s = w % L::QS;
                if (w >= L::QS && !wait_bar(bar_qe + 8 * s, (w / L::QS - 1) & 1, lim.wait_ns, abort_flag)) {
                    ok = false;
                    break;
                }
                const int row = (b * a.Hq + g * a.rep + w / tiles) * a.Lq + base + (w % tiles) * 128;
                const uint32_t dst = sb + L::kOffQ + s * 2 * L::kTile;
                mbar_expect_tx(bar_qf + 8 * s, 2 * L::kTile);
                load_tile(&tmQ, dst, bar_qf + 8 * s, row);
                load_tile(&tmD, dst + L::kTile, bar_qf + 8 * s, row);
            }
            if (!ok) fail();
            wait_bar(bar_k, 0, lim.drain_ns, nullptr);
            for (int t = max(0, w - L::QS); t < w; ++t)
                wait_bar(bar_qf + 8 * (t % L::QS), (t / L::QS) & 1, lim.drain_ns, nullptr);
        }
    } else if (warp == kSoftWarps + 1) {
        // ------------------------------------------------------------ MMA issuer
        if (nu > 0) {
            constexpr uint32_t kIdS = idesc_i8(128, kStep);
            constexpr uint32_t kIdHi = idesc_i8(128, DP, false, true);
            constexpr uint32_t kIdLo = idesc_i8(128, DP, false, true) & ~(1u << 7);
            auto wait = [&](uint32_t bar, uint32_t parity) {
                return (bool)__all_sync(0xffffffffu, wait_bar(bar, parity, lim.wait_ns, abort_flag));
            };
            bool ok = wait(bar_k, 0);
            // walk of the steps: tile index w and half within the tile, for the scores and for the products
            int sw = 0, sh = 0, sk = 0, pw = 0, ph = 0, pk_ = 0;  // sk, pk_: step within the head
            auto scores = [&](int u) {
                const int s = sw % L::QS;
                if (sh == 0 && !wait(bar_qf + 8 * s, (sw / L::QS) & 1)) return false;
                tc_fence_after();
                const uint32_t q = sb + L::kOffQ + s * 2 * L::kTile + sh * kStep * 64;
                const uint64_t dk = smem_desc_kmajor(sb, 64), dv = smem_desc_kmajor(sb + L::kOffV, 64);
                const uint64_t dq = smem_desc_kmajor(q, 64), dd = smem_desc_kmajor(q + L::kTile, 64);
                const uint32_t col = tm + (u & 1) * 128;
                if (elect_one()) {
#pragma unroll
                    for (int x = 0; x < 2 * H; ++x) {
                        const int o = (x >> 1) * (kHalfTile >> 4) + 2 * (x & 1);
                        umma_i8(col, dk + o, dq + o, kIdS, x ? 1u : 0u);
                    }
                    if (MODE & 2) {
#pragma unroll
                        for (int x = 0; x < 2 * H; ++x) {
                            const int o = (x >> 1) * (kHalfTile >> 4) + 2 * (x & 1);
                            umma_i8(col + kStep, dv + o, dd + o, kIdS, x ? 1u : 0u);
                        }
                    }
                    umma_commit(bar_sf + 8 * (u & 1));
                }
                __syncwarp();
                if (++sk == per) sk = 0, sh = 0, ++sw;
                else if ((sh ^= 1) == 0) ++sw;
                return true;
            };
            if (ok) ok = scores(0);
            for (int u = 0; u < nu && ok; ++u) {
                if (u + 1 < nu) {
                    if (u > 0) ok = wait(bar_ee, (u - 1) & 1);
                    if (!ok || !(ok = scores(u + 1))) break;
                }
                if (!(ok = wait(bar_ef + 8 * (u & 1), (u >> 1) & 1))) break;
                tc_fence_after();
                const int s = pw % L::QS;
                const uint32_t q = sb + L::kOffQ + s * 2 * L::kTile + ph * kStep * 64;
                const uint64_t dq = smem_desc_mnmajor64(q, kHalfTile), dd = smem_desc_mnmajor64(q + L::kTile, kHalfTile);
                const uint32_t e0 = tm + (u & 1) * 128, first = u ? 1u : 0u;
                const bool done = pk_ + 1 == per || ph == 1;
                constexpr int kDk = MODE == 3 ? kAccCol + 2 * DP : kAccCol;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        if (MODE & 1) {
                            umma_i8_ta(tm + kAccCol, e0 + kk * 32, dd + 128 * kk, kIdHi, kk ? 1u : first);
                            umma_i8_ta(tm + kAccCol + DP, e0 + kk * 32 + 8, dd + 128 * kk, kIdLo, kk ? 1u : first);
                        }
                        if (MODE & 2) {
                            umma_i8_ta(tm + kDk, e0 + kStep + kk * 32, dq + 128 * kk, kIdHi, kk ? 1u : first);
                            umma_i8_ta(tm + kDk + DP, e0 + kStep + kk * 32 + 8, dq + 128 * kk, kIdLo, kk ? 1u : first);
                        }
                    }
                    if (done) umma_commit(bar_qe + 8 * s);
                    umma_commit(bar_ee);
                }
                __syncwarp();
                if (++pk_ == per) pk_ = 0, ph = 0, ++pw;
                else if ((ph ^= 1) == 0) ++pw;
            }
            if (!ok && lane == 0) fail();
            if (elect_one()) {
                umma_commit(bar_of);
                umma_commit(bar_dr);
            }
            __syncwarp();
            wait_bar(bar_dr, 0, lim.drain_ns, nullptr);
        }
    } else if (warp == kSoftWarps + 2) {
        // ------------------------------------------------------------ the queries' vectors
        // two queries per lane and step, read one step ahead
        int2 st[2], rw[2];
        auto fetch = [&](int u) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int i = base + (u % per) * kStep + 2 * lane + k;
                st[k] = rw[k] = make_int2(0, 0);
                if (u < nu && i < nq) {
                    const int64_t at = ((int64_t)b * a.Hq + g * a.rep + u / per) * a.Lq + i;
                    st[k] = a.stats[at];
                    if (MODE & 2) rw[k] = a.row[at];
                }
            }
        };
        bool ok = true;
        if (nu > 0) fetch(0);
        for (int u = 0; u < nu && ok; ++u) {
            float m[2], r[2], d[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                // a query that sees nothing, or none: every score lies below its maximum, and r = 0
                m[k] = -(kAttnMagic + (st[k].y > 0 ? (float)st[k].x : 4194304.0f));
                r[k] = attn_rho(st[k].y, pi);
                d[k] = -(kAttnMagic + (float)rw[k].x);
            }
            fetch(u + 1);
            const int s = u & 3;
            if (u >= 4) ok = __all_sync(0xffffffffu, wait_bar(bar_ce + 8 * s, ((u >> 2) - 1) & 1, lim.wait_ns, abort_flag));
            float *v = (float *)(smem + L::kOffVec) + s * 3 * kStep + 2 * lane;
            *reinterpret_cast<float2 *>(v) = make_float2(m[0], m[1]);
            *reinterpret_cast<float2 *>(v + kStep) = make_float2(r[0], r[1]);
            *reinterpret_cast<float2 *>(v + 2 * kStep) = make_float2(d[0], d[1]);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_cf + 8 * s);
        }
        if (!ok && lane == 0) fail();
    } else {
        // ------------------------------------------------------------ softmax: lane = key
        const int wg = warp >> 2, et = threadIdx.x & 127, j = j0 + et, pair = wg >> 1, c0 = (wg & 1) * 32;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const f2 f = pk(attn_factor(a, bg)), sc = pk(pow2f(-cexp));
        const int lo_i = a.causal ? j - off : 0;  // the first query that sees this key
        const int lo_max = warp_max(lo_i);
        bool ok = true;
        int k_in = pair % max(per, 1);
        for (int u = pair; u < nu && ok; u += 2) {
            ok = __all_sync(0xffffffffu, wait_bar(bar_sf + 8 * pair, (u >> 1) & 1, lim.wait_ns, abort_flag) &&
                                             wait_bar(bar_cf + 8 * (u & 3), (u >> 2) & 1, lim.wait_ns, abort_flag));
            if (!ok) break;
            tc_fence_after();
            const float *vec = (const float *)(smem + L::kOffVec) + (u & 3) * 3 * kStep + c0;
            const int i = base + k_in * kStep + c0;
            const uint32_t mine = tm + lanes + pair * 128 + c0;
#pragma unroll 1
            for (int c = 0; c < 32; c += 16) {
                uint32_t vs[16], vd[16], plo[4], phi[4], ulo[4], uhi[4];
                tmem_ld16(mine + c, vs);
                if (MODE & 2) tmem_ld16(mine + kStep + c, vd);
                tmem_ld_wait();
                tmem_tie(vs);
                if (MODE & 2) tmem_tie(vd);
                if (i + c >= lo_max) dkv16<false, MODE>(vs, vd, vec + c, f, sc, 0, plo, phi, ulo, uhi);
                else dkv16<true, MODE>(vs, vd, vec + c, f, sc, lo_i - i - c, plo, phi, ulo, uhi);
                if (MODE & 1) {  // in the place of scores already read
                    tmem_st4(mine + c / 4, phi);
                    tmem_st4(mine + 8 + c / 4, plo);
                }
                if (MODE & 2) {
                    tmem_st4(mine + kStep + c / 4, uhi);
                    tmem_st4(mine + kStep + 8 + c / 4, ulo);
                }
            }
            tmem_st_wait();
            warp_arrive(bar_ef + 8 * pair);
            if (lane == 0) mbar_arrive(bar_ce + 8 * (u & 3));
            if ((k_in += 2) >= per) k_in %= per;
        }
        if (nu > 0 && ok) {
            ok = __all_sync(0xffffffffu, wait_bar(bar_of, 0, lim.wait_ns, abort_flag));
            tc_fence_after();
        }
        if (!ok && lane == 0) fail();
        const bool live = j < a.Lk, read = nu > 0 && ok;
        const int ed = attn_top(a, OPD, bg), ev = attn_top(a, OPV, bg), eq = attn_top(a, OPQ, bg);
        // 32 columns of one gradient per warpgroup
        const bool is_k = MODE == 3 ? wg >= 2 : MODE == 2;
        const int cc = MODE == 3 ? (wg & 1) * 32 : wg * 32, acc = MODE == 3 && is_k ? kAccCol + 2 * DP : kAccCol;
        float2 *gm = (float2 *)(smem + L::kOffRed) + (MODE == 3 && is_k ? 8 * 128 : 0) + et;
        const int64_t row = (int64_t)b * a.Lk + j;
        const int den = read && j < nk ? 1 : 0;
        const bool narrow = (int64_t)nq * a.rep <= 1024;
        const int bar = MODE == 3 ? 1 + (wg >> 1) : 1, nthr = MODE == 3 ? 256 : 32 * kSoftWarps;
        const AttnOut &out = is_k ? a.dk : a.dv;
        const int mul = is_k ? a.mul : 1, r = is_k ? cexp - pi - a.shift + ed + ev + eq : ed - pi;
        fit_row_tmem<2>(a, out, row, g, cc, den, mul, r, live, narrow, gm, 128, bar, nthr, AccCols{tm + lanes + acc, DP, read});
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kSoftWarps + 1) tmem_dealloc(tm, 512);
}

}  // namespace ict
