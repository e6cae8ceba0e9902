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
// Steps of 64 columns in two or three buffers; two pairs of softmax warpgroups take alternate
// steps, each warpgroup 32 columns.  One block per SM (512 TMEM columns: two or three buffers of
// 64 + 64 scores and 256 or 128 columns of accumulators).  For heads wider than 64 columns dV and
// dK do not fit side by side: one block computes dV, another dK.
// Bound by the elementwise work: per (query, key) about 9 instructions for dQ and 11 for dK and
// dV beside one exponential each, with 16 warps to hide their latencies (half of the issue slots
// are used); the tensor pipe is busy 15 % of the time.  A step of 128 keys x 64 queries takes 1.1
// us; rounding an item's outputs about 4 thousand clocks, for half of which the accumulators are
// blocked, which counts for short items (64 x 12 heads of 197 tokens: dQ 53 us, dK and dV 85 us).
// 3 x 8 causal heads of up to 2048 tokens on 2 key heads: 40 and 64 us.
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

// The row's head columns [c0, c0 + n) of a row that nothing contributes to.
__device__ __forceinline__ void zero_row(const AttnArgs &a, const AttnOut &out, int64_t row, int h, int c0, int n) {
    const int col = out.col + h * a.D, end = min(a.D, c0 + n);
    for (int c = c0; c < end; c += 16) {
        *reinterpret_cast<uint4 *>(out.mant + row * out.ld + col + c) = make_uint4(0, 0, 0, 0);
        if (c % out.G == 0) out.exp[row * out.ngc + out.gcol + h * out.dg + c / out.G] = (int8_t)kEZero;
    }
}

template <int DP>
struct DqCfg {
    static constexpr int H = DP / 64, kTile = H * kHalfTile, QS = 2, KS = 3, VS = 2;
    static constexpr int NB = DP == 64 ? 3 : 2;               // score buffers (128 columns each)
    static constexpr int kAcc = DP == 64 ? 384 : 256;         // dQ's column
    static constexpr int kOffK = QS * 2 * kTile, kOffV = kOffK + KS * kTile;  // Q stage: Q tile, dO tile
    static constexpr int kOffRed = kOffV + VS * kTile;  // [2][8][128] float2, [4][4][128] int
    static constexpr int kOffBar = kOffRed + 2 * 8 * 128 * 8 + 4 * 4 * 128 * 4;
    static constexpr int kBars = 2 * (QS + KS + VS) + 3 * NB + 4;
    static constexpr int kBytes = kOffBar + kBars * 8 + 16 + 1024;
    static constexpr int kThreads = 32 * kSoftWarps + 64;
};

// Persistent blocks, as the forward's.  Two pairs of softmax warpgroups take alternate steps; the
// pairs also take turns at the items' outputs, so that one pair starts the next item meanwhile.
// Score buffers go round over the steps of all items (step G in buffer G % NB; the pair
// G & 1 takes it, so that a pair never waits for a phase whose forerunner is still open).
template <int DP>
__global__ void __launch_bounds__(DqCfg<DP>::kThreads, 1)
    attn_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmD,
                   const __grid_constant__ AttnArgs a, const __grid_constant__ AttnLimits lim, int items) {
    using L = DqCfg<DP>;
    constexpr int H = L::H, NS = 32 * kSoftWarps;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t sb = smem_u32(smem);
    const uint32_t bar_qf = sb + L::kOffBar, bar_qe = bar_qf + 8 * L::QS;
    const uint32_t bar_kf = bar_qe + 8 * L::QS, bar_ke = bar_kf + 8 * L::KS;
    const uint32_t bar_vf = bar_ke + 8 * L::KS, bar_ve = bar_vf + 8 * L::VS;
    const uint32_t bar_sf = bar_ve + 8 * L::VS, bar_ef = bar_sf + 8 * L::NB;  // scores full, T written (per buffer)
    const uint32_t bar_ee = bar_ef + 8 * L::NB, bar_of = bar_ee + 8 * L::NB, bar_oe = bar_of + 16, bar_dr = bar_oe + 8;
    volatile int *misc = (volatile int *)(smem + L::kOffBar + L::kBars * 8);
    volatile int *abort_flag = &misc[1];
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == NS) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        prefetch_tmap(&tmD);
        for (int s = 0; s < L::QS; ++s) mbar_init(bar_qf + 8 * s, 1), mbar_init(bar_qe + 8 * s, 1);
        for (int s = 0; s < L::KS; ++s) mbar_init(bar_kf + 8 * s, 1), mbar_init(bar_ke + 8 * s, 1);
        for (int s = 0; s < L::VS; ++s) mbar_init(bar_vf + 8 * s, 1), mbar_init(bar_ve + 8 * s, 1);
        for (int s = 0; s < L::NB; ++s) {
            mbar_init(bar_sf + 8 * s, 1), mbar_init(bar_ef + 8 * s, kSoftWarps / 2), mbar_init(bar_ee + 8 * s, 1);
        }
        for (int s = 0; s < 2; ++s) mbar_init(bar_of + 8 * s, 1);  // per pair: each sees every other output
        mbar_init(bar_oe, kSoftWarps / 2);
        mbar_init(bar_dr, 1);
        misc[1] = 0;
        fence_barrier_init();
    }
    __syncthreads();
    auto fail = [&]() {
        *abort_flag = 1;
        raise_status(ICT_ERR_DEVICE_TIMEOUT);
    };

    if (warp == kSoftWarps) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            auto load_tile = [&](const CUtensorMap *m, uint32_t dst, uint32_t bar, int row) {
                for (int x = 0; x < H; ++x) tma_load_2d(dst + x * kHalfTile, m, bar, 64 * x, row);
            };
            auto free = [&](uint32_t bar, int n, int stages) {  // the n-th use of a ring's stage
                return n < stages || wait_bar(bar + 8 * (n % stages), (n / stages - 1) & 1, lim.wait_ns, abort_flag);
            };
            bool ok = true;
            int qn = 0, kn = 0, vn = 0;
            for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
                const AttnItem w = attn_item(a, item);
                if (w.nt == 0) continue;
                if (!(ok = free(bar_qe, qn, L::QS))) break;
                const uint32_t dst = sb + (qn % L::QS) * 2 * L::kTile, bar = bar_qf + 8 * (qn % L::QS);
                mbar_expect_tx(bar, 2 * L::kTile);
                load_tile(&tmQ, dst, bar, w.bh * a.Lq + w.i0);
                load_tile(&tmD, dst + L::kTile, bar, w.bh * a.Lq + w.i0);
                ++qn;
                const int krow = (w.b * a.Hkv + w.g) * a.Lk;
                for (int t = 0; t < w.nt; ++t) {
                    if (!(ok = free(bar_ke, kn, L::KS))) break;
                    mbar_expect_tx(bar_kf + 8 * (kn % L::KS), L::kTile);
                    load_tile(&tmK, sb + L::kOffK + (kn % L::KS) * L::kTile, bar_kf + 8 * (kn % L::KS), krow + t * 128);
                    ++kn;
                    if (!(ok = free(bar_ve, vn, L::VS))) break;
                    mbar_expect_tx(bar_vf + 8 * (vn % L::VS), L::kTile);
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
    } else if (warp == kSoftWarps + 1) {
        // ------------------------------------------------------------ TMEM and MMA issue
        tmem_alloc(smem_u32((const void *)&misc[0]), 512);
        tmem_relinquish();
        tc_fence_before();
        named_bar_sync(5, NS + 32);
        tc_fence_after();
        const uint32_t tm = __shfl_sync(0xffffffffu, (uint32_t)misc[0], 0);
        constexpr uint32_t kIdS = idesc_i8(128, kStep);
        constexpr uint32_t kIdHi = idesc_i8(128, DP, false, true);              // signed high plane
        constexpr uint32_t kIdLo = idesc_i8(128, DP, false, true) & ~(1u << 7);  // unsigned low plane
        auto wait = [&](uint32_t bar, int parity) {
            return (bool)__all_sync(0xffffffffu, wait_bar(bar, (uint32_t)(parity & 1), lim.wait_ns, abort_flag));
        };
        bool ok = true;
        int qn = 0, kn = 0, k0 = 0, vn = 0, sn = 0, pn = 0, on = 0;  // kn, sn: K tiles, steps whose scores, k0, pn: whose products are issued
        for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
            const AttnItem w = attn_item(a, item);
            if (w.nt == 0) continue;
            const int nu = (w.most + kStep - 1) / kStep;
            const uint32_t qt = sb + (qn % L::QS) * 2 * L::kTile;
            if (!(ok = wait(bar_qf + 8 * (qn % L::QS), qn / L::QS))) break;
            // S and dP of the item's step u; the buffer's last T planes (NB steps ago) are used
            auto scores = [&](int u) {
                const int s = kn % L::KS, v = vn % L::VS, half = u & 1, buf = sn % L::NB;
                if (sn >= L::NB && !wait(bar_ee + 8 * buf, sn / L::NB - 1)) return false;
                if (half == 0 && (!wait(bar_kf + 8 * s, kn / L::KS) || !wait(bar_vf + 8 * v, vn / L::VS))) return false;
                tc_fence_after();
                const bool done = half == 1 || u + 1 == nu;
                const uint64_t dq = smem_desc_kmajor(qt, 64), dd = smem_desc_kmajor(qt + L::kTile, 64);
                const uint64_t dk = smem_desc_kmajor(sb + L::kOffK + s * L::kTile + half * kStep * 64, 64);
                const uint64_t dv = smem_desc_kmajor(sb + L::kOffV + v * L::kTile + half * kStep * 64, 64);
                const uint32_t col = tm + buf * 128;
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
                    if (done) umma_commit(bar_ve + 8 * v);
                    if (u + 1 == nu) umma_commit(bar_qe + 8 * (qn % L::QS));
                    umma_commit(bar_sf + 8 * buf);
                }
                __syncwarp();
                ++sn;
                if (done) ++kn, ++vn;
                return true;
            };
            for (int u = 0; u < L::NB - 1 && u < nu && ok; ++u) ok = scores(u);
            for (int u = 0; u < nu && ok; ++u) {
                if (u + L::NB - 1 < nu && !(ok = scores(u + L::NB - 1))) break;
                const int buf = pn % L::NB;
                if (!(ok = wait(bar_ef + 8 * buf, pn / L::NB))) break;
                if (u == 0 && on > 0 && !(ok = wait(bar_oe, on - 1))) break;  // the last item's dQ is read
                tc_fence_after();
                const int s = k0 % L::KS, ks = (min(kStep, w.most - u * kStep) + 31) / 32;
                const uint64_t dk = smem_desc_mnmajor64(sb + L::kOffK + s * L::kTile + (u & 1) * kStep * 64, kHalfTile);
                const uint32_t e0 = tm + buf * 128, first = u ? 1u : 0u;
                const bool done = (u & 1) || u + 1 == nu;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk)
                        if (kk < ks) {
                            umma_i8_ta(tm + L::kAcc, e0 + kk * 32, dk + 128 * kk, kIdHi, kk ? 1u : first);
                            umma_i8_ta(tm + L::kAcc + DP, e0 + kk * 32 + 8, dk + 128 * kk, kIdLo, kk ? 1u : first);
                        }
                    if (done) umma_commit(bar_ke + 8 * s);
                    umma_commit(bar_ee + 8 * buf);
                    if (u + 1 == nu) umma_commit(bar_of + 8 * (on & 1));
                }
                __syncwarp();
                ++pn;
                if (done) ++k0;
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
        named_bar_sync(5, NS + 32);
        tc_fence_after();
        const uint32_t tm = (uint32_t)misc[0];
        const int wg = warp >> 2, et = threadIdx.x & 127, pair = wg >> 1, c0 = (wg & 1) * 32;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        bool ok = true;
        int on = 0, gn = 0;  // outputs, steps of the items so far
        for (int item = blockIdx.x; item < items; item += gridDim.x) {  // (outputs are written after a failure too)
            const AttnItem w = attn_item(a, item);
            const int i = w.i0 + et, nu = (w.most + kStep - 1) / kStep, bg = w.b * a.Hkv + w.g;
            const int see = i >= w.nq ? 0 : (a.causal ? max(0, min(w.nk, i + w.nk - w.nq + 1)) : w.nk);
            const int see_max = warp_max(see), see_min = -warp_max(-see);
            const bool live = i < a.Lq;
            const int64_t at = (int64_t)w.bh * a.Lq + (live ? i : 0);
            int2 st = make_int2(0, 0), rw = make_int2(0, 0);
            if (live && w.nt > 0) st = a.stats[at], rw = a.row[at];
            const int tau = 32 - __clz(rw.y);
            const f2 nm = pk(-(kAttnMagic + (float)st.x)), nd = pk(-(kAttnMagic + (float)rw.x));
            const f2 f = pk(attn_factor(a, bg)), sc = pk(pow2f(-tau));
            int tmax = 0x4B400000, tmin = 0x4B400000;
            for (int u = (pair ^ gn) & 1; u < nu && ok; u += 2) {
                const int buf = (gn + u) % L::NB;
                ok = __all_sync(0xffffffffu, wait_bar(bar_sf + 8 * buf, ((gn + u) / L::NB) & 1, lim.wait_ns, abort_flag));
                if (!ok) break;
                tc_fence_after();
                const int col = u * kStep + c0;
                if (c0 < w.most - u * kStep) {
                    const uint32_t mine = tm + lanes + buf * 128 + c0;
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
                warp_arrive(bar_ef + 8 * buf);
            }
            gn += nu;
            if (w.nt == 0) {
                if (pair == 0 && live) zero_row(a, a.o, (int64_t)w.b * a.Lq + i, w.h, (wg & 1) * (DP / 2), DP / 2);
                if (wg == 0 && live) a.tmax[at] = 0;
                continue;
            }
            // the item's output is this turn's pair's; the other leaves its maxima and goes on
            const int turn = on & 1;
            // four of these in turn: a warp may still read this output's maxima when another leaves those of the
            // output after the next, but not once both have met again at that one's barrier
            int *red = (int *)(smem + L::kOffRed + 2 * 8 * 128 * 8) + (on & 3) * 4 * 128;
            red[wg * 128 + et] = max(tmax - 0x4B400000, 0x4B400000 - tmin);
            if (pair != turn) {
                named_bar_arrive(3 + turn, NS);
                ++on;
                continue;
            }
            named_bar_sync(3 + turn, NS);
            if (wg == 2 * turn && live) a.tmax[at] = max(max(red[et], red[128 + et]), max(red[256 + et], red[384 + et]));
            const RowOut out = row_out(a, a.o, (int64_t)w.b * a.Lq + i, w.h, st.y, a.mul, live);
            const int r = tau + attn_top(a, OPD, bg) + attn_top(a, OPV, bg) + attn_top(a, OPK, bg) - a.shift;
            if (ok) ok = __all_sync(0xffffffffu, wait_bar(bar_of + 8 * turn, (on >> 1) & 1, lim.wait_ns, abort_flag));
            tc_fence_after();
            float2 *gm = (float2 *)(smem + L::kOffRed) + turn * 8 * 128 + et;
            fit_row_tmem<DP / 32>(a, a.o, out, (wg & 1) * (DP / 2), r, w.nk <= 1024, gm, (int *)(gm - et) + et, 128, 1 + turn, NS / 2,
                                  AccCols{tm + lanes + L::kAcc, DP, ok}, bar_oe);
            ++on;
        }
        if (!ok && lane == 0) fail();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kSoftWarps + 1) tmem_dealloc(__shfl_sync(0xffffffffu, (uint32_t)misc[0], 0), 512);
}

// rn24(2^pi / rn24(S)) of a row; 0 for a row that sees no key
__device__ __forceinline__ float attn_rho(int S, int pi) { return S > 0 ? __fdiv_rn(pow2f(pi), (float)S) : 0.0f; }
// no |P x| of the row is larger
__device__ __forceinline__ int64_t attn_bound(float rho, int tmax, int X) {
    return (int64_t)floor((double)rho * (double)(tmax + 1) * pow2d(32 - __clz(X))) + X;
}

template <int DP>
struct DkvCfg {
    static constexpr int H = DP / 64, kTile = H * kHalfTile, KS = 2, QS = 2;
    static constexpr int kOffQ = KS * 2 * kTile;                           // K stage: K tile, V tile; Q stage: Q tile, dO tile
    static constexpr int kVec = 3 * kStep + 4;                             // a step's floats: see dkv16, then f and 2^-c
    static constexpr int kOffVec = kOffQ + QS * 2 * kTile;                 // [4][kVec] floats
    static constexpr int kOffRed = kOffVec + 4 * kVec * 4;                 // [8][128] float2, [2][8][128] int
    static constexpr int kOffBar = kOffRed + 8 * 128 * 8 + 2 * 8 * 128 * 4;
    static constexpr int kBars = 2 * (KS + QS) + 2 + 2 + 4 + 4 + 5;
    static constexpr int kBytes = kOffBar + kBars * 8 + 16 + 1024;
    static constexpr int kThreads = 32 * kSoftWarps + 96;
};

// One work item: a block of keys of one key/value head, or a part of the queries that see it (tiles
// of 128 queries, head after head).  Heavy causal blocks come first.
struct KeyItem {
    int b, g, bg, j0, nq, nk, off, i0, n, base, tiles, per, slot, join, part, t0, nw, u0, nu;
};
__device__ __forceinline__ KeyItem key_item(const AttnArgs &a, int item) {
    KeyItem w;
    const int heads = a.B * a.Hkv, Jp = a.heads_kv(item);  // J parts + part
    const int J = a.parts == 1 ? Jp : Jp / a.parts, part = Jp - J * a.parts;
    w.part = part;
    w.bg = item - Jp * heads;
    w.b = a.hkv(w.bg);
    w.g = w.bg - w.b * a.Hkv;
    w.j0 = J * kKeyBlock;
    w.slot = J * heads + w.bg;
    w.nq = clamp_len(a.op[OPQ].lens, w.b, a.Lq);
    w.nk = clamp_len(a.op[OPK].lens, w.b, a.Lk);
    w.off = w.nk - w.nq;
    w.i0 = a.causal ? max(0, w.j0 - w.off) : 0;          // first query that sees the block
    w.n = w.j0 < w.nk ? max(0, w.nq - w.i0) : 0;         // such queries of one head
    w.base = w.i0 & ~(kStep - 1);
    w.tiles = w.n > 0 ? (w.nq - w.base + 127) / 128 : 0;
    w.per = w.n > 0 ? (w.nq - w.base + kStep - 1) / kStep : 0;  // steps of one head
    const int all = w.tiles * a.rep;
    w.join = min(a.parts, max(all, 1));  // parts with work (one for a block that no query sees)
    w.t0 = w.u0 = 0;
    w.nw = all, w.nu = w.per * a.rep;
    if (a.parts == 1) return w;
    w.nw = w.nu = 0;
    if (part < w.join && all > 0) {
        const int t1 = all * (part + 1) / w.join;
        w.t0 = all * part / w.join;
        w.nw = t1 - w.t0;
        w.u0 = (w.t0 / w.tiles) * w.per + 2 * (w.t0 % w.tiles);
        w.nu = (t1 / w.tiles) * w.per + 2 * (t1 % w.tiles) - w.u0;
    } else if (part >= w.join) {
        w.join = 0;  // nothing to do
    }
    return w;
}

// The exponents of every key block: pi from the smallest sum of weights, c from the largest bound,
// over the queries that see the block and have a gradient; those of the accumulators of dV and dK.  One block of threads
// each, of up to 1024.  A query with X = 0 (dO aligned to zeros, and with it every x) adds nothing to dV and dK whatever
// its P is, and P that pass 16 bits there do no harm; counted, one such query with all its weight on one key would
// leave flat queries over 65536 keys no digit.
__global__ void __launch_bounds__(1024) attn_exps_kernel(const __grid_constant__ AttnArgs a) {
    __shared__ int smin;
    __shared__ unsigned long long bmax;
    const int heads = a.B * a.Hkv, J = blockIdx.x / heads, bg = blockIdx.x - J * heads, b = bg / a.Hkv;
    const int nq = clamp_len(a.op[OPQ].lens, b, a.Lq), nk = clamp_len(a.op[OPK].lens, b, a.Lk), j0 = J * kKeyBlock;
    const int i0 = j0 < nk ? (a.causal ? max(0, j0 - (nk - nq)) : 0) : nq, n = nq - i0, total = n > 0 ? n * a.rep : 0;
    const int64_t head0 = (int64_t)bg * a.rep * a.Lq + i0;
    auto row = [&](int t) {
        const int r = t / n;
        return head0 + (int64_t)r * a.Lq + (t - r * n);
    };
    if (threadIdx.x == 0) smin = INT_MAX, bmax = 0;
    __syncthreads();
    int m = INT_MAX;
#pragma unroll 4
    for (int t = threadIdx.x; t < total; t += blockDim.x) {
        const int64_t at = row(t);
        const int S = a.stats[at].y;
        m = S > 0 && a.row[at].y > 0 ? min(m, S) : m;
    }
    m = -warp_max(-m);
    if ((threadIdx.x & 31) == 0) atomicMin(&smin, m);
    __syncthreads();
    m = smin;
    const int pi = m == INT_MAX ? 0 : 31 - __clz(m);
    unsigned long long x = 0;
#pragma unroll 4
    for (int t = threadIdx.x; t < total; t += blockDim.x) {
        const int64_t at = row(t);
        const int S = a.stats[at].y, tmax = a.tmax[at], X = a.row[at].y;
        if (S > 0 && X > 0) x = max(x, (unsigned long long)attn_bound(attn_rho(S, pi), tmax, X));
    }
    for (int o = 16; o > 0; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
    if ((threadIdx.x & 31) == 0) atomicMax(&bmax, x);
    __syncthreads();
    if (threadIdx.x == 0) {
        const int c = max(0, 64 - __clzll((long long)bmax) - 14);
        const int ed = attn_top(a, OPD, bg), ev = attn_top(a, OPV, bg), eq = attn_top(a, OPQ, bg);
        a.exps[blockIdx.x] = make_int4(pi, c, ed - pi, c - pi - a.shift + ed + ev + eq);
    }
}

// A part leaves its sums in memory; the last part to come (true) adds the others' to its
// accumulators.  Whole numbers below 2^31 in total, so their order does not matter.  sums: this
// thread's row in [part][64 columns in fours][128 keys], 32 columns of the high and, lo_cols / 4
// further on, of the low plane.  (Atomics into one place are bound by L2: 75 us against 44 us for
// 12 causal heads of 2048 tokens in three parts and in one.)
constexpr int64_t kPartSums = 64 * 128;  // uint4 of a part: 256 columns
__device__ __noinline__ bool join_parts(const AccCols acc, int c0, uint4 *sums, int lo_cols, int part, int *tickets, int join,
                                        volatile int *shared, int bar, int nthreads) {
    uint4 *mine = sums + part * kPartSums;
#pragma unroll 1
    for (int c = 0; c < 32; c += 16) {
        uint32_t hi[16], lo[16];
        acc.load16(c0 + c, hi, lo);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            mine[(c / 4 + q) * 128] = make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
            mine[(lo_cols / 4 + c / 4 + q) * 128] = make_uint4(lo[4 * q], lo[4 * q + 1], lo[4 * q + 2], lo[4 * q + 3]);
        }
    }
    __threadfence();
    named_bar_sync(bar, nthreads);
    if (tickets) *shared = atomicAdd(tickets, 1);
    named_bar_sync(bar, nthreads);
    if (*shared != join - 1) return false;
    __threadfence();
    // 16 columns of a plane at a time, four parts' loads in flight (its own among them)
#pragma unroll 1
    for (int z = 0; z < 4; ++z) {
        const uint4 *src = sums + ((z >> 1) * lo_cols + (z & 1) * 16) / 4 * 128;
        uint32_t t[4][4] = {};
#pragma unroll 1
        for (int k = 0; k < join; k += 4) {
            uint4 v[4][4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    v[u][q] = k + u < join ? __ldcg(src + (k + u) * kPartSums + q * 128) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int q = 0; q < 4; ++q) t[q][0] += v[u][q].x, t[q][1] += v[u][q].y, t[q][2] += v[u][q].z, t[q][3] += v[u][q].w;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_st4(acc.hi + (z >> 1) * acc.lo + c0 + (z & 1) * 16 + 4 * q, t[q]);
    }
    tmem_st_wait();
    tc_fence_before();  // other warpgroups may read these columns (AccCols::exact) behind their next barrier
    return true;
}

// MODE: 3 computes dV and dK (heads of 64 columns), 1 only dV, 2 only dK.  Persistent blocks.
template <int DP, int MODE>
__global__ void __launch_bounds__(DkvCfg<DP>::kThreads, 1)
    attn_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmD,
                    const __grid_constant__ AttnArgs a, const __grid_constant__ AttnLimits lim, int items) {
    using L = DkvCfg<DP>;
    constexpr int H = L::H, NS = 32 * kSoftWarps;
    static_assert(MODE != 3 || DP == 64, "both gradients: 256 accumulator columns");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t sb = smem_u32(smem);
    const uint32_t bar_kf = sb + L::kOffBar, bar_ke = bar_kf + 8 * L::KS;
    const uint32_t bar_qf = bar_ke + 8 * L::KS, bar_qe = bar_qf + 8 * L::QS;
    const uint32_t bar_sf = bar_qe + 8 * L::QS, bar_ef = bar_sf + 16;
    const uint32_t bar_cf = bar_ef + 16, bar_ce = bar_cf + 32;  // the queries' vectors full / empty
    const uint32_t bar_ee = bar_ce + 32, bar_of = bar_ee + 16, bar_oe = bar_of + 8, bar_dr = bar_oe + 8;
    volatile int *misc = (volatile int *)(smem + L::kOffBar + L::kBars * 8);  // tmem, abort, ticket
    volatile int *abort_flag = &misc[1];
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == NS) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        prefetch_tmap(&tmD);
        for (int s = 0; s < L::KS; ++s) mbar_init(bar_kf + 8 * s, 1), mbar_init(bar_ke + 8 * s, 1);
        for (int s = 0; s < L::QS; ++s) mbar_init(bar_qf + 8 * s, 1), mbar_init(bar_qe + 8 * s, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar_sf + 8 * s, 1);
            mbar_init(bar_ef + 8 * s, kSoftWarps / 2);
            mbar_init(bar_ee + 8 * s, 1);
        }
        for (int s = 0; s < 4; ++s) mbar_init(bar_cf + 8 * s, 1), mbar_init(bar_ce + 8 * s, kSoftWarps / 2);
        mbar_init(bar_of, 1);
        mbar_init(bar_oe, kSoftWarps);
        mbar_init(bar_dr, 1);
        misc[1] = 0;
        fence_barrier_init();
    }
    __syncthreads();
    auto fail = [&]() {
        *abort_flag = 1;
        raise_status(ICT_ERR_DEVICE_TIMEOUT);
    };
    // step u of a key block (an item has nu from u0 on): query head g rep + u / per, queries base + (u % per) 64 ...
    if (warp == kSoftWarps) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            auto load_tile = [&](const CUtensorMap *m, uint32_t dst, uint32_t bar, int row) {
                for (int x = 0; x < H; ++x) tma_load_2d(dst + x * kHalfTile, m, bar, 64 * x, row);
            };
            auto free = [&](uint32_t bar, int n, int stages) {
                return n < stages || wait_bar(bar + 8 * (n % stages), (n / stages - 1) & 1, lim.wait_ns, abort_flag);
            };
            bool ok = true;
            int kn = 0, qn = 0;
            for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
                const KeyItem w = key_item(a, item);
                if (w.nu == 0) continue;
                if (!(ok = free(bar_ke, kn, L::KS))) break;
                const uint32_t dst = sb + (kn % L::KS) * 2 * L::kTile, bar = bar_kf + 8 * (kn % L::KS);
                mbar_expect_tx(bar, 2 * L::kTile);
                load_tile(&tmK, dst, bar, w.bg * a.Lk + w.j0);
                load_tile(&tmV, dst + L::kTile, bar, w.bg * a.Lk + w.j0);
                ++kn;
                for (int t = w.t0; t < w.t0 + w.nw; ++t) {
                    if (!(ok = free(bar_qe, qn, L::QS))) break;
                    const int row = (w.b * a.Hq + w.g * a.rep + t / w.tiles) * a.Lq + w.base + (t % w.tiles) * 128;
                    const uint32_t q = sb + L::kOffQ + (qn % L::QS) * 2 * L::kTile, bq = bar_qf + 8 * (qn % L::QS);
                    mbar_expect_tx(bq, 2 * L::kTile);
                    load_tile(&tmQ, q, bq, row);
                    load_tile(&tmD, q + L::kTile, bq, row);
                    ++qn;
                }
            }
            if (!ok) fail();
            for (int t = max(0, kn - L::KS); t < kn; ++t)
                wait_bar(bar_kf + 8 * (t % L::KS), (t / L::KS) & 1, lim.drain_ns, nullptr);
            for (int t = max(0, qn - L::QS); t < qn; ++t)
                wait_bar(bar_qf + 8 * (t % L::QS), (t / L::QS) & 1, lim.drain_ns, nullptr);
        }
    } else if (warp == kSoftWarps + 1) {
        // ------------------------------------------------------------ TMEM and MMA issue
        tmem_alloc(smem_u32((const void *)&misc[0]), 512);
        tmem_relinquish();
        tc_fence_before();
        named_bar_sync(5, NS + 32);
        tc_fence_after();
        const uint32_t tm = __shfl_sync(0xffffffffu, (uint32_t)misc[0], 0);
        constexpr uint32_t kIdS = idesc_i8(128, kStep);
        constexpr uint32_t kIdHi = idesc_i8(128, DP, false, true);
        constexpr uint32_t kIdLo = idesc_i8(128, DP, false, true) & ~(1u << 7);
        constexpr int kDk = MODE == 3 ? kAccCol + 2 * DP : kAccCol;
        auto wait = [&](uint32_t bar, int parity) {
            return (bool)__all_sync(0xffffffffu, wait_bar(bar, (uint32_t)(parity & 1), lim.wait_ns, abort_flag));
        };
        bool ok = true;
        int kn = 0, pn = 0, on = 0, sw = 0, pw = 0;  // sw, pw: query tiles whose scores, products are done
        int sn = 0;  // steps whose scores are issued (step G of all items in buffer G & 1)
        for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
            const KeyItem w = key_item(a, item);
            if (w.nu == 0) continue;
            const uint32_t kt = sb + (kn % L::KS) * 2 * L::kTile;
            if (!(ok = wait(bar_kf + 8 * (kn % L::KS), kn / L::KS))) break;
            // half within the tile and step within the head, for the scores and for the products
            int sh = 0, sk = w.u0 % w.per, ph = 0, pk_ = sk;
            auto scores = [&](int u) {
                const int s = sw % L::QS, buf = sn & 1;
                if (sn >= 2 && !wait(bar_ee + 8 * buf, (sn >> 1) - 1)) return false;  // the buffer's last planes are used
                if (sh == 0 && !wait(bar_qf + 8 * s, sw / L::QS)) return false;
                tc_fence_after();
                const uint32_t q = sb + L::kOffQ + s * 2 * L::kTile + sh * kStep * 64;
                const uint64_t dk = smem_desc_kmajor(kt, 64), dv = smem_desc_kmajor(kt + L::kTile, 64);
                const uint64_t dq = smem_desc_kmajor(q, 64), dd = smem_desc_kmajor(q + L::kTile, 64);
                const uint32_t col = tm + buf * 128;
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
                    if (u + 1 == w.nu) umma_commit(bar_ke + 8 * (kn % L::KS));
                    umma_commit(bar_sf + 8 * buf);
                }
                __syncwarp();
                ++sn;
                if (++sk == w.per) sk = 0, sh = 0, ++sw;
                else if ((sh ^= 1) == 0) ++sw;
                return true;
            };
            ok = scores(0);
            for (int u = 0; u < w.nu && ok; ++u) {
                if (u + 1 < w.nu && !(ok = scores(u + 1))) break;
                const int buf = pn & 1;
                if (!(ok = wait(bar_ef + 8 * buf, pn >> 1))) break;
                if (u == 0 && on > 0 && !(ok = wait(bar_oe, on - 1))) break;  // the last item's gradients are read
                tc_fence_after();
                const int s = pw % L::QS;
                const uint32_t q = sb + L::kOffQ + s * 2 * L::kTile + ph * kStep * 64;
                const uint64_t dq = smem_desc_mnmajor64(q, kHalfTile), dd = smem_desc_mnmajor64(q + L::kTile, kHalfTile);
                const uint32_t e0 = tm + buf * 128, first = u ? 1u : 0u;
                const bool done = pk_ + 1 == w.per || ph == 1;
                const int ks = (min(kStep, w.nq - w.base - pk_ * kStep) + 31) / 32;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        if (kk >= ks) break;
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
                    umma_commit(bar_ee + 8 * buf);
                    if (u + 1 == w.nu) umma_commit(bar_of);
                }
                __syncwarp();
                ++pn;
                if (++pk_ == w.per) pk_ = 0, ph = 0, ++pw;
                else if ((ph ^= 1) == 0) ++pw;
            }
            ++kn;
            ++on;
        }
        if (!ok && lane == 0) fail();
        if (elect_one()) umma_commit(bar_dr);
        __syncwarp();
        wait_bar(bar_dr, 0, lim.drain_ns, nullptr);
    } else if (warp == kSoftWarps + 2) {
        // ------------------------------------------------------------ the queries' vectors
        bool ok = true;
        int cn = 0;  // steps
        for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
            const KeyItem w = key_item(a, item);
            if (w.nu == 0) continue;
            const int64_t row0 = ((int64_t)w.b * a.Hq + w.g * a.rep) * a.Lq;
            const int4 ex = a.exps[w.slot];
            const int pi = ex.x;
            const float2 fs = make_float2(attn_factor(a, w.bg), pow2f(-ex.y));
            // two queries per lane and step, read one step ahead
            int2 st[2], rw[2];
            auto fetch = [&](int u) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int i = w.base + ((w.u0 + u) % w.per) * kStep + 2 * lane + k;
                    st[k] = rw[k] = make_int2(0, 0);
                    if (u < w.nu && i < w.nq) {
                        const int64_t at = row0 + (int64_t)((w.u0 + u) / w.per) * a.Lq + i;
                        st[k] = a.stats[at];
                        if (MODE & 2) rw[k] = a.row[at];
                    }
                }
            };
            fetch(0);
            for (int u = 0; u < w.nu && ok; ++u) {
                float mm[2], r[2], d[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    // a query that sees nothing, or none: every score lies below its maximum, and r = 0
                    mm[k] = -(kAttnMagic + (st[k].y > 0 ? (float)st[k].x : 4194304.0f));
                    r[k] = attn_rho(st[k].y, pi);
                    d[k] = -(kAttnMagic + (float)rw[k].x);
                }
                fetch(u + 1);
                const int s = cn & 3;
                if (cn >= 4) ok = __all_sync(0xffffffffu, wait_bar(bar_ce + 8 * s, ((cn >> 2) - 1) & 1, lim.wait_ns, abort_flag));
                float *v = (float *)(smem + L::kOffVec) + s * L::kVec + 2 * lane;
                *reinterpret_cast<float2 *>(v) = make_float2(mm[0], mm[1]);
                *reinterpret_cast<float2 *>(v + kStep) = make_float2(r[0], r[1]);
                *reinterpret_cast<float2 *>(v + 2 * kStep) = make_float2(d[0], d[1]);
                if (lane == 0) *reinterpret_cast<float2 *>(v + 3 * kStep) = fs;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_cf + 8 * s);
                ++cn;
            }
        }
        if (!ok && lane == 0) fail();
    } else {
        // ------------------------------------------------------------ softmax: lane = key
        named_bar_sync(5, NS + 32);
        tc_fence_after();
        const uint32_t tm = (uint32_t)misc[0];
        const int wg = warp >> 2, et = threadIdx.x & 127, pair = wg >> 1, c0 = (wg & 1) * 32;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        bool ok = true;
        int on = 0, cn = 0;  // outputs, steps of the items so far
        for (int item = blockIdx.x; item < items; item += gridDim.x) {  // (outputs are written after a failure too)
            const KeyItem w = key_item(a, item);
            if (w.join == 0) continue;
            const int j = w.j0 + et;
            const int lo_i = a.causal ? j - w.off : 0;  // the first query that sees this key
            const int lo_max = warp_max(lo_i);
            const int u0 = (pair ^ cn) & 1;
            int k_in = w.per > 0 ? (w.u0 + u0) % w.per : 0;
            for (int u = u0; u < w.nu && ok; u += 2) {
                const int cs = (cn + u) & 3, buf = (cn + u) & 1;
                ok = __all_sync(0xffffffffu, wait_bar(bar_sf + 8 * buf, ((cn + u) >> 1) & 1, lim.wait_ns, abort_flag) &&
                                                 wait_bar(bar_cf + 8 * cs, ((cn + u) >> 2) & 1, lim.wait_ns, abort_flag));
                if (!ok) break;
                tc_fence_after();
                const float *vec = (const float *)(smem + L::kOffVec) + cs * L::kVec + c0;
                const float2 fs = *reinterpret_cast<const float2 *>(vec - c0 + 3 * kStep);
                const f2 f = pk(fs.x), sc = pk(fs.y);
                const int i = w.base + k_in * kStep + c0;
                const uint32_t mine = tm + lanes + buf * 128 + c0;
#pragma unroll 1
                for (int c = 0; c < 32 && i < w.nq; c += 16) {  // (the MMAs read no 32 columns behind the last query)
                    uint32_t vs[16], vd[16], plo[4], phi[4], ulo[4], uhi[4];
                    tmem_ld16(mine + c, vs);
                    if (MODE & 2) tmem_ld16(mine + kStep + c, vd);
                    tmem_ld_wait();
                    tmem_tie(vs);
                    if (MODE & 2) tmem_tie(vd);
                    if (i + c >= w.nq) {  // no such query
#pragma unroll
                        for (int q = 0; q < 4; ++q) plo[q] = phi[q] = ulo[q] = uhi[q] = 0;
                    } else if (i + c >= lo_max) dkv16<false, MODE>(vs, vd, vec + c, f, sc, 0, plo, phi, ulo, uhi);
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
                warp_arrive(bar_ef + 8 * buf);
                if (lane == 0) mbar_arrive(bar_ce + 8 * cs);
                if ((k_in += 2) >= w.per) k_in %= w.per;
            }
            cn += w.nu;
            const bool live = j < a.Lk;
            const int64_t row = (int64_t)w.b * a.Lk + j;
            if (w.nu == 0) {
                if (pair == 0 && live) {
                    if ((MODE & 1) && (wg == 0 || MODE != 3)) zero_row(a, a.dv, row, w.g, MODE == 3 ? 0 : wg * 64, 64);
                    if ((MODE & 2) && (wg == 1 || MODE != 3)) zero_row(a, a.dk, row, w.g, MODE == 3 ? 0 : wg * 64, 64);
                }
                continue;
            }
            // 32 columns of one gradient per warpgroup
            const bool is_k = MODE == 3 ? wg >= 2 : MODE == 2;
            const int cc = MODE == 3 ? (wg & 1) * 32 : wg * 32, acc = MODE == 3 && is_k ? kAccCol + 2 * DP : kAccCol;
            const int4 ex = a.exps[w.slot];
            const RowOut out = row_out(a, is_k ? a.dk : a.dv, row, w.g, j < w.nk ? 1 : 0, is_k ? a.mul : 1, live);
            if (ok) ok = __all_sync(0xffffffffu, wait_bar(bar_of, on & 1, lim.wait_ns, abort_flag));
            ++on;
            tc_fence_after();
            const AccCols sums{tm + lanes + acc, DP, ok};
            if (w.join > 1) {
                // [block][part]; heads of 128: dV's after dK's
                const int64_t at = (MODE == 1 ? a.blocks : 0) + w.slot;
                uint4 *row_sums = a.join + at * a.parts * kPartSums + ((MODE == 3 && is_k ? 128 : 0) + cc) / 4 * 128 + et;
                if (!join_parts(sums, cc, row_sums, DP, w.part, threadIdx.x == 0 ? a.tickets + at : nullptr, w.join, misc + 2, 1, NS)) {
                    warp_arrive(bar_oe);
                    continue;
                }
            }
            const int half = (MODE == 3 && is_k ? 4 * 128 : 0) + et;
            float2 *gm = (float2 *)(smem + L::kOffRed) + half;
            // two of these in turn: a warp may read its group's maxima after the accumulators are released
            int *gi = (int *)(smem + L::kOffRed + 8 * 128 * 8) + (on & 1) * 8 * 128 + half;
            fit_row_tmem<2>(a, is_k ? a.dk : a.dv, out, cc, is_k ? ex.w : ex.z, (int64_t)w.nq * a.rep <= 1024, gm, gi, 128,
                            MODE == 3 ? 2 + (wg >> 1) : 1, MODE == 3 ? NS / 2 : NS, sums, bar_oe);
        }
        if (!ok && lane == 0) fail();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kSoftWarps + 1) tmem_dealloc(__shfl_sync(0xffffffffu, (uint32_t)misc[0], 0), 512);
}

}  // namespace ict
