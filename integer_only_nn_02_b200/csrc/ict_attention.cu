// ict_attention.cu -- attention on (C,e) tensors, forward and backward (include/ict.h).
#include <string.h>

#include <algorithm>
#include <cmath>

#include "ict_attention.cuh"
#include "ict_attention_bwd.cuh"
#include "ict_attention_few.cuh"
#include "ict_attention_fwd.cuh"
#include "ict_host.h"

namespace ict {
namespace {

// ------------------------------------------------------------------ aligned operands

// Shared by the two kernels below: the rows [l0, l1) of one operand of one sequence and
// key/value head.  A vector is 16 columns; vectors of one row lie side by side.
struct OperandRows {
    const AttnOperand &o;
    int b, g, per, l0, l1, nvd;  // query heads of the group, rows, vectors of a head's columns
    __device__ __forceinline__ int exponent(int l, int h, int v) const {
        const int vec = o.col / 16 + h * nvd + v;
        return o.exp[((int64_t)b * o.L + l) * o.ngc + (o.gsh >= 0 ? vec >> o.gsh : vec / o.gv)];
    }
};

// largest exponent of the rows' groups that are not zero, over the block
__device__ __forceinline__ int block_top(const OperandRows &r, int *scratch) {
    int m = kNoExp;
    const int n = (r.l1 - r.l0) * r.nvd;
    for (int k = 0; k < r.per; ++k)
        for (int t = threadIdx.x; t < n; t += blockDim.x) {
            const int l = t / r.nvd, e = r.exponent(r.l0 + l, r.g * r.per + k, t - l * r.nvd);
            if (e != kEZero) m = max(m, e);
        }
    m = warp_max(m);
    if (threadIdx.x == 0) *scratch = kNoExp;
    __syncthreads();
    if ((threadIdx.x & 31) == 0 && m > kNoExp) atomicMax(scratch, m);
    __syncthreads();
    return *scratch;
}

// The rows' aligned copies [B][heads][L][Dp]: RNE(C 2^(e - e*)), zeros beyond the sequence's
// length and the head's width.  rows: the copy's rows [l0, lend), of which [l0, l1) are valid.
template <int NV>
__device__ __forceinline__ void copy_rows(const AttnArgs &a, const OperandRows &r, int lend, int es) {
    for (int k = 0; k < r.per; ++k) {
        const int h = r.g * r.per + k;
        int8_t *dst = r.o.copy + (((int64_t)r.b * r.o.heads + h) * r.o.L) * a.Dp;
        const int8_t *src = r.o.mant + (int64_t)r.b * r.o.L * r.o.ld + r.o.col + h * a.D;
        for (int t = threadIdx.x; t < (lend - r.l0) * NV; t += blockDim.x) {
            const int l = r.l0 + t / NV, v = t % NV;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (l < r.l1 && v < r.nvd) {
                w = *reinterpret_cast<const uint4 *>(src + (int64_t)l * r.o.ld + v * 16);
                const int e = r.exponent(l, h, v);
                if (e != es) w = rne_shift16(w, rne_index(es, e));
            }
            *reinterpret_cast<uint4 *>(dst + (int64_t)l * a.Dp + v * 16) = w;
        }
    }
}

constexpr int kTopRows = 128;      // rows of a block of the two-kernel form
constexpr int kFuseVecs = 2048;    // see align_operands

// Largest group exponent of every operand's valid rows, per sequence and key/value head
// (a.top, very negative before).  Grid (row block, sequence and head, operand).
__global__ void __launch_bounds__(256) attn_top_kernel(const __grid_constant__ AttnArgs a) {
    __shared__ int m;
    const AttnOperand &o = a.op[blockIdx.z];
    const int bg = blockIdx.x, b = bg / a.Hkv, n = clamp_len(o.lens, b, o.L), l0 = blockIdx.y * kTopRows;
    if (l0 >= n) return;
    const int e = block_top(OperandRows{o, b, bg - b * a.Hkv, o.heads / a.Hkv, l0, min(n, l0 + kTopRows), a.D / 16}, &m);
    if (threadIdx.x == 0 && e > kNoExp) atomicMax(&a.top[(blockIdx.z * a.B + b) * a.Hkv + bg % a.Hkv], e);
}
template <int NV>
__global__ void __launch_bounds__(256) attn_copy_kernel(const __grid_constant__ AttnArgs a) {
    const AttnOperand &o = a.op[blockIdx.z];
    const int bg = blockIdx.x, b = bg / a.Hkv, n = clamp_len(o.lens, b, o.L), l0 = blockIdx.y * kTopRows;
    if (l0 >= o.L) return;
    const int lend = min(o.L, l0 + kTopRows);
    copy_rows<NV>(a, OperandRows{o, b, bg - b * a.Hkv, o.heads / a.Hkv, l0, max(l0, min(n, lend)), a.D / 16}, lend,
                  a.top[blockIdx.z * a.B * a.Hkv + bg]);
}
// Both in one kernel, a block per sequence, key/value head and operand: the exponents are
// scanned by the block that copies.  One launch and one pass instead of a memset and two
// launches; for heads of 197 x 64 the three operands of 768 heads take 17 us against 34 us.
template <int NV>
__global__ void __launch_bounds__(256) attn_align_kernel(const __grid_constant__ AttnArgs a) {
    __shared__ int m;
    const AttnOperand &o = a.op[blockIdx.y];
    const int bg = blockIdx.x, b = bg / a.Hkv, n = clamp_len(o.lens, b, o.L), per = o.heads / a.Hkv;
    const OperandRows r{o, b, bg - b * a.Hkv, per, 0, n, a.D / 16};
    constexpr int U = 4;
    const int rows = per * o.L;
    if (rows * NV <= U * 256) {  // the vectors wait in registers for the block's largest exponent
        uint4 w[U];
        int e[U], mx = kNoExp;
        if (threadIdx.x == 0) m = kNoExp;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = threadIdx.x + u * 256, rw = t / NV, v = t % NV, k = per == 1 ? 0 : rw / o.L, l = rw - k * o.L;
            w[u] = make_uint4(0, 0, 0, 0);
            e[u] = kEZero;
            if (rw < rows && l < n && v < r.nvd) {
                const int h = r.g * per + k;
                w[u] = *reinterpret_cast<const uint4 *>(o.mant + ((int64_t)b * o.L + l) * o.ld + o.col + h * a.D + v * 16);
                e[u] = r.exponent(l, h, v);
                if (e[u] != kEZero) mx = max(mx, e[u]);
            }
        }
        mx = warp_max(mx);
        if ((threadIdx.x & 31) == 0 && mx > kNoExp) atomicMax(&m, mx);
        __syncthreads();
        const int es = m;
        int8_t *dst = o.copy + ((int64_t)b * o.heads + r.g * per) * o.L * a.Dp;  // the group's heads lie one after the other
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = threadIdx.x + u * 256;
            if (t >= rows * NV) continue;
            if (e[u] != es) w[u] = rne_shift16(w[u], rne_index(es, e[u]));
            *reinterpret_cast<uint4 *>(dst + (int64_t)t * 16) = w[u];
        }
        if (threadIdx.x == 0) a.top[blockIdx.y * a.B * a.Hkv + bg] = es;
        return;
    }
    const int es = block_top(r, &m);
    copy_rows<NV>(a, r, o.L, es);
    if (threadIdx.x == 0) a.top[blockIdx.y * a.B * a.Hkv + bg] = es;
}

// ------------------------------------------------------------------ backward

// d = clamp(RNE(sum_d AdO AO 2^(eO - eV))), X = 127 sum |AdO| + |d|: a lane per 16 columns.
template <int NL>
__global__ void __launch_bounds__(256) attn_row_kernel(const __grid_constant__ AttnArgs a) {
    const int v = threadIdx.x % NL;
    const int64_t rows = (int64_t)a.B * a.Hq * a.Lq, at = (int64_t)blockIdx.x * (256 / NL) + threadIdx.x / NL;
    const int64_t r = min(at, rows - 1);
    const int i = (int)(r % a.Lq), bh = (int)(r / a.Lq), h = bh % a.Hq, b = bh / a.Hq;
    const int64_t row = (int64_t)b * a.Lq + i;
    const int vec = (h * a.D) / 16 + v;
    const bool on = v < a.D / 16 && i < clamp_len(a.op[OPQ].lens, b, a.Lq);
    const int e = on ? a.o_exp[row * a.o_ngc + vec / a.o_gv] : kEZero;
    uint4 w = make_uint4(0, 0, 0, 0), d = w;
    if (on) {
        w = *reinterpret_cast<const uint4 *>(a.o_mant + row * a.o_ld + (int64_t)vec * 16);
        d = *reinterpret_cast<const uint4 *>(a.op[OPD].copy + r * a.Dp + v * 16);
    }
    int es = e == kEZero ? kNoExp : e;
    for (int o = NL / 2; o > 0; o >>= 1) es = max(es, __shfl_xor_sync(0xffffffffu, es, o));
    w = rne_shift16(w, rne_index(es, e));
    const uint32_t o4[4] = {w.x, w.y, w.z, w.w}, d4[4] = {d.x, d.y, d.z, d.w};
    int dot = 0, sum = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        dot = __dp4a((int)o4[q], (int)d4[q], dot);
        sum = __dp4a((int)__vabs4(d4[q]), 0x01010101, sum);
    }
    for (int o = NL / 2; o > 0; o >>= 1) {
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (v == 0 && at < rows) {
        const int k = es <= kNoExp ? 0 : es - attn_top(a, OPV, b * a.Hkv + h / a.rep);
        int delta;
        if (k >= 0) {
            const int64_t x = (int64_t)dot << min(k, 24);  // |dot| < 2^22: beyond 24 only the bound remains
            delta = (int)max((int64_t)-kDeltaMax, min((int64_t)kDeltaMax, x));
        } else {
            delta = rne_shr32(dot, -k);
        }
        a.row[r] = make_int2(delta, 127 * sum + abs(delta));
    }
}

// ------------------------------------------------------------------ host

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

// Few key blocks leave SMs without work, and causal ones differ in length: the queries of a key
// block are then shared by parts whose sums are joined.  The time in tiles of 128 queries (2.2 us):
// a block of threads costs about 3 beside its tiles, a part 6 and 0.6 for every part that the last
// one adds up; blocks run in waves, unequal (causal) ones as SMs become free.  Heads of 64 columns,
// one part against the chosen number: 3 x 8 causal heads of 2048 tokens on 2, 144 us against 81 us;
// 3 causal heads of 4096, 77 against 52 us; 8 heads of 512 on one, 75 against 31 us.  Where one
// part is chosen, two cost more: 12 heads of 1024 tokens 25 against 42 us, causal 24 against 28 us.
// Heads of 128 columns have two kernels and about 1.6 times the time of all of these, so that the same numbers serve
// (whole backward passes, one part, the chosen number, the best of 1 to 16): 371, 268 and 268 us; 240, 201 and 201 us;
// 203, 131 and 129 us; with one part chosen 107 against 139 us, causal 104 against 117 us.  The count of SMs is the
// B200's and not asked for: the workspace's size, which depends on the parts, is asked for without a device.
int split_parts(const AttnArgs &a) {
    const double tiles = (double)host::cdiv(a.Lq, 128) * a.rep, blocks = a.blocks, sms = 148;
    // of the queries, those that a key sees on average
    const double mean = a.Lk <= a.Lq ? (double)a.Lk / (2.0 * std::max(a.Lq, 1)) : 1.0 - (double)a.Lq / (2.0 * a.Lk);
    int best = 1;
    double least = 0;
    for (int p = 1; p <= 32 && (p == 1 || 2 * p <= tiles); ++p) {
        const double beside = p == 1 ? 3 : 6 + 0.6 * p, longest = tiles / p + beside, n = blocks * p;
        const double all = a.causal ? n * (tiles * mean / p + beside) / sms : 0;
        const double t = a.causal ? std::max(longest, all) : std::ceil(n / sms) * longest;
        if (p == 1 || t < (best == 1 ? 0.9 : 1.0) * least) best = p, least = t;
    }
    return best;
}

Div divide_by(int d) {  // d >= 1
    int l = 0;
    while ((1u << l) < (unsigned)d) ++l;
    return Div{(uint32_t)(((1ull << 32) * ((1ull << l) - (unsigned)d)) / (unsigned)d + 1), l};
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
    if ((int64_t)d->batch * d->heads_q * host::cdiv(std::max(d->len_q, d->len_k), 128) > 0x7fffffff) return ICT_ERR_LAYOUT;
    if (back && (int64_t)d->len_q * (d->heads_q / d->heads_kv) > 65536) return ICT_ERR_LAYOUT;
    memset(&a, 0, sizeof(a));
    a.B = d->batch, a.Hq = d->heads_q, a.Hkv = d->heads_kv, a.rep = a.Hq / a.Hkv, a.Lq = d->len_q, a.Lk = d->len_k;
    a.D = d->head_dim, a.Dp = a.D <= 64 ? 64 : 128, a.causal = d->causal, a.mul = d->scale_mul, a.shift = d->scale_shift;
    a.fmul = (float)((double)d->scale_mul * 12102203.0);  // log2(e) 2^23
    a.n_op = back ? 4 : 3;
    a.blocks = (int)(host::cdiv(a.Lk, kKeyBlock) * a.B * a.Hkv);
    a.parts = back ? split_parts(a) : 1;
    a.heads_q = divide_by(std::max(1, a.B * a.Hq)), a.hq = divide_by(a.Hq), a.by_rep = divide_by(a.rep);
    a.heads_kv = divide_by(std::max(1, a.B * a.Hkv)), a.hkv = divide_by(a.Hkv);
    return ICT_OK;
}

// A few queries per key/value head over many keys take the kernels that read K and V in place: at
// 16 sequences of up to 16384 keys (4 heads of 64, 3 queries each) take 70 us against 369 us with
// the tensor-core kernel; below kFewKeys keys, or with more queries (K and V are read once per
// kFewQ of them), the tiles win.
bool few_queries_path(const AttnArgs &a, bool back) {
    return !back && (int64_t)a.rep * a.Lq <= 2 * kFewQ && a.Lk >= kFewKeys;
}

struct Scratch {
    size_t top, copy[OPN], row, tmax, total;
    size_t scores, mx, sum, acc;  // the few-queries path (scores apart, the others cleared before use)
    size_t exps, join, tickets;   // backward (tickets are cleared before use)
};
Scratch scratch(const AttnArgs &a, bool back) {
    Scratch s = {};
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t p = at;
        at += (size_t)host::round_up(std::max<int64_t>(bytes, 1), 1024);
        return p;
    };
    const int64_t q = (int64_t)a.B * a.Hq * a.Lq, k = (int64_t)a.B * a.Hkv * a.Lk;
    s.top = take((int64_t)OPN * a.B * a.Hkv * 4);
    if (few_queries_path(a, back)) {
        const int64_t n = (int64_t)a.B * a.Hq * a.Lq;
        s.mx = take(n * 4);
        s.sum = take(n * 4);
        s.acc = take(n * a.Dp * 8);
        s.scores = take(n * host::round_up(a.Lk, 4) * 4);
        s.total = at;
        return s;
    }
    s.copy[OPQ] = take(q * a.Dp);
    s.copy[OPK] = take(k * a.Dp);
    s.copy[OPV] = take(k * a.Dp);
    s.copy[OPD] = take(back ? q * a.Dp : 0);
    s.row = take(back ? q * 8 : 0);
    s.tmax = take(back ? q * 4 : 0);
    s.exps = take(back ? (int64_t)a.blocks * 16 : 0);
    if (back && a.parts > 1) {
        const int64_t n = (int64_t)a.blocks * (a.Dp / 64);
        s.tickets = take(n * 4);
        s.join = take(n * a.parts * kPartSums * 16);
    }
    s.total = at;
    return s;
}

void operand(AttnOperand &o, const ict_tensor *t, int col, int heads, int L, const int32_t *lens, int8_t *copy) {
    o.mant = t->mant, o.exp = t->exp, o.ld = t->ld, o.ngc = host::groups_per_row(t), o.gv = host::vec_per_group(t);
    o.gsh = (o.gv & (o.gv - 1)) == 0 ? __builtin_ctz((unsigned)o.gv) : -1;
    o.col = col, o.heads = heads, o.L = L, o.lens = lens, o.copy = copy;
}
void output(AttnOut &o, const ict_tensor *t, int col, int D) {
    o.mant = t->mant, o.exp = t->exp, o.ld = t->ld, o.ngc = host::groups_per_row(t);
    o.G = (int)std::min<int64_t>(t->g_cols, t->cols), o.col = col;
    o.gcol = col / o.G, o.dg = D / o.G;
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

template <int NV>
int align_operands(const AttnArgs &a, cudaStream_t s) {
    const int L = std::max(a.Lq, a.Lk);
    const int64_t vecs = std::max((int64_t)a.rep * a.Lq, (int64_t)a.Lk) * NV;
    const unsigned bg = (unsigned)(a.B * a.Hkv);
    int sms = 148;
    host::device_info(&sms);
    // Few vectors per block of threads, or enough heads to fill the SMs: one kernel.  12 heads of 64
    // columns: 512 rows 7.0 us against 6.7 us in three launches, 1024 rows 11.9 against 6.9; 192 heads:
    // 1024 rows 30 against 38 us, 2048 rows 58 against 68 us.
    if (vecs <= kFuseVecs || (bg >= (unsigned)sms && vecs <= 16 * kFuseVecs)) {
        attn_align_kernel<NV><<<dim3(bg, (unsigned)a.n_op), 256, 0, s>>>(a);
        host::counted(1);
        return host::launch_status();
    }
    if (cudaMemsetAsync(a.top, 0x80, (size_t)OPN * a.B * a.Hkv * 4, s) != cudaSuccess) return ICT_ERR_CUDA;
    const dim3 grid(bg, (unsigned)host::cdiv(L, kTopRows), (unsigned)a.n_op);
    attn_top_kernel<<<grid, 256, 0, s>>>(a);
    attn_copy_kernel<NV><<<grid, 256, 0, s>>>(a);
    host::counted(2);
    return host::launch_status();
}

// [rows][Dp] aligned copy of an operand as boxes of 128 rows and 64 columns
int copy_map(CUtensorMap *m, const AttnArgs &a, int op) {
    const AttnOperand &o = a.op[op];
    return host::tmap_2d(m, o.copy, (uint64_t)a.Dp, (uint64_t)std::max<int64_t>((int64_t)a.B * o.heads * o.L, 1), (uint64_t)a.Dp,
                         64, 128, CU_TENSOR_MAP_SWIZZLE_64B);
}

// Blocks of a persistent kernel: as many as run at once, unless an item is long: then one per
// item, which the hardware hands out as blocks finish (2 x 12 causal heads of 4096: 114 us against
// 129 us with a fixed share of unequal items per block; 64 x 12 heads of 197 tokens: 65 us against
// 55 us, before later steps took 10 us from both).
unsigned blocks_for(int64_t items, int per_sm, int len) {
    int sms = 148;
    host::device_info(&sms);
    return (unsigned)(len > 512 ? items : std::min<int64_t>(items, (int64_t)sms * per_sm));
}

template <int DP>
int launch_fwd(const AttnArgs &a, cudaStream_t s) {
    using L = FwdCfg<DP>;
    CUtensorMap q, k, v;
    int st;
    if ((st = copy_map(&q, a, OPQ)) || (st = copy_map(&k, a, OPK)) || (st = copy_map(&v, a, OPV))) return st;
    if ((st = host::allow_smem<attn_fwd_kernel<DP>, L::kBytes>())) return st;
    AttnLimits lim;
    host::wait_limits(&lim.wait_ns, &lim.drain_ns);
    const int64_t items = host::cdiv(a.Lq, kQTile) * a.B * a.Hq;
    const unsigned blocks = blocks_for(items, DP == 64 ? 2 : 1, a.Lk);
    attn_fwd_kernel<DP><<<blocks, L::kThreads, L::kBytes, s>>>(q, k, v, a, lim, (int)items);
    host::counted(1);
    return host::launch_status();
}

template <int NV>
int launch_few(const AttnArgs &a, const Scratch &w, cudaStream_t s) {
    FewArgs p;
    p.a = a;
    p.R = a.rep * a.Lq;
    p.ldk = host::round_up(a.Lk, 4);
    uint8_t *base = (uint8_t *)a.top - w.top;
    p.top = a.top;
    p.mx = (int32_t *)(base + w.mx);
    p.sum = (int32_t *)(base + w.sum);
    p.acc = (unsigned long long *)(base + w.acc);
    p.scores = (int32_t *)(base + w.scores);
    // the exponents, maxima and sums lie before the scores
    if (cudaMemsetAsync(p.top, 0, w.scores - w.top, s) != cudaSuccess) return ICT_ERR_CUDA;
    const unsigned chunks = (unsigned)host::cdiv(a.Lk, kFewKeys), bg = (unsigned)(a.B * a.Hkv);
    const unsigned qs = (unsigned)host::cdiv(p.R, kFewQ);
    few_top_kernel<<<dim3((unsigned)a.B, chunks, 2), 256, 0, s>>>(p);
    few_scores_kernel<NV><<<dim3(bg, chunks, qs), 256, 0, s>>>(p);
    // as many queries per block as there are, or an even share of them
    switch (p.R <= kFewQ ? p.R : (int)host::cdiv(p.R, qs)) {
        case 1: few_values_kernel<NV, 1><<<dim3(bg, chunks, 1), 128, 0, s>>>(p); break;
        case 2: few_values_kernel<NV, 2><<<dim3(bg, chunks, 1), 128, 0, s>>>(p); break;
        case 3: few_values_kernel<NV, 3><<<dim3(bg, chunks, (unsigned)host::cdiv(p.R, 3)), 128, 0, s>>>(p); break;
        default: few_values_kernel<NV, 4><<<dim3(bg, chunks, qs), 128, 0, s>>>(p); break;
    }
    few_out_kernel<<<(unsigned)host::cdiv((int64_t)bg * p.R, 8), 256, 0, s>>>(p);
    host::counted(4);
    return host::launch_status();
}

template <int DP>
int launch_bwd(const AttnArgs &a, cudaStream_t s) {
    CUtensorMap q, k, v, d;
    int st;
    if ((st = copy_map(&q, a, OPQ)) || (st = copy_map(&k, a, OPK)) || (st = copy_map(&v, a, OPV)) || (st = copy_map(&d, a, OPD)))
        return st;
    AttnLimits lim;
    host::wait_limits(&lim.wait_ns, &lim.drain_ns);
    const int64_t rows = (int64_t)a.B * a.Hq * a.Lq;
    if (rows > 0) {
        using L = DqCfg<DP>;
        constexpr int NL = DP / 16;
        attn_row_kernel<NL><<<(unsigned)host::cdiv(rows, 256 / NL), 256, 0, s>>>(a);
        if ((st = host::allow_smem<attn_dq_kernel<DP>, L::kBytes>())) return st;
        const int64_t items = host::cdiv(a.Lq, kQTile) * a.B * a.Hq;
        attn_dq_kernel<DP><<<blocks_for(items, 1, a.Lk), L::kThreads, L::kBytes, s>>>(q, k, v, d, a, lim, (int)items);
        host::counted(2);
    }
    if ((int64_t)a.B * a.Lk > 0) {
        using L = DkvCfg<DP>;
        const int64_t items = (int64_t)a.blocks * a.parts;
        const unsigned blocks = blocks_for(items, 1, a.Lq * a.rep);
        const unsigned threads = (unsigned)std::min<int64_t>(1024, host::round_up((int64_t)a.Lq * a.rep / 2 + 1, 64));
        attn_exps_kernel<<<(unsigned)a.blocks, threads, 0, s>>>(a);
        host::counted(1);
        if (a.parts > 1) {
            if (cudaMemsetAsync(a.tickets, 0, (size_t)a.blocks * (DP / 64) * 4, s) != cudaSuccess) return ICT_ERR_CUDA;
        }
        if constexpr (DP == 64) {
            if ((st = host::allow_smem<attn_dkv_kernel<64, 3>, L::kBytes>())) return st;
            attn_dkv_kernel<64, 3><<<blocks, L::kThreads, L::kBytes, s>>>(q, k, v, d, a, lim, (int)items);
            host::counted(1);
        } else {
            if ((st = host::allow_smem<attn_dkv_kernel<DP, 1>, L::kBytes>()) || (st = host::allow_smem<attn_dkv_kernel<DP, 2>, L::kBytes>()))
                return st;
            attn_dkv_kernel<DP, 2><<<blocks, L::kThreads, L::kBytes, s>>>(q, k, v, d, a, lim, (int)items);
            attn_dkv_kernel<DP, 1><<<blocks, L::kThreads, L::kBytes, s>>>(q, k, v, d, a, lim, (int)items);
            host::counted(2);
        }
    }
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
    output(a.o, O, 0, a.D);
    const int64_t rows = (int64_t)a.B * a.Hq * a.Lq;
    if (rows == 0) return ICT_OK;
    cudaStream_t s = (cudaStream_t)stream;
    host::Timer kt(s, ICT_KC_GEMM, 4.0 * (double)rows * a.Lk * a.D);
    if (few_queries_path(a, false)) return a.Dp == 64 ? launch_few<4>(a, w, s) : launch_few<8>(a, w, s);
    if ((st = a.Dp == 64 ? align_operands<4>(a, s) : align_operands<8>(a, s))) return st;
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
    if (host::share_columns(dQ, d->q_col, wq, dK, d->k_col, wk) || host::share_columns(dQ, d->q_col, wq, dV, d->v_col, wk) ||
        host::share_columns(dK, d->k_col, wk, dV, d->v_col, wk))
        return ICT_ERR_INVALID_ARG;
    if ((st = host::device_info(nullptr))) return st;
    uint8_t *base = (uint8_t *)ws;
    operand(a.op[OPD], dO, 0, a.Hq, a.Lq, lens_q, (int8_t *)(base + w.copy[OPD]));
    a.o_mant = O->mant, a.o_exp = O->exp, a.o_ld = O->ld, a.o_ngc = host::groups_per_row(O), a.o_gv = host::vec_per_group(O);
    output(a.o, dQ, d->q_col, a.D);
    output(a.dk, dK, d->k_col, a.D);
    output(a.dv, dV, d->v_col, a.D);
    a.row = (int2 *)(base + w.row);
    a.tmax = (int32_t *)(base + w.tmax);
    a.exps = (int4 *)(base + w.exps);
    if (a.parts > 1) a.tickets = (int32_t *)(base + w.tickets), a.join = (uint4 *)(base + w.join);
    if (rq == 0 && rk == 0) return ICT_OK;
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t rows = rq * a.Hq;
    host::Timer kt(s, ICT_KC_GEMM, 10.0 * (double)rows * a.Lk * a.D);
    if ((st = a.Dp == 64 ? align_operands<4>(a, s) : align_operands<8>(a, s))) return st;
    return a.Dp == 64 ? launch_bwd<64>(a, s) : launch_bwd<128>(a, s);
}

}  // extern "C"
