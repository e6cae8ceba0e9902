// ict_host.h -- host-side services of ict_api.cu that the library's other source files use.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/ict.h"

namespace ict {
namespace host {

int device_info(int *sms);  // ICT_OK on sm_100, and its SM count
int int8_only();            // ICT_ERR_LAYOUT while the mantissa width is not 8
int launch_status();
void counted(int n);        // n kernels launched
int check_tensor(const ict_tensor *t);
int check_vec(const ict_tensor *t);  // 16-byte vectors: pointer, ld, cols, group width
int tmap_2d(CUtensorMap *m, const void *base, uint64_t inner, uint64_t outer, uint64_t stride, uint32_t box_inner,
            uint32_t box_outer, CUtensorMapSwizzle sw);
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }
// of a tensor that check_vec has passed: groups of a row, 16-column vectors of a group
inline int groups_per_row(const ict_tensor *t) { return (int)cdiv(t->cols, t->g_cols); }
inline int vec_per_group(const ict_tensor *t) { return (int)((t->g_cols >= t->cols ? t->cols : t->g_cols) / 16); }
// columns [c, c + w) of `rows` rows of bytes, ld apart
struct Bytes {
    intptr_t at;
    int64_t rows, ld, w;
};
inline Bytes mantissas(const ict_tensor *t, int64_t c, int64_t w) { return {(intptr_t)t->mant + c, t->rows, t->ld, w}; }
inline Bytes exponents(const ict_tensor *t, int64_t c, int64_t w) {
    const int64_t g0 = c / t->g_cols;
    return {(intptr_t)t->exp + g0, cdiv(t->rows, t->g_rows), groups_per_row(t), cdiv(c + w, t->g_cols) - g0};
}
// a and b share a byte.  Rows of one ld repeat the pattern of the first two; rows of different ld whose ranges
// meet count as shared.
inline bool meet(const Bytes &a, const Bytes &b) {
    if (a.at > b.at) return meet(b, a);
    if (a.rows == 0 || b.rows == 0 || a.w == 0 || b.w == 0) return false;
    const int64_t d = b.at - a.at;
    if (d >= (a.rows - 1) * a.ld + a.w) return false;
    return a.ld != b.ld || d % a.ld < a.w || d % a.ld + b.w > a.ld;
}
// columns [ca, ca + wa) of a and [cb, cb + wb) of b share memory, mantissas or exponents
inline bool share_columns(const ict_tensor *a, int64_t ca, int64_t wa, const ict_tensor *b, int64_t cb, int64_t wb) {
    const Bytes x[2] = {mantissas(a, ca, wa), exponents(a, ca, wa)}, y[2] = {mantissas(b, cb, wb), exponents(b, cb, wb)};
    return meet(x[0], y[0]) || meet(x[0], y[1]) || meet(x[1], y[0]) || meet(x[1], y[1]);
}
void wait_limits(uint64_t *wait_ns, uint64_t *drain_ns);

// Dynamic shared memory of a kernel, set once per device (the call costs a microsecond of every launch).  The size is
// the kernel's largest, whatever a call needs: threads that meet here set the same value, and it never goes down.
template <auto Kernel, int Bytes>
int allow_smem() {
    static std::atomic<bool> set[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return ICT_ERR_CUDA;
    if (set[dev].load(std::memory_order_acquire)) return ICT_OK;
    if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Bytes) != cudaSuccess) return ICT_ERR_CUDA;
    set[dev].store(true, std::memory_order_release);
    return ICT_OK;
}

// the source files' device status words, OR-ed into *v and cleared (the stream is idle)
int take_status_attention(int32_t *v);
int take_status_norm(int32_t *v);

// brackets the launches made during its lifetime with a pair of events (ict_timing_enable)
struct Timer {
    Timer(cudaStream_t s, int kernel_class, double work);
    ~Timer();
    Timer(const Timer &) = delete;
    Timer &operator=(const Timer &) = delete;

private:
    alignas(8) unsigned char mem[48];
    void *impl;
};


}  // namespace host
}  // namespace ict
