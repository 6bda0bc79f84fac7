// dropout.hip -- dropout whose mask is a function of (seed, stream, row,
// column) and never stored, with an optional residual add:
// y = [residual +] (kept ? x * scale : 0), in binary32, rounded once.
//
// HBM-bound: each input read and the output written once.  A thread takes
// kPerThread chunks of eight elements, kThreads apart, with all their loads
// issued before the first Philox call.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4q_internal.h"
#include "row_ops.h"

namespace fp4q {

namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 4;

template <typename T, bool kRes, bool kTail>
__global__ __launch_bounds__(kThreads) void dropout_kernel(const T *x, const T *res, T *y, uint32_t cols, int64_t ld_x,
                                                           int64_t ld_r, int64_t ld_y, uint32_t nchunks, FastDiv cpr_div,
                                                           uint32_t cpr, Dropout d)
{
    const uint64_t base = (uint64_t)blockIdx.x * (kThreads * kPerThread) + threadIdx.x;
    Chunk<T> q[kPerThread], s[kPerThread];
    uint32_t row[kPerThread], col[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const uint64_t at = base + i * kThreads;
        const uint32_t c = at < nchunks ? (uint32_t)at : 0u;
        row[i] = fast_div(c, cpr_div);
        col[i] = c - row[i] * cpr;
        load_chunk<T, kTail>(x + row[i] * ld_x, col[i], cols, q[i]);
        if (kRes) load_chunk<T, kTail>(res + row[i] * ld_r, col[i], cols, s[i]);
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        float v[8];
        q[i].get(v);
        if (d.drop) apply_dropout(d, row[i], col[i], v);
        if (kRes) {
            float r[8];
            s[i].get(r);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = r[j] + v[j];
        }
        q[i].set(v);
        if (base + i * kThreads < nchunks) store_chunk<T, kTail>(y + row[i] * ld_y, col[i], cols, q[i]);
    }
}

template <typename T>
int launch(const DropoutArgs &a, hipStream_t st)
{
    const uint32_t cols = (uint32_t)a.cols, cpr = (cols + 7) / 8;
    const uint32_t nchunks = (uint32_t)(a.rows * cpr);
    const unsigned grid = (unsigned)(((uint64_t)nchunks + kThreads * kPerThread - 1) / (kThreads * kPerThread));
    const Dropout d = dropout_of(a.p, a.seed, a.stream_id);
    const FastDiv fd = fast_div_for(cpr);
#define FP4Q_DROP(RES, TAIL)                                                                                       \
    hipLaunchKernelGGL((dropout_kernel<T, RES, TAIL>), dim3(grid), dim3(kThreads), 0, st,                          \
                       reinterpret_cast<const T *>(a.x), reinterpret_cast<const T *>(a.residual),                  \
                       reinterpret_cast<T *>(a.y), cols, a.ld_x, a.ld_r, a.ld_y, nchunks, fd, cpr, d)
    if (a.residual) {
        if (cols % 8) FP4Q_DROP(true, true); else FP4Q_DROP(true, false);
    } else {
        if (cols % 8) FP4Q_DROP(false, true); else FP4Q_DROP(false, false);
    }
#undef FP4Q_DROP
    return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace

int launch_dropout(const DropoutArgs &a, hipStream_t st)
{
    return a.bf16 ? launch<bf16_t>(a, st) : launch<float>(a, st);
}

}  // namespace fp4q
