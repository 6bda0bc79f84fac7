// dropout.hip -- dropout whose mask is a function of (seed, stream, row,
// column) and never stored, with an optional residual add:
// y = [residual +] (kept ? x * scale : 0), in binary32, rounded once.
//
// HBM-bound: each input read and the output written once.  A thread takes
// kPerThread chunks of eight elements, kThreads apart, and makes their random
// words (one Philox call of ten rounds per chunk, about half the time that
// the memory takes) while the loads are under way.  8192 x 14336 bf16: 75.4
// us, 6.2 TB/s, as without dropout (p = 0: 75.2); 64 x 4096: 4.0 us a call,
// launch and latency.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4q_internal.h"
#include "row_ops.h"

namespace fp4q {

namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 4;

// a span whose row pointer already stands at its first element
__device__ __forceinline__ Span here(Span s)
{
    s.from = 0u;
    return s;
}

template <typename T, bool kRes, Edge kEdge>
__global__ __launch_bounds__(kThreads) void dropout_kernel(const T *x, const T *res, T *y, uint32_t cols, int64_t ld_x,
                                                           int64_t ld_r, int64_t ld_y, uint32_t nchunks, FastDiv cpr_div,
                                                           uint32_t cpr, Dropout d)
{
    const uint64_t base = (uint64_t)blockIdx.x * (kThreads * kPerThread) + threadIdx.x;
    Chunk<T> q[kPerThread], s[kPerThread];
    uint32_t row[kPerThread], col[kPerThread];
    Span sp[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const uint64_t at = base + i * kThreads;
        const uint32_t c = at < nchunks ? (uint32_t)at : 0u;
        row[i] = fast_div(c, cpr_div);
        col[i] = c - row[i] * cpr;
        sp[i] = span_of<kEdge>(col[i], cols);
        load_chunk<T, kEdge, kStream<T>>(x + (row[i] * ld_x + sp[i].from), here(sp[i]), cols, q[i]);
        if (kRes) load_chunk<T, kEdge, kStream<T>>(res + (row[i] * ld_r + sp[i].from), here(sp[i]), cols, s[i]);
    }
    __builtin_amdgcn_sched_barrier(0);
    Draws w[kPerThread];
    if (d.drop) {
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) w[i] = draws_of<kEdge>(d, row[i], col[i], sp[i]);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        float v[8];
        q[i].get(v);
        if (d.drop) apply_dropout(d, w[i], v);
        if (kRes) {
            float r[8];
            s[i].get(r);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = r[j] + v[j];
        }
        q[i].set(v);
        if (base + i * kThreads < nchunks) store_chunk<T, kEdge, kStream<T>>(y + (row[i] * ld_y + sp[i].from), here(sp[i]), q[i]);
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
#define FP4Q_DROP(RES, EDGE)                                                                                       \
    hipLaunchKernelGGL((dropout_kernel<T, RES, EDGE>), dim3(grid), dim3(kThreads), 0, st,                          \
                       reinterpret_cast<const T *>(a.x), reinterpret_cast<const T *>(a.residual),                  \
                       reinterpret_cast<T *>(a.y), cols, a.ld_x, a.ld_r, a.ld_y, nchunks, fd, cpr, d)
#define FP4Q_DROP_R(EDGE) \
    do { if (a.residual) FP4Q_DROP(true, EDGE); else FP4Q_DROP(false, EDGE); } while (0)
    switch (edge_of(a.cols)) {
    case kWhole: FP4Q_DROP_R(kWhole); break;
    case kRagged: FP4Q_DROP_R(kRagged); break;
    case kTiny: FP4Q_DROP_R(kTiny); break;
    }
#undef FP4Q_DROP_R
#undef FP4Q_DROP
    return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace

int launch_dropout(const DropoutArgs &a, hipStream_t st)
{
    return a.bf16 ? launch<bf16_t>(a, st) : launch<float>(a, st);
}

}  // namespace fp4q
