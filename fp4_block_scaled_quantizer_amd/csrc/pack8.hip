// pack8.hip -- rows to 8-bit block-scaled rows and back (the format is in
// pack8.h): what a training step keeps of its activations for the backward
// pass, in 33/64 of the bf16 bytes.
//
// HBM-bound: each element read once and written once.  A thread takes
// kPerThread chunks of eight elements, kThreads apart, so that a wave's loads
// and stores are whole cache lines; the packed side is dense whatever the
// other side's pitch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4q_internal.h"
#include "pack8.h"

namespace fp4q {

namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 4;

template <typename T>
__global__ __launch_bounds__(kThreads) void pack8_kernel(const T *x, uint8_t *codes, uint8_t *scales, int64_t ld,
                                                         uint32_t nchunks, uint32_t cpr, FastDiv cpr_div)
{
    const uint64_t base = (uint64_t)blockIdx.x * (kThreads * kPerThread) + threadIdx.x;
    Chunk<T> q[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const uint64_t at = base + i * kThreads;
        const uint32_t c = at < nchunks ? (uint32_t)at : 0u;
        const uint32_t row = fast_div(c, cpr_div);
        q[i].template load<kStream<T>>(x + (row * ld + (c - row * cpr) * 8u));
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const uint64_t at = base + i * kThreads;
        const bool in = at < nchunks;
        const Packed8 p = pack8(q[i]);
        const uint32_t lane16 = threadIdx.x & 15u;
        store_scales8(scales + (at >> 2), p.scale, lane16, (at | 15u) < nchunks, in);
        if (in) store_vec<true>(reinterpret_cast<u32x2v *>(codes + at * 8u), p.q);
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void unpack8_kernel(const uint8_t *codes, const uint8_t *scales, T *y, int64_t ld,
                                                           uint32_t nchunks, uint32_t cpr, FastDiv cpr_div)
{
    const uint64_t base = (uint64_t)blockIdx.x * (kThreads * kPerThread) + threadIdx.x;
    Packed8 p[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const uint64_t at = base + i * kThreads;
        p[i].load<true>(codes, scales, at < nchunks ? at : 0u);
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const uint64_t at = base + i * kThreads;
        if (at >= nchunks) continue;
        const uint32_t c = (uint32_t)at, row = fast_div(c, cpr_div);
        float v[8];
        Chunk<T> q;
        p[i].get(v);
        q.set(v);
        q.template store<kStream<T>>(y + (row * ld + (c - row * cpr) * 8u));
    }
}

}  // namespace

int launch_pack8(const Pack8Args &a, hipStream_t st)
{
    const uint32_t cpr = (uint32_t)(a.cols / 8), nchunks = (uint32_t)(a.rows * cpr);
    const unsigned grid = (unsigned)(((uint64_t)nchunks + kThreads * kPerThread - 1) / (kThreads * kPerThread));
    const FastDiv fd = fast_div_for(cpr);
    uint8_t *codes = reinterpret_cast<uint8_t *>(a.codes), *scales = reinterpret_cast<uint8_t *>(a.scales);
#define FP4Q_PACK8(KERNEL, T, ...) \
    hipLaunchKernelGGL((KERNEL<T>), dim3(grid), dim3(kThreads), 0, st, __VA_ARGS__, a.ld, nchunks, cpr, fd)
    if (a.unpack && a.bf16)
        FP4Q_PACK8(unpack8_kernel, bf16_t, codes, scales, reinterpret_cast<bf16_t *>(a.x));
    else if (a.unpack)
        FP4Q_PACK8(unpack8_kernel, float, codes, scales, reinterpret_cast<float *>(a.x));
    else if (a.bf16)
        FP4Q_PACK8(pack8_kernel, bf16_t, reinterpret_cast<const bf16_t *>(a.x), codes, scales);
    else
        FP4Q_PACK8(pack8_kernel, float, reinterpret_cast<const float *>(a.x), codes, scales);
#undef FP4Q_PACK8
    return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace fp4q
