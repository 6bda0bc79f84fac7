// pack8.hip -- rows to 8-bit block-scaled rows and back (the format is in
// pack8.h): what a training step keeps of its activations for the backward
// pass, in 33/64 of the bf16 bytes.
//
// HBM-bound: each element read once and written once.  A thread takes
// kPerThread chunks of eight elements, kThreads apart, so that a wave's loads
// and stores are whole cache lines; the packed side is dense whatever the
// other side's pitch.
//   Matrices from memory, where a copy reaches 6.3 TB/s: pack 8192 x 28672 bf16
// 112.7 us, 6.3 TB/s, 8192 x 4096 bf16 18.6 and binary32 30.2, 5.5; unpack 8192
// x 4096 to bf16 18.1, 5.6, to binary32 29.0, 5.8; 1537 x 4096 to bf16 4.6 us a
// call, launch and latency.
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

// kElements of a thread's piece: 16 bytes of y, so that a wave's store is whole
// cache lines (binary32 by eights, two stores that each touch every line:
// 8192 x 4096 38.2 us, 29.2 by fours).
template <typename T> constexpr int kElements = 16 / sizeof(T);

template <typename T>
__global__ __launch_bounds__(kThreads) void unpack8_kernel(const uint8_t *codes, const uint8_t *scales, T *y, int64_t ld,
                                                           uint64_t npieces, uint32_t per_row, FastDiv row_div,
                                                           uint32_t rows_once)
{
    typedef typename std::conditional<sizeof(T) == 2, u32x2v, uint32_t>::type Codes;
    constexpr int kE = kElements<T>;
    // grid.y: rows_once rows each, of fewer than 2^32 pieces together
    const uint64_t base = (uint64_t)blockIdx.x * (kThreads * kPerThread) + threadIdx.x;
    const int64_t row0 = (int64_t)blockIdx.y * rows_once;
    const uint64_t from = (uint64_t)row0 * per_row, here = min((uint64_t)rows_once * per_row, npieces - from);
    Codes q[kPerThread];
    uint32_t scale[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const uint64_t at = base + i * kThreads, c = from + (at < here ? at : 0u);
        q[i] = load_vec<true>(reinterpret_cast<const Codes *>(codes) + c);
        scale[i] = scales[c / (32 / kE)];
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const uint64_t at = base + i * kThreads;
        if (at >= here) continue;
        const uint32_t row = fast_div((uint32_t)at, row_div), piece = (uint32_t)at - row * per_row;
        T *to = y + ((row0 + row) * ld + (int64_t)piece * kE);
        const float s = mx_scale_f32(scale[i]);
        if constexpr (sizeof(T) == 2) {
            Packed8 p;
            p.q = q[i];
            p.scale = scale[i];
            float v[8];
            Chunk<bf16_t> out;
            p.get(v);
            out.set(v);
            out.template store<true>(to);
        } else {
            const f32x2v lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q[i], s, false);
            const f32x2v hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q[i], s, true);
            store_vec<true>(reinterpret_cast<u32x4_a4 *>(to), (u32x4v){f2u(lo[0]), f2u(lo[1]), f2u(hi[0]), f2u(hi[1])});
        }
    }
}

template <typename T>
void run_pack8(const Pack8Args &a, hipStream_t st)
{
    const uint32_t cpr = (uint32_t)(a.cols / 8), nchunks = (uint32_t)(a.rows * cpr);
    const unsigned grid = (unsigned)(((uint64_t)nchunks + kThreads * kPerThread - 1) / (kThreads * kPerThread));
    hipLaunchKernelGGL((pack8_kernel<T>), dim3(grid), dim3(kThreads), 0, st, reinterpret_cast<const T *>(a.x),
                       reinterpret_cast<uint8_t *>(a.codes), reinterpret_cast<uint8_t *>(a.scales), a.ld, nchunks, cpr,
                       fast_div_for(cpr));
}

template <typename T>
void run_unpack8(const Pack8Args &a, hipStream_t st)
{
    const uint32_t per_row = (uint32_t)(a.cols / kElements<T>);
    int64_t rows = ((int64_t)1 << 31) / per_row;
    if (rows < 1) rows = 1;
    if (rows > a.rows) rows = a.rows;
    const dim3 grid((unsigned)(((uint64_t)rows * per_row + kThreads * kPerThread - 1) / (kThreads * kPerThread)),
                    (unsigned)((a.rows + rows - 1) / rows));
    hipLaunchKernelGGL((unpack8_kernel<T>), grid, dim3(kThreads), 0, st, reinterpret_cast<const uint8_t *>(a.codes),
                       reinterpret_cast<const uint8_t *>(a.scales), reinterpret_cast<T *>(a.x), a.ld,
                       (uint64_t)a.rows * per_row, per_row, fast_div_for(per_row), (uint32_t)rows);
}

}  // namespace

int launch_pack8(const Pack8Args &a, hipStream_t st)
{
    if (a.unpack)
        a.bf16 ? run_unpack8<bf16_t>(a, st) : run_unpack8<float>(a, st);
    else
        a.bf16 ? run_pack8<bf16_t>(a, st) : run_pack8<float>(a, st);
    return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace fp4q
