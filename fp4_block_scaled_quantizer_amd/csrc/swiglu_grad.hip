// swiglu_grad.hip -- the gradient of SwiGLU, h = g sigma(g) u:
//   dg = dh u (sigma + h_g (1 - sigma)) with h_g = g sigma,   du = dh h_g,
// sigma(g) = 1 / (1 + e^-g), and optionally h itself again (the weight
// gradient of the down projection needs it and then need not keep it).
// C's columns interleave gate and up as in swiglu.hip; dC has the same order.
//
// C may come as 8-bit rows: its values through the same steps.
//
// HBM-bound: 6 bytes read (4.06 with 8-bit rows) and 4 (6 with h) written per
// hidden element.  A thread takes eight hidden columns of one row: three loads
// (16 bytes each, of 8-bit rows 8) and two or three stores, whose pieces of 64
// bytes (pair = 32) the caches join, so nothing is streamed past them
// (non-temporal loads: 250 us instead of 237).
// 8192 x 14336 with h: 238 us, 5.9 TB/s; without h 196 us, 6.0 TB/s; 64 x
// 14336: 4.2 us a call, launch and latency.  C as 8-bit rows: 8192 x 14336 with
// h 202 us, without 164, 5.8 TB/s; 64 x 14336 4.7.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4q_internal.h"
#include "pack8.h"
#include "row_ops.h"

namespace fp4q {

namespace {

constexpr int kThreads = 256;

// sigma(x) and 1 - sigma(x) from e = e^-|x| and r = 1 / (1 + e): neither
// loses digits far from zero (1 - sigma by subtraction would).  e is the
// hardware's exp2, which flushes subnormal results: below 2^-126 it is taken
// 64 binades higher and scaled down.  exp2 and reciprocal are off by about
// one unit in the last place and the exponent by |x| 2^-24, far below the
// bf16 rounding of what is made of them.
__device__ __forceinline__ void sigmoid_pair(float x, float &s, float &c)
{
    const float t = __builtin_fabsf(x) * -0x1.715476p+0f;
    const bool low = t < -126.0f;
    const float e = __builtin_amdgcn_exp2f(low ? t + 64.0f : t) * (low ? 0x1p-64f : 1.0f);
    const float r = __builtin_amdgcn_rcpf(1.0f + e), er = e * r;
    s = x >= 0.0f ? r : er;
    c = x >= 0.0f ? er : r;
}

// A thread takes one chunk of eight hidden columns.  kRows: a workgroup is
// within one row, whose address is then the same for all its threads; where
// a row's chunks do not divide into workgroups, they run on over the rows
// instead, so that none is left part empty.  grid.y: `rows` rows each, of
// fewer than 2^31 chunks together; `row_div` divides by a row's workgroups
// or chunks (`per_row`), `pair_div` by a group's chunks.  Workgroups within a
// row / chunks run on, with h: 8192 x 14336 237 / 242 us; with the last
// workgroup of a row part empty / run on, 8192 x 11008 210 / 183, 16384 x
// 2080 111 / 73, 65536 x 64 55 / 13.
template <bool kH, bool kRows, bool kPack8>
__global__ __launch_bounds__(kThreads) void swiglu_grad_kernel(const uint16_t *dh, const uint16_t *c,
                                                               const uint8_t *codes, const uint8_t *scales,
                                                               uint16_t *dc, uint16_t *h, int64_t M, int64_t ld_dh,
                                                               int64_t ldc, int64_t ld_dc, int64_t ldh, uint32_t rows,
                                                               uint32_t per_row, FastDiv row_div, uint32_t pair_chunks,
                                                               FastDiv pair_div)
{
    const int64_t row0 = (int64_t)blockIdx.y * rows, pair = (int64_t)pair_chunks * 8;
    const uint32_t at = kRows ? blockIdx.x : blockIdx.x * (uint32_t)kThreads + threadIdx.x;
    const uint32_t r = fast_div(at, row_div), rest = at - r * per_row;
    const uint32_t k = kRows ? rest * kThreads + threadIdx.x : rest;
    const bool in = r < rows && row0 + r < M;
    const int64_t m = in ? row0 + r : row0;  // past the end: a chunk of the first row, not stored
    const int64_t j = (int64_t)k * 8, gcol = j + (int64_t)fast_div(k, pair_div) * pair;
    typename std::conditional<kPack8, Packed8, Chunk<bf16_t>>::type g, u;
    if constexpr (kPack8) {  // dense rows
        const uint64_t at = (uint64_t)(m * ldc + gcol) >> 3;
        g.load(codes, scales, at);
        u.load(codes, scales, at + pair_chunks);
    } else {
        const uint16_t *row = c + m * ldc;
        g.q = *reinterpret_cast<const u32x4v *>(row + gcol);
        u.q = *reinterpret_cast<const u32x4v *>(row + gcol + pair);
    }
    const u32x4v d = *reinterpret_cast<const u32x4v *>(dh + m * ld_dh + j);
    u32x4v og, ou, oh;
    float gs[8], us[8];
    g.get(gs);
    u.get(us);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a[2], b[2], e[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float gv = gs[2 * i + n], uv = us[2 * i + n];
            const float dv = n ? bf16_hi(d[i]) : bf16_lo(d[i]);
            float sg, cg;
            sigmoid_pair(gv, sg, cg);
            const float act = gv * sg;
            a[n] = dv * uv * __builtin_fmaf(act, cg, sg);
            b[n] = dv * act;
            if (kH) e[n] = silu_f32(gv) * uv;  // as the forward kernels compute it
        }
        og[i] = pack_bf16x2(a[0], a[1]);
        ou[i] = pack_bf16x2(b[0], b[1]);
        if (kH) oh[i] = pack_bf16x2(e[0], e[1]);
    }
    if (!in) return;
    uint16_t *out = dc + m * ld_dc + gcol;
    *reinterpret_cast<u32x4v *>(out) = og;
    *reinterpret_cast<u32x4v *>(out + pair) = ou;
    if (kH) *reinterpret_cast<u32x4v *>(h + m * ldh + j) = oh;
}

template <bool kH, bool kRows, bool kPack8>
void run(const SwigluGradArgs &a, hipStream_t st)
{
    const uint32_t chunks = (uint32_t)(a.F / 8), pair_chunks = (uint32_t)(a.pair / 8);
    const uint32_t per_row = kRows ? chunks / kThreads : chunks;
    int64_t rows = ((int64_t)1 << 31) / chunks;
    if (rows > a.M) rows = a.M;
    const dim3 grid((unsigned)((rows * chunks + kThreads - 1) / kThreads), (unsigned)((a.M + rows - 1) / rows));
    hipLaunchKernelGGL((swiglu_grad_kernel<kH, kRows, kPack8>), grid, dim3(kThreads), 0, st,
                       reinterpret_cast<const uint16_t *>(a.dh), reinterpret_cast<const uint16_t *>(a.c),
                       a.c_codes, a.c_scales, reinterpret_cast<uint16_t *>(a.dc), reinterpret_cast<uint16_t *>(a.h),
                       a.M, a.ld_dh, kPack8 ? 2 * a.F : a.ldc, a.ld_dc, a.ldh, (uint32_t)rows, per_row, fast_div_for(per_row),
                       pair_chunks,
                       fast_div_for(pair_chunks));
}

template <bool kPack8>
void pick(const SwigluGradArgs &a, hipStream_t st)
{
    const bool whole = a.F % (8 * kThreads) == 0;
    if (a.h)
        whole ? run<true, true, kPack8>(a, st) : run<true, false, kPack8>(a, st);
    else
        whole ? run<false, true, kPack8>(a, st) : run<false, false, kPack8>(a, st);
}

}  // namespace

int launch_swiglu_grad(const SwigluGradArgs &a, hipStream_t st)
{
    a.c_codes ? pick<true>(a, st) : pick<false>(a, st);
    return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace fp4q
