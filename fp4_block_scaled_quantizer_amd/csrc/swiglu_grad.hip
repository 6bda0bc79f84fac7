// swiglu_grad.hip -- the gradient of SwiGLU, h = g sigma(g) u:
//   dg = dh u (sigma + h_g (1 - sigma)) with h_g = g sigma,   du = dh h_g,
// sigma(g) = 1 / (1 + e^-g), and optionally h itself again (the weight
// gradient of the down projection needs it and then need not keep it).
// C's columns interleave gate and up as in swiglu.hip; dC has the same order.
//
// HBM-bound: 6 bytes read and 4 (6 with h) written per hidden element.  A
// thread takes eight hidden columns of one row: three 16-byte loads and two
// or three stores, whose pieces of 64 bytes (pair = 32) the caches join, so
// nothing is streamed past them (non-temporal loads: 250 us instead of 237).
// 8192 x 14336 with h: 237 us, 5.9 TB/s; without h 195 us, 6.0 TB/s; 64 x
// 14336: 4.2 us a call, launch and latency.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4q_internal.h"
#include "row_ops.h"

namespace fp4q {

namespace {

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

// grid.x covers F / 8 column chunks, grid.y strides over rows
template <bool kH>
__global__ __launch_bounds__(256) void swiglu_grad_kernel(const uint16_t *dh, const uint16_t *c,
                                                          uint16_t *dc, uint16_t *h, int64_t M, int64_t F,
                                                          int64_t ld_dh, int64_t ldc, int64_t ld_dc, int64_t ldh,
                                                          int64_t pair)
{
    const int64_t j = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (j >= F) return;
    const int64_t gcol = (j / pair) * 2 * pair + (j % pair);
    for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
        const uint16_t *row = c + m * ldc + gcol;
        const u32x4v g = *reinterpret_cast<const u32x4v *>(row);
        const u32x4v u = *reinterpret_cast<const u32x4v *>(row + pair);
        const u32x4v d = *reinterpret_cast<const u32x4v *>(dh + m * ld_dh + j);
        u32x4v og, ou, oh;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a[2], b[2], e[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float gv = k ? bf16_hi(g[i]) : bf16_lo(g[i]);
                const float uv = k ? bf16_hi(u[i]) : bf16_lo(u[i]);
                const float dv = k ? bf16_hi(d[i]) : bf16_lo(d[i]);
                float sg, cg;
                sigmoid_pair(gv, sg, cg);
                const float act = gv * sg;
                a[k] = dv * uv * __builtin_fmaf(act, cg, sg);
                b[k] = dv * act;
                if (kH) e[k] = silu_f32(gv) * uv;  // as the forward kernels compute it
            }
            og[i] = pack_bf16x2(a[0], a[1]);
            ou[i] = pack_bf16x2(b[0], b[1]);
            if (kH) oh[i] = pack_bf16x2(e[0], e[1]);
        }
        uint16_t *out = dc + m * ld_dc + gcol;
        *reinterpret_cast<u32x4v *>(out) = og;
        *reinterpret_cast<u32x4v *>(out + pair) = ou;
        if (kH) *reinterpret_cast<u32x4v *>(h + m * ldh + j) = oh;
    }
}

}  // namespace

int launch_swiglu_grad(const SwigluGradArgs &a, hipStream_t st)
{
    const int64_t chunks = a.F / 8;
    const unsigned gx = (unsigned)((chunks + 255) / 256);
    const unsigned gy = (unsigned)(a.M < 65535 ? a.M : 65535);
    const uint16_t *dh = reinterpret_cast<const uint16_t *>(a.dh), *c = reinterpret_cast<const uint16_t *>(a.c);
    uint16_t *dc = reinterpret_cast<uint16_t *>(a.dc), *h = reinterpret_cast<uint16_t *>(a.h);
    if (h)
        hipLaunchKernelGGL(swiglu_grad_kernel<true>, dim3(gx, gy), dim3(256), 0, st, dh, c, dc, h, a.M, a.F, a.ld_dh,
                           a.ldc, a.ld_dc, a.ldh, a.pair);
    else
        hipLaunchKernelGGL(swiglu_grad_kernel<false>, dim3(gx, gy), dim3(256), 0, st, dh, c, dc, h, a.M, a.F, a.ld_dh,
                           a.ldc, a.ld_dc, a.ldh, a.pair);
    return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace fp4q
