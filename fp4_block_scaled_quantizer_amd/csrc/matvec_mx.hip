// matvec_mx.hip -- products of few rows with MXFP4 weights (matvec.h), and of no
// columns, with either format's.
#include "matvec.h"

namespace fp4q {

namespace {

constexpr uint32_t kZeroThreads = 256, kZeroPerThread = 4;

// Y = 0.  grid.y: rows.  A workgroup has 1024 columns, so that a launch's
// threads along x are below 2^32 at any N.
template <typename T>
__global__ __launch_bounds__(kZeroThreads) void zero_rows_kernel(T *y, uint32_t N, int64_t ld)
{
    const uint32_t n = blockIdx.x * (kZeroThreads * kZeroPerThread) + threadIdx.x;
#pragma unroll
    for (uint32_t i = 0; i < kZeroPerThread; ++i)
        if (n + i * kZeroThreads < N) y[blockIdx.y * ld + n + i * kZeroThreads] = (T)0;
}

}  // namespace

int launch_matvec_zero(const MatvecArgs &g, hipStream_t st)
{
    const uint32_t N = (uint32_t)g.N, once = kZeroThreads * kZeroPerThread;
    const dim3 grid((N + once - 1u) / once, (unsigned)g.M);
    if (g.y_bf16)
        hipLaunchKernelGGL(zero_rows_kernel<uint16_t>, grid, dim3(kZeroThreads), 0, st, reinterpret_cast<uint16_t *>(g.y), N, g.ld_y);
    else
        hipLaunchKernelGGL(zero_rows_kernel<float>, grid, dim3(kZeroThreads), 0, st, reinterpret_cast<float *>(g.y), N, g.ld_y);
    return hipGetLastError() == hipSuccess ? 0 : 1;
}

int launch_matvec_mx(const MatvecArgs &g, hipStream_t st)
{
    const int units = device_cu_count();
    if (units <= 0) return 1;
    const Matvec a = matvec_of(g);
    if (g.x_scales)
        pick_matvec<kMx, true>(a, !g.tiled, (uint32_t)units, st);
    else
        pick_matvec<kMx, false>(a, !g.tiled, (uint32_t)units, st);
    return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace fp4q
