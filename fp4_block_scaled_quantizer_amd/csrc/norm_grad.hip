// norm_grad.hip -- the gradient of the norms (norm_grad.h) for rows of their
// own type, and the joining of the weights' sums.
#include "norm_grad.h"

namespace fp4q {

namespace {

// out[which][col] = sum of the workgroups' parts.  64 columns of a workgroup
// times 16 slices of the parts, the slices joined in LDS.
__global__ __launch_bounds__(1024) void norm_grad_weights_kernel(const float *__restrict__ parts, uint32_t nparts,
                                                                 uint32_t cols, float *dgamma, float *dbeta)
{
    __shared__ float s[16][64];
    const uint32_t col = blockIdx.x * 64u + (threadIdx.x & 63u), slice = threadIdx.x >> 6, which = blockIdx.y;
    float *out = which ? dbeta : dgamma;
    float v = 0.0f;
    if (col < cols && out) {
#pragma unroll 16
        for (uint32_t p = slice; p < nparts; p += 16) v += parts[((size_t)p * 2 + which) * cols + col];
    }
    s[slice][threadIdx.x & 63u] = v;
    __syncthreads();
    if (slice == 0 && col < cols && out) {
#pragma unroll
        for (int i = 1; i < 16; ++i) v += s[i][threadIdx.x];
        out[col] = v;
    }
}

}  // namespace

size_t norm_grad_workspace_bytes(int64_t rows, int64_t cols, bool bf16)
{
    return rows <= 0 || cols <= 0 ? 0 : (size_t)grad_plan(rows, cols, bf16, true).parts * 2u * (size_t)cols * sizeof(float);
}

int launch_norm_grad(const NormGradArgs &a, float *dgamma, float *dbeta, hipStream_t st)
{
    const bool sums = dgamma || dbeta;
    const GradPlan g = grad_plan(a.rows, a.cols, a.bf16, sums);
    if (a.rows > 0) {
        const int rc = a.h_codes ? norm_grad_rows_pack8(a, dgamma, dbeta, st) : norm_grad_rows<false>(a, dgamma, dbeta, st);
        if (rc != 0) return rc;
        if (!sums || g.sums == kBeside) return 0;
    }
    // joins the parts, or with no rows writes zeros
    hipLaunchKernelGGL(norm_grad_weights_kernel, dim3((unsigned)((a.cols + 63) / 64), dbeta ? 2 : 1), dim3(1024), 0, st,
                       a.parts, (uint32_t)(a.rows > 0 ? g.parts : 0), (uint32_t)a.cols, dgamma, dbeta);
    return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace fp4q
