// norm.hip -- layer norm and RMS norm over rows, with the residual add and
// dropout in front of them and the MXFP4 producer behind them, and their
// gradient with the weights' reduction.
//
// Forward, per row of n columns:
//   h = [residual +] dropout(x), rounded to the element type;
//   mean = sum h / n (RMS: 0), rstd = 1 / sqrt(sum (h - mean)^2 / n + eps);
//   y = (h - mean) rstd gamma + beta, rounded; optionally the MXFP4 operand
//   of y along rows, byte for byte what the row producer makes of y.
// A row stays in registers between its two sums (the second one of the
// centred values, so that a large mean costs no precision), and each input
// is read and each output written once: HBM-bound.
//
// Gradient, with xh = (h - mean) rstd and g = dy gamma:
//   dh = [dres +] rstd (g - sum g / n - xh sum(g xh) / n) (RMS: no second
//   term), dx = dropout(dh); dgamma = sum over rows of dy xh, dbeta = of dy.
// A workgroup walks rows and keeps its columns' weight sums in registers;
// the workgroups' sums go to the workspace and a second kernel adds them in
// a fixed order (no atomics: two runs give the same bits).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4q_internal.h"
#include "row_ops.h"

namespace fp4q {

namespace {

// The weights are read once per row from cache, in their own type.
template <bool kTail>
__device__ __forceinline__ void load_weight(const void *w, bool bf16, uint32_t c, uint32_t cols, float v[8])
{
    if (bf16) {
        Chunk<bf16_t> q;
        load_chunk<bf16_t, kTail>(reinterpret_cast<const bf16_t *>(w), c, cols, q);
        q.get(v);
    } else {
        Chunk<float> q;
        load_chunk<float, kTail>(reinterpret_cast<const float *>(w), c, cols, q);
        q.get(v);
    }
}

// Sum over the kTpr threads of a row: a wave by itself, or the waves of the
// row's group through LDS (`slot`: one float per wave of the workgroup, of
// its own for each sum of a row).  kTpr > 64: every thread of the workgroup
// must call it.
template <int kTpr>
__device__ __forceinline__ float row_sum(float v, float *slot)
{
    v = wave_sum(v);
    if (kTpr <= 64) return v;
    constexpr int kWaves = kTpr / 64 > 0 ? kTpr / 64 : 1;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) slot[wave] = v;
    __syncthreads();
    const int first = wave / kWaves * kWaves;
    v = slot[first];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) v += slot[first + i];
    return v;
}

template <int kMask>
__device__ __forceinline__ uint32_t quad_max(uint32_t v)
{
    constexpr int ctrl = kMask == 1 ? 0xB1 : 0x4E;  // quad_perm [1,0,3,2] / [2,3,0,1]
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xF, 0xF, false));
}

// Chunk c (eight bf16 values) of row `row` of an MXFP4 operand along rows;
// the four chunks of a block sit in four neighbouring lanes.
__device__ __forceinline__ void store_mx(const NormArgs &a, int64_t row, uint32_t c, uint32_t cols,
                                         const Chunk<bf16_t> &y)
{
    const uint32_t w[4] = {y.q[0], y.q[1], y.q[2], y.q[3]};
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) amax = max(amax, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
    amax = quad_max<1>(amax);
    amax = quad_max<2>(amax);
    const uint32_t sbyte = mx_scale_byte(amax << 16);
    const float scale = mx_scale_f32(sbyte);
    uint32_t code = 0;
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(code, __builtin_bit_cast(bf16x2v, w[0]), scale, 0);
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(code, __builtin_bit_cast(bf16x2v, w[1]), scale, 1);
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(code, __builtin_bit_cast(bf16x2v, w[2]), scale, 2);
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(code, __builtin_bit_cast(bf16x2v, w[3]), scale, 3);
    if (c * 8u >= cols) return;
    uint8_t *codes = reinterpret_cast<uint8_t *>(a.codes), *scales = reinterpret_cast<uint8_t *>(a.scales);
    const uint64_t r = (uint64_t)row;
    if (a.tiled) {
        *reinterpret_cast<uint32_t *>(codes + ((r >> 5) * (cols >> 6) + (c >> 3)) * 1024u +
                                      ((r & 31u) + 32u * ((c >> 2) & 1u)) * 16u + (c & 3u) * 4u) = code;
        if ((c & 3u) == 0) scales[((uint64_t)(c >> 4) * (uint64_t)a.rows_out + r) * 4u + ((c >> 2) & 3u)] = (uint8_t)sbyte;
    } else {
        *reinterpret_cast<uint32_t *>(codes + r * (cols >> 1) + c * 4u) = code;
        if ((c & 3u) == 0) scales[r * (cols >> 5) + (c >> 2)] = (uint8_t)sbyte;
    }
}

// kTpr threads per row, kC chunks of eight elements per thread.
template <typename T, int kTpr, int kC, bool kRes, bool kTail, bool kMx>
__global__ __launch_bounds__(kTpr < 256 ? 256 : kTpr) void norm_kernel(const NormArgs a, const Dropout d,
                                                                            const void *__restrict__ gamma,
                                                                            const void *__restrict__ beta)
{
    constexpr int kRows = kTpr < 256 ? 256 / kTpr : 1;  // rows of a workgroup at a time
    static_assert(kTpr == 64 || kRows == 1, "a workgroup's waves share a row's barriers or need none");
    __shared__ float red[2][2][kTpr / 64 * kRows];  // a row's slots stay apart from the next row's
    const uint32_t t = threadIdx.x % kTpr, cols = (uint32_t)a.cols;
    const float inv_n = 1.0f / (float)cols;
    int parity = 0;
    // tiled output: the padding rows up to rows_out get zero codes and scales
    for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kTpr; row < a.rows_out;
         row += (int64_t)gridDim.x * kRows, parity ^= 1) {
        if (kMx && row >= a.rows) {
            Chunk<bf16_t> z;
            z.q = (u32x4v){0u, 0u, 0u, 0u};
#pragma unroll
            for (int i = 0; i < kC; ++i) store_mx(a, row, i * kTpr + t, cols, z);
            continue;
        }
        Chunk<T> q[kC];
        const T *x = reinterpret_cast<const T *>(a.x) + row * a.ld_x;
#pragma unroll
        for (int i = 0; i < kC; ++i) load_chunk<T, kTail>(x, i * kTpr + t, cols, q[i]);
        if (kRes || d.drop || a.h) {
            Chunk<T> s[kRes ? kC : 1];
            if (kRes) {
                const T *res = reinterpret_cast<const T *>(a.residual) + row * a.ld_r;
#pragma unroll
                for (int i = 0; i < kC; ++i) load_chunk<T, kTail>(res, i * kTpr + t, cols, s[i]);
            }
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                const uint32_t c = i * kTpr + t;
                float v[8];
                q[i].get(v);
                if (d.drop) apply_dropout(d, (uint32_t)row, c, v);
                if (kRes) {
                    float r[8];
                    s[i].get(r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = r[j] + v[j];
                }
                q[i].set(v);
                if (a.h) store_chunk<T, kTail>(reinterpret_cast<T *>(a.h) + row * a.ld_h, c, cols, q[i]);
            }
        }
        float mean = 0.0f;
        if (a.layer) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                float v[8];
                q[i].get(v);
                sum += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
            }
            mean = row_sum<kTpr>(sum, red[parity][0]) * inv_n;
        }
        float sq = 0.0f;
#pragma unroll
        for (int i = 0; i < kC; ++i) {
            const uint32_t at = (i * kTpr + t) * 8u;
            float v[8];
            q[i].get(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = kTail ? at + j < cols : at < cols;
                const float e = in ? v[j] - mean : 0.0f;
                sq = __builtin_fmaf(e, e, sq);
            }
        }
        const float rstd = 1.0f / __builtin_sqrtf(row_sum<kTpr>(sq, red[parity][1]) * inv_n + a.eps);
        if (t == 0) {
            if (a.layer && a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int i = 0; i < kC; ++i) {
            const uint32_t c = i * kTpr + t;
            float v[8];
            q[i].get(v);
            float w[8], b[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 1.0f, b[j] = 0.0f;
            if (gamma) load_weight<kTail>(gamma, a.w_bf16, c, cols, w);
            if (beta) load_weight<kTail>(beta, a.w_bf16, c, cols, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __builtin_fmaf((v[j] - mean) * rstd, w[j], b[j]);
            Chunk<T> out;
            out.set(v);
            if (a.y) store_chunk<T, kTail>(reinterpret_cast<T *>(a.y) + row * a.ld_y, c, cols, out);
            if constexpr (kMx) {
                out.mask(c * 8u < cols);
                store_mx(a, row, c, cols, out);
            }
        }
    }
}

template <typename T, int kTpr, int kC, bool kMx>
void run_norm(const NormArgs &a, const Dropout &d, hipStream_t st)
{
    constexpr int kThreads = kTpr < 256 ? 256 : kTpr, kRows = kThreads / kTpr;
    const int64_t need = (a.rows_out + kRows - 1) / kRows;
    const dim3 grid((unsigned)(need < (1 << 20) ? need : (1 << 20))), block(kThreads);
    const bool tail = a.cols % 8 != 0;
    if constexpr (kMx) {  // cols % 32 == 0
        if (a.residual)
            hipLaunchKernelGGL((norm_kernel<T, kTpr, kC, true, false, true>), grid, block, 0, st, a, d, a.gamma, a.beta);
        else
            hipLaunchKernelGGL((norm_kernel<T, kTpr, kC, false, false, true>), grid, block, 0, st, a, d, a.gamma, a.beta);
    } else {
        if (a.residual) {
            if (tail)
                hipLaunchKernelGGL((norm_kernel<T, kTpr, kC, true, true, false>), grid, block, 0, st, a, d, a.gamma, a.beta);
            else
                hipLaunchKernelGGL((norm_kernel<T, kTpr, kC, true, false, false>), grid, block, 0, st, a, d, a.gamma, a.beta);
        } else {
            if (tail)
                hipLaunchKernelGGL((norm_kernel<T, kTpr, kC, false, true, false>), grid, block, 0, st, a, d, a.gamma, a.beta);
            else
                hipLaunchKernelGGL((norm_kernel<T, kTpr, kC, false, false, false>), grid, block, 0, st, a, d, a.gamma, a.beta);
        }
    }
}

template <typename T, bool kMx>
void pick_norm(const NormArgs &a, const Dropout &d, hipStream_t st)
{
    const int64_t chunks = (a.cols + 7) / 8;
    if (chunks <= 64)
        run_norm<T, 64, 1, kMx>(a, d, st);
    else if (chunks <= 128)
        run_norm<T, 64, 2, kMx>(a, d, st);
    else if (chunks <= 256)
        run_norm<T, 256, 1, kMx>(a, d, st);
    else if (chunks <= 512)
        run_norm<T, 256, 2, kMx>(a, d, st);
    else if (chunks <= 1024)
        run_norm<T, 256, 4, kMx>(a, d, st);
    else if (chunks <= 2048)
        run_norm<T, 512, 4, kMx>(a, d, st);
    else
        run_norm<T, 1024, 4, kMx>(a, d, st);
}

// ------------------------------------------------------------------ gradient

constexpr int kGradThreads = 1024;
constexpr int kMaxParts = 256;  // workgroups that keep weight sums: one per compute unit

// A workgroup of 1024 threads takes 1024 / kTpr rows at a time; its weight
// sums are folded over those row groups in LDS at the end.
template <typename T, int kTpr, int kC, bool kRes, bool kDx, bool kTail>
__global__ __launch_bounds__(kGradThreads) void norm_grad_kernel(const NormGradArgs a, const Dropout d)
{
    constexpr int kGroups = kGradThreads / kTpr;
    __shared__ float red[2][2][kGradThreads / 64];
    __shared__ float fold[kGroups > 1 ? kC * 8 * kGradThreads : 1];
    const uint32_t t = threadIdx.x % kTpr, g = threadIdx.x / kTpr, cols = (uint32_t)a.cols;
    const float inv_n = 1.0f / (float)cols;
    float w[kC][8], sum_w[kC][8], sum_b[kC][8];
#pragma unroll
    for (int i = 0; i < kC; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[i][j] = 1.0f, sum_w[i][j] = 0.0f, sum_b[i][j] = 0.0f;
        if (a.gamma) load_weight<kTail>(a.gamma, a.w_bf16, i * kTpr + t, cols, w[i]);
    }
    const int64_t stride = (int64_t)gridDim.x * kGroups;
    int parity = 0;
    for (int64_t base = (int64_t)blockIdx.x * kGroups; base < a.rows; base += stride, parity ^= 1) {
        const bool live = base + g < a.rows;  // the same on every lane of a wave
        const int64_t row = live ? base + g : a.rows - 1;
        Chunk<T> dy[kC], h[kC], res[kRes ? kC : 1];
#pragma unroll
        for (int i = 0; i < kC; ++i) {
            load_chunk<T, kTail>(reinterpret_cast<const T *>(a.dy) + row * a.ld_dy, i * kTpr + t, cols, dy[i]);
            load_chunk<T, kTail>(reinterpret_cast<const T *>(a.h) + row * a.ld_h, i * kTpr + t, cols, h[i]);
            if (kRes)
                load_chunk<T, kTail>(reinterpret_cast<const T *>(a.dres) + row * a.ld_dres, i * kTpr + t, cols, res[i]);
        }
        const float mean = a.layer ? a.mean[row] : 0.0f, rstd = a.rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < kC; ++i) {
            float e[8], v[8];
            dy[i].get(e);
            h[i].get(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float xh = (v[j] - mean) * rstd, gj = e[j] * w[i][j];
                s1 = __builtin_fmaf(gj, xh, s1);
                s2 += gj;
                if (live) {
                    sum_w[i][j] = __builtin_fmaf(e[j], xh, sum_w[i][j]);
                    sum_b[i][j] += e[j];
                }
            }
        }
        // both sums with one barrier; the two parities keep a row's slots
        // apart from the next row's
        s1 = wave_sum(s1);
        s2 = wave_sum(s2);
        if (kTpr > 64) {
            constexpr int kWaves = kTpr / 64;
            const int wave = threadIdx.x >> 6, first = wave / kWaves * kWaves;
            if ((threadIdx.x & 63) == 0) red[parity][0][wave] = s1, red[parity][1][wave] = s2;
            __syncthreads();
            s1 = red[parity][0][first];
            s2 = red[parity][1][first];
#pragma unroll
            for (int i = 1; i < kWaves; ++i) {
                s1 += red[parity][0][first + i];
                s2 += red[parity][1][first + i];
            }
        }
        const float c1 = s1 * inv_n, c2 = a.layer ? s2 * inv_n : 0.0f;
        if (live) {
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                const uint32_t c = i * kTpr + t;
                float e[8], v[8];
                dy[i].get(e);
                h[i].get(v);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float xh = (v[j] - mean) * rstd;
                    v[j] = __builtin_fmaf(-xh, c1, __builtin_fmaf(e[j], w[i][j], -c2)) * rstd;
                }
                if (kRes) {
                    float r[8];
                    res[i].get(r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = r[j] + v[j];
                }
                Chunk<T> out;
                if (a.dh) {
                    out.set(v);
                    store_chunk<T, kTail>(reinterpret_cast<T *>(a.dh) + row * a.ld_dh, c, cols, out);
                }
                if (kDx) {
                    if (d.drop) apply_dropout(d, (uint32_t)row, c, v);
                    out.set(v);
                    store_chunk<T, kTail>(reinterpret_cast<T *>(a.dx) + row * a.ld_dx, c, cols, out);
                }
            }
        }
    }
    if (!a.parts) return;
    // parts[workgroup][gamma, beta][cols]
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (which == 1 && !a.layer_beta) break;
        float *part = a.parts + ((size_t)blockIdx.x * 2 + which) * cols;
        if (kGroups == 1) {
#pragma unroll
            for (int i = 0; i < kC; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t col = (i * kTpr + t) * 8u + j;
                    if (col < cols) part[col] = which ? sum_b[i][j] : sum_w[i][j];
                }
        } else {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kC; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) fold[(i * 8 + j) * kGradThreads + threadIdx.x] = which ? sum_b[i][j] : sum_w[i][j];
            __syncthreads();
            for (uint32_t col = threadIdx.x; col < cols; col += kGradThreads) {
                const uint32_t c = col >> 3, at = ((c / kTpr) * 8u + (col & 7u)) * kGradThreads + c % kTpr;
                float s = fold[at];
                for (int k = 1; k < kGroups; ++k) s += fold[at + k * kTpr];
                part[col] = s;
            }
        }
    }
}

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
#pragma unroll 4
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

int grad_rows_at_once(int64_t cols)
{
    const int64_t chunks = (cols + 7) / 8;
    return chunks <= 128 ? 16 : chunks <= 256 ? 8 : chunks <= 512 ? 4 : chunks <= 1024 ? 2 : 1;
}

template <typename T, int kTpr, int kC>
void run_norm_grad(const NormGradArgs &a, const Dropout &d, unsigned grid, hipStream_t st)
{
    const bool tail = a.cols % 8 != 0;
#define FP4Q_NORM_GRAD(RES, DX, TAIL)                                                                             \
    hipLaunchKernelGGL((norm_grad_kernel<T, kTpr, kC, RES, DX, TAIL>), dim3(grid), dim3(kGradThreads), 0, st, a, d)
#define FP4Q_NORM_GRAD_T(RES, DX) \
    do { if (tail) FP4Q_NORM_GRAD(RES, DX, true); else FP4Q_NORM_GRAD(RES, DX, false); } while (0)
    if (a.dres) {
        if (a.dx) FP4Q_NORM_GRAD_T(true, true); else FP4Q_NORM_GRAD_T(true, false);
    } else {
        if (a.dx) FP4Q_NORM_GRAD_T(false, true); else FP4Q_NORM_GRAD_T(false, false);
    }
#undef FP4Q_NORM_GRAD_T
#undef FP4Q_NORM_GRAD
}

template <typename T>
void pick_norm_grad(const NormGradArgs &a, const Dropout &d, unsigned grid, hipStream_t st)
{
    const int64_t chunks = (a.cols + 7) / 8;
    if (chunks <= 128)
        run_norm_grad<T, 64, 2>(a, d, grid, st);
    else if (chunks <= 256)
        run_norm_grad<T, 128, 2>(a, d, grid, st);
    else if (chunks <= 512)
        run_norm_grad<T, 256, 2>(a, d, grid, st);
    else if (chunks <= 1024)
        run_norm_grad<T, 512, 2>(a, d, grid, st);
    else if (chunks <= 2048)
        run_norm_grad<T, 1024, 2>(a, d, grid, st);
    else
        run_norm_grad<T, 1024, 4>(a, d, grid, st);
}

}  // namespace

int launch_norm(const NormArgs &a, hipStream_t st)
{
    const Dropout d = dropout_of(a.p, a.seed, a.stream_id);
    if (a.codes)
        pick_norm<bf16_t, true>(a, d, st);
    else if (a.bf16)
        pick_norm<bf16_t, false>(a, d, st);
    else
        pick_norm<float, false>(a, d, st);
    return hipGetLastError() == hipSuccess ? 0 : 1;
}

// Workgroups of the gradient kernel, each of which keeps one row of sums.
static int64_t grad_parts(int64_t rows, int64_t cols)
{
    const int at_once = grad_rows_at_once(cols);
    const int64_t need = (rows + at_once - 1) / at_once;
    return need < kMaxParts ? need : kMaxParts;
}

size_t norm_grad_workspace_bytes(int64_t rows, int64_t cols)
{
    return rows <= 0 || cols <= 0 ? 0 : (size_t)grad_parts(rows, cols) * 2u * (size_t)cols * sizeof(float);
}

int launch_norm_grad(NormGradArgs a, float *dgamma, float *dbeta, hipStream_t st)
{
    const Dropout d = dropout_of(a.p, a.seed, a.stream_id);
    const unsigned grid = (unsigned)grad_parts(a.rows, a.cols);
    if (!dgamma && !dbeta) a.parts = nullptr;
    a.layer_beta = dbeta != nullptr;
    if (grid > 0) {
        if (a.bf16)
            pick_norm_grad<bf16_t>(a, d, grid, st);
        else
            pick_norm_grad<float>(a, d, grid, st);
        if (hipGetLastError() != hipSuccess) return 1;
    }
    if (dgamma || dbeta)
        hipLaunchKernelGGL(norm_grad_weights_kernel, dim3((unsigned)((a.cols + 63) / 64), dbeta ? 2 : 1), dim3(1024), 0,
                           st, a.parts, grid, (uint32_t)a.cols, dgamma, dbeta);
    return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace fp4q
