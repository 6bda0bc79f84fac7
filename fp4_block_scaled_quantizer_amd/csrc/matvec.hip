// matvec.hip -- products of few rows with FP4 weights, y = alpha x W^T: the
// linear layers of a decoding step, x a token's activations (or a few tokens')
// in bf16 or as 8-bit rows, W an MXFP4 or NVFP4 operand as the GEMMs take it.
//
// What bounds it is reading W once (17/32 byte an MXFP4 weight, 9/16 NVFP4).
// A wave takes 16 rows of W (kR times) and 128 columns a step: lane l holds
// the 16 bytes of row l mod 16, columns 32 (l / 16) .. + 31, which is a run of
// whole scale blocks in every layout, makes the 32 weights' exact bf16 values
// (an E2M1 code times a power of two, or times an E4M3 scale, has at most six
// significant bits) and multiplies them on v_mfma_f32_16x16x32_bf16 with the
// same columns of 16 rows of x, in binary32 sums.  (The scaled FP4 x FP8
// MFMA would take both without a convert, but sums 8-bit products with fewer
// bits: up to 8e-5 of sum |x w| off, measured, against 1e-7.)  The
// order of the columns inside an MFMA's sum does not matter as long as both
// operands have the same, so neither is rearranged.  The waves of a workgroup
// split the columns and join their sums through LDS in a fixed order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4q_internal.h"
#include "pack8.h"

namespace fp4q {

namespace {

typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));
typedef float f32x4v __attribute__((ext_vector_type(4)));

// Where the layouts have row n's piece q of step s: codes at n / 32 *
// code_group + n mod 32 * code_row + q / 2 * code_pair + q mod 2 * code_q + s *
// code_step, scales alike.
struct Weights4 {
    const uint8_t *codes, *scales;
    int64_t code_group, code_row, scale_group, scale_row;
    uint32_t code_pair, code_q, scale_q;
    int64_t code_step, scale_step;
};
struct Matvec {
    Weights4 w;
    const uint8_t *x, *x_scales;
    const float *tensor_scale;
    int64_t ld_x, ld_y;  // elements
    uint32_t M, N, steps;
    float alpha;
    void *y;
    bool y_bf16;
};

// Eight weights, a word of codes, as bf16.
__device__ __forceinline__ bf16x8v weights8_mx(uint32_t w, float scale)
{
    const bf16x2v a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
    const bf16x2v b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
    const bf16x2v c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
    const bf16x2v d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
    return (bf16x8v){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// The scaled converts take a scale's exponent only, so an E4M3 scale is
// multiplied in binary32 (the products are exact).
__device__ __forceinline__ bf16x8v weights8_nv(uint32_t w, float scale)
{
    const f32x2v a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    const f32x2v b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const f32x2v c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    const f32x2v d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    const u32x4v q = {pack_bf16x2(a[0] * scale, a[1] * scale), pack_bf16x2(b[0] * scale, b[1] * scale),
                      pack_bf16x2(c[0] * scale, c[1] * scale), pack_bf16x2(d[0] * scale, d[1] * scale)};
    return __builtin_bit_cast(bf16x8v, q);
}
// Eight elements of an 8-bit row as bf16.
__device__ __forceinline__ bf16x8v rows8(uint32_t lo, uint32_t hi, float scale)
{
    const bf16x2v a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf16x2v b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2v c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf16x2v d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return (bf16x8v){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

enum Format { kMx, kNvGlobal, kNvTile };

// What a wave loads of one step.
template <Format kFormat, bool kX8, int kMT, int kR>
struct Step {
    u32x4v codes[kR];
    uint32_t scales[kR];
    float tile[kFormat == kNvTile ? kR : 1];
    u32x4v x[kMT][kX8 ? 2 : 4];
    uint32_t x_scale[kX8 ? kMT : 1];
};

// kMT: 16 rows of x each; kR: 16 rows of W each.  grid.x: groups of 16 kR
// rows of W.
template <Format kFormat, bool kX8, int kMT, int kR>
__global__ __launch_bounds__(kMT <= 2 ? 1024 : 512) void matvec_kernel(const Matvec a)
{
    extern __shared__ __attribute__((aligned(16))) float parts[];  // [waves][kR * kMT][64][4]
    constexpr int kTiles = kR * kMT;
    const uint32_t lane = threadIdx.x & 63u, r = lane & 15u, q = lane >> 4;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), waves = blockDim.x >> 6;
    const uint32_t n0 = blockIdx.x * (16u * kR);
    const uint32_t from = a.steps * wave / waves, to = a.steps * (wave + 1u) / waves;

    const uint8_t *codes[kR], *scales[kR], *x[kMT], *x_scales[kX8 ? kMT : 1];
    const float *tile[kFormat == kNvTile ? kR : 1];
#pragma unroll
    for (int j = 0; j < kR; ++j) {  // past W's end: its last row again, not stored
        const uint32_t n = min(n0 + 16u * j + r, a.N - 1u);
        codes[j] = a.w.codes + (int64_t)(n >> 5) * a.w.code_group + (int64_t)(n & 31u) * a.w.code_row +
                   (q >> 1) * a.w.code_pair + (q & 1u) * a.w.code_q;
        scales[j] = a.w.scales + (int64_t)(n >> 5) * a.w.scale_group + (int64_t)(n & 31u) * a.w.scale_row + q * a.w.scale_q;
        // 16 rows are within one 128 x 128 tile
        if (kFormat == kNvTile) tile[j] = a.tensor_scale + (int64_t)(min(n0 + 16u * j, a.N - 1u) >> 7) * a.steps;
    }
#pragma unroll
    for (int i = 0; i < kMT; ++i) {  // past x's end: its last row again, in columns of D that are not stored
        const uint32_t m = min(16u * i + r, a.M - 1u);
        x[i] = a.x + (int64_t)m * a.ld_x * (kX8 ? 1 : 2) + q * (kX8 ? 32u : 64u);
        if (kX8) x_scales[i] = a.x_scales + (int64_t)m * (a.steps * 4u) + q;
    }
    typedef Step<kFormat, kX8, kMT, kR> S;
    const auto fetch = [&](uint32_t step, S &s) {
#pragma unroll
        for (int j = 0; j < kR; ++j) {
            s.codes[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4v *>(codes[j] + step * a.w.code_step));
            const uint8_t *p = scales[j] + step * a.w.scale_step;
            s.scales[j] = kFormat == kMx ? (uint32_t)*p : (uint32_t)*reinterpret_cast<const uint16_t *>(p);
            if (kFormat == kNvTile) s.tile[j] = tile[j][step];
        }
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
            const u32x4v *p = reinterpret_cast<const u32x4v *>(x[i] + step * (kX8 ? 128u : 256u));
#pragma unroll
            for (int k = 0; k < (kX8 ? 2 : 4); ++k) s.x[i][k] = p[k];
            if (kX8) s.x_scale[i] = x_scales[i][step * 4u];
        }
    };
    f32x4v acc[kR][kMT];
#pragma unroll
    for (int j = 0; j < kR; ++j) {
#pragma unroll
        for (int i = 0; i < kMT; ++i) acc[j][i] = (f32x4v){0.0f, 0.0f, 0.0f, 0.0f};
    }
    const auto multiply = [&](const S &s) {
        bf16x8v b[kMT][4];
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
            const float xs = kX8 ? mx_scale_f32(s.x_scale[i]) : 1.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                b[i][k] = kX8 ? rows8(s.x[i][k >> 1][2 * (k & 1)], s.x[i][k >> 1][2 * (k & 1) + 1], xs)
                              : __builtin_bit_cast(bf16x8v, s.x[i][kX8 ? 0 : k]);
        }
#pragma unroll
        for (int j = 0; j < kR; ++j) {
            const f32x2v nv = __builtin_amdgcn_cvt_pk_f32_fp8(s.scales[j], false);
            f32x4v sum[kMT];
#pragma unroll
            for (int i = 0; i < kMT; ++i) sum[i] = kFormat == kNvTile ? (f32x4v){0.0f, 0.0f, 0.0f, 0.0f} : acc[j][i];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bf16x8v w = kFormat == kMx ? weights8_mx(s.codes[j][k], mx_scale_f32(s.scales[j]))
                                                 : weights8_nv(s.codes[j][k], nv[k >> 1]);
#pragma unroll
                for (int i = 0; i < kMT; ++i) sum[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, b[i][k], sum[i], 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kMT; ++i) {
                if (kFormat == kNvTile) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][i][e] = __builtin_fmaf(sum[i][e], s.tile[kFormat == kNvTile ? j : 0], acc[j][i][e]);
                } else {
                    acc[j][i] = sum[i];
                }
            }
        }
    };
    if (from < to) {
        S one, two;
        fetch(from, one);
        for (uint32_t step = from; step < to; step += 2u) {  // past the wave's last step: it again, not used
            fetch(min(step + 1u, to - 1u), two);
            multiply(one);
            if (step + 1u >= to) break;
            fetch(min(step + 2u, to - 1u), one);
            multiply(two);
        }
    }
    f32x4v *mine = reinterpret_cast<f32x4v *>(parts) + wave * (kTiles * 64u) + lane;
#pragma unroll
    for (int j = 0; j < kR; ++j) {
#pragma unroll
        for (int i = 0; i < kMT; ++i) mine[(j * kMT + i) * 64] = acc[j][i];
    }
    __syncthreads();
    const float scale = kFormat == kNvGlobal ? a.tensor_scale[0] : 1.0f;
    for (uint32_t t = wave; t < (uint32_t)kTiles; t += waves) {
        const f32x4v *p = reinterpret_cast<const f32x4v *>(parts) + t * 64u + lane;
        f32x4v sum = p[0];
        for (uint32_t k = 1; k < waves; ++k) sum += p[k * (kTiles * 64u)];
        // lane l has rows 4 (l / 16) .. + 3 of the tile's 16 of W, row l mod 16 of x
        const uint32_t n = n0 + t / kMT * 16u + q * 4u, m = t % kMT * 16u + r;
        if (m >= a.M) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = sum[e] * scale * a.alpha;
        const int64_t at = (int64_t)m * a.ld_y + n;
        if (a.y_bf16) {
            bf16_t *y = reinterpret_cast<bf16_t *>(a.y) + at;
            const u32x2v v = {pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3])};
            if (n + 3u < a.N) {
                *reinterpret_cast<u32x2_a2 *>(y) = v;
            } else {
#pragma unroll
                for (uint32_t e = 0; e < 4u; ++e)
                    if (n + e < a.N) y[e].bits = (uint16_t)(v[e >> 1] >> (16u * (e & 1u)));
            }
        } else {
            float *y = reinterpret_cast<float *>(a.y) + at;
            if (n + 3u < a.N) {
                *reinterpret_cast<u32x4_a4 *>(y) = __builtin_bit_cast(u32x4v, sum);
            } else {
#pragma unroll
                for (uint32_t e = 0; e < 4u; ++e)
                    if (n + e < a.N) y[e] = sum[e];
            }
        }
    }
}

template <Format kFormat, bool kX8, int kMT, int kR>
void run_matvec(const Matvec &a, uint32_t waves, hipStream_t st)
{
    const unsigned grid = (a.N + 16u * kR - 1u) / (16u * kR);
    hipLaunchKernelGGL((matvec_kernel<kFormat, kX8, kMT, kR>), dim3(grid), dim3(waves * 64u), waves * kR * kMT * 1024u, st, a);
}

template <Format kFormat, bool kX8>
void pick_matvec(const Matvec &a, hipStream_t st)
{
    const uint32_t blocks = (a.N + 15u) / 16u;
    uint32_t waves = a.steps < 16u ? (a.steps > 0u ? a.steps : 1u) : 16u;
    if (a.M <= 16) {
        if (blocks >= 1024u)
            run_matvec<kFormat, kX8, 1, 2>(a, waves, st);
        else
            run_matvec<kFormat, kX8, 1, 1>(a, waves, st);
    } else if (a.M <= 32) {
        if (blocks >= 1024u)
            run_matvec<kFormat, kX8, 2, 2>(a, waves, st);
        else
            run_matvec<kFormat, kX8, 2, 1>(a, waves, st);
    } else {
        if (waves > 8u) waves = 8u;
        if (blocks >= 1024u)
            run_matvec<kFormat, kX8, 4, 2>(a, waves, st);
        else
            run_matvec<kFormat, kX8, 4, 1>(a, waves, st);
    }
}

Matvec matvec_of(const MatvecArgs &g)
{
    Matvec a{};
    const int64_t K = g.K;
    const bool nv = g.tensor_scale != nullptr;
    a.w.codes = reinterpret_cast<const uint8_t *>(g.codes);
    a.w.scales = reinterpret_cast<const uint8_t *>(g.scales);
    const int64_t scale_bytes = K / (nv ? 16 : 32);
    a.w.code_pair = 32;
    a.w.code_q = 16;
    a.w.scale_q = nv ? 2 : 1;
    if (!g.tiled) {
        a.w.code_row = K / 2;
        a.w.scale_row = scale_bytes;
        a.w.code_step = 64;
        a.w.scale_step = nv ? 8 : 4;
    } else if (nv) {  // [Rp/32][K/128][32][64] and [Rp/32][K/128][32][8]
        a.w.code_row = 64;
        a.w.scale_row = 8;
        a.w.code_step = 2048;
        a.w.scale_step = 256;
    } else {  // [Rp/32][K/64][2][32][16] and [K/128][Rp][4]
        a.w.code_row = 16;
        a.w.code_pair = 1024;
        a.w.code_q = 512;
        a.w.scale_row = 4;
        a.w.code_step = 2048;
        a.w.scale_step = (g.N + 31) / 32 * 128;
    }
    a.w.code_group = 16 * K;
    a.w.scale_group = g.tiled && !nv ? 128 : 32 * scale_bytes;
    a.x = reinterpret_cast<const uint8_t *>(g.x);
    a.x_scales = reinterpret_cast<const uint8_t *>(g.x_scales);
    a.tensor_scale = g.tensor_scale;
    a.ld_x = g.ld_x;
    a.ld_y = g.ld_y;
    a.M = (uint32_t)g.M;
    a.N = (uint32_t)g.N;
    a.steps = (uint32_t)(K / 128);
    a.alpha = g.alpha;
    a.y = g.y;
    a.y_bf16 = g.y_bf16;
    return a;
}

}  // namespace

int launch_matvec(const MatvecArgs &g, hipStream_t st)
{
    const Matvec a = matvec_of(g);
    if (g.tensor_scale && g.nv_domain == 0)
        pick_matvec<kNvGlobal, false>(a, st);
    else if (g.tensor_scale)
        pick_matvec<kNvTile, false>(a, st);
    else if (g.x_scales)
        pick_matvec<kMx, true>(a, st);
    else
        pick_matvec<kMx, false>(a, st);
    return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace fp4q
