// matvec.h -- products of few rows with FP4 weights, y = alpha x W^T: the
// linear layers of a decoding step, x a token's activations (or a few tokens')
// in bf16 or as 8-bit rows, W an MXFP4 or NVFP4 operand as the GEMMs take it.
//
// What bounds it is reading W once (17/32 byte an MXFP4 weight, 9/16 NVFP4).
// A wave takes 16 rows of W (kR times) and 128 columns a step: lane l holds
// the 16 bytes of row l mod 16, columns 32 (l / 16) .. + 31, which is a run of
// whole scale blocks in every layout, makes the 32 weights' exact bf16 values
// (an E2M1 code times a power of two, or times an E4M3 scale, has at most six
// significant bits; those of 2^128 and more: large_rows) and multiplies them
// on v_mfma_f32_16x16x32_bf16 with the same columns of 16 rows of x, in
// binary32 sums.  (The scaled FP4 x FP8
// MFMA would take both without a convert, but sums 8-bit products with fewer
// bits: up to 8e-5 of sum |x w| off, measured, against 1e-7.)  The
// order of the columns inside an MFMA's sum does not matter as long as both
// operands have the same, so neither is rearranged.  The waves of a workgroup
// take the columns' steps in turn and join their sums through LDS in a fixed
// order.
//   Weights from memory (where a copy reads and writes 6.3 TB/s), us a call:
// one row of x, MXFP4 tiled 4096 x 4096 4.6 (launch), 28672 x 4096 12.1 (5.2
// TB/s, HBM; in rows 14.7, NVFP4 tiles 14.4), 4096 x 14336 8.0; 5 rows, NVFP4 4096
// x 14336 tiled 10.1, in rows 12.0 (a compute unit has 16 rows of W, whose start,
// 85 vector instructions a step of 128 columns and join are not hidden: four
// fifths of those are the products of codes and scales, twice MXFP4's); 28672 x
// 4096 MXFP4 with 16 rows 12.9, 32 8-bit rows 15.3, 64 rows 23.2 (x's way from
// the L2 through LDS, the converts and the MFMAs, 5 to 7 us each, overlap in
// part); 32 rows, 4096 x 14336 14.3 (where a compute unit reads 448 KiB of x and
// 238 of W).  The first kernel, whose lanes loaded x in the MFMA's layout
// instead of whole lines, took 33 us for the 32 rows and 81 for the 64.
#pragma once

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
// code_step, scales alike (modulo 2^32 but for the steps).
struct Weights4 {
    const uint8_t *codes, *scales;
    uint32_t code_group, code_row, scale_group, scale_row;
    int64_t code_step, scale_step;
    uint32_t code_pair, code_q, scale_q, N;
};
struct Matvec {
    Weights4 w;
    const uint8_t *x, *x_scales;
    const float *tensor_scale;
    int64_t ld_x;  // elements
    uint32_t M, steps;
    int64_t ld_y;
    void *y;
    float alpha;
    bool y_bf16;
    uint32_t groups;  // of rows of x, each a workgroup's
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

// Four neighbouring elements of row m of Y.
__device__ __forceinline__ void store4(const Matvec &a, uint32_t m, uint32_t n, const f32x4v &v)
{
    const int64_t at = (int64_t)m * a.ld_y + n;
    if (a.y_bf16) {
        bf16_t *y = reinterpret_cast<bf16_t *>(a.y) + at;
        const u32x2v w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        if (n + 3u < a.w.N) {
            *reinterpret_cast<u32x2_a2 *>(y) = w;
        } else {
#pragma unroll
            for (uint32_t e = 0; e < 4u; ++e)
                if (n + e < a.w.N) y[e].bits = (uint16_t)(w[e >> 1] >> (16u * (e & 1u)));
        }
    } else {
        float *y = reinterpret_cast<float *>(a.y) + at;
        if (n + 3u < a.w.N) {
            *reinterpret_cast<u32x4_a4 *>(y) = __builtin_bit_cast(u32x4v, v);
        } else {
#pragma unroll
            for (uint32_t e = 0; e < 4u; ++e)
                if (n + e < a.w.N) y[e] = v[e];
        }
    }
}

// bf16 ends at 2^128, and an MXFP4 weight of a scale byte above 252 (which the
// producers do not write) may reach 1.5 * 2^129: it was infinite in the MFMA,
// and NaN times a zero.  So where a sum is not finite, the wave looks through
// the scales of the tile's 16 rows of W for such a byte (large_rows), and the
// elements of those rows that are not finite are summed again, each by its
// lane in binary64 (again4).  What an element becomes is thus a matter of its
// own row of x and of W, and the loop over W has no part in it.
//   28672 x 4096 tiled, us without / with this: one row of x 12.0 / 12.1, 64
// rows 22.7 / 23.1; with a NaN in a row of x (W from the caches) 11.1 / 13.0 and
// 22.6 / 33.3.

// Bit r: row n + r of W has a scale byte of 253 or 254.  The whole wave must
// call it.
__device__ __forceinline__ uint32_t large_rows(const Matvec &a, uint32_t n, uint32_t r, uint32_t q)
{
    const uint32_t row = min(n + r, a.w.N - 1u);
    const uint8_t *scales = a.w.scales + ((row >> 5) * a.w.scale_group + (row & 31u) * a.w.scale_row);
    bool large = false;
    for (uint32_t s = q; s < a.steps; s += 4u) {  // a step's four bytes side by side
        const uint32_t four = *reinterpret_cast<const uint32_t *>(scales + s * a.w.scale_step);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t byte = four >> (8 * k) & 255u;
            large |= byte == 253u || byte == 254u;
        }
    }
    const uint64_t b = __ballot(large);
    return (uint32_t)(b | b >> 16 | b >> 32 | b >> 48) & 0xFFFFu;
}

// Elements (m, n + j) of Y, bit j of `which` set, where they are not finite.
template <bool kX8>
__device__ __forceinline__ void again4(const Matvec &a, uint32_t m, uint32_t n, uint32_t which)
{
    const uint8_t *x = a.x + m * (a.ld_x * (kX8 ? 1 : 2)), *x_scales = kX8 ? a.x_scales + m * (a.steps * 4ull) : nullptr;
    for (uint32_t i = n; i < n + 4u && i < a.w.N; ++i) {
        if (!(which >> (i - n) & 1u)) continue;
        const int64_t to = (int64_t)m * a.ld_y + i;
        const float was = a.y_bf16 ? as_float(reinterpret_cast<const bf16_t *>(a.y)[to]) : reinterpret_cast<const float *>(a.y)[to];
        if (was - was == 0.0f) continue;
        const uint8_t *codes = a.w.codes + ((i >> 5) * a.w.code_group + (i & 31u) * a.w.code_row);
        const uint8_t *scales = a.w.scales + ((i >> 5) * a.w.scale_group + (i & 31u) * a.w.scale_row);
        double v = 0.0;
        for (uint32_t at = 0; at < a.steps * 16u; ++at) {  // eight columns, a word of codes
            const uint32_t s = at >> 4, q = at >> 2 & 3u, byte = scales[s * a.w.scale_step + q];
            const double unit = byte == 255u ? (double)__builtin_nanf("") : __builtin_ldexp(1.0, (int)byte - 127);
            const uint32_t w = *reinterpret_cast<const uint32_t *>(
                codes + s * a.w.code_step + (q >> 1) * a.w.code_pair + (q & 1u) * a.w.code_q + (at & 3u) * 4u);
            bf16x8v e;
            if constexpr (kX8) {
                const u32x2v b = *reinterpret_cast<const u32x2v *>(x + at * 8ull);
                e = rows8(b[0], b[1], mx_scale_f32(x_scales[at >> 2]));
            } else {
                e = *reinterpret_cast<const bf16x8v *>(x + at * 16ull);
            }
            const bf16x8v f = weights8_mx(w, 1.0f);
#pragma unroll
            for (int k = 0; k < 8; ++k) v = __builtin_fma((double)(float)f[k] * unit, (double)(float)e[k], v);
        }
        const float y = (float)v * a.alpha;
        if (a.y_bf16)
            reinterpret_cast<bf16_t *>(a.y)[to].bits = (uint16_t)pack_bf16x2(y, y);
        else
            reinterpret_cast<float *>(a.y)[to] = y;
    }
}

// What a wave loads of one step of kP * 128 columns.  kMQ: groups of four rows
// of x, of which a load (16 bytes a lane, 64 lanes) takes one for each 128
// columns in bf16 and two in 8 bits, whole cache lines either way.
template <Format kFormat, bool kX8, int kMQ, int kR, int kP>
struct Step {
    static constexpr int kLoads = kX8 ? (kMQ * kP + 1) / 2 : kMQ * kP;
    u32x4v x[kLoads];
    uint32_t x_scale[kX8 ? kLoads : 1];
    u32x4v codes[kR][kP];
    uint32_t scales[kR];
    float tile[kFormat == kNvTile ? kR : 1];
};

// How a kernel is made: rows of x and bytes of each that a wave keeps in LDS,
// steps that it has in flight, and the most waves of a workgroup (four where
// a wave needs more than half of its registers).
template <Format kFormat, bool kX8, int kMQ, int kR, int kP>
struct Shape {
    static constexpr int kMT = (kMQ + 3) / 4, kTiles = kR * kMT;  // 16 x 16 results
    static constexpr int kRows = kMQ * 4;
    static constexpr uint32_t kPitch = 256 * kP + 16;  // 16 rows' pieces lie in all banks alike
    static constexpr int kAhead = kMQ <= 4 || (kMQ == 8 && kR * kP <= 4) ? 2 : 1;
    static constexpr bool kWide = (kMQ == 16 && kR > (kFormat == kNvTile ? 2 : 4)) ||
                                  (kP == 2 && ((kMQ == 8 && kR > 5) || (kMQ == 4 && kR > 6)));
    static constexpr int kMost = !kWide && kRows * kPitch * 8 <= 160 * 1024 ? 8 : 4;
    static constexpr int kWaves = kR == 1 && kMQ <= 4 && kP == 1 ? 16 : kMost;
    static constexpr int kAtOnce = kTiles < 64 / kWaves ? kTiles : 64 / kWaves;  // tiles joined, in 64 KiB at most
    static uint32_t lds_bytes(uint32_t waves)
    {
        const uint32_t x = waves * kRows * kPitch, sums = waves * kAtOnce * 1024u;
        return x > sums ? x : sums;
    }
};

// kR: 16 rows of W each; grid.x: groups of 16 kR rows of W (or a few more, with
// nothing to store), grid.y: of 4 kMQ rows of x.  kP = 2 is for W in
// rows (the linear layout): a lane then takes 32 neighbouring bytes, so that a
// wave's two loads are 128 bytes of each row, and all its scales with one.
template <Format kFormat, bool kX8, int kMQ, int kR, int kP>
__global__ __launch_bounds__((Shape<kFormat, kX8, kMQ, kR, kP>::kWaves * 64)) void matvec_kernel(const Matvec a)
{
    typedef Step<kFormat, kX8, kMQ, kR, kP> S;
    typedef Shape<kFormat, kX8, kMQ, kR, kP> H;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    // all arguments wanted at once, and none between them that is not: the
    // compiler loads others over those it does not need, and waits for them one
    // after the other (0.25 us a call and wait)
    asm volatile("" ::"s"(a.w.codes), "s"(a.w.scales), "s"(a.w.code_group), "s"(a.w.code_row), "s"(a.w.scale_group),
                 "s"(a.w.scale_row), "s"(a.w.code_step), "s"(a.w.scale_step), "s"(a.x), "s"(a.ld_x), "s"(a.M),
                 "s"(a.w.N), "s"(a.steps), "s"(a.w.scale_q), "s"(a.w.code_pair), "s"(a.w.code_q), "s"(a.x_scales),
                 "s"(a.tensor_scale), "s"((uint32_t)blockDim.x));
    const uint32_t lane = threadIdx.x & 63u, r = lane & 15u, q = lane >> 4;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), waves = blockDim.x >> 6;
    const uint32_t n0 = blockIdx.x * (16u * kR), m0 = blockIdx.y * H::kRows, M = min(a.M - m0, (uint32_t)H::kRows);
    const uint32_t steps = a.steps / kP;
    // the wave's steps: `wave` and every `waves`-th after it, so that those of
    // the workgroup that are under way are neighbours (each wave a run of its
    // own: 5 x 4096 x 14336 NVFP4 in rows 12.7 us instead of 12.2)
    const uint32_t count = (steps + waves - 1u - wave) / waves;

    // bytes from the step's start, below 2^32 as all of W is: the start is the
    // wave's, in scalar registers
    uint32_t codes[kR], scales[kR];
    const float *tile[kFormat == kNvTile ? kR : 1];
#pragma unroll
    for (int j = 0; j < kR; ++j) {  // past W's end: its last row again, not stored
        const uint32_t n = min(n0 + 16u * j + r, a.w.N - 1u);
        codes[j] = (n >> 5) * a.w.code_group + (n & 31u) * a.w.code_row +
                   (kP == 2 ? q * 32u : (q >> 1) * a.w.code_pair + (q & 1u) * a.w.code_q);
        scales[j] = (n >> 5) * a.w.scale_group + (n & 31u) * a.w.scale_row +
                    q * a.w.scale_q * kP;
        // 16 rows are within one 128 x 128 tile
        if (kFormat == kNvTile) tile[j] = a.tensor_scale + (int64_t)(min(n0 + 16u * j, a.w.N - 1u) >> 7) * a.steps;
    }
    // A load of x takes 64 / kPer rows, the last ones of M where it would go
    // past them (the rows before M are then there twice, the same; those of
    // LDS from M on hold anything, for columns of the result not stored): the
    // rows' place is the same for the wave, a lane's own part of the address
    // the same for all loads.
    constexpr uint32_t kPer = (kX8 ? 8 : 16) * kP, kOnce = 64u / kPer;
    const uint32_t row = min(lane / kPer, M - 1u), piece = lane % kPer;
    const uint32_t last = M > kOnce ? M - kOnce : 0u;
    // made anew in each step where the loads are many: kept over the loop, their
    // addresses spill
    const auto fresh = [](uint32_t v) {
        if constexpr (kMQ >= 2) {
            v = (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
            asm volatile("" : "+s"(v));
        }
        return v;
    };
    const int64_t x_row = a.ld_x * (kX8 ? 1 : 2), x_scale_row = a.steps * 4u;
    const uint8_t *x = a.x + (m0 + row) * x_row + piece * 16u;
    const uint8_t *x_scales = kX8 ? a.x_scales + (m0 + row) * x_scale_row + piece / 2u : nullptr;
    const auto fetch = [&](uint32_t i, S &s) {
        const uint32_t step = wave + i * waves;
        const uint8_t *step_codes = a.w.codes + step * kP * a.w.code_step;
        const uint8_t *step_scales = a.w.scales + step * kP * a.w.scale_step;
        const uint32_t end = fresh(last);
#pragma unroll
        for (int i = 0; i < S::kLoads; ++i) {
            const uint32_t m = min(i * kOnce, end);
            s.x[i] = *reinterpret_cast<const u32x4v *>(x + (m * x_row + step * ((kX8 ? 128u : 256u) * kP)));
            if (kX8) s.x_scale[i] = x_scales[m * x_scale_row + step * (4u * kP)];
        }
#pragma unroll
        for (int j = 0; j < kR; ++j) {
            const u32x4v *p = reinterpret_cast<const u32x4v *>(step_codes + codes[j]);
#pragma unroll
            for (int k = 0; k < kP; ++k) s.codes[j][k] = load_vec<kP == 1>(p + k);
            const uint8_t *b = step_scales + scales[j];
            constexpr int kBytes = (kFormat == kMx ? 1 : 2) * kP;
            if constexpr (kBytes == 1)
                s.scales[j] = *b;
            else if constexpr (kBytes == 2)
                s.scales[j] = *reinterpret_cast<const uint16_t *>(b);
            else
                s.scales[j] = *reinterpret_cast<const uint32_t *>(b);
            if (kFormat == kNvTile) s.tile[j] = tile[j][step];
        }
    };
    f32x4v acc[kR][H::kMT];
#pragma unroll
    for (int j = 0; j < kR; ++j) {
#pragma unroll
        for (int i = 0; i < H::kMT; ++i) acc[j][i] = (f32x4v){0.0f, 0.0f, 0.0f, 0.0f};
    }
    // A wave's step of x goes through its own part of LDS, as bf16, from the
    // lanes that loaded it to those that multiply it.  A wave's LDS accesses
    // are done in their order, so no wait but the fences that keep the
    // compiler to it.
    uint8_t *own = lds + wave * (H::kRows * H::kPitch);
    uint8_t *to0 = own + row * H::kPitch + piece * (kX8 ? 32u : 16u);
    const uint8_t *mine = own + (kMQ < 4 ? r % (kMQ * 4u) : r) * H::kPitch + q * (64u * kP);
    const auto multiply = [&](const S &s) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const uint32_t end = fresh(last);
#pragma unroll
        for (int i = 0; i < S::kLoads; ++i) {
            uint8_t *to = to0 + min(i * kOnce, end) * H::kPitch;
            if constexpr (kX8) {
                const float scale = mx_scale_f32(s.x_scale[i]);
                *reinterpret_cast<bf16x8v *>(to) = rows8(s.x[i][0], s.x[i][1], scale);
                *reinterpret_cast<bf16x8v *>(to + 16) = rows8(s.x[i][2], s.x[i][3], scale);
            } else {
                *reinterpret_cast<u32x4v *>(to) = s.x[i];
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int p = 0; p < kP; ++p) {
            bf16x8v b[H::kMT][4];
#pragma unroll
            for (int i = 0; i < H::kMT; ++i) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    b[i][k] = *reinterpret_cast<const bf16x8v *>(mine + i * (16u * H::kPitch) + p * 64u + k * 16u);
            }
#pragma unroll
            for (int j = 0; j < kR; ++j) {
                const uint32_t scales = kFormat == kMx ? s.scales[j] >> (8 * p) & 255u : s.scales[j] >> (16 * p);
                const f32x2v nv = __builtin_amdgcn_cvt_pk_f32_fp8(scales, false);
                f32x4v sum[H::kMT];
#pragma unroll
                for (int i = 0; i < H::kMT; ++i)
                    sum[i] = kFormat == kNvTile ? (f32x4v){0.0f, 0.0f, 0.0f, 0.0f} : acc[j][i];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const bf16x8v w = kFormat == kMx ? weights8_mx(s.codes[j][p][k], mx_scale_f32(scales))
                                                     : weights8_nv(s.codes[j][p][k], nv[k >> 1]);
#pragma unroll
                    for (int i = 0; i < H::kMT; ++i)
                        sum[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, b[i][k], sum[i], 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < H::kMT; ++i) {
                    if (kFormat == kNvTile) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[j][i][e] = __builtin_fmaf(sum[i][e], s.tile[kFormat == kNvTile ? j : 0], acc[j][i][e]);
                    } else {
                        acc[j][i] = sum[i];
                    }
                }
            }
        }
    };
    // kA steps in flight.  The main loop's loads are under no condition: under
    // one, the wait for a step could not tell how many loads came after it, and
    // waited for all of them.
    constexpr uint32_t kA = H::kAhead;
    S s[kA];
    uint32_t step = 0;
    if (kA == 1u) {
        if (count > 0u) fetch(0, s[0]);
        for (; step < count; ++step) {
            multiply(s[0]);
            __builtin_amdgcn_sched_barrier(0);
            if (step + 1u < count) fetch(step + 1u, s[0]);
            __builtin_amdgcn_sched_barrier(0);
        }
    } else if (count >= kA) {
#pragma unroll
        for (uint32_t d = 0; d < kA; ++d) fetch(d, s[d]);
        for (; step + 2u * kA <= count; step += kA) {
#pragma unroll
            for (uint32_t d = 0; d < kA; ++d) {
                multiply(s[d]);
                __builtin_amdgcn_sched_barrier(0);
                fetch(step + kA + d, s[d]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (uint32_t d = 0; d < kA; ++d) {  // fewer than kA steps are not loaded yet
            multiply(s[d]);
            __builtin_amdgcn_sched_barrier(0);
            if (step + kA + d < count) fetch(step + kA + d, s[d]);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (uint32_t d = 0; d + 1u < kA; ++d)
            if (step + kA + d < count) multiply(s[d]);
    } else {
        for (; step < count; ++step) {
            fetch(step, s[0]);
            multiply(s[0]);
        }
    }
    __syncthreads();  // the sums take x's place
    f32x4v *parts = reinterpret_cast<f32x4v *>(lds);  // [tiles][waves][64]
    const float scale = kFormat == kNvGlobal ? a.tensor_scale[0] : 1.0f;
    uint32_t again = 0;  // bit j kMT + i: this lane's part of that tile has a sum that is not finite
#pragma unroll
    for (int t0 = 0; t0 < H::kTiles; t0 += H::kAtOnce) {
        if (t0 > 0) __syncthreads();
#pragma unroll
        for (int t = t0; t < t0 + H::kAtOnce && t < H::kTiles; ++t)
            parts[((t - t0) * waves + wave) * 64u + lane] = acc[t / H::kMT][t % H::kMT];
        __syncthreads();
        for (uint32_t t = wave; t < (uint32_t)H::kAtOnce && t + t0 < (uint32_t)H::kTiles; t += waves) {
            const f32x4v *p = parts + t * waves * 64u + lane;
            f32x4v sum = p[0];
            for (uint32_t k = 1; k < waves; ++k) sum += p[k * 64u];
            // lane l has rows 4 (l / 16) .. + 3 of the tile's 16 of W, row l mod 16 of x
            const uint32_t n = n0 + (t + t0) / H::kMT * 16u + q * 4u, m = (t + t0) % H::kMT * 16u + r;
            if (m >= M) continue;
            if (kFormat == kMx) {
                float any = 0.0f;  // NaN where one is not finite
#pragma unroll
                for (int e = 0; e < 4; ++e) any = __builtin_fmaf(sum[e], 0.0f, any);
                again |= any != any ? 1u << (t + t0) : 0u;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = sum[e] * scale * a.alpha;
            store4(a, m0 + m, n, sum);
        }
    }
    if constexpr (kFormat == kMx) {
        if (__ballot(again != 0u) == 0u) return;
        for (uint32_t j = 0; j < (uint32_t)kR; ++j) {
            const uint32_t mine_again = again >> (j * H::kMT) & ((1u << H::kMT) - 1u), n = n0 + 16u * j;
            if (__ballot(mine_again != 0u) == 0u) continue;
            const uint32_t which = large_rows(a, n, r, q) >> (4u * q) & 15u;
            for (uint32_t i = 0; i < (uint32_t)H::kMT; ++i)
                if (mine_again >> i & 1u) again4<kX8>(a, m0 + 16u * i + r, n + 4u * q, which);
        }
    }
}

template <Format kFormat, bool kX8, int kMQ, int kR, int kP>
void run_matvec(const Matvec &a, uint32_t most, hipStream_t st)
{
    typedef Shape<kFormat, kX8, kMQ, kR, kP> H;
    const uint32_t steps = a.steps / kP, limit = most < (uint32_t)H::kWaves ? most : (uint32_t)H::kWaves;
    const uint32_t waves = steps < limit ? steps : limit;  // at least one of each
    unsigned grid = (a.w.N + 16u * kR - 1u) / (16u * kR);
    // workgroup i runs on XCD i mod 8: the groups that read the same rows of W on one
    if (a.groups > 1u) grid = (grid + 7u) / 8u * 8u;
    hipLaunchKernelGGL((matvec_kernel<kFormat, kX8, kMQ, kR, kP>), dim3(grid, a.groups), dim3(waves * 64u), H::lds_bytes(waves),
                       st, a);
}

template <Format kFormat, bool kX8, int kMQ, int kP, int kR>
void pick_rows(const Matvec &a, uint32_t r, uint32_t most, hipStream_t st)
{
    // with fewer rows of W to a unit, x's are in groups of 32 at most (group_rows)
    if constexpr (kR > (kMQ < 16 ? 1 : kFormat == kMx ? 4 : 3)) {
        if (r < (uint32_t)kR) return pick_rows<kFormat, kX8, kMQ, kP, kR - 1>(a, r, most, st);
    }
    run_matvec<kFormat, kX8, kMQ, kR, kP>(a, most, st);
}

// Rows of W to a wave: x is loaded, and goes through LDS, once for them, so a
// compute unit gets one workgroup of as many rows as it has to do, or where
// those are more than registers hold as few workgroups of the same rows.  With
// at most four rows of x, which cost little, 16 rows of W each are as good at
// any size.  Waves: four, of two steps in flight each; eight where a unit has
// only 16 rows of W, or (with more than 16 rows of x, and registers for them)
// only one step fits in flight; 16 with at most 16 rows of x on few but long
// rows of W, whose loads are all that is under way.  The waves, and so the
// order of the sums, do not depend on x's rows up to 16.
//   Measured in us on weights from memory, K = 4096, MXFP4 tiled unless named.
// Rows of W to a wave: 16 rows of x, 16 / 32 / 48 / 64 / 80 / 112: 8192 rows of W
// 8.0 / 6.4, 11008 10.7 / 9.7 / 7.3 / 8.0, 28672 - / 17.2 / 16.5 / 14.3 / 16.1 /
// 12.9 (in rows - / - / - / 19.3 / 22.5 / 18.5), 40000, 80 each for two workgroups
// and one of 112 for a first and most of a second round, - / - / - / 19.8 / 17.5
// / 20.4; 28672 rows of W, 64 / 80 / 112: 32 rows of x 18.8 / 22.2 / 16.2, in rows
// 27.4 / 31.3 / 21.7 (NVFP4 tiles 21.7 / 24.5, and 112, not kept, 22.9); 64 rows
// of x 26.0 / 36.4 / 23.5, in rows 35.5 / 40.1 / 27.7, NVFP4 tiles 42.4 / 46.8 / 30.0.  One row
// of x, 16 / 32: 11008 6.5 / 7.2, 28672 12.1 / 12.3, 60000 22.4 / 21.7; four rows,
// 28672 13.0 / 12.5.
//   Waves, four / eight: 16 rows of x 4096 rows of W 5.7 / 5.4, 8192 7.3 / 7.4, 14336
// 8.4 / 8.9, 28672 12.9 / 13.2; 32 rows of x, two steps in flight, 14336 10.9 /
// 11.2, one step, 20480 14.0 / 13.1, 28672 16.8 / 16.2; 64 rows of x, 12000 NVFP4
// 16.7 / 15.1.  Four / eight / sixteen, one row of x, 4096 rows of W 5.1 / 4.3 / 4.3,
// with K = 14336 12.0 / 8.4 / 7.9 (16 rows of x 13.2 / 12.6 / 12.7: they keep one
// row's waves).
template <Format kFormat, bool kX8, int kMQ, int kP>
void pick_waves(const Matvec &a, uint32_t units, hipStream_t st)
{
    constexpr uint32_t kMost = kMQ == 8 && kFormat == kNvTile ? 5 : 7;
    const uint32_t blocks = (a.w.N + 15u) / 16u, each = (blocks * a.groups + units - 1u) / units;
    const uint32_t waves = each > 1u ? 4u : kP == 1 && a.steps >= 64u ? 16u : 8u;
    if constexpr (kMQ == 1) {
        run_matvec<kFormat, kX8, 1, 1, kP>(a, waves, st);
    } else {
        const uint32_t groups = (each + kMost - 1u) / kMost, r = (each + groups - 1u) / groups;
        const bool eight = groups == 1u && ((kMQ == 8 && r * kP > 4u) || (kMQ == 16 && r == 3u));
        pick_rows<kFormat, kX8, kMQ, kP, kMost>(a, r, eight ? 8u : waves, st);
    }
}

template <Format kFormat, bool kX8, int kMQ>
void pick_layout(const Matvec &a, bool linear, uint32_t units, hipStream_t st)
{
    if constexpr (kFormat != kNvTile) {  // (a lane's 64 columns side by side: four lanes meet two tiles)
        if (linear && a.steps % 2 == 0) return pick_waves<kFormat, kX8, kMQ, 2>(a, units, st);
    }
    pick_waves<kFormat, kX8, kMQ, 1>(a, units, st);
}

// Rows of x to a workgroup.  Where a unit has few rows of W, x of many rows is
// most of what it reads and stages; groups of x's rows in workgroups of their
// own read W again (from the L2, being on one XCD and under way together).
// The cost of a unit's rows of W (16 each) and of x (four each) is weighed as
// measured: NVFP4's converts, and W in rows, count for more.  x's type does not
// (8-bit rows may not be summed in another order than the rows unpacked; four
// for them with W in rows instead of eight: 32 x 4096 x 4096 7.0 us instead of
// 6.1, 64 x 8192 x 4096 13.9 instead of 11.2).  More groups have to win a
// sixteenth: any less, and 20 x 2000 x 4096 in rows takes 5.7 us instead of 5.1,
// 48 x 6144 x 4096 11.0 instead of 9.9, 20 x 11008 x 4096 tiled 9.6 instead of 8.7
// (the other way, 48 x 5000 x 4096 NVFP4 tiled 9.4 instead of 10.7).
//   us from memory, one group / as many as this gives: 32 rows of x, MXFP4 tiled
// 512 x 8192 11.1 / 5.2, 4096 x 4096 7.5 / 6.0, 4096 x 14336 18.4 / 14.3, 8192 x
// 4096 8.4 / 7.7, NVFP4 2000 x 14336 18.6 / 12.5; 64 rows, MXFP4 4096 x 4096 11.2 /
// 7.2; 16 rows 512 x 8192 7.7 / 5.3.  24 rows, in two groups where this gives
// one: MXFP4 12000 x 8192 15.1 / 16.2, in rows 20.4 / 23.8.
uint32_t group_rows(const Matvec &a, bool nv, bool linear, uint32_t units)
{
    uint32_t whole = 4u;
    while (whole < a.M) whole *= 2u;
    const uint32_t blocks = (a.w.N + 15u) / 16u, of_w = nv ? 24u : linear ? 14u : 9u, of_x = 8u;
    uint32_t best = whole, least = 0u;
    for (uint32_t rows = whole; rows >= 4u; rows /= 2u) {
        const uint32_t groups = (a.M + rows - 1u) / rows, each = (blocks * groups + units - 1u) / units;
        // up to 16 rows the order of the sums stays that of one row, whose waves are chosen by `each`
        if (groups > 1u && each > 1u && (a.M <= 16u || rows == 4u)) break;
        const uint32_t r = (each + (each + 6u) / 7u - 1u) / ((each + 6u) / 7u), wide = (blocks + r - 1u) / r;
        const uint32_t workgroups = groups > 1u ? (wide + 7u) / 8u * 8u * groups : wide;
        const uint32_t cost = (workgroups + units - 1u) / units * (r * of_w + rows / 4u * of_x);
        if (rows == whole || cost * 16u < least * 15u) least = cost, best = rows;
    }
    return best;
}

template <Format kFormat, bool kX8>
void pick_matvec(const Matvec &a, bool linear, uint32_t units, hipStream_t st)
{
    Matvec g = a;
    const uint32_t rows = group_rows(a, kFormat != kMx, linear, units);
    g.groups = (a.M + rows - 1u) / rows;
    if (rows <= 4u)
        pick_layout<kFormat, kX8, 1>(g, linear, units, st);
    else if (rows <= 8u)
        pick_layout<kFormat, kX8, 2>(g, linear, units, st);
    else if (rows <= 16u)
        pick_layout<kFormat, kX8, 4>(g, linear, units, st);
    else if (rows <= 32u)
        pick_layout<kFormat, kX8, 8>(g, linear, units, st);
    else
        pick_layout<kFormat, kX8, 16>(g, linear, units, st);
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
        a.w.code_row = (uint32_t)(K / 2);
        a.w.scale_row = (uint32_t)scale_bytes;
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
    a.w.code_group = (uint32_t)(16 * K);
    a.w.scale_group = g.tiled && !nv ? 128u : (uint32_t)(32 * scale_bytes);
    a.x = reinterpret_cast<const uint8_t *>(g.x);
    a.x_scales = reinterpret_cast<const uint8_t *>(g.x_scales);
    a.tensor_scale = g.tensor_scale;
    a.ld_x = g.ld_x;
    a.ld_y = g.ld_y;
    a.M = (uint32_t)g.M;
    a.w.N = (uint32_t)g.N;
    a.steps = (uint32_t)(K / 128);
    a.alpha = g.alpha;
    a.y = g.y;
    a.y_bf16 = g.y_bf16;
    return a;
}

}  // namespace

}  // namespace fp4q
