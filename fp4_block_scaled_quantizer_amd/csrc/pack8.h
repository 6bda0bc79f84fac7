// pack8.h -- 8-bit block-scaled rows: OCP FP8 E4M3 codes [rows x cols] and one
// E8M0 scale per 32 elements along the row [rows x cols/32], both dense.
//
// A block's scale is 2^E with E the least integer that brings its largest
// finite magnitude to E4M3's largest value, 448, or below (the floor(log2) - 8
// of the MX specification lets (448, 512) 2^E saturate, off by up to an
// eighth; here no element is off by more than half a step, 2^-4 of its value).
// E stops at 119, so that no code stands for 2^128 or more: elements above 448
// 2^119 become that.  NaN and infinities do not count towards the scale and
// become E4M3's NaN.
#pragma once

#include "row_ops.h"

namespace fp4q {

typedef short s16x2v __attribute__((ext_vector_type(2)));
constexpr uint32_t kPack8TopByte = 119 + 127;

// E8M0 byte E + 127 of a block whose largest finite magnitude has the binary32
// bits `amax`: with a significand of 1.75 or less amax 2^-E lies in (224, 448]
// for E = floor(log2 amax) - 8, above that one more is needed.
FP4Q_HD uint32_t pack8_scale_byte(uint32_t amax)
{
    const uint32_t e = (amax >> 23) + ((amax & 0x7FFFFFu) > 0x600000u ? 1u : 0u);
    const uint32_t byte = e > 8u ? e - 8u : 0u;
    return byte < kPack8TopByte ? byte : kPack8TopByte;
}

template <int kMask>
__device__ __forceinline__ uint32_t quad_max(uint32_t v)
{
    constexpr int ctrl = kMask == 1 ? 0xB1 : 0x4E;  // quad_perm [1,0,3,2] / [2,3,0,1]
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xF, 0xF, false));
}

// Eight packed elements and their block's scale byte.
struct Packed8 {
    u32x2v q;
    uint32_t scale;
    // chunk `c` of all rows' (eight elements each, rows being dense)
    __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *scales, uint64_t c)
    {
        q = load_vec<false>(reinterpret_cast<const u32x2v *>(codes + c * 8u));
        scale = scales[c >> 2];
    }
    __device__ __forceinline__ void get(float v[8]) const
    {
        const float s = mx_scale_f32(scale);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const f32x2v lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q[i], s, false);
            const f32x2v hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q[i], s, true);
            v[4 * i] = lo[0], v[4 * i + 1] = lo[1], v[4 * i + 2] = hi[0], v[4 * i + 3] = hi[1];
        }
    }
};

// The largest magnitude of a chunk as binary32 bits; with kFinite, of its
// finite elements.
template <bool kFinite>
__device__ __forceinline__ uint32_t chunk_amax(const Chunk<bf16_t> &x)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = (i & 1 ? x.q[i >> 1] >> 16 : x.q[i >> 1]) & 0x7FFFu;
        m = max(m, kFinite && b >= 0x7F80u ? 0u : b);
    }
    return m << 16;
}
template <bool kFinite>
__device__ __forceinline__ uint32_t chunk_amax(const Chunk<float> &x)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = (i < 4 ? x.a[i & 3] : x.b[i & 3]) & 0x7FFFFFFFu;
        m = max(m, kFinite && b >= 0x7F800000u ? 0u : b);
    }
    return m;
}

// x / 2^E in E4M3, round to nearest even, by gfx950's scaled converts (all
// codes checked against the rule; a magnitude above 464 would become NaN).
__device__ __forceinline__ void convert8(const Chunk<bf16_t> &x, float scale, u32x2v &q)
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = x.q[2 * i], hi = x.q[2 * i + 1];
        s16x2v w = {0, 0};
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(bf16x2v, lo), scale, false);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(bf16x2v, hi), scale, true);
        q[i] = __builtin_bit_cast(uint32_t, w);
    }
}
__device__ __forceinline__ void convert8(const Chunk<float> &x, float scale, u32x2v &q)
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const u32x4v v = i ? x.b : x.a;
        s16x2v w = {0, 0};
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, u2f(v[0]), u2f(v[1]), scale, false);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, u2f(v[2]), u2f(v[3]), scale, true);
        q[i] = __builtin_bit_cast(uint32_t, w);
    }
}

// A chunk packed; the four chunks of a block sit in four neighbouring lanes,
// which all come here.
template <typename T>
__device__ __forceinline__ Packed8 pack8(Chunk<T> x)
{
    Packed8 p;
    uint32_t amax = chunk_amax<false>(x);
    amax = quad_max<2>(quad_max<1>(amax));
    if (amax >= 0x7F800000u) {  // the same in the four lanes
        amax = chunk_amax<true>(x);
        amax = quad_max<2>(quad_max<1>(amax));
        float v[8];  // the converts keep an infinity's sign, not a NaN's
        x.get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = v[j] != v[j] ? __builtin_copysignf(__builtin_inff(), v[j]) : v[j];
        x.set(v);
    }
    p.scale = pack8_scale_byte(amax);
    if (p.scale == kPack8TopByte) {
        float v[8];
        x.get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = f2u(v[j]) & 0x7FFFFFFFu;  // 448 * 2^119: 0x7F600000
            v[j] = b > 0x7F600000u && b < 0x7F800000u ? __builtin_copysignf(u2f(0x7F600000u), v[j]) : v[j];
        }
        x.set(v);
    }
    convert8(x, mx_scale_f32(p.scale), p.q);
    return p;
}

// Stores the scale bytes of 16 neighbouring lanes' chunks, four blocks, with
// one instruction by the first lane where `whole` says that all are there, or
// each by its block's first.  to: the scale of this lane's block; c: its
// chunk, lane 0 of each 16 having a multiple of four.
__device__ __forceinline__ void store_scales8(uint8_t *to, uint32_t byte, uint32_t lane16, bool whole, bool in)
{
    uint32_t word = byte;
    word |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)byte, 0x104, 0xF, 0xF, true) << 8;   // row_shl:4
    word |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)byte, 0x108, 0xF, 0xF, true) << 16;  // row_shl:8
    word |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)byte, 0x10C, 0xF, 0xF, true) << 24;  // row_shl:12
    if (!in) return;
    if (whole) {
        if (lane16 == 0u) *reinterpret_cast<u32_a1 *>(to) = word;
    } else if ((lane16 & 3u) == 0u) {
        *to = (uint8_t)byte;
    }
}

}  // namespace fp4q
