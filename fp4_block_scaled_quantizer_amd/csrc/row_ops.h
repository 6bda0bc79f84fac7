// row_ops.h -- building blocks of the row-wise operators between the FP4
// GEMMs (norm and its gradient, dropout, SwiGLU's gradient, rotary
// positions): eight-element chunks of bf16 or binary32 rows at any element
// alignment, reductions over a wave, and dropout's keep rule.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4q_device.h"

namespace fp4q {

typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
// gfx950 loads and stores 16 bytes at any byte address; the alignment the
// type promises is the element's, so rows of odd pitch take the same path
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
typedef float f32x2v __attribute__((ext_vector_type(2)));

struct bf16_t { uint16_t bits; };  // storage of a bf16 element

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2v){lo, hi}, bf16x2v));  // v_cvt_pk_bf16_f32, RNE
}

// Eight consecutive elements of a row in registers, as stored.
template <typename T> struct Chunk;
template <> struct Chunk<bf16_t> {
    u32x4v q;
    __device__ __forceinline__ void load(const bf16_t *p)
    {
        q = *reinterpret_cast<const u32x4_a2 *>(p);
    }
    __device__ __forceinline__ void store(bf16_t *p) const { *reinterpret_cast<u32x4_a2 *>(p) = q; }
    __device__ __forceinline__ void mask(bool keep)
    {
        const uint32_t m = keep ? ~0u : 0u;
        q = (u32x4v){q[0] & m, q[1] & m, q[2] & m, q[3] & m};
    }
    __device__ __forceinline__ void get(float v[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(q[i]);
            v[2 * i + 1] = bf16_hi(q[i]);
        }
    }
    __device__ __forceinline__ void set(const float v[8])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    }
    static __device__ __forceinline__ float load1(const bf16_t *p) { return u2f((uint32_t)p->bits << 16); }
    __device__ __forceinline__ void store_first(bf16_t *p, uint32_t n) const
    {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < (int)n) p[j].bits = (uint16_t)(q[j >> 1] >> (16 * (j & 1)));
    }
};
template <> struct Chunk<float> {
    u32x4v a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = *reinterpret_cast<const u32x4_a4 *>(p);
        b = *reinterpret_cast<const u32x4_a4 *>(p + 4);
    }
    __device__ __forceinline__ void store(float *p) const
    {
        *reinterpret_cast<u32x4_a4 *>(p) = a;
        *reinterpret_cast<u32x4_a4 *>(p + 4) = b;
    }
    __device__ __forceinline__ void mask(bool keep)
    {
        const uint32_t m = keep ? ~0u : 0u;
        a = (u32x4v){a[0] & m, a[1] & m, a[2] & m, a[3] & m};
        b = (u32x4v){b[0] & m, b[1] & m, b[2] & m, b[3] & m};
    }
    __device__ __forceinline__ void get(float v[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = u2f(a[i]);
            v[4 + i] = u2f(b[i]);
        }
    }
    __device__ __forceinline__ void set(const float v[8])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = f2u(v[i]);
            b[i] = f2u(v[4 + i]);
        }
    }
    static __device__ __forceinline__ float load1(const float *p) { return *p; }
    __device__ __forceinline__ void store_first(float *p, uint32_t n) const
    {
        float v[8];
        get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < (int)n) p[j] = v[j];
    }
};

// Chunk c of a row of `cols` elements (cols >= 1).  A chunk past the row's
// end gives zeros.  The loads themselves are unconditional, from clamped
// in-bounds addresses, because a load under a branch is waited for inside
// it; what they fetch beyond the chunk is masked.  kTail: cols % 8 != 0;
// the row's last chunk then loads the row's last eight elements and moves
// its own to the front (rows shorter than eight are loaded one by one).
template <typename T, bool kTail>
__device__ __forceinline__ void load_chunk(const T *row, uint32_t c, uint32_t cols, Chunk<T> &q)
{
    const uint32_t at = c * 8u;
    const bool in = at < cols;
    if constexpr (!kTail) {
        q.load(row + (in ? at : 0u));
        q.mask(in);
    } else if (cols >= 8u) {
        const uint32_t from = min(at, cols - 8u);
        q.load(row + from);
        const uint32_t by = at - from;  // the chunk's own elements start here (>= 8: none)
        if (by != 0u) {
            float v[8];
            q.get(v);
#pragma unroll
            for (int s = 4; s >= 1; s >>= 1) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float w = j + s < 8 ? v[j + s] : 0.0f;
                    v[j] = (by & (uint32_t)s) ? w : v[j];
                }
            }
            q.set(v);
            q.mask(by < 8u);
        }
    } else {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float w = Chunk<T>::load1(row + min(at + j, cols - 1u));
            v[j] = at + j < cols ? w : 0.0f;
        }
        q.set(v);
    }
}
template <typename T, bool kTail>
__device__ __forceinline__ void store_chunk(T *row, uint32_t c, uint32_t cols, const Chunk<T> &q)
{
    const uint32_t at = c * 8u;
    if (!kTail || at + 8u <= cols) {
        if (at < cols) q.store(row + at);
    } else if (at < cols) {
        q.store_first(row + at, cols - at);
    }
}

// Sum over the 64 lanes of a wave, the same on every lane: DPP shifts inside
// the rows of 16, then two broadcasts across rows (a fixed order, no LDS).
template <int kCtrl, int kRowMask>
__device__ __forceinline__ float dpp_add(float v)
{
    return v + u2f((uint32_t)__builtin_amdgcn_update_dpp(0, (int)f2u(v), kCtrl, kRowMask, 0xF, true));
}
__device__ __forceinline__ float wave_sum(float v)
{
    v = dpp_add<0x111, 0xF>(v);  // row_shr:1
    v = dpp_add<0x112, 0xF>(v);  // row_shr:2
    v = dpp_add<0x114, 0xF>(v);  // row_shr:4
    v = dpp_add<0x118, 0xF>(v);  // row_shr:8 -- lane 15 of a row holds its sum
    v = dpp_add<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
    v = dpp_add<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
    return u2f((uint32_t)__builtin_amdgcn_readlane((int)f2u(v), 63));
}

// Dropout.  Element (r, k) draws 16 bits as stochastic rounding does, from
// Philox4x32-10 under counter {k / 8, r, stream_id, 1} (the 1 keeps the two
// uses apart) and is kept iff they are >= drop = rint(p 2^16); kept values
// are scaled by 2^16 / (2^16 - drop), which is unbiased for the probability
// that the 16 bits give.  Nothing is stored: the gradient draws the same bits.
struct Dropout {
    uint32_t drop;  // 0: off
    float scale;
    uint32_t key0, key1, stream;
};
inline Dropout dropout_of(float p, uint64_t seed, uint32_t stream_id)
{
    Dropout d{};
    d.drop = (uint32_t)__builtin_rint((double)p * 65536.0);
    d.scale = d.drop >= 65536u ? 0.0f : (float)(65536.0 / (double)(65536u - d.drop));
    d.key0 = (uint32_t)seed;
    d.key1 = (uint32_t)(seed >> 32);
    d.stream = stream_id;
    return d;
}
__device__ __forceinline__ void apply_dropout(const Dropout &d, uint32_t r, uint32_t c, float v[8])
{
    uint32_t w[4];
    philox4x32_10(c, r, d.stream, 1u, d.key0, d.key1, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = r16_of(w, j) >= d.drop ? v[j] * d.scale : 0.0f;
}

}  // namespace fp4q
