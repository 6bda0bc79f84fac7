// row_ops.h -- building blocks of the row-wise operators between the FP4
// GEMMs (norm and its gradient, dropout, SwiGLU's gradient, rotary
// positions): eight-element chunks of bf16 or binary32 rows at any element
// alignment, reductions over a wave, and dropout's keep rule.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fp4q_device.h"

namespace fp4q {

typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
// gfx950 loads and stores 16 bytes at any byte address; the alignment the
// type promises is the element's, so rows of odd pitch take the same path
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x2_a4 __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));
typedef uint32_t u32_a2 __attribute__((aligned(2)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
typedef float f32x2v __attribute__((ext_vector_type(2)));

// Non-temporal or not.  What a kernel streams -- read or written once, whole
// cache lines by each wave instruction -- is marked non-temporal: bf16 chunks
// are (16 bytes a lane, 1 KiB a wave), binary32 chunks are not (two loads
// each touch every line of 2 KiB, and the second one finds the line gone).
// Measured on matrices that do not fit the caches: dropout 8192 x 14336 bf16
// 75.5 us with, 80.7 without; with residual 8192 x 4096 binary32 74.0 with,
// 69.8 without.
template <typename T> constexpr bool kStream = sizeof(T) == 2;
template <bool kNt, typename V>
__device__ __forceinline__ V load_vec(const V *p)
{
    if constexpr (kNt)
        return __builtin_nontemporal_load(p);
    else
        return *p;
}
template <bool kNt, typename V, typename W>
__device__ __forceinline__ void store_vec(V *p, W v)
{
    if constexpr (kNt)
        __builtin_nontemporal_store((V)v, p);
    else
        *p = v;
}

struct bf16_t { uint16_t bits; };  // storage of a bf16 element
__device__ __forceinline__ float as_float(bf16_t v) { return u2f((uint32_t)v.bits << 16); }
__device__ __forceinline__ float as_float(float v) { return v; }

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2v){lo, hi}, bf16x2v));  // v_cvt_pk_bf16_f32, RNE
}

// Eight consecutive elements of a row in registers, as stored.
template <typename T> struct Chunk;
template <> struct Chunk<bf16_t> {
    u32x4v q;
    template <bool kNt> __device__ __forceinline__ void load(const bf16_t *p)
    {
        q = load_vec<kNt>(reinterpret_cast<const u32x4_a2 *>(p));
    }
    template <bool kNt> __device__ __forceinline__ void store(bf16_t *p) const
    {
        store_vec<kNt>(reinterpret_cast<u32x4_a2 *>(p), q);
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
    // the elements lo .. hi - 1 only: they move to the front, and then four,
    // two and one of them are stored
    __device__ __forceinline__ void store_own(bf16_t *p, uint32_t lo, uint32_t hi) const
    {
        uint32_t v[4] = {q[0], q[1], q[2], q[3]};
        if (lo & 4u) v[0] = v[2], v[1] = v[3];
        if (lo & 2u) v[0] = v[1], v[1] = v[2], v[2] = v[3];
        if (lo & 1u) {
            v[0] = v[0] >> 16 | v[1] << 16;
            v[1] = v[1] >> 16 | v[2] << 16;
            v[2] = v[2] >> 16 | v[3] << 16;
            v[3] = v[3] >> 16;
        }
        const uint32_t n = hi - lo;
        p += lo;
        if (n & 4u) {
            *reinterpret_cast<u32x2_a2 *>(p) = (u32x2v){v[0], v[1]};
            v[0] = v[2], v[1] = v[3];
            p += 4;
        }
        if (n & 2u) {
            *reinterpret_cast<u32_a2 *>(p) = v[0];
            v[0] = v[1];
            p += 2;
        }
        if (n & 1u) p->bits = (uint16_t)v[0];
    }
};
template <> struct Chunk<float> {
    u32x4v a, b;
    template <bool kNt> __device__ __forceinline__ void load(const float *p)
    {
        a = load_vec<kNt>(reinterpret_cast<const u32x4_a4 *>(p));
        b = load_vec<kNt>(reinterpret_cast<const u32x4_a4 *>(p + 4));
    }
    template <bool kNt> __device__ __forceinline__ void store(float *p) const
    {
        store_vec<kNt>(reinterpret_cast<u32x4_a4 *>(p), a);
        store_vec<kNt>(reinterpret_cast<u32x4_a4 *>(p + 4), b);
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
    __device__ __forceinline__ void store_own(float *p, uint32_t lo, uint32_t hi) const
    {
        uint32_t v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
        for (int s = 4; s >= 1; s >>= 1)
            if (lo & (uint32_t)s) {
#pragma unroll
                for (int j = 0; j + s < 8; ++j) v[j] = v[j + s];
            }
        const uint32_t n = hi - lo;
        p += lo;
        if (n & 4u) {
            *reinterpret_cast<u32x4_a4 *>(p) = (u32x4v){v[0], v[1], v[2], v[3]};
            v[0] = v[4], v[1] = v[5], v[2] = v[6];
            p += 4;
        }
        if (n & 2u) {
            *reinterpret_cast<u32x2_a4 *>(p) = (u32x2v){v[0], v[1]};
            v[0] = v[2];
            p += 2;
        }
        if (n & 1u) *p = u2f(v[0]);
    }
};

// How a width divides into chunks of eight: kWhole, evenly; kRagged, with a
// rest; kTiny, below eight.
enum Edge { kWhole, kRagged, kTiny };
inline Edge edge_of(int64_t cols) { return cols % 8 == 0 ? kWhole : cols > 8 ? kRagged : kTiny; }

// Chunk c of a row of `cols` elements (cols >= 1): eight consecutive columns
// from `from`, of which lo .. hi - 1 are the chunk's own.  A load covers all
// eight, from an in-bounds place, whatever the chunk: a load under a branch
// is waited for inside it.  A chunk past the row's end owns nothing and reads
// the row's start (kWhole) or end; a ragged row's last chunk reads the row's
// last eight columns, the first of them its neighbour's; a tiny row is read
// one by one.  Sums leave out, and stores keep off, what is not the chunk's
// own; a NaN read beside it is in the same row.
struct Span {
    uint32_t from, lo, hi;
    __device__ __forceinline__ bool own(int j) const { return (uint32_t)j >= lo && (uint32_t)j < hi; }
    __device__ __forceinline__ bool any() const { return lo < hi; }
};
template <Edge kEdge>
__device__ __forceinline__ Span span_of(uint32_t c, uint32_t cols)
{
    const uint32_t at = c * 8u;
    const bool in = at < cols;
    Span s;
    if (kEdge == kWhole) {
        s.from = in ? at : 0u;
        s.lo = 0u;
        s.hi = in ? 8u : 0u;
    } else if (kEdge == kRagged) {
        s.from = min(at, cols - 8u);
        s.lo = min(at - s.from, 8u);
        s.hi = in ? 8u : 0u;
    } else {
        s.from = 0u;
        s.lo = 0u;
        s.hi = in ? cols : 0u;
    }
    return s;
}

// Element `from` of a row: a 32-bit byte offset, so that a row whose address
// is the same for the whole wave is addressed from scalar registers.  Rows
// are below 2^30 elements.
template <typename T>
__device__ __forceinline__ T *in_row(T *row, uint32_t from)
{
    typedef typename std::conditional<std::is_const<T>::value, const char, char>::type Byte;
    return reinterpret_cast<T *>(reinterpret_cast<Byte *>(row) + (uint32_t)(from * (uint32_t)sizeof(T)));
}
template <typename T, Edge kEdge, bool kNt = false>
__device__ __forceinline__ void load_chunk(const T *row, const Span &s, uint32_t cols, Chunk<T> &q)
{
    if (kEdge != kTiny) {
        q.template load<kNt>(in_row(row, s.from));
    } else {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = as_float(row[min((uint32_t)j, cols - 1u)]);
        q.set(v);
    }
}
template <typename T, Edge kEdge, bool kNt = false>
__device__ __forceinline__ void store_chunk(T *row, const Span &s, const Chunk<T> &q)
{
    if (kEdge == kWhole || (s.lo == 0u && s.hi == 8u)) {
        if (s.hi != 0u) q.template store<kNt>(in_row(row, s.from));
    } else if (s.any()) {
        q.store_own(in_row(row, s.from), s.lo, s.hi);
    }
}

// A chunk of a weight vector of either type, loaded where it is used.
template <Edge kEdge>
__device__ __forceinline__ void weights_now(const void *w, bool bf16, const Span &s, uint32_t cols, float v[8])
{
    if (bf16) {
        Chunk<bf16_t> q;
        load_chunk<bf16_t, kEdge>(reinterpret_cast<const bf16_t *>(w), s, cols, q);
        q.get(v);
    } else {
        Chunk<float> q;
        load_chunk<float, kEdge>(reinterpret_cast<const float *>(w), s, cols, q);
        q.get(v);
    }
}

// Sums by DPP, in a fixed order and without LDS: shifts inside the rows of 16
// lanes, then for the whole wave two broadcasts across rows.
template <int kCtrl, int kRowMask>
__device__ __forceinline__ float dpp_add(float v)
{
    return v + u2f((uint32_t)__builtin_amdgcn_update_dpp(0, (int)f2u(v), kCtrl, kRowMask, 0xF, true));
}
// The sum of each row of 16 lanes, in its lane 15.
__device__ __forceinline__ float sum16(float v)
{
    v = dpp_add<0x111, 0xF>(v);  // row_shr:1
    v = dpp_add<0x112, 0xF>(v);  // row_shr:2
    v = dpp_add<0x114, 0xF>(v);  // row_shr:4
    return dpp_add<0x118, 0xF>(v);  // row_shr:8
}
__device__ __forceinline__ float lane_value(float v, int lane)
{
    return u2f((uint32_t)__builtin_amdgcn_readlane((int)f2u(v), lane));
}
// The sum of all 64 lanes, on every lane.
__device__ __forceinline__ float wave_sum(float v)
{
    v = sum16(v);
    v = dpp_add<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
    v = dpp_add<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
    return lane_value(v, 63);
}

// The sum of each group of kLanes neighbouring lanes (16, 32 or 64), on every
// lane of it: rotations inside a row of 16 and one exchange between two rows.
template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v)
{
    if (kLanes == 64) return wave_sum(v);
    v = dpp_add<0x128, 0xF>(v);  // row_ror:8
    v = dpp_add<0x124, 0xF>(v);  // row_ror:4
    v = dpp_add<0x122, 0xF>(v);  // row_ror:2
    v = dpp_add<0x121, 0xF>(v);  // row_ror:1
    if (kLanes == 32) v += u2f((uint32_t)__builtin_amdgcn_ds_swizzle((int)f2u(v), 0x401F));  // lane ^ 16
    return v;
}
// How many lanes a short row takes (one chunk each); 64 above 256 columns.
inline int lanes_of(int64_t cols) { return cols <= 128 ? 16 : cols <= 256 ? 32 : 64; }

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
// The random words of chunk c of row r, element j of the registers (the
// chunk's element j - lo) drawing half j; and what they do to its values.
// Apart, so that the words can be made while the values are on their way.
struct Draws {
    uint32_t w[4];
};
template <Edge kEdge>
__device__ __forceinline__ Draws draws_of(const Dropout &d, uint32_t r, uint32_t c, const Span &s)
{
    Draws x;
    uint32_t(&w)[4] = x.w;
    philox4x32_10(c, r, d.stream, 1u, d.key0, d.key1, w);
    if (kEdge == kRagged && s.lo != 0u) {  // the random halves move up by lo places
        if (s.lo & 4u) w[3] = w[1], w[2] = w[0];
        if (s.lo & 2u) w[3] = w[2], w[2] = w[1], w[1] = w[0];
        if (s.lo & 1u) {
            w[3] = w[3] << 16 | w[2] >> 16;
            w[2] = w[2] << 16 | w[1] >> 16;
            w[1] = w[1] << 16 | w[0] >> 16;
            w[0] = w[0] << 16;
        }
    }
    return x;
}
__device__ __forceinline__ void apply_dropout(const Dropout &d, const Draws &x, float v[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = r16_of(x.w, j) >= d.drop ? v[j] * d.scale : 0.0f;
}

}  // namespace fp4q
