// norm.hip -- layer norm and RMS norm over rows, with the residual add and
// dropout in front of them and the producers of the MXFP4 operand and of 8-bit
// rows behind them.
//
// Per row of n columns:
//   h = [residual +] dropout(x), rounded to the element type;
//   mean = sum h / n (RMS: 0), rstd = 1 / sqrt(sum (h - mean)^2 / n + eps);
//   y = (h - mean) rstd gamma + beta, rounded; optionally the MXFP4 operand
//   of y along rows and its 8-bit rows, byte for byte what the row producer
//   and the packing make of y.
// A row stays in registers between its two sums (the second one of the
// centred values, so that a large mean costs no precision), and each input
// is read and each output written once: HBM-bound.  One workgroup per row, a
// chunk of eight elements per thread (two above 4096 columns, four above
// 16384; at 1024 and below a wave per row, at 256 half a wave and at 128, the
// norms of single heads, a quarter), many workgroups to a compute unit, so
// that one row's loads run under another's sums and stores.
// Measured a call, matrices from memory, where a copy reaches 6.3 TB/s:
//   8192 x 4096 bf16, layer norm, dropout, residual: 44.7 us, 6.0 TB/s;
//   327680 x 128 bf16, layer norm: 32.9 us, 5.2 TB/s (a wave per row 80; 32768
//   x 256 9.4, a wave per row 12.6);
//   1537 x 5003 binary32, layer norm: 18.6 us, 3.3 TB/s, or 13.4 where three
//   such in turn fit the last-level cache (1536 rows at once, six workgroups
//   to a compute unit: the loads of all, the stores of all, and one row more);
//   4097 x 4099 bf16: 23.9 us, 2.8 TB/s (rows share cache lines, and two chunks
//   a thread leave a fifth of the places empty);
//   1 x 4096 bf16: 4.8 us a call, launch and latency;
//   8192 x 4096 to 8-bit rows and no y: bf16 RMS norm with residual 38.5 us, 6.1
//   TB/s (with the MXFP4 operand too, in rows 42.8 for 39.7, tiled 44.8); binary32
//   layer norm 37.5, 4.5; 1 x 4096 5.7 us a call.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4q_internal.h"
#include "pack8.h"
#include "row_ops.h"

namespace fp4q {

namespace {

// Eight weights as stored, in either type: the loads are the same whatever
// the type (bf16 reads its 16 bytes twice), so that nothing waits for them
// under a branch; get() is where they have to be there.
struct Weights {
    u32x4v a, b;
    __device__ __forceinline__ void get(bool bf16, float v[8]) const
    {
        Chunk<bf16_t> h;
        Chunk<float> f;
        h.q = a;
        f.a = a;
        f.b = b;
        if (bf16)
            h.get(v);
        else
            f.get(v);
    }
};
template <Edge kEdge>
__device__ __forceinline__ void load_weights(const void *w, bool bf16, const Span &s, uint32_t cols, Weights &q)
{
    if (kEdge != kTiny) {
        const char *p = reinterpret_cast<const char *>(w) + (s.from << (bf16 ? 1 : 2));
        q.a = *reinterpret_cast<const u32x4_a2 *>(p);
        q.b = *reinterpret_cast<const u32x4_a2 *>(p + (bf16 ? 0 : 16));
    } else if (bf16) {
        Chunk<bf16_t> h;
        load_chunk<bf16_t, kEdge>(reinterpret_cast<const bf16_t *>(w), s, cols, h);
        q.a = q.b = h.q;
    } else {
        Chunk<float> f;
        load_chunk<float, kEdge>(reinterpret_cast<const float *>(w), s, cols, f);
        q.a = f.a;
        q.b = f.b;
    }
}

// Sum over the `waves` waves (at most 16) of a workgroup, through LDS
// (`slot`: a float per wave, for this sum alone).  Every thread must call it.
__device__ __forceinline__ float row_sum(float v, float *slot, uint32_t wave, uint32_t waves)
{
    v = wave_sum(v);
    const uint32_t lane = threadIdx.x & 63u;
    if (lane == 0) slot[wave] = v;
    __syncthreads();
    v = lane < waves ? slot[lane] : 0.0f;
    return lane_value(sum16(v), 15);
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
    // the scale bytes of four blocks, 16 lanes, as one word in the first lane
    uint32_t word = sbyte;
    word |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)sbyte, 0x104, 0xF, 0xF, true) << 8;   // row_shl:4
    word |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)sbyte, 0x108, 0xF, 0xF, true) << 16;  // row_shl:8
    word |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)sbyte, 0x10C, 0xF, 0xF, true) << 24;  // row_shl:12
    if (c * 8u >= cols) return;
    uint8_t *codes = reinterpret_cast<uint8_t *>(a.codes), *scales = reinterpret_cast<uint8_t *>(a.scales);
    const uint64_t r = (uint64_t)row;
    if (a.tiled) {  // cols % 128 == 0
        *reinterpret_cast<uint32_t *>(codes + ((r >> 5) * (cols >> 6) + (c >> 3)) * 1024u +
                                      ((r & 31u) + 32u * ((c >> 2) & 1u)) * 16u + (c & 3u) * 4u) = code;
        if ((c & 15u) == 0)
            *reinterpret_cast<uint32_t *>(scales + ((uint64_t)(c >> 4) * (uint64_t)a.rows_out + r) * 4u) = word;
    } else {
        *reinterpret_cast<uint32_t *>(codes + r * (cols >> 1) + c * 4u) = code;
        uint8_t *to = scales + r * (cols >> 5) + (c >> 2);
        if (cols % 128u == 0) {
            if ((c & 15u) == 0) *reinterpret_cast<u32_a1 *>(to) = word;
        } else if ((c & 3u) == 0) {
            *to = (uint8_t)sbyte;
        }
    }
}

// Chunk c of row `row` of y's 8-bit rows.
template <typename T>
__device__ __forceinline__ void store_pack8(const NormArgs &a, int64_t row, uint32_t c, uint32_t cols, const Chunk<T> &y)
{
    const Packed8 p = pack8(y);
    const uint64_t cpr = cols >> 3, at = (uint64_t)row * cpr + c;
    const bool in = c < cpr;
    store_scales8(reinterpret_cast<uint8_t *>(a.scales8) + (at >> 2), p.scale, c & 15u, (c | 15u) < cpr, in);
    if (in) *reinterpret_cast<u32x2v *>(reinterpret_cast<uint8_t *>(a.codes8) + at * 8u) = p.q;
}

// What a norm leaves of y beside its rows: nothing, the MXFP4 operand, or its
// 8-bit rows and, if asked for, the operand too.
enum Made { kRowsOnly, kMxOperand, kPack8Rows };

// kC chunks of eight elements per thread.  kLanes > 0: that many lanes of a
// wave have a row to themselves (256 / kLanes rows to a workgroup, no
// barriers); 0: a workgroup of as many waves as the row needs has it.
template <typename T, int kLanes, int kC, bool kRes, Edge kEdge, Made kMade>
__global__ __launch_bounds__(kLanes ? 256 : 1024) void norm_kernel(const NormArgs a, const Dropout d,
                                                                  const void *__restrict__ gamma,
                                                                  const void *__restrict__ beta)
{
    __shared__ float red[2][16];
    constexpr bool kEarlyW = kC == 1;
    constexpr bool kMx = kMade == kMxOperand || (kMade == kPack8Rows && sizeof(T) == 2);
    const bool mx = kMade == kMxOperand || (kMx && a.codes);
    constexpr bool kGroup = kLanes == 0;
    constexpr int kRows = kGroup ? 1 : 256 / kLanes;  // of a workgroup
    const uint32_t tpr = kGroup ? blockDim.x : kLanes, t = kGroup ? threadIdx.x : threadIdx.x % tpr;
    const uint32_t cols = (uint32_t)a.cols, waves = blockDim.x >> 6;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));  // rows in scalar registers
    const auto sum_of = [&](float v, float *slot) {
        if constexpr (kGroup)
            return row_sum(v, slot, wave, waves);
        else
            return lanes_sum<kLanes>(v);
    };
    const float inv_n = 1.0f / (float)cols;
    // whether each lane of the wave has a full chunk of its own in place i
    const auto whole = [&](int i) { return (i * tpr + (kGroup ? wave * 64u + 64u : tpr)) * 8u <= cols; };
    // no loop over rows: what a loop would keep ready for its next turn
    // (Philox's keys among it) spills
    int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (mx && a.tiled) {
        // 32 rows share the tiled operand's cache lines, 16 bytes each:
        // workgroup b runs on XCD b mod 8, and of 256 rows each XCD gets 32
        // together, so that its L2 puts the lines together
        constexpr int64_t kRun = 32 / kRows;
        block = block / (8 * kRun) * (8 * kRun) + block % 8 * kRun + block / 8 % kRun;
    }
    const int64_t row = block * kRows + (kGroup ? 0u : kLanes == 64 ? wave : threadIdx.x / tpr);
    if (row >= a.rows_out) return;
    if (mx && row >= a.rows) {  // tiled output's padding rows: zero codes and scales
        Chunk<bf16_t> z;
        z.q = (u32x4v){0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < kC; ++i) store_mx(a, row, i * tpr + t, cols, z);
        return;
    }
    Span sp[kC];
    Chunk<T> q[kC], s[kRes ? kC : 1];
    const T *px = reinterpret_cast<const T *>(a.x) + row * a.ld_x;
    const T *res = reinterpret_cast<const T *>(a.residual) + row * a.ld_r;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
        sp[i] = span_of<kEdge>(i * tpr + t, cols);
        load_chunk<T, kEdge, kStream<T>>(px, sp[i], cols, q[i]);
        if (kRes) load_chunk<T, kEdge, kStream<T>>(res, sp[i], cols, s[i]);
    }
    // behind the row, so that they have come when its sums are done
    Weights wg, wb;
    if (kEarlyW) {
        if (gamma) load_weights<kEdge>(gamma, a.w_bf16, sp[0], cols, wg);
        if (beta) load_weights<kEdge>(beta, a.w_bf16, sp[0], cols, wb);
    }
    if (kRes || d.drop || a.h) {
        // the random words are made while the row is on its way
        __builtin_amdgcn_sched_barrier(0);
        Draws x[kC];
        if (d.drop) {
#pragma unroll
            for (int i = 0; i < kC; ++i) x[i] = draws_of<kEdge>(d, (uint32_t)row, i * tpr + t, sp[i]);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kC; ++i) {
            float v[8];
            q[i].get(v);
            if (d.drop) apply_dropout(d, x[i], v);
            if (kRes) {
                float r[8];
                s[i].get(r);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = r[j] + v[j];
            }
            q[i].set(v);
            if (a.h) store_chunk<T, kEdge, kStream<T>>(reinterpret_cast<T *>(a.h) + row * a.ld_h, sp[i], q[i]);
        }
    }
    float mean = 0.0f;
    if (a.layer) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kC; ++i) {
            float v[8];
            q[i].get(v);
            if (kEdge != kWhole && !whole(i)) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = sp[i].own(j) ? v[j] : 0.0f;
            }
            const float e = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
            sum += kEdge != kWhole || sp[i].any() ? e : 0.0f;
        }
        mean = sum_of(sum, red[0]) * inv_n;
    }
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
        float v[8], e = 0.0f;
        q[i].get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] -= mean;
        if (kEdge != kWhole && !whole(i)) {  // after the mean is taken off: it may be infinite
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = sp[i].own(j) ? v[j] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) e = __builtin_fmaf(v[j], v[j], e);
        sq += kEdge != kWhole || sp[i].any() ? e : 0.0f;
    }
    const float rstd = 1.0f / __builtin_sqrtf(sum_of(sq, red[1]) * inv_n + a.eps);
    if (t == 0) {
        if (a.layer && a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < kC; ++i) {
        float v[8], w[8], b[8];
        q[i].get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 1.0f, b[j] = 0.0f;
        if (kEarlyW) {
            if (gamma) wg.get(a.w_bf16, w);
            if (beta) wb.get(a.w_bf16, b);
        } else {
            if (gamma) weights_now<kEdge>(gamma, a.w_bf16, sp[i], cols, w);
            if (beta) weights_now<kEdge>(beta, a.w_bf16, sp[i], cols, b);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __builtin_fmaf((v[j] - mean) * rstd, w[j], b[j]);
        q[i].set(v);
        // y is left to the caches for the GEMM's producer that reads it next
        // (norm and producer 8192 x 4096: 56.9 us; with y streamed past them
        // 59.6); h is read a sub-block later
        if (a.y) store_chunk<T, kEdge>(reinterpret_cast<T *>(a.y) + row * a.ld_y, sp[i], q[i]);
        if constexpr (kMx) {
            if (mx) store_mx(a, row, i * tpr + t, cols, q[i]);
        }
        if constexpr (kMade == kPack8Rows) store_pack8(a, row, i * tpr + t, cols, q[i]);
    }
}

template <typename T, int kLanes, int kC, Made kMade>
void run_norm(const NormArgs &a, const Dropout &d, hipStream_t st)
{
    const int64_t chunks = (a.cols + 7) / 8, rows = a.codes && a.tiled ? (a.rows_out + 255) / 256 * 256 : a.rows_out;
    constexpr int kRows = kLanes ? 256 / kLanes : 1;
    const int64_t need = (rows + kRows - 1) / kRows;
    const int64_t wide = 1 << 20;  // a launch's threads along x are below 2^32
    const dim3 grid((unsigned)(need < wide ? need : wide), (unsigned)((need + wide - 1) / wide));
    const dim3 block(kLanes ? 256 : (unsigned)((chunks + 64 * kC - 1) / (64 * kC) * 64));
#define FP4Q_NORM(EDGE)                                                                                           \
    do {                                                                                                          \
        if (a.residual)                                                                                           \
            hipLaunchKernelGGL((norm_kernel<T, kLanes, kC, true, EDGE, kMade>), grid, block, 0, st, a, d, a.gamma, a.beta);  \
        else                                                                                                      \
            hipLaunchKernelGGL((norm_kernel<T, kLanes, kC, false, EDGE, kMade>), grid, block, 0, st, a, d, a.gamma, a.beta); \
    } while (0)
    const Edge edge = edge_of(a.cols);  // an operand's is kWhole, and only short rows are tiny
    if constexpr (kLanes == 16 && kMade == kRowsOnly) {
        if (edge == kTiny) FP4Q_NORM(kTiny);
    }
    if constexpr (kMade == kRowsOnly) {
        if (edge == kRagged) FP4Q_NORM(kRagged);
    }
    if (edge == kWhole) FP4Q_NORM(kWhole);
#undef FP4Q_NORM
}

template <typename T, Made kMade>
void pick_norm(const NormArgs &a, const Dropout &d, hipStream_t st)
{
    if (a.cols <= 128)
        run_norm<T, 16, 1, kMade>(a, d, st);
    else if (a.cols <= 256)
        run_norm<T, 32, 1, kMade>(a, d, st);
    else if (a.cols <= 512)
        run_norm<T, 64, 1, kMade>(a, d, st);
    else if (a.cols <= 1024)
        run_norm<T, 64, 2, kMade>(a, d, st);
    else if (a.cols <= 4096)
        run_norm<T, 0, 1, kMade>(a, d, st);
    else if (a.cols <= 16384)
        run_norm<T, 0, 2, kMade>(a, d, st);
    else
        run_norm<T, 0, 4, kMade>(a, d, st);
}

}  // namespace

int launch_norm(const NormArgs &a, hipStream_t st)
{
    const Dropout d = dropout_of(a.p, a.seed, a.stream_id);
    if (a.codes8 && a.bf16)
        pick_norm<bf16_t, kPack8Rows>(a, d, st);
    else if (a.codes8)
        pick_norm<float, kPack8Rows>(a, d, st);
    else if (a.codes)
        pick_norm<bf16_t, kMxOperand>(a, d, st);
    else if (a.bf16)
        pick_norm<bf16_t, kRowsOnly>(a, d, st);
    else
        pick_norm<float, kRowsOnly>(a, d, st);
    return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace fp4q
