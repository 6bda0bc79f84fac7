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
//   1 x 4096 bf16: 4.8 us a call, launch and latency.
//
// Gradient, with xh = (h - mean) rstd and g = dy gamma:
//   dh = [dres +] rstd (g - sum g / n - xh sum(g xh) / n) (RMS: no second
//   term), dx = dropout(dh); dgamma = sum over rows of dy xh, dbeta = of dy.
// A workgroup per compute unit walks rows and keeps its columns' weight sums
// in registers (above 8192 columns in LDS); the workgroups' sums go to the
// workspace and a second kernel adds them in a fixed order (no atomics: two
// runs give the same bits).  More workgroups would hide more latency but
// leave more sums to write and read: 512 took 69 us where 256 take 63.
//   8192 x 4096 bf16, layer norm, dropout, dres: 64.6 us, 5.2 TB/s (62.6 the
//   rows' kernel, 4.9 the second); 2047 x 14336 binary32: 77.2 us, 4.6 TB/s
//   (eight rows to a compute unit, of which the first one's loads and the
//   sums' 59 MB are not hidden); 327680 x 128 bf16, dres: 63.7 us, 5.3 TB/s (a
//   wave per row 94); 96 x 1024: 4.8 us a call.
// Above 8192 columns some kernels do not fit a workgroup's 128 registers and
// spill: two chunks a thread up to 46 (16384 columns bf16 with dres and dropout
// 19: 4096 rows 145 us, 4.6 TB/s), four chunks up to 16 for bf16 and 63 for
// binary32, ragged 131 (4096 x 24000 bf16 199 us, 4096 x 24001 508: there the
// rows' kernel moves more than three times its rows' bytes).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4q_internal.h"
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

// ... and loaded where they are used, which takes fewer registers.
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

// kC chunks of eight elements per thread.  kLanes > 0: that many lanes of a
// wave have a row to themselves (256 / kLanes rows to a workgroup, no
// barriers); 0: a workgroup of as many waves as the row needs has it.
template <typename T, int kLanes, int kC, bool kRes, Edge kEdge, bool kMx>
__global__ __launch_bounds__(kLanes ? 256 : 1024) void norm_kernel(const NormArgs a, const Dropout d,
                                                                  const void *__restrict__ gamma,
                                                                  const void *__restrict__ beta)
{
    __shared__ float red[2][16];
    constexpr bool kEarlyW = kC == 1;
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
    if (kMx && a.tiled) {
        // 32 rows share the tiled operand's cache lines, 16 bytes each:
        // workgroup b runs on XCD b mod 8, and of 256 rows each XCD gets 32
        // together, so that its L2 puts the lines together
        constexpr int64_t kRun = 32 / kRows;
        block = block / (8 * kRun) * (8 * kRun) + block % 8 * kRun + block / 8 % kRun;
    }
    const int64_t row = block * kRows + (kGroup ? 0u : kLanes == 64 ? wave : threadIdx.x / tpr);
    if (row >= a.rows_out) return;
    if (kMx && row >= a.rows) {  // tiled output's padding rows: zero codes and scales
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
        if constexpr (kMx) store_mx(a, row, i * tpr + t, cols, q[i]);
    }
}

template <typename T, int kLanes, int kC, bool kMx>
void run_norm(const NormArgs &a, const Dropout &d, hipStream_t st)
{
    const int64_t chunks = (a.cols + 7) / 8, rows = kMx && a.tiled ? (a.rows_out + 255) / 256 * 256 : a.rows_out;
    constexpr int kRows = kLanes ? 256 / kLanes : 1;
    const int64_t need = (rows + kRows - 1) / kRows;
    const int64_t wide = 1 << 20;  // a launch's threads along x are below 2^32
    const dim3 grid((unsigned)(need < wide ? need : wide), (unsigned)((need + wide - 1) / wide));
    const dim3 block(kLanes ? 256 : (unsigned)((chunks + 64 * kC - 1) / (64 * kC) * 64));
#define FP4Q_NORM(EDGE)                                                                                           \
    do {                                                                                                          \
        if (a.residual)                                                                                           \
            hipLaunchKernelGGL((norm_kernel<T, kLanes, kC, true, EDGE, kMx>), grid, block, 0, st, a, d, a.gamma, a.beta);  \
        else                                                                                                      \
            hipLaunchKernelGGL((norm_kernel<T, kLanes, kC, false, EDGE, kMx>), grid, block, 0, st, a, d, a.gamma, a.beta); \
    } while (0)
    const Edge edge = edge_of(a.cols);  // an operand's is kWhole, and only short rows are tiny
    if constexpr (kLanes == 16 && !kMx) {
        if (edge == kTiny) FP4Q_NORM(kTiny);
    }
    if constexpr (!kMx) {
        if (edge == kRagged) FP4Q_NORM(kRagged);
    }
    if (edge == kWhole) FP4Q_NORM(kWhole);
#undef FP4Q_NORM
}

template <typename T, bool kMx>
void pick_norm(const NormArgs &a, const Dropout &d, hipStream_t st)
{
    if (a.cols <= 128)
        run_norm<T, 16, 1, kMx>(a, d, st);
    else if (a.cols <= 256)
        run_norm<T, 32, 1, kMx>(a, d, st);
    else if (a.cols <= 512)
        run_norm<T, 64, 1, kMx>(a, d, st);
    else if (a.cols <= 1024)
        run_norm<T, 64, 2, kMx>(a, d, st);
    else if (a.cols <= 4096)
        run_norm<T, 0, 1, kMx>(a, d, st);
    else if (a.cols <= 16384)
        run_norm<T, 0, 2, kMx>(a, d, st);
    else
        run_norm<T, 0, 4, kMx>(a, d, st);
}

// ------------------------------------------------------------------ gradient

constexpr int kMaxParts = 256;  // workgroups that walk the rows (and keep weight sums): one per compute unit

// The weight sums of 64 columns over every `nslices`-th run of 128 rows, by
// a workgroup of 1024 threads: eight lanes side by side take the columns,
// the other 128 the rows.  They need the rows' statistics but not their
// sums, so this part can run beside the rows' own work.
template <typename T, Edge kEdge>
__device__ __forceinline__ void weight_sums(const NormGradArgs &a, uint32_t block, uint32_t slice, uint32_t nslices,
                                            float *dgamma, float *dbeta)
{
    __shared__ float s[2][16][64];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6, cols = (uint32_t)a.cols;
    const Span sp = span_of<kEdge>(block * 8u + (lane & 7u), cols);
    float sum_w[8], sum_b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sum_w[j] = 0.0f, sum_b[j] = 0.0f;
#pragma unroll(kEdge == kTiny ? 1 : 4)
    for (int64_t row = (int64_t)slice * 128 + (threadIdx.x >> 3); row < a.rows; row += (int64_t)nslices * 128) {
        Chunk<T> dy, h;
        load_chunk<T, kEdge, kStream<T>>(reinterpret_cast<const T *>(a.dy) + row * a.ld_dy, sp, cols, dy);
        load_chunk<T, kEdge, kStream<T>>(reinterpret_cast<const T *>(a.h) + row * a.ld_h, sp, cols, h);
        const float mean = a.layer ? a.mean[row] : 0.0f, rstd = a.rstd[row];
        float e[8], v[8];
        dy.get(e);
        h.get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sum_w[j] = __builtin_fmaf(e[j], (v[j] - mean) * rstd, sum_w[j]);
            sum_b[j] += e[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int m = 8; m < 64; m <<= 1) {
            sum_w[j] += __shfl_xor(sum_w[j], m);
            sum_b[j] += __shfl_xor(sum_b[j], m);
        }
    }
    if (lane < 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s[0][wave][lane * 8 + j] = sum_w[j];
            s[1][wave][lane * 8 + j] = sum_b[j];
        }
    }
    __syncthreads();
    if (threadIdx.x < 128) {
        const uint32_t which = threadIdx.x >> 6;
        float v = s[which][0][lane];
#pragma unroll
        for (int i = 1; i < 16; ++i) v += s[which][i][lane];
        // the last chunk's own columns start at its lo
        const Span o = span_of<kEdge>(block * 8u + (lane >> 3), cols);
        float *out = which ? dbeta : dgamma;
        if (out && o.own(lane & 7u)) out[o.from + (lane & 7u)] = v;
    }
}

// A workgroup takes a.groups rows at a time, a.waves waves each (kLanes < 64:
// one wave takes 64 / kLanes rows), and loads the next ones before it works
// on those it has (kAhead).  Weight sums:
// kInRegs and kInLds, each workgroup keeps those of its rows and leaves them
// in the workspace; kNone, where they are asked for, the workgroups from
// a.row_blocks on take them from all rows (weight_sums), 64 columns each, and
// a workgroup ends with its first rows; kWalk has no sums and walks the rows
// like kInRegs.
enum Sums { kNone, kWalk, kInRegs, kInLds };
template <typename T, int kC, bool kAhead, int kLanes, Sums kSums, bool kRes, bool kDx, Edge kEdge>
__global__ __launch_bounds__(1024) void norm_grad_kernel(const NormGradArgs a, const Dropout d, float *dgamma,
                                                         float *dbeta)
{
    const uint32_t block = blockIdx.y * gridDim.x + blockIdx.x;
    if constexpr (kSums == kNone) {
        if (block >= a.row_blocks) {
            if (dgamma || dbeta) weight_sums<T, kEdge>(a, block - a.row_blocks, 0, 1, dgamma, dbeta);
            return;
        }
    }
    __shared__ float red[2][2][16];
    // the sums in LDS, or folded there over the groups at the end; a
    // thread's eight of a chunk are two groups of four, each wave-contiguous
    __shared__ __attribute__((aligned(16))) float keep[kSums <= kWalk ? 1 : (kSums == kInLds ? 2 : 1) * kC * 8 * 1024];
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));  // rows in scalar registers
    const uint32_t lane = threadIdx.x & 63u, cols = (uint32_t)a.cols;
    constexpr bool kShort = kLanes < 64;
    const auto same_in_wave = [](uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); };
    const uint32_t g = kShort ? threadIdx.x / kLanes : same_in_wave(wave / a.waves), first = g * a.waves;
    const uint32_t tpr = kShort ? kLanes : a.waves * 64u, t = kShort ? threadIdx.x % kLanes : threadIdx.x - first * 64u;
    const float inv_n = 1.0f / (float)cols;
    // wide rows read the weights again for each row rather than hold them
    constexpr bool kHoldW = kC <= 2;
    constexpr int kRegs = kSums == kInRegs ? kC : 1;
    float w[kHoldW ? kC : 1][8], sum_w[kRegs][8], sum_b[kRegs][8];
    Span sp[kC];
    const auto weight = [&](int i, float v[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 1.0f;
        if (a.gamma) weights_now<kEdge>(a.gamma, a.w_bf16, sp[i], cols, v);
    };
    const auto kept = [&](int which, int i, int half) {
        return reinterpret_cast<float4 *>(keep) + ((which * kC + i) * 2 + half) * 1024 + threadIdx.x;
    };
#pragma unroll
    for (int i = 0; i < kC; ++i) {
        // (a wave past the last group: one past the row's end, a load of one line)
        sp[i] = span_of<kEdge>(kSums == kNone && g >= a.groups ? cols : i * tpr + t, cols);
        if (kSums == kInRegs) {
#pragma unroll
            for (int j = 0; j < 8; ++j) sum_w[kRegs > i ? i : 0][j] = 0.0f, sum_b[kRegs > i ? i : 0][j] = 0.0f;
        }
        if (kSums == kInLds) {
#pragma unroll
            for (int k = 0; k < 4; ++k) *kept(k >> 1, i, k & 1) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        if (kHoldW) weight(i, w[i]);
    }
    struct Row {
        Chunk<T> dy[kC], h[kC], res[kRes ? kC : 1];
        float mean, rstd;
    };
    const uint32_t rows = (uint32_t)a.rows;
    const float *means = a.layer ? a.mean : a.rstd;
    const auto fetch = [&](uint32_t base, Row &r) {  // past the end: the last row again
        const uint32_t at = min(base + g, rows - 1u);
        const int64_t row = kShort ? at : same_in_wave(at);
#pragma unroll
        for (int i = 0; i < kC; ++i) {
            load_chunk<T, kEdge, kStream<T>>(reinterpret_cast<const T *>(a.dy) + row * a.ld_dy, sp[i], cols, r.dy[i]);
            load_chunk<T, kEdge, kStream<T>>(reinterpret_cast<const T *>(a.h) + row * a.ld_h, sp[i], cols, r.h[i]);
            if (kRes)
                load_chunk<T, kEdge, kStream<T>>(reinterpret_cast<const T *>(a.dres) + row * a.ld_dres, sp[i], cols,
                                                 r.res[i]);
        }
        r.mean = means[row];
        r.rstd = a.rstd[row];
    };
    // rows < 2^31 and three strides (where there is a loop) < 2^16: below 2^32
    const uint32_t stride = a.row_blocks * a.groups, base0 = block * a.groups;
    // whether each lane of the wave has a full chunk of its own in place i
    const auto whole = [&](int i) { return (i * tpr + (kShort ? kLanes : (wave - first) * 64u + 64u)) * 8u <= cols; };
    int parity = 0;
    const auto work = [&](uint32_t base, const Row &cur) {
        const int64_t row = kShort ? base + g : same_in_wave(base + g);
        // the same on every lane of a row; waves past the last group (the
        // workgroups beside this one need 1024 threads) have no row
        const bool live = row < a.rows && g < a.groups;
        Draws x[kC];
        if (kDx && d.drop) {
            // the key made anew for each row: the rounds' keys, kept over the
            // loop, would spill
            Dropout k = d;
            asm volatile("" : "+s"(k.key0), "+s"(k.key1));
#pragma unroll
            for (int i = 0; i < kC; ++i) x[i] = draws_of<kEdge>(k, (uint32_t)row, i * tpr + t, sp[i]);
        }
        const float mean = a.layer ? cur.mean : 0.0f, rstd = cur.rstd;
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < kC; ++i) {
            float e[8], v[8], wi[8], p1 = 0.0f, p2 = 0.0f;
            cur.dy[i].get(e);
            cur.h[i].get(v);
            if (!kHoldW) weight(i, wi);
            if (kEdge != kWhole && !whole(i)) {
#pragma unroll
                for (int j = 0; j < 8; ++j) e[j] = sp[i].own(j) ? e[j] : 0.0f, v[j] = sp[i].own(j) ? v[j] : mean;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = (v[j] - mean) * rstd;
                const float gj = e[j] * (kHoldW ? w[kHoldW ? i : 0][j] : wi[j]);
                p1 = __builtin_fmaf(gj, v[j], p1);
                p2 += gj;
                if (kSums == kInRegs && live) {
                    sum_w[kRegs > i ? i : 0][j] = __builtin_fmaf(e[j], v[j], sum_w[kRegs > i ? i : 0][j]);
                    sum_b[kRegs > i ? i : 0][j] += e[j];
                }
            }
            if (kSums == kInLds && live) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float *pe = e + 4 * half, *pv = v + 4 * half;
                    float4 m = *kept(0, i, half);
                    m.x = __builtin_fmaf(pe[0], pv[0], m.x);
                    m.y = __builtin_fmaf(pe[1], pv[1], m.y);
                    m.z = __builtin_fmaf(pe[2], pv[2], m.z);
                    m.w = __builtin_fmaf(pe[3], pv[3], m.w);
                    *kept(0, i, half) = m;
                    m = *kept(1, i, half);
                    m.x += pe[0], m.y += pe[1], m.z += pe[2], m.w += pe[3];
                    *kept(1, i, half) = m;
                }
            }
            s1 += kEdge != kWhole || sp[i].any() ? p1 : 0.0f;
            s2 += kEdge != kWhole || sp[i].any() ? p2 : 0.0f;
        }
        // both sums with one barrier, lanes 0-15 the one and 16-31 the other;
        // the two parities keep a row's slots apart from the next row's
        s1 = lanes_sum<kLanes>(s1);
        s2 = lanes_sum<kLanes>(s2);
        if (!kShort && a.waves > 1) {
            if (lane == 0) red[parity][0][wave] = s1, red[parity][1][wave] = s2;
            __syncthreads();
            const uint32_t k = lane & 15u;
            const float v = sum16(k < a.waves && g < a.groups ? red[parity][(lane >> 4) & 1u][first + k] : 0.0f);
            s1 = lane_value(v, 15);
            s2 = lane_value(v, 31);
        }
        const float c1 = s1 * inv_n, c2 = a.layer ? s2 * inv_n : 0.0f;
        if (live) {
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                float e[8], v[8], wi[8];
                cur.dy[i].get(e);
                cur.h[i].get(v);
                if (!kHoldW) weight(i, wi);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float xh = (v[j] - mean) * rstd, gj = kHoldW ? w[kHoldW ? i : 0][j] : wi[j];
                    v[j] = __builtin_fmaf(-xh, c1, __builtin_fmaf(e[j], gj, -c2)) * rstd;
                }
                if (kRes) {
                    float r[8];
                    cur.res[i].get(r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = r[j] + v[j];
                }
                Chunk<T> out;
                if (a.dh) {
                    out.set(v);
                    store_chunk<T, kEdge, kStream<T>>(reinterpret_cast<T *>(a.dh) + row * a.ld_dh, sp[i], out);
                }
                if (kDx) {
                    if (d.drop) apply_dropout(d, x[i], v);
                    out.set(v);
                    store_chunk<T, kEdge, kStream<T>>(reinterpret_cast<T *>(a.dx) + row * a.ld_dx, sp[i], out);
                }
            }
        }
        parity ^= 1;
    };
    // two rows in registers: the one after the next is asked for as soon as
    // a row is done, before the next one has to be there
    Row one, two;
    fetch(base0, one);
    if constexpr (kSums == kNone) {
        work(base0, one);
        return;
    }
    if (kAhead) fetch(base0 + stride, two);
    for (uint32_t base = base0; base < rows; base += kAhead ? 2 * stride : stride) {
        work(base, one);
        if (kAhead) {
            fetch(base + 2 * stride, one);
            if (base + stride >= rows) break;
            work(base + stride, two);
            fetch(base + 3 * stride, two);
        } else {
            fetch(base + stride, one);
        }
    }
    if constexpr (kSums > kWalk) {  // parts[workgroup][gamma, beta][cols]
        if constexpr (kShort) {  // the sums of a wave's rows
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int k = kLanes; k < 64; k *= 2) {
                    sum_w[0][j] += __shfl_xor(sum_w[0][j], k);
                    sum_b[0][j] += __shfl_xor(sum_b[0][j], k);
                }
            }
        }
        const uint32_t folds = kShort ? 16u : a.groups, apart = kShort ? 64u : tpr;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            if (which == 1 && !dbeta) break;
            if (kSums == kInRegs && folds > 1) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kC; ++i) {
                    const float *v = which ? sum_b[kRegs > i ? i : 0] : sum_w[kRegs > i ? i : 0];
#pragma unroll
                    for (int half = 0; half < 2; ++half)
                        *kept(0, i, half) = make_float4(v[4 * half], v[4 * half + 1], v[4 * half + 2], v[4 * half + 3]);
                }
            }
            if (folds > 1) __syncthreads();
            if (g == 0) {  // the first group's threads add the others' sums
                float *part = a.parts + ((size_t)block * 2 + which) * cols;
#pragma unroll
                for (int i = 0; i < kC; ++i) {
                    float v[8];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float4 m;
                        if (kSums == kInLds) {
                            m = *kept(which, i, half);
                        } else {
                            const float *r = (which ? sum_b[kRegs > i ? i : 0] : sum_w[kRegs > i ? i : 0]) + 4 * half;
                            m = make_float4(r[0], r[1], r[2], r[3]);
                        }
                        for (uint32_t k = 1; k < folds; ++k) {
                            const float4 o = kept(kSums == kInLds ? which : 0, i, half)[k * apart];
                            m.x += o.x, m.y += o.y, m.z += o.z, m.w += o.w;
                        }
                        v[4 * half] = m.x, v[4 * half + 1] = m.y, v[4 * half + 2] = m.z, v[4 * half + 3] = m.w;
                    }
                    Chunk<float> out;
                    out.set(v);
                    store_chunk<float, kEdge>(part, sp[i], out);
                }
            }
        }
    }
}

// The weight sums by themselves: into the workspace in gridDim.y slices, or
// as one slice into their place (parts null).
template <typename T, Edge kEdge>
__global__ __launch_bounds__(1024) void norm_weight_sums_kernel(const NormGradArgs a, float *parts, float *dgamma,
                                                                float *dbeta)
{
    if (parts) {
        dgamma = parts + (size_t)blockIdx.y * 2 * (uint32_t)a.cols;
        dbeta = dgamma + (uint32_t)a.cols;
    }
    weight_sums<T, kEdge>(a, blockIdx.x, blockIdx.y, gridDim.y, dgamma, dbeta);
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

// How a call is run.  Weight sums are made
//   in the rows' own kernel (kInRows), each workgroup leaving its own;
//   beside it (kBeside) in workgroups of their own, which read the rows again:
//     few rows, where the workgroups' sums are as many as the rows and a
//     second launch costs more than the reading.  The row counts are about
//     where the two meet, beside / in rows: bf16 96 x 1024 4.8 / 8.2 us, 768 x
//     4096 12.7 / 13.5, 768 x 8192 19.0 / 20.3, 400 x 5000 (10 of 16 waves)
//     11.0 / 14.2, 512 x 5000 14.0 / 15.0, but 1000 x 1000 13.2 / 11.0; two
//     chunks a thread 256 x 16384 12.0 / 25.0, 640 x 12000 22.5 / 25.6;
//     binary32 in 16 waves 640 x 8192 22.8 / 22.6, 768 x 8192 27.3 / 23.9;
//   by a kernel of their own before the rows' (kApart): rows too wide for a
//     workgroup to keep their sums (beside / apart 1024 x 20000 66 / 78, 2048
//     x 20000 123 / 122, 4096 x 16392 226 / 206), and in place of kBeside
//     where the rows' results overwrite what it reads.
// Without them a workgroup per compute unit walks the rows as for kInRows
// (kRowsWalked), whose loads then never pause; up to 3 * 2^20 elements, where
// there is little to walk, each workgroup has its first rows only (kNoSums).
// Walked / not, us, bf16: 8192 x 4096 36.2 / 50.7, 2048 x 4096 11.8 / 14.7,
// 365 x 8192 6.8 / 7.1 (with dres and dropout 9.4 / 8.8), 2048 x 1024 5.5 /
// 4.7, but 3072 x 1024 6.1 / 7.2, 10000 x 256 6.2 / 5.9; two chunks a thread
// 400 x 9000 7.4 / 8.3, 219 x 14336 7.6 / 5.9; binary32 512 x 4096 8.0 / 7.7,
// 768 x 4096 10.9 / 11.7.
enum How { kNoSums, kRowsWalked, kInRows, kBeside, kApart };
struct GradPlan {
    How sums;
    int chunks_per_thread;
    int lanes;
    uint32_t waves, groups;
    int64_t row_blocks, parts;
};
GradPlan grad_plan(int64_t rows, int64_t cols, bool bf16, bool sums)
{
    const int64_t waves1 = (cols + 511) / 512;  // waves of a row at one chunk per thread
    GradPlan g{};
    // 16 waves fit a workgroup
    g.chunks_per_thread = waves1 > 32 ? 4 : waves1 > 16 ? 2 : 1;
    g.waves = (uint32_t)((waves1 + g.chunks_per_thread - 1) / g.chunks_per_thread);
    g.lanes = lanes_of(cols);
    g.groups = 16 / g.waves * (64 / g.lanes);
    const int64_t need = (rows + g.groups - 1) / g.groups;
    const int64_t few = g.chunks_per_thread == 4                                ? 1024
                        : g.chunks_per_thread == 2 || (g.waves == 16 && !bf16) ? 640
                        : 16 % g.waves == 0                                     ? 768
                                                                                : 400;
    if (sums)
        g.sums = rows <= few ? kBeside : g.chunks_per_thread == 4 ? kApart : kInRows;
    else
        g.sums = g.chunks_per_thread == 4 || rows * cols <= (3 << 20) ? kNoSums : kRowsWalked;
    g.row_blocks = (g.sums == kInRows || g.sums == kRowsWalked) && need > kMaxParts ? kMaxParts : need;
    const int64_t runs = (rows + 127) / 128;
    g.parts = g.sums == kInRows ? g.row_blocks : g.sums == kApart ? (runs < 4 ? runs : 4) : 0;
    return g;
}

template <typename T, int kC, Sums kSums, int kLanes = 64>
void run_norm_grad(const NormGradArgs &a, const Dropout &d, How how, float *dgamma, float *dbeta, hipStream_t st)
{
    const unsigned blocks = a.row_blocks + (how == kBeside ? (unsigned)((a.cols + 63) / 64) : 0u);
    const unsigned wide = 1u << 20;  // a launch's threads along x are below 2^32
    const dim3 grid(blocks < wide ? blocks : wide, (blocks + wide - 1) / wide);
    const dim3 block(how == kBeside ? 1024 : a.waves * a.groups * kLanes);
    const Edge edge = edge_of(a.cols);
#define FP4Q_NORM_GRAD(RES, DX, EDGE)                                                                          \
    hipLaunchKernelGGL((norm_grad_kernel<T, kC, kC == 1 || (kC == 2 && (sizeof(T) == 2 || !RES)), kLanes, kSums, RES,  \
                                         DX, EDGE>),                                                                  \
                       grid, block, 0, st, a, d, dgamma, dbeta)
#define FP4Q_NORM_GRAD_E(RES, DX)                            \
    do {                                                     \
        if (edge == kWhole)                                  \
            FP4Q_NORM_GRAD(RES, DX, kWhole);                 \
        else if (edge == kRagged)                            \
            FP4Q_NORM_GRAD(RES, DX, kRagged);                \
        else if constexpr (kLanes == 16)                     \
            FP4Q_NORM_GRAD(RES, DX, kTiny);                  \
    } while (0)
    if (a.dres) {
        if (a.dx) FP4Q_NORM_GRAD_E(true, true); else FP4Q_NORM_GRAD_E(true, false);
    } else {
        if (a.dx) FP4Q_NORM_GRAD_E(false, true); else FP4Q_NORM_GRAD_E(false, false);
    }
#undef FP4Q_NORM_GRAD_E
#undef FP4Q_NORM_GRAD
}

template <typename T, Sums kOne, Sums kTwo>
void run_norm_grad_n(const NormGradArgs &a, const Dropout &d, const GradPlan &g, How how, float *dgamma, float *dbeta,
                     hipStream_t st)
{
    if (g.chunks_per_thread == 2)
        run_norm_grad<T, 2, kTwo>(a, d, how, dgamma, dbeta, st);
    else if (g.lanes == 64)
        run_norm_grad<T, 1, kOne>(a, d, how, dgamma, dbeta, st);
    else if (g.lanes == 32)
        run_norm_grad<T, 1, kOne, 32>(a, d, how, dgamma, dbeta, st);
    else
        run_norm_grad<T, 1, kOne, 16>(a, d, how, dgamma, dbeta, st);
}

template <typename T>
void pick_norm_grad(const NormGradArgs &a, const Dropout &d, const GradPlan &g, float *dgamma, float *dbeta,
                    hipStream_t st)
{
    How how = g.sums;
    const bool overwritten = (a.dh && (a.dh == a.dy || a.dh == a.h)) || (a.dx && (a.dx == a.dy || a.dx == a.h));
    if (how == kApart || (how == kBeside && overwritten)) {
        float *parts = how == kApart ? a.parts : nullptr;
        const dim3 grid((unsigned)((a.cols + 63) / 64), how == kApart ? (unsigned)g.parts : 1u);
        switch (edge_of(a.cols)) {
        case kWhole:
            hipLaunchKernelGGL((norm_weight_sums_kernel<T, kWhole>), grid, dim3(1024), 0, st, a, parts, dgamma, dbeta);
            break;
        case kRagged:
            hipLaunchKernelGGL((norm_weight_sums_kernel<T, kRagged>), grid, dim3(1024), 0, st, a, parts, dgamma, dbeta);
            break;
        case kTiny:
            hipLaunchKernelGGL((norm_weight_sums_kernel<T, kTiny>), grid, dim3(1024), 0, st, a, parts, dgamma, dbeta);
            break;
        }
        how = kNoSums;
    }
    if (how == kNoSums) dgamma = dbeta = nullptr;  // not the rows' kernel's
    if (g.chunks_per_thread == 4)
        run_norm_grad<T, 4, kNone>(a, d, how, dgamma, dbeta, st);
    else if (how == kNoSums || how == kBeside)
        run_norm_grad_n<T, kNone, kNone>(a, d, g, how, dgamma, dbeta, st);
    else if (how == kRowsWalked)
        run_norm_grad_n<T, kWalk, kWalk>(a, d, g, how, dgamma, dbeta, st);
    else
        run_norm_grad_n<T, kInRegs, kInLds>(a, d, g, how, dgamma, dbeta, st);
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

size_t norm_grad_workspace_bytes(int64_t rows, int64_t cols, bool bf16)
{
    return rows <= 0 || cols <= 0 ? 0 : (size_t)grad_plan(rows, cols, bf16, true).parts * 2u * (size_t)cols * sizeof(float);
}

int launch_norm_grad(NormGradArgs a, float *dgamma, float *dbeta, hipStream_t st)
{
    const Dropout d = dropout_of(a.p, a.seed, a.stream_id);
    const bool sums = dgamma || dbeta;
    const GradPlan g = grad_plan(a.rows, a.cols, a.bf16, sums);
    a.waves = g.waves;
    a.groups = g.groups;
    a.row_blocks = (uint32_t)g.row_blocks;
    if (a.rows > 0) {
        if (a.bf16)
            pick_norm_grad<bf16_t>(a, d, g, dgamma, dbeta, st);
        else
            pick_norm_grad<float>(a, d, g, dgamma, dbeta, st);
        if (hipGetLastError() != hipSuccess) return 1;
        if (!sums || g.sums == kBeside) return 0;
    }
    // joins the parts, or with no rows writes zeros
    hipLaunchKernelGGL(norm_grad_weights_kernel, dim3((unsigned)((a.cols + 63) / 64), dbeta ? 2 : 1), dim3(1024), 0, st,
                       a.parts, (uint32_t)(a.rows > 0 ? g.parts : 0), (uint32_t)a.cols, dgamma, dbeta);
    return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace fp4q
