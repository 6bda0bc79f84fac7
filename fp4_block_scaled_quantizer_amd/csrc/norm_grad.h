// norm_grad.h -- the gradient of layer norm and RMS norm with the weights'
// reduction: kernels for rows of their own type and for 8-bit rows, each
// compiled in a source of its own.
//
// With xh = (h - mean) rstd and g = dy gamma:
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
// The normed rows in 8 bits are 33/64 of their bf16 bytes to read:
//   8192 x 4096 bf16, layer norm, dres: 46.6 us, 5.1 TB/s (binary32 rows, RMS
//   norm 59.5, 5.1); 640 x 4096 12.6 us (beside their weights' sums the rows are
//   read twice); 96 x 1024: 4.9 us a call.
// Above 8192 columns some kernels do not fit a workgroup's 128 registers and
// spill: two chunks a thread up to 46 (16384 columns bf16 with dres and dropout
// 19: 4096 rows 145 us, 4.6 TB/s), four chunks up to 16 for bf16 and 63 for
// binary32, ragged 131 (4096 x 24000 bf16 199 us, 4096 x 24001 508: there the
// rows' kernel moves more than three times its rows' bytes).
// Two chunks of 8-bit rows beside bf16 dy (two rows in flight, each with a
// scale register a chunk) spill more than bf16 rows: with sums, dres 15 against
// 7, dropout 17 / 2, both 31 / 19; walked without sums, both 17 / 1 (binary32 dy,
// with sums, dropout 18 / 12, both 10 / 4).  4096 x 16384, RMS norm, 8-bit / own
// rows, us: bf16 72 / 83, dres 103 / 104, dropout 115 / 105, both 155 / 136, so that
// with dropout the bytes saved do not pay; binary32 117 / 154, 166 / 207, 218 /
// 231, 232 / 255.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4q_internal.h"
#include "pack8.h"
#include "row_ops.h"

namespace fp4q {

namespace {

constexpr int kMaxParts = 256;  // workgroups that walk the rows (and keep weight sums): one per compute unit

// The rows that were normed, as the call has them: a matrix of its own, or
// 8-bit rows (always of whole chunks).
template <typename T, bool kPack8> using NormedChunk = typename std::conditional<kPack8, Packed8, Chunk<T>>::type;
template <typename T, Edge kEdge, bool kPack8>
__device__ __forceinline__ void load_normed(const NormGradArgs &a, int64_t row, const Span &s, uint32_t cols,
                                            NormedChunk<T, kPack8> &q)
{
    if constexpr (kPack8) {
        const uint32_t cpr = cols >> 3, c = s.from >> 3;
        q.q = load_vec<true>(reinterpret_cast<const u32x2v *>(a.h_codes + row * cols + s.from));
        q.scale = (a.h_scales + row * (cpr >> 2))[c >> 2];
    } else {
        load_chunk<T, kEdge, kStream<T>>(reinterpret_cast<const T *>(a.h) + row * a.ld_h, s, cols, q);
    }
}

// The weight sums of 64 columns over every `nslices`-th run of 128 rows, by
// a workgroup of 1024 threads: eight lanes side by side take the columns,
// the other 128 the rows.  They need the rows' statistics but not their
// sums, so this part can run beside the rows' own work.
template <typename T, Edge kEdge, bool kPack8>
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
        Chunk<T> dy;
        NormedChunk<T, kPack8> h;
        load_chunk<T, kEdge, kStream<T>>(reinterpret_cast<const T *>(a.dy) + row * a.ld_dy, sp, cols, dy);
        load_normed<T, kEdge, kPack8>(a, row, sp, cols, h);
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
template <typename T, int kC, bool kAhead, int kLanes, Sums kSums, bool kRes, bool kDx, Edge kEdge, bool kPack8>
__global__ __launch_bounds__(1024) void norm_grad_kernel(const NormGradArgs a, const Dropout d, float *dgamma,
                                                         float *dbeta)
{
    const uint32_t block = blockIdx.y * gridDim.x + blockIdx.x;
    if constexpr (kSums == kNone) {
        if (block >= a.row_blocks) {
            if (dgamma || dbeta) weight_sums<T, kEdge, kPack8>(a, block - a.row_blocks, 0, 1, dgamma, dbeta);
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
        Chunk<T> dy[kC], res[kRes ? kC : 1];
        NormedChunk<T, kPack8> h[kC];
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
            load_normed<T, kEdge, kPack8>(a, row, sp[i], cols, r.h[i]);
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
template <typename T, Edge kEdge, bool kPack8>
__global__ __launch_bounds__(1024) void norm_weight_sums_kernel(const NormGradArgs a, float *parts, float *dgamma,
                                                                float *dbeta)
{
    if (parts) {
        dgamma = parts + (size_t)blockIdx.y * 2 * (uint32_t)a.cols;
        dbeta = dgamma + (uint32_t)a.cols;
    }
    weight_sums<T, kEdge, kPack8>(a, blockIdx.x, blockIdx.y, gridDim.y, dgamma, dbeta);
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
// 365 x 8192 6.8 / 7.1 (with dres and dropout 9.4 / 8.8), 2048 x 1024 5.4 /
// 4.5, but 3000 x 1024 6.0 / 7.3 (with dres and dropout 8.6 / 9.1), 10000 x 256
// 6.0 / 5.7; two chunks a thread 400 x 9000 7.4 / 8.3, 219 x 14336 7.6 / 5.6;
// binary32 512 x 4096 7.5 / 7.1, 768 x 4096 11.0 / 11.8.  The limit lies between
// the calls' kinds: with one to two workgroups a unit, 22 widths of 8 to 16384,
// walked takes 0.80 to 1.06 of the other's time, with dres and dropout 0.88 to
// 1.21 (8-bit rows 0.79 to 1.05, and 0.88 to 1.74).
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

template <typename T, bool kPack8, int kC, Sums kSums, int kLanes = 64>
void run_norm_grad(const NormGradArgs &a, const Dropout &d, How how, float *dgamma, float *dbeta, hipStream_t st)
{
    const unsigned blocks = a.row_blocks + (how == kBeside ? (unsigned)((a.cols + 63) / 64) : 0u);
    const unsigned wide = 1u << 20;  // a launch's threads along x are below 2^32
    const dim3 grid(blocks < wide ? blocks : wide, (blocks + wide - 1) / wide);
    const dim3 block(how == kBeside ? 1024 : a.waves * a.groups * kLanes);
    const Edge edge = edge_of(a.cols);
#define FP4Q_NORM_GRAD(RES, DX, EDGE)                                                                          \
    hipLaunchKernelGGL((norm_grad_kernel<T, kC, kC == 1 || (kC == 2 && (sizeof(T) == 2 || !RES)), kLanes, kSums, RES,  \
                                         DX, EDGE, kPack8>),                                                          \
                       grid, block, 0, st, a, d, dgamma, dbeta)
#define FP4Q_NORM_GRAD_E(RES, DX)                            \
    do {                                                     \
        if (edge == kWhole) {                                \
            FP4Q_NORM_GRAD(RES, DX, kWhole);                 \
        } else if constexpr (!kPack8) {                      \
            if (edge == kRagged)                             \
                FP4Q_NORM_GRAD(RES, DX, kRagged);            \
            else if constexpr (kLanes == 16)                 \
                FP4Q_NORM_GRAD(RES, DX, kTiny);              \
        }                                                    \
    } while (0)
    if (a.dres) {
        if (a.dx) FP4Q_NORM_GRAD_E(true, true); else FP4Q_NORM_GRAD_E(true, false);
    } else {
        if (a.dx) FP4Q_NORM_GRAD_E(false, true); else FP4Q_NORM_GRAD_E(false, false);
    }
#undef FP4Q_NORM_GRAD_E
#undef FP4Q_NORM_GRAD
}

template <typename T, bool kPack8, Sums kOne, Sums kTwo>
void run_norm_grad_n(const NormGradArgs &a, const Dropout &d, const GradPlan &g, How how, float *dgamma, float *dbeta,
                     hipStream_t st)
{
    if (g.chunks_per_thread == 2)
        run_norm_grad<T, kPack8, 2, kTwo>(a, d, how, dgamma, dbeta, st);
    else if (g.lanes == 64)
        run_norm_grad<T, kPack8, 1, kOne>(a, d, how, dgamma, dbeta, st);
    else if (g.lanes == 32)
        run_norm_grad<T, kPack8, 1, kOne, 32>(a, d, how, dgamma, dbeta, st);
    else
        run_norm_grad<T, kPack8, 1, kOne, 16>(a, d, how, dgamma, dbeta, st);
}

template <typename T, bool kPack8>
void pick_norm_grad(const NormGradArgs &a, const Dropout &d, const GradPlan &g, float *dgamma, float *dbeta,
                    hipStream_t st)
{
    How how = g.sums;
    const bool overwritten = (a.dh && (a.dh == a.dy || a.dh == a.h)) || (a.dx && (a.dx == a.dy || a.dx == a.h));
    if (how == kApart || (how == kBeside && overwritten)) {
        float *parts = how == kApart ? a.parts : nullptr;
        const dim3 grid((unsigned)((a.cols + 63) / 64), how == kApart ? (unsigned)g.parts : 1u);
#define FP4Q_NORM_WEIGHT_SUMS(EDGE)                                                                               \
    hipLaunchKernelGGL((norm_weight_sums_kernel<T, EDGE, kPack8>), grid, dim3(1024), 0, st, a, parts, dgamma, dbeta)
        const Edge edge = edge_of(a.cols);
        if (edge == kWhole) {
            FP4Q_NORM_WEIGHT_SUMS(kWhole);
        } else if constexpr (!kPack8) {
            if (edge == kRagged)
                FP4Q_NORM_WEIGHT_SUMS(kRagged);
            else
                FP4Q_NORM_WEIGHT_SUMS(kTiny);
        }
#undef FP4Q_NORM_WEIGHT_SUMS
        how = kNoSums;
    }
    if (how == kNoSums) dgamma = dbeta = nullptr;  // not the rows' kernel's
    if (g.chunks_per_thread == 4)
        run_norm_grad<T, kPack8, 4, kNone>(a, d, how, dgamma, dbeta, st);
    else if (how == kNoSums || how == kBeside)
        run_norm_grad_n<T, kPack8, kNone, kNone>(a, d, g, how, dgamma, dbeta, st);
    else if (how == kRowsWalked)
        run_norm_grad_n<T, kPack8, kWalk, kWalk>(a, d, g, how, dgamma, dbeta, st);
    else
        run_norm_grad_n<T, kPack8, kInRegs, kInLds>(a, d, g, how, dgamma, dbeta, st);
}

// The rows' part of a call, in kernels for h as it is given.
template <bool kPack8>
int norm_grad_rows(NormGradArgs a, float *dgamma, float *dbeta, hipStream_t st)
{
    const GradPlan g = grad_plan(a.rows, a.cols, a.bf16, dgamma || dbeta);
    const Dropout d = dropout_of(a.p, a.seed, a.stream_id);
    a.waves = g.waves;
    a.groups = g.groups;
    a.row_blocks = (uint32_t)g.row_blocks;
    if (a.bf16)
        pick_norm_grad<bf16_t, kPack8>(a, d, g, dgamma, dbeta, st);
    else
        pick_norm_grad<float, kPack8>(a, d, g, dgamma, dbeta, st);
    return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace

}  // namespace fp4q
