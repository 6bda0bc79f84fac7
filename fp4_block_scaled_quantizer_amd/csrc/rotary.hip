// rotary.hip -- rotary position embedding of query and key heads, forward
// and (with the angle negated) backward.
//
// Pair i of a head turns by angle = position * inv_freq[i]:
//   (a, b) -> scale (a cos - b sin, b cos + a sin),
// a and b being elements i and i + rot / 2 of the head (half style) or 2 i
// and 2 i + 1 (interleaved); elements from rot on are copied.
//
// The angle is reduced to a fraction of a turn in binary64 (53 bits: at a
// position of a million a frequency of 1 is off by 2^-35 of a turn, at 2^31
// by 2^-24), so long contexts lose no precision; sine and cosine of the
// fraction are binary32.
// A workgroup evaluates them once per token, into LDS, for all its heads.
// HBM-bound: each element read and written once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4q_internal.h"
#include "row_ops.h"

namespace fp4q {

namespace {

constexpr int kThreads = 256;
constexpr int kAngles = 1024;    // angles of a workgroup: tokens * pairs, pairs rounded up to 8

template <typename T>
__device__ __forceinline__ void load8(const T *p, uint32_t n, float v[8])
{
    Chunk<T> q;
    if (n >= 8u) {
        q.load(p);
        q.get(v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < (int)n ? Chunk<T>::load1(p + j) : 0.0f;
    }
}
template <typename T>
__device__ __forceinline__ void store8(T *p, uint32_t n, const float v[8])
{
    Chunk<T> q;
    q.set(v);
    if (n >= 8u)
        q.store(p);
    else
        q.store_first(p, n);
}

// grid.x: groups of a.tokens_at_once tokens.  An item is one chunk of one
// head of one token: eight pairs, or eight elements to copy.
template <typename T, bool kInter>
__global__ __launch_bounds__(kThreads) void rotary_kernel(const RotaryArgs a, FastDiv per_token_div, FastDiv per_head_div)
{
    __shared__ __attribute__((aligned(16))) float cs[kAngles], sn[kAngles];
    const uint32_t half = a.rot >> 1, hc = (half + 7) / 8;  // chunks of pairs
    const uint32_t cc = a.copy ? (a.dim - a.rot + 7) / 8 : 0;  // chunks to copy
    const uint32_t per_head = hc + cc, per_token = per_head * a.heads;
    for (int64_t tok0 = (int64_t)blockIdx.x * a.tokens_at_once; tok0 < a.tokens;
         tok0 += (int64_t)gridDim.x * a.tokens_at_once) {
    const uint32_t ntok = (uint32_t)min((int64_t)a.tokens_at_once, a.tokens - tok0);
    for (uint32_t i = threadIdx.x; i < ntok * hc * 8; i += kThreads) {
        const uint32_t tk = i / (hc * 8), k = i - tk * (hc * 8);
        float c = 0.0f, s = 0.0f;
        if (k < half) {
            const int64_t pos = a.pos64 ? reinterpret_cast<const int64_t *>(a.positions)[tok0 + tk]
                                        : (int64_t) reinterpret_cast<const int32_t *>(a.positions)[tok0 + tk];
            double turns = (double)pos * ((double)a.inv_freq[k] * 0.15915494309189533577);
            turns -= __builtin_rint(turns);
            const float f = 2.0f * (float)turns;
            sincospif(f, &s, &c);
            c *= a.scale;
            s *= a.inverse ? -a.scale : a.scale;
        }
        cs[i] = c;
        sn[i] = s;
    }
    __syncthreads();
    const T *x = reinterpret_cast<const T *>(a.x);
    T *y = reinterpret_cast<T *>(a.y);
    for (uint32_t it = threadIdx.x; it < ntok * per_token; it += kThreads) {
        const uint32_t tk = fast_div(it, per_token_div), in_tok = it - tk * per_token;
        const uint32_t head = fast_div(in_tok, per_head_div), ch = in_tok - head * per_head;
        const T *px = x + (tok0 + tk) * a.x_token + (int64_t)head * a.x_head;
        T *py = y + (tok0 + tk) * a.y_token + (int64_t)head * a.y_head;
        if (ch < hc) {
            const uint32_t k0 = ch * 8, n = min(8u, half - k0);
            float c[8], s[8], u[8], v[8];
            const uint32_t at = (tk * hc + ch) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = cs[at + j], s[j] = sn[at + j];
            if (kInter) {
                const uint32_t n2 = 2 * n;
                load8(px + 2 * k0, min(n2, 8u), u);
                load8(px + 2 * k0 + 8, n2 > 8u ? n2 - 8u : 0u, v);
                float p[8], q[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    p[2 * j] = u[2 * j] * c[j] - u[2 * j + 1] * s[j];
                    p[2 * j + 1] = u[2 * j + 1] * c[j] + u[2 * j] * s[j];
                    q[2 * j] = v[2 * j] * c[4 + j] - v[2 * j + 1] * s[4 + j];
                    q[2 * j + 1] = v[2 * j + 1] * c[4 + j] + v[2 * j] * s[4 + j];
                }
                store8(py + 2 * k0, min(n2, 8u), p);
                store8(py + 2 * k0 + 8, n2 > 8u ? n2 - 8u : 0u, q);
            } else {
                load8(px + k0, n, u);
                load8(px + half + k0, n, v);
                float p[8], q[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    p[j] = u[j] * c[j] - v[j] * s[j];
                    q[j] = v[j] * c[j] + u[j] * s[j];
                }
                store8(py + k0, n, p);
                store8(py + half + k0, n, q);
            }
        } else {
            const uint32_t e = a.rot + (ch - hc) * 8;
            float u[8];
            load8(px + e, min(8u, a.dim - e), u);
            store8(py + e, min(8u, a.dim - e), u);
        }
    }
    __syncthreads();  // the next tokens' angles take the same place
    }
}

}  // namespace

int launch_rotary(RotaryArgs a, hipStream_t st)
{
    const uint32_t half = a.rot / 2, hc = (half + 7) / 8;
    const uint32_t cc = a.copy ? (a.dim - a.rot + 7) / 8 : 0;
    const uint32_t per_head = hc + cc, per_token = per_head * a.heads;
    int64_t at_once = kAngles / (hc * 8);
    if (at_once > 4) at_once = 4;
    while (at_once > 1 && (a.tokens + at_once - 1) / at_once < 1024) at_once >>= 1;
    a.tokens_at_once = (uint32_t)at_once;
    const int64_t groups = (a.tokens + at_once - 1) / at_once;
    const dim3 grid((unsigned)(groups < (1 << 20) ? groups : (1 << 20)));
    const FastDiv dt = fast_div_for(per_token), dh = fast_div_for(per_head);
#define FP4Q_ROTARY(T, INTER) hipLaunchKernelGGL((rotary_kernel<T, INTER>), grid, dim3(kThreads), 0, st, a, dt, dh)
    if (a.bf16) {
        if (a.interleaved) FP4Q_ROTARY(bf16_t, true); else FP4Q_ROTARY(bf16_t, false);
    } else {
        if (a.interleaved) FP4Q_ROTARY(float, true); else FP4Q_ROTARY(float, false);
    }
#undef FP4Q_ROTARY
    return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace fp4q
