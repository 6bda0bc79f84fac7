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
// A workgroup evaluates them once per token, into LDS, for all its heads,
// while its first elements are on their way.
// HBM-bound: each element read and written once.  8192 tokens x 40 heads x
// 128 bf16 out of QKV rows, from memory: 32.8 us, 5.1 TB/s; on three sets in
// turn, which the last-level cache holds in part, 28.6 (angles before loads and
// plain loads 37).  Interleaved 35.6, heads of whole tokens 35.0, both from
// memory.  32 tokens: 4.2 us a call, launch and latency.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4q_internal.h"
#include "row_ops.h"

namespace fp4q {

namespace {

constexpr int kThreads = 256;
constexpr int kAngles = 1024;  // angles of a workgroup: tokens * pairs, pairs rounded up to 8

// How the last chunk of a part (of a head) that eight does not divide is
// made: kAgain, as the part's last eight elements, some of them a second
// time; kOwn, in place, the same but stored without those, which their
// chunk may have turned already; kShort, parts below eight, element by
// element.  kOwn against element by
// element for all rests in place, 8192 x 32 heads bf16: half style, 24 of 96
// turned 19.1 / 29.1 us; interleaved, 100 of 100 24.7 / 35.4, 50 of 100 30.8 /
// 30.5, 250 of 256 72.1 / 67.8.
enum Rest { kAgain, kOwn, kShort };
template <typename T, Rest kRest, bool kNt>
__device__ __forceinline__ void load8(const T *p, uint32_t n, Chunk<T> &q)
{
    if (kRest != kShort || n >= 8u) {
        q.template load<kNt>(p);
    } else {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < (int)n ? as_float(p[j]) : 0.0f;
        q.set(v);
    }
}
template <typename T, Rest kRest>
__device__ __forceinline__ void store8(T *p, uint32_t lo, uint32_t n, const float v[8])
{
    Chunk<T> q;
    q.set(v);
    if (kRest == kAgain || (lo == 0u && n >= 8u))
        q.template store<false>(p);
    else if (lo < n)
        q.store_own(p, lo, n);
}

// An item is one chunk of one head of one token: eight pairs (half style),
// eight elements that are four pairs (interleaved), or eight elements to copy.
struct Item {
    int64_t x, y;           // the head's first element
    uint32_t first, lo, n;  // the chunk's first element, and which of its eight are its own
    uint32_t angle;         // of its first pair
    bool copy;
};

// grid.x: groups of a.tokens_at_once tokens.
template <typename T, bool kInter, Rest kRest>
__global__ __launch_bounds__(kThreads) void rotary_kernel(const RotaryArgs a, FastDiv per_token_div, FastDiv per_head_div)
{
    __shared__ __attribute__((aligned(16))) float cs[kAngles], sn[kAngles];
    constexpr bool kNt = kStream<T>;
    const uint32_t half = a.rot >> 1, angles = (half + 7u) & ~7u;  // of a token
    const uint32_t turned = kInter ? (a.rot + 7u) >> 3 : angles >> 3;  // chunks of a head to turn
    const uint32_t per_head = turned + (a.copy ? (a.dim - a.rot + 7u) >> 3 : 0u), per_token = per_head * a.heads;
    const T *x = reinterpret_cast<const T *>(a.x);
    T *y = reinterpret_cast<T *>(a.y);
    const int64_t tok0 = (int64_t)(blockIdx.y * gridDim.x + blockIdx.x) * a.tokens_at_once;
    if (tok0 >= a.tokens) return;
    const uint32_t ntok = (uint32_t)min((int64_t)a.tokens_at_once, a.tokens - tok0), total = ntok * per_token;
    const auto item = [&](uint32_t it) {
        const uint32_t tk = fast_div(it, per_token_div), in_tok = it - tk * per_token;
        const uint32_t head = fast_div(in_tok, per_head_div), ch = in_tok - head * per_head;
        Item m;
        m.x = (tok0 + tk) * a.x_token + (int64_t)head * a.x_head;
        m.y = (tok0 + tk) * a.y_token + (int64_t)head * a.y_head;
        m.copy = ch >= turned;
        const uint32_t from = m.copy ? a.rot : 0u, to = m.copy ? a.dim : kInter ? a.rot : half;
        const uint32_t start = from + (ch - (m.copy ? turned : 0u)) * 8u;
        m.first = kRest == kShort ? start : min(start, to - 8u);
        m.lo = kRest == kOwn ? start - m.first : 0u;
        m.n = min(8u, to - m.first);
        m.angle = tk * angles + (kInter ? m.first >> 1 : m.first);
        return m;
    };
    const auto fetch = [&](const Item &m, Chunk<T> &u, Chunk<T> &v) {
        load8<T, kRest, kNt>(x + m.x + m.first, m.n, u);
        if (!kInter) load8<T, kRest, kNt>(x + m.x + m.first + (m.copy ? 0u : half), m.n, v);
    };
    // the first item is on its way while the angles are made
    uint32_t it = min(threadIdx.x, total - 1u);
    Item m = item(it);
    Chunk<T> u, v;
    fetch(m, u, v);
    for (uint32_t i = threadIdx.x; i < ntok * angles; i += kThreads) {
        const uint32_t tk = i / angles, k = i - tk * angles;
        float c = 0.0f, s = 0.0f;
        if (k < half) {
            const int64_t pos = a.pos64 ? reinterpret_cast<const int64_t *>(a.positions)[tok0 + tk]
                                        : (int64_t) reinterpret_cast<const int32_t *>(a.positions)[tok0 + tk];
            double turns = (double)pos * ((double)a.inv_freq[k] * 0.15915494309189533577);
            turns -= __builtin_rint(turns);
            sincospif(2.0f * (float)turns, &s, &c);
            c *= a.scale;
            s *= a.inverse ? -a.scale : a.scale;
        }
        cs[i] = c;
        sn[i] = s;
    }
    __syncthreads();
    for (it = threadIdx.x; it < total; it += kThreads) {
        const Item next = item(min(it + kThreads, total - 1u));
        Chunk<T> nu, nv;
        fetch(next, nu, nv);  // in place: the last item again, after its store perhaps, but then it is not used
        float p[8], q[8], o[8], r[8];
        u.get(p);
        T *out = y + m.y + m.first;
        if (m.copy) {
            store8<T, kRest>(out, m.lo, m.n, p);
        } else if (kInter) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float c = cs[m.angle + j], s = sn[m.angle + j];
                o[2 * j] = p[2 * j] * c - p[2 * j + 1] * s;
                o[2 * j + 1] = p[2 * j + 1] * c + p[2 * j] * s;
            }
            store8<T, kRest>(out, m.lo, m.n, o);
        } else {
            v.get(q);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float c = cs[m.angle + j], s = sn[m.angle + j];
                o[j] = p[j] * c - q[j] * s;
                r[j] = q[j] * c + p[j] * s;
            }
            store8<T, kRest>(out, m.lo, m.n, o);
            store8<T, kRest>(out + half, m.lo, m.n, r);
        }
        m = next;
        u = nu;
        v = nv;
    }
}

}  // namespace

int launch_rotary(RotaryArgs a, hipStream_t st)
{
    const uint32_t half = a.rot / 2, angles = (half + 7) / 8 * 8;
    const uint32_t turned = a.interleaved ? (a.rot + 7) / 8 : angles / 8;
    const uint32_t per_head = turned + (a.copy ? (a.dim - a.rot + 7) / 8 : 0), per_token = per_head * a.heads;
    // four tokens to a workgroup, or as many as give its threads an item each
    // (one head of 64, 65536 tokens: 8.7 us, four tokens at once 18.9), but at
    // least about four workgroups to a compute unit. Binary32 items of the half
    // style, 64 bytes in and out, go to half the threads (16384 tokens of two
    // heads of 128: 9.8 us, to all 11.0, four tokens 10.2; of three 14.6, 16.0,
    // 13.2; interleaved, 32 bytes, to all 10.4, to half 10.9)
    const int64_t items = a.bf16 || a.interleaved ? kThreads : kThreads / 2;
    const int64_t cap = (items + per_token - 1) / per_token;
    int64_t at_once = kAngles / angles;
    if (at_once > (cap > 4 ? cap : 4)) at_once = cap > 4 ? cap : 4;
    while (at_once > 1 && (a.tokens + at_once - 1) / at_once < 1024) at_once >>= 1;
    a.tokens_at_once = (uint32_t)at_once;
    const int64_t groups = (a.tokens + at_once - 1) / at_once, wide = 1 << 20;  // a launch's threads along x are below 2^32
    const dim3 grid((unsigned)(groups < wide ? groups : wide), (unsigned)((groups + wide - 1) / wide));
    const FastDiv dt = fast_div_for(per_token), dh = fast_div_for(per_head);
    const uint32_t part = a.interleaved ? a.rot : half, rest = a.copy ? a.dim - a.rot : 0;
    const Rest last = part < 8 || (rest > 0 && rest < 8) ? kShort : part % 8 != 0 && a.x == a.y ? kOwn : kAgain;
#define FP4Q_ROTARY(T, INTER, REST) \
    hipLaunchKernelGGL((rotary_kernel<T, INTER, REST>), grid, dim3(kThreads), 0, st, a, dt, dh)
#define FP4Q_ROTARY_R(T, INTER)                               \
    do {                                                      \
        switch (last) {                                       \
        case kAgain: FP4Q_ROTARY(T, INTER, kAgain); break;    \
        case kOwn: FP4Q_ROTARY(T, INTER, kOwn); break;        \
        case kShort: FP4Q_ROTARY(T, INTER, kShort); break;    \
        }                                                     \
    } while (0)
#define FP4Q_ROTARY_T(T)                                                        \
    do {                                                                        \
        if (a.interleaved) FP4Q_ROTARY_R(T, true); else FP4Q_ROTARY_R(T, false); \
    } while (0)
    if (a.bf16)
        FP4Q_ROTARY_T(bf16_t);
    else
        FP4Q_ROTARY_T(float);
#undef FP4Q_ROTARY_T
#undef FP4Q_ROTARY_R
#undef FP4Q_ROTARY
    return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace fp4q
