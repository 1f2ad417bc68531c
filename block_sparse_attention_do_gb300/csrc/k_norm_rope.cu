// k_norm_rope.cu -- RMS norm of every query and key head and the rotation by
// its token's position, in one pass over q and k; and its gradients.
//
// Per head vector x of D elements, with r = (mean x^2 + eps)^(-1/2):
//   y = r w x,   pairs (y_a, y_b) of the first R dimensions become
//   (y_a c - y_b s, y_b c + y_a s),  c, s = cos, sin of position * inv_freq
// so an output element is r (x w c + x' w' s'), x' its pair's other element and
// s' = -s for the first, +s for the second of a pair: w c and w' s' are the
// same for all heads of a token.  Backward, from dz:
//   dy = dz c - dz' s',  dw = sum over tokens and heads of dy x r,
//   u = dy w,  dx = r (u - x r^2 mean(u x))
//
// What bounds it: the bytes, each read or written once.  A warp takes one
// token's heads, 16 bytes per lane and head, the next loads under way while it
// computes, over the end of a token too; the token's angles are computed once, a
// lane each, and shared through shared memory.  Measured, without the 4 us of a launch
// from a graph: 12,572 packed tokens of 40 heads of 128 in bf16, 258 MB, 47 us, 5.4 TB/s (80%
// of a plain copy's rate); gradients of 8192 tokens of 34 heads, 214 MB, 43 us, 5.0 TB/s;
// the latter's forward and gradients in fp32, 285 MB, 48 us, and 428 MB, 72 us, 5.9 TB/s; one
// token 2 us.  Loads into registers, two under way within a token: 51 and 52.
// Rings of 2, 3, 4, 5, 6, 8 vectors: 51, 47, 47, 48, 49, 50 and 47, 43, 43, 43, 43,
// 44 us; 2 or 4 CTAs an SM instead of 3: 57 and 60, 1 or 3 instead of 2: 56 and 61
// (registers spill).  A CTA's angles shared by its four tokens' warps behind a
// barrier took 60 and 57 us.
#include <math.h>

#include "cache_common.cuh"
#include "launch.h"
#include "tc_common.cuh"

namespace nsa {

namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;

constexpr int kDepth = 4;                   // vectors of a warp under way
constexpr int kFwdCtas = 3, kBwdCtas = 2;   // of an SM
constexpr int kRounds = 3;      // units of a warp, at least, before a unit is a whole token
constexpr int kMaxHalf = 64;    // angles of a token: D / 2

struct RopeArgs {
    Geo g;
    Strides sqr, skr;            // the rotated q and k (backward: their gradients)
    const void *q, *k;
    const float *qw, *kw;        // norm weights [D], or nullptr: ones
    const float *freq;           // [rot / 2]
    const int *pos;              // [ntok], or nullptr: a token's place in its sequence
    void *qr, *kr;               // forward: written; backward: read
    void *dq, *dk;
    float *part;                 // backward: [gridDim.x][2][D] sums of the weights' gradients
    int rot, pairs;
    float eps;
    int cq, ck;                  // vectors of a token: of its query and of its key heads
    int parts, per, units;       // units of a token, vectors of a unit, units of the call
};

// f as a fraction of 2^64 of a turn: f's 24 bits times 2^64 / 2 pi, shifted by
// its exponent; what passes 2^64 are whole turns.
__device__ __forceinline__ uint64_t turns_of(float f)
{
    constexpr uint64_t kInv = 0x28be60db9391054aull;  // 2^64 / 2 pi
    const uint32_t u = __float_as_uint(f), ex = u >> 23 & 255u;
    const uint64_t m = (u & 0x7fffffu) | (ex ? 0x800000u : 0u), lo = m * kInv, hi = __umul64hi(m, kInv);
    const int sh = 150 - (int)max(ex, 1u);  // f = m 2^-sh
    const uint64_t per = sh >= 128 ? 0 : sh >= 64 ? hi >> (sh - 64) : sh > 0 ? lo >> sh | hi << (64 - sh) : sh > -64 ? lo << -sh : 0;
    return u >> 31 ? 0 - per : per;
}

// cos and sin of pos * f, f given by turns_of.  A float product would leave a far
// position's angle no digits (position 10^6: 0.03 radians off); modulo 2^64 the
// product drops whole turns exactly.  turns_of is off by its truncation, one 2^-64 turn,
// and f times the rounding of 2^64 / 2 pi: the product by at most |pos| (1 + f) 2^-64
// turns, 2^-32 for f up to 1, and the 32 bits that are kept by 2^-26 once a float.
__device__ __forceinline__ float2 cos_sin(int pos, uint64_t per)
{
    const int turns = (int)((uint64_t)(int64_t)pos * per >> 32);  // of 2^-32, -1/2 .. 1/2
    float2 cs;
    sincospif((float)turns * 4.656612873077393e-10f, &cs.y, &cs.x);  // half turns: 2^-31
    return cs;
}

// 16 bytes of a head as pairs of floats (packed arithmetic: two a instruction).
template <typename T> struct Vec;
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4 &w, uint64_t (&x)[4])
    {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = tc::f2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
    }
    static __device__ __forceinline__ uint4 put(const uint64_t (&x)[4])
    {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo, hi;
            tc::f2_split(x[i], lo, hi);
            u[i] = tc::pack_bf16(lo, hi);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(const uint4 &w, uint64_t (&x)[2])
    {
        x[0] = tc::f2(__uint_as_float(w.x), __uint_as_float(w.y));
        x[1] = tc::f2(__uint_as_float(w.z), __uint_as_float(w.w));
    }
    static __device__ __forceinline__ uint4 put(const uint64_t (&x)[2])
    {
        float f[4];
        tc::f2_split(x[0], f[0], f[1]);
        tc::f2_split(x[1], f[2], f[3]);
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

__device__ __forceinline__ float both(uint64_t x)
{
    float lo, hi;
    tc::f2_split(x, lo, hi);
    return lo + hi;
}

// The lane's share of a head: elements d0 .. d0 + N of D, and where their
// pairs' other elements lie.  PAIRS: neighbours, else half the turning part away.
template <typename T, int D, bool PAIRS> struct Share {
    static constexpr int N = Vec<T>::N, P = N / 2, L = D / N, ROWS = 32 / L;  // pairs of floats; lanes of a head, heads of a warp
    int row, d0, other, d_other;  // other: the lane that holds the pairs' other elements, d_other: its first
    bool turns;
    __device__ __forceinline__ Share(const RopeArgs &a, int lane)
        : row(lane / L), d0(lane % L * N), other(lane), d_other(lane % L * N), turns(lane % L * N < a.rot)
    {
        if (turns && !PAIRS) {
            const int away = d0 < a.rot / 2 ? a.rot / 2 : -(a.rot / 2);
            other += away / N;
            d_other += away;
        }
    }
    // x': the pairs' other elements (an element that does not turn is its own)
    __device__ __forceinline__ void others(const uint4 &w, const uint64_t (&x)[P], uint64_t (&y)[P]) const
    {
        if constexpr (PAIRS) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float lo, hi;
                tc::f2_split(x[i], lo, hi);
                y[i] = turns ? tc::f2(hi, lo) : x[i];
            }
        } else {
            Vec<T>::get(make_uint4(__shfl_sync(0xffffffffu, w.x, other), __shfl_sync(0xffffffffu, w.y, other),
                                   __shfl_sync(0xffffffffu, w.z, other), __shfl_sync(0xffffffffu, w.w, other)), y);
        }
    }
    // the angles of dimensions d0 ..: c, and s with its sign (1 and 0 where nothing turns)
    __device__ __forceinline__ void angles(const float2 *table, uint64_t (&c)[P], uint64_t (&s)[P]) const
    {
        const bool second = !PAIRS && d_other < d0;
        const float4 *at = (const float4 *)(table + (PAIRS ? d0 / 2 : second ? d_other : d0));  // two angles
        const float4 none = make_float4(1.f, 0.f, 1.f, 0.f);
        if constexpr (PAIRS) {
#pragma unroll
            for (int i = 0; i < P; i += 2) {
                const float4 x = turns ? at[i / 2] : none;
                c[i] = tc::f2(x.x, x.x);
                s[i] = tc::f2(-x.y, x.y);
                c[i + 1] = tc::f2(x.z, x.z);
                s[i + 1] = tc::f2(-x.w, x.w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float4 x = turns ? at[i] : none;
                c[i] = tc::f2(x.x, x.z);
                s[i] = second ? tc::f2(x.y, x.w) : tc::f2(-x.y, -x.w);
            }
        }
    }
    // the weights of dimensions d0 .., and of their pairs' other elements (w: 16-byte aligned shared memory)
    __device__ __forceinline__ void weights(const float *w, uint64_t (&x)[P], uint64_t (&y)[P]) const
    {
#pragma unroll
        for (int i = 0; i < P; i += 2) {
            const float4 m = *(const float4 *)(w + d0 + 2 * i);
            const float4 o = PAIRS ? make_float4(m.y, m.x, m.w, m.z) : *(const float4 *)(w + d_other + 2 * i);
            x[i] = tc::f2(m.x, m.y);
            x[i + 1] = tc::f2(m.z, m.w);
            y[i] = tc::f2(o.x, o.y);
            y[i + 1] = tc::f2(o.z, o.w);
        }
    }
};

// over the lanes of a head
template <int L> __device__ __forceinline__ float head_sum(float x)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Token tok's place: its sequence (packed: 0) and token; false for a token in
// front of the first sequence or behind the last, and behind the call's last.
__device__ __forceinline__ bool place_of(const Geo &g, int tok, int &b, int &t)
{
    b = 0;
    t = tok;
    if (tok >= g.ntok || (g.thd && (tok < g.cu[0] || tok >= g.cu[g.B])))
        return false;
    if (!g.thd) {
        b = tok / g.T;
        t = tok - b * g.T;
    }
    return true;
}

// What the units of a warp share: its angles' frequencies (lane i has pairs i and
// i + 32) and room for a token's angles, and both norm weights.
template <int D> struct RopeSmem {
    float2 table[kWarps][kMaxHalf];
    float w[2][D];
};
template <int D> __device__ __forceinline__ void load_weights(const RopeArgs &a, RopeSmem<D> &sm)
{
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        const float *w = i < D ? a.qw : a.kw;
        sm.w[i / D][i % D] = w ? w[i % D] : 1.f;
    }
    __syncthreads();
}

// A unit: vectors [v0, v1) of a token, a vector being ROWS heads of q (the first
// a.cq vectors) or of k.
struct RopeUnit {
    int tok, b, t, v0, v1;
    bool live;
};
__device__ __forceinline__ RopeUnit unit_of(const RopeArgs &a, int unit)
{
    RopeUnit u;
    u.tok = a.parts == 1 ? unit : unit / a.parts;
    u.v0 = (unit - u.tok * a.parts) * a.per;
    u.v1 = min(u.v0 + a.per, a.cq + a.ck);
    u.live = place_of(a.g, u.tok, u.b, u.t);
    return u;
}
__device__ __forceinline__ void unit_angles(const RopeArgs &a, const RopeUnit &u, const uint64_t (&per)[2], int lane, float2 *table)
{
    const Geo &g = a.g;
    const int pos = a.pos ? a.pos[u.tok] : g.thd ? u.t - g.cu[seq_of_token(g, u.t)] : u.t, half = a.rot / 2;
    __syncwarp();  // (the unit before has read its own)
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (lane + i * 32 < half)
            table[lane + i * 32] = cos_sin(pos, per[i]);
    __syncwarp();
}

// A walk over a warp's vectors, unit after unit: where the lane's 16 bytes of the
// next one lie, in one or two tensors with q's and k's heads.
template <typename T, typename S, int TENSORS> struct Walk {
    int unit, v, v1, b, t;
    const T *q[TENSORS], *k[TENSORS];  // the token's first heads of the lane's row
    // sets the walk to the first unit from `unit` on that has a token; false: none is left
    __device__ __forceinline__ bool settle(const RopeArgs &a, const S &sh, const void *const (&qb)[TENSORS], const void *const (&kb)[TENSORS],
                                           const Strides *const (&qs)[TENSORS], const Strides *const (&ks)[TENSORS])
    {
        for (; unit < a.units; unit += (int)gridDim.x * kWarps) {
            const RopeUnit u = unit_of(a, unit);
            if (!u.live)
                continue;
            v = u.v0;
            v1 = u.v1;
            b = u.b;
            t = u.t;
#pragma unroll
            for (int i = 0; i < TENSORS; ++i) {
                q[i] = (const T *)qb[i] + (int64_t)b * qs[i]->b + (int64_t)t * qs[i]->t + (int64_t)sh.row * qs[i]->h + sh.d0;
                k[i] = (const T *)kb[i] + (int64_t)b * ks[i]->b + (int64_t)t * ks[i]->t + (int64_t)sh.row * ks[i]->h + sh.d0;
            }
            return true;
        }
        return false;
    }
};

// Units of a warp one after another, each lane's loads kDepth vectors ahead into a
// ring of its own in shared memory: cp.async of 16 bytes, which the same lane reads.
template <typename T, int D, bool PAIRS> __global__ void __launch_bounds__(kThreads, kFwdCtas) norm_rope_fwd_kernel(const RopeArgs a)
{
    using S = Share<T, D, PAIRS>;
    constexpr int P = S::P, R = S::ROWS;
    __shared__ __align__(16) RopeSmem<D> sm;
    __shared__ uint4 rings[kWarps][kDepth][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    dependents_may_start();
    dependency_wait();
    const Geo &g = a.g;
    const S sh(a, lane);
    const void *const qb[1] = {a.q}, *const kb[1] = {a.k};
    const Strides *const qs[1] = {&g.sq}, *const ks[1] = {&g.skv};
    Walk<T, S, 1> ahead;
    ahead.unit = blockIdx.x * kWarps + warp;
    bool more = ahead.settle(a, sh, qb, kb, qs, ks);
    auto fetch = [&](int stage) {
        if (more) {
            const bool key = ahead.v >= a.cq;
            const int h0 = (key ? ahead.v - a.cq : ahead.v) * R;
            const T *from = (key ? ahead.k[0] : ahead.q[0]) + h0 * (key ? g.skv.h : g.sq.h);
            if (h0 + sh.row < (key ? g.Hkv : g.Hq))
                tc::cp_async_16(tc::smem_u32(&rings[warp][stage][lane]), from, 16);
            if (++ahead.v == ahead.v1) {
                ahead.unit += (int)gridDim.x * kWarps;
                more = ahead.settle(a, sh, qb, kb, qs, ks);
            }
        }
        tc::cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth; ++i)
        fetch(i);
    load_weights(a, sm);
    uint64_t per[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        per[i] = lane + i * 32 < a.rot / 2 ? turns_of(a.freq[lane + i * 32]) : 0;
    int stage = 0;
    for (int unit = blockIdx.x * kWarps + warp; unit < a.units; unit += gridDim.x * kWarps) {
        const RopeUnit u = unit_of(a, unit);
        if (!u.live)
            continue;
        unit_angles(a, u, per, lane, sm.table[warp]);
        uint64_t c[P], s[P];
        T *dst = nullptr;
        for (int v = u.v0; v < u.v1; ++v) {
            const bool key = v >= a.cq;
            const int h = (key ? v - a.cq : v) * R + sh.row;
            const Strides &to = key ? a.skr : a.sqr;
            if (v == u.v0 || v == a.cq) {  // the unit's query heads begin, or its key heads
                dst = (T *)(key ? a.kr : a.qr) + (int64_t)u.b * to.b + (int64_t)u.t * to.t + (int64_t)h * to.h + sh.d0;
                sh.angles(sm.table[warp], c, s);
                uint64_t x[P], y[P];
                sh.weights(sm.w[key], x, y);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    c[i] = tc::f2_mul(c[i], x[i]);
                    s[i] = tc::f2_mul(s[i], y[i]);
                }
            }
            tc::cp_async_wait<kDepth - 1>();
            const uint4 w = rings[warp][stage][lane];
            fetch(stage);
            stage = stage == kDepth - 1 ? 0 : stage + 1;
            uint64_t x[P], y[P], sum;
            Vec<T>::get(w, x);
            sh.others(w, x, y);
            sum = tc::f2_mul(x[0], x[0]);
#pragma unroll
            for (int e = 1; e < P; ++e)
                sum = tc::f2_fma(x[e], x[e], sum);
            const float r = rsqrtf(fmaf(head_sum<S::L>(both(sum)), 1.f / D, a.eps));
            const uint64_t rr = tc::f2(r, r);
#pragma unroll
            for (int e = 0; e < P; ++e)
                x[e] = tc::f2_mul(tc::f2_fma(x[e], c[e], tc::f2_mul(y[e], s[e])), rr);
            if (h < (key ? g.Hkv : g.Hq))
                *(uint4 *)dst = Vec<T>::put(x);
            dst += R * to.h;
        }
    }
    tc::cp_async_wait<0>();
}

// As the forward.  A lane's sums of the weights' gradients stay in its registers
// to the end; a CTA's sums are one row of a.part, added up by
// norm_rope_sum_kernel: the order is fixed by the grid alone.
template <typename T, int D, bool PAIRS> __global__ void __launch_bounds__(kThreads, kBwdCtas) norm_rope_bwd_kernel(const RopeArgs a)
{
    using S = Share<T, D, PAIRS>;
    constexpr int N = S::N, P = S::P, R = S::ROWS;
    __shared__ __align__(16) RopeSmem<D> sm;
    extern __shared__ uint4 ring_raw[];  // [kWarps][kDepth][2][32]
    float(*sums)[2][D] = (float(*)[2][D])ring_raw;  // [kWarps]: at the end
    static_assert(sizeof(float) * kWarps * 2 * D <= sizeof(uint4) * kWarps * kDepth * 2 * 32, "");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint4 *ring = ring_raw + warp * kDepth * 2 * 32;
    dependents_may_start();
    dependency_wait();
    const Geo &g = a.g;
    const S sh(a, lane);
    const void *const qb[2] = {a.q, a.qr}, *const kb[2] = {a.k, a.kr};
    const Strides *const qs[2] = {&g.sq, &a.sqr}, *const ks[2] = {&g.skv, &a.skr};
    Walk<T, S, 2> ahead;
    ahead.unit = blockIdx.x * kWarps + warp;
    bool more = ahead.settle(a, sh, qb, kb, qs, ks);
    auto fetch = [&](int stage) {
        if (more) {
            const bool key = ahead.v >= a.cq;
            const int h0 = (key ? ahead.v - a.cq : ahead.v) * R;
            const bool have = h0 + sh.row < (key ? g.Hkv : g.Hq);
            const T *x = (key ? ahead.k[0] : ahead.q[0]) + h0 * (key ? g.skv.h : g.sq.h), *z = (key ? ahead.k[1] : ahead.q[1]) + h0 * (key ? a.skr.h : a.sqr.h);
            if (have) {
                tc::cp_async_16(tc::smem_u32(&ring[stage * 64 + lane]), x, 16);
                tc::cp_async_16(tc::smem_u32(&ring[stage * 64 + 32 + lane]), z, 16);
            } else  // (zeros, which add nothing)
                ring[stage * 64 + lane] = ring[stage * 64 + 32 + lane] = make_uint4(0, 0, 0, 0);
            if (++ahead.v == ahead.v1) {
                ahead.unit += (int)gridDim.x * kWarps;
                more = ahead.settle(a, sh, qb, kb, qs, ks);
            }
        }
        tc::cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth; ++i)
        fetch(i);
    load_weights(a, sm);
    uint64_t per[2], dqw[P], dkw[P];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        per[i] = lane + i * 32 < a.rot / 2 ? turns_of(a.freq[lane + i * 32]) : 0;
#pragma unroll
    for (int e = 0; e < P; ++e)
        dqw[e] = dkw[e] = 0;
    int stage = 0;
    for (int unit = blockIdx.x * kWarps + warp; unit < a.units; unit += gridDim.x * kWarps) {
        const RopeUnit u = unit_of(a, unit);
        if (!u.live)
            continue;
        unit_angles(a, u, per, lane, sm.table[warp]);
        uint64_t c[P], s[P];
        sh.angles(sm.table[warp], c, s);
#pragma unroll
        for (int e = 0; e < P; ++e)
            s[e] ^= 0x8000000080000000ull;  // turned back
        for (int part = u.v0 >= a.cq; part < 2; ++part) {  // the unit's query heads, then its key heads
            const bool key = part == 1;
            const int v0 = key ? max(u.v0 - a.cq, 0) : u.v0, v1 = key ? u.v1 - a.cq : min(u.v1, a.cq), heads = key ? g.Hkv : g.Hq;
            const Strides &to = key ? g.sdkv : g.sdq;
            int h = v0 * R + sh.row;
            T *dst = (T *)(key ? a.dk : a.dq) + (int64_t)u.b * to.b + (int64_t)u.t * to.t + (int64_t)h * to.h + sh.d0;
            uint64_t w[P], dw[P];
            {
                uint64_t y[P];
                sh.weights(sm.w[key], w, y);
            }
#pragma unroll
            for (int e = 0; e < P; ++e)
                dw[e] = 0;
            for (int v = v0; v < v1; ++v) {
                tc::cp_async_wait<kDepth - 1>();
                const uint4 xw = ring[stage * 64 + lane], zw = ring[stage * 64 + 32 + lane];
                fetch(stage);
                stage = stage == kDepth - 1 ? 0 : stage + 1;
                uint64_t x[P], z[P], y[P], xx = 0, ux = 0;
                Vec<T>::get(xw, x);
                Vec<T>::get(zw, z);
                sh.others(zw, z, y);
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    z[e] = tc::f2_fma(z[e], c[e], tc::f2_mul(y[e], s[e]));  // dy
                    xx = tc::f2_fma(x[e], x[e], xx);
                    y[e] = tc::f2_mul(z[e], w[e]);  // u
                    ux = tc::f2_fma(y[e], x[e], ux);
                }
                const float r = rsqrtf(fmaf(head_sum<S::L>(both(xx)), 1.f / D, a.eps));
                const float m = head_sum<S::L>(both(ux)) * r * (r * (1.f / D));  // (each factor in range: u x r is of u's size)
                const uint64_t rr = tc::f2(r, r), mm = tc::f2(-m, -m);
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    dw[e] = tc::f2_fma(tc::f2_mul(z[e], rr), x[e], dw[e]);
                    x[e] = tc::f2_mul(tc::f2_fma(mm, x[e], y[e]), rr);
                }
                if (h < heads)
                    *(uint4 *)dst = Vec<T>::put(x);
                h += R;
                dst += R * to.h;
            }
#pragma unroll
            for (int e = 0; e < P; ++e) {
                dqw[e] = tc::f2_add(dqw[e], key ? 0ull : dw[e]);
                dkw[e] = tc::f2_add(dkw[e], key ? dw[e] : 0ull);
            }
        }
    }
    tc::cp_async_wait<0>();
    if (!a.part)
        return;
    __syncthreads();  // the rings are used up
#pragma unroll
    for (int e = 0; e < N; ++e)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float lo, hi;
            tc::f2_split(i ? dkw[e / 2] : dqw[e / 2], lo, hi);
            float x = e & 1 ? hi : lo;
#pragma unroll
            for (int o = S::L; o < 32; o <<= 1)
                x += __shfl_xor_sync(0xffffffffu, x, o);
            if (sh.row == 0)
                sums[warp][i][sh.d0 + e] = x;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            x += sums[w][i / D][i % D];
        a.part[(int64_t)blockIdx.x * 2 * D + i] = x;
    }
}

// dqw, dkw [D] (either may be nullptr) from n rows of sums: a block for 32 of
// the 2 D columns, its warps taking the rows in turn.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(kSumWarps * 32) norm_rope_sum_kernel(const float *part, int n, int D, float *dqw, float *dkw)
{
    __shared__ float sums[kSumWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = blockIdx.x * 32 + lane;
    dependents_may_start();
    dependency_wait();
    float x = 0.f;
#pragma unroll 8
    for (int i = warp; i < n; i += kSumWarps)
        x += part[(int64_t)i * 2 * D + col];
    sums[warp][lane] = x;
    __syncthreads();
    float *dst = col < D ? dqw : dkw;
    if (warp != 0 || !dst)
        return;
#pragma unroll
    for (int w = 1; w < kSumWarps; ++w)
        x += sums[w][lane];
    dst[col % D] = x;
}

int bwd_grid() { return num_sms() * kBwdCtas; }

// The call's units for `ctas` CTAs' warps: a token each, cut up (as far as single
// vectors) until every warp has about kRounds: a token alone is spread over as
// many warps as it has vectors, and the last round of many costs little (3 rounds
// 55.2 and 55.7 us on the cases above, 6 56.7 and 60.1).  Returns the grid.
int cut_units(RopeArgs &a, int rows, int ctas)
{
    a.cq = (a.g.Hq + rows - 1) / rows;
    a.ck = (a.g.Hkv + rows - 1) / rows;
    const int n = a.cq + a.ck;
    const int64_t want = (int64_t)ctas * kWarps * kRounds, ntok = a.g.ntok;
    a.parts = (int)min((int64_t)n, max((int64_t)1, (want + ntok - 1) / ntok));
    a.per = (n + a.parts - 1) / a.parts;
    a.parts = (n + a.per - 1) / a.per;
    a.units = (int)(ntok * a.parts);  // (below ntok * (Hq + Hkv): checked)
    return (int)min((int64_t)ctas, ((int64_t)a.units + kWarps - 1) / kWarps);
}

template <typename T, int D, bool PAIRS> cudaError_t fwd_t(RopeArgs &a, cudaStream_t st)
{
    const int grid = cut_units(a, Share<T, D, PAIRS>::ROWS, num_sms() * kFwdCtas);
    return launch_dependent(norm_rope_fwd_kernel<T, D, PAIRS>, dim3(grid), dim3(kThreads), 0, st, a);
}

template <typename T, int D, bool PAIRS> cudaError_t bwd_t(RopeArgs &a, float *dqw, float *dkw, cudaStream_t st)
{
    const int grid = cut_units(a, Share<T, D, PAIRS>::ROWS, bwd_grid());
    constexpr int ring = kWarps * kDepth * 2 * 32 * (int)sizeof(uint4);
    static_assert(ring + sizeof(RopeSmem<D>) <= 48 * 1024, "what a kernel has without asking");
    cudaError_t e = launch_dependent(norm_rope_bwd_kernel<T, D, PAIRS>, dim3(grid), dim3(kThreads), ring, st, a);
    if (e != cudaSuccess || !a.part)
        return e;
    return launch_dependent(norm_rope_sum_kernel, dim3(2 * D / 32), dim3(kSumWarps * 32), 0, st, (const float *)a.part, grid, D, dqw, dkw);
}

RopeArgs rope_args(const Geo &g, const Rope &r)
{
    RopeArgs a = {};
    a.g = g;
    a.sqr = r.sqr;
    a.skr = r.skr;
    a.q = r.q;
    a.k = r.k;
    a.qw = r.qw;
    a.kw = r.kw;
    a.freq = r.freq;
    a.pos = r.pos;
    a.rot = r.rot;
    a.pairs = r.pairs;
    a.eps = r.eps;
    return a;
}

}  // namespace

size_t norm_rope_bwd_ws_bytes(const Geo &g) { return sizeof(float) * 2 * g.D * (size_t)bwd_grid(); }

cudaError_t launch_norm_rope_fwd(const Geo &g, const Rope &r, void *qr, void *kr, int dtype, cudaStream_t st)
{
    RopeArgs a = rope_args(g, r);
    a.qr = qr;
    a.kr = kr;
#define NSA_ROPE(T, D) (a.pairs ? fwd_t<T, D, true>(a, st) : fwd_t<T, D, false>(a, st))
    if (dtype == NSA_DTYPE_BF16)
        return g.D == 128 ? NSA_ROPE(__nv_bfloat16, 128) : g.D == 64 ? NSA_ROPE(__nv_bfloat16, 64) : NSA_ROPE(__nv_bfloat16, 32);
    return g.D == 128 ? NSA_ROPE(float, 128) : g.D == 64 ? NSA_ROPE(float, 64) : NSA_ROPE(float, 32);
#undef NSA_ROPE
}

cudaError_t launch_norm_rope_bwd(const Geo &g, const Rope &r, const void *dqr, const void *dkr, void *dq, void *dk, float *dqw, float *dkw,
                                 float *part, int dtype, cudaStream_t st)
{
    RopeArgs a = rope_args(g, r);
    a.qr = (void *)dqr;
    a.kr = (void *)dkr;
    a.dq = dq;
    a.dk = dk;
    a.part = dqw || dkw ? part : nullptr;
#define NSA_ROPE(T, D) (a.pairs ? bwd_t<T, D, true>(a, dqw, dkw, st) : bwd_t<T, D, false>(a, dqw, dkw, st))
    if (dtype == NSA_DTYPE_BF16)
        return g.D == 128 ? NSA_ROPE(__nv_bfloat16, 128) : g.D == 64 ? NSA_ROPE(__nv_bfloat16, 64) : NSA_ROPE(__nv_bfloat16, 32);
    return g.D == 128 ? NSA_ROPE(float, 128) : g.D == 64 ? NSA_ROPE(float, 64) : NSA_ROPE(float, 32);
#undef NSA_ROPE
}

}  // namespace nsa
