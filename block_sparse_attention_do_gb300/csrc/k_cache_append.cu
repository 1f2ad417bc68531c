// k_cache_append.cu -- new tokens' keys and values rounded to e4m3 with one
// scale per (page, head) and written into their pages.
//
// For a page of head h that gets new tokens x: s = the least power of two
// with max|x| <= 448 s over the finite x; where the page already holds
// tokens, s = max(s, its scale) and, if that grew, their codes are rounded
// again by (old scale / s).  code = e4m3(x / s).  Each (page, head, k or v)
// is one group of threads' work: the new values stay in registers between
// the maximum and the rounding, so the input is read once and the codes are
// written once; a page's earlier codes are touched only when its scale grew.
//
// What bounds it: prompts, the bytes (keys and values, 2 in and 1 out each:
// 172 MB of 8 prompts of up to 8192 tokens in 31 us, 5.5 TB/s); single tokens,
// the launch (64 rows: 5.5 us, of which 4 are any launch's).
#include <math.h>

#include "cache_common.cuh"
#include "launch.h"
#include "tc_common.cuh"

namespace nsa {

namespace {

constexpr int kCta = 128;

// A 16-byte vector of the element type: as floats; as floats times a power of
// two (exact: bf16 has float's exponents, and what falls below its normal range
// is far below the least code); and the running maximum of its magnitudes,
// which order as their bits do.
template <typename T> struct Vec16;
template <> struct Vec16<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void scaled(const uint4 &w, float by, float (&x)[8])
    {
        const __nv_bfloat162 f = __float2bfloat162_rn(by);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        uint32_t y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __hmul2(*(const __nv_bfloat162 *)&u[i], f);
            y[i] = *(const uint32_t *)&p;
        }
        get(make_uint4(y[0], y[1], y[2], y[3]), x);
    }
    static __device__ __forceinline__ uint32_t top(uint32_t t, const uint4 &w)
    {
        t = __vmaxu2(__vmaxu2(t, w.x & 0x7fff7fffu), w.y & 0x7fff7fffu);
        return __vmaxu2(__vmaxu2(t, w.z & 0x7fff7fffu), w.w & 0x7fff7fffu);
    }
    static __device__ __forceinline__ uint32_t top_bits(uint32_t t) { return max(t << 16, t & 0xffff0000u); }  // a float's
    static __device__ __forceinline__ void get(const uint4 &w, float (&x)[8])
    {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
};
template <> struct Vec16<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void scaled(const uint4 &w, float by, float (&x)[4])
    {
        get(w, x);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] *= by;
    }
    static __device__ __forceinline__ uint32_t top(uint32_t t, const uint4 &w)
    {
        return max(max(max(t, w.x & 0x7fffffffu), max(w.y & 0x7fffffffu, w.z & 0x7fffffffu)), w.w & 0x7fffffffu);
    }
    static __device__ __forceinline__ uint32_t top_bits(uint32_t t) { return t; }
    static __device__ __forceinline__ void get(const uint4 &w, float (&x)[4])
    {
        x[0] = __uint_as_float(w.x);
        x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z);
        x[3] = __uint_as_float(w.w);
    }
};

// the reciprocal of a power of two (exact: a product with it is the
// quotient), or 0 for a scale that is none
__device__ __forceinline__ float pow2_inverse(float scale)
{
    const uint32_t u = __float_as_uint(scale);
    return (u & 0x7fffffu) == 0 && (u >> 23) > 1 && (u >> 23) < 253 ? __uint_as_float((254u - (u >> 23)) << 23) : 0.f;
}

// N floats to N codes
template <int N> __device__ __forceinline__ void store_codes(uint8_t *p, const float (&x)[N])
{
    uint32_t u[N / 4];
#pragma unroll
    for (int e = 0; e < N / 4; ++e)
        u[e] = e4m3_pack2(x[4 * e], x[4 * e + 1]) | e4m3_pack2(x[4 * e + 2], x[4 * e + 3]) << 16;
    if constexpr (N == 8)
        *(uint2 *)p = make_uint2(u[0], u[1]);
    else
        *(uint32_t *)p = u[0];
}

// the new tokens of row b: their count and first position; false where the
// row's length or packed range cannot hold them
__device__ __forceinline__ bool places(const Geo &g, const Cache &c, int b, int &n, int &start)
{
    const int len = c.lens[b];
    n = new_tokens(g, b);
    start = n >= 0 && len >= n ? len - n : -1;
    return start >= 0 && (int64_t)len <= (int64_t)c.cols * c.bs;
}

// a page that new tokens may go into: in the pool, and no other row's
__device__ __forceinline__ bool writable(const Cache &c, int page)
{
    return page >= 0 && page < c.pages && (!c.ref || c.ref[page] == 1);
}

// Every row and every page that the call writes, checked by one block of the
// launch, which alone writes the error word: it needs no clearing.  A thread
// takes one (row, touched page) at a time, so its few dependent reads are
// under way for all of them together.
__device__ void append_check(const Geo &g, const Cache &c, int per_row, int *err)
{
    int bad = 0;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < (int64_t)c.rows * per_row; i += kCta) {
        const int b = (int)(i / per_row), j = (int)(i % per_row);
        int n, start;
        if (!places(g, c, b, n, start))
            bad = 1;
        else if (n > 0 && (start >> c.bsh) + j <= (start + n - 1) >> c.bsh)
            bad |= !writable(c, c.table[(int64_t)b * c.cols + (start >> c.bsh) + j]);
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0)
        *err = bad ? NSA_ERR_BAD_INDEX : NSA_OK;
}

// Blocks of an SM that the registers leave room for: as many as hold a
// thread's vectors without spilling (8 prompts of up to 8192 tokens, 8 vectors
// a thread: 31.0 us with 10 blocks, 34.8 with 6, 36.9 with 12; one vector: any
// number serves).
template <typename T, int VPT> constexpr int append_ctas() { return VPT == 1 ? 4 : VPT * sizeof(T) <= 16 ? 10 : 6; }

// GROUP threads per head of k or v of a touched page; VPT vectors of the
// page's new tokens per thread (VPT * GROUP * N elements cover a page, or
// the call's few new tokens).
template <typename T, int GROUP, int VPT>
__global__ void __launch_bounds__(kCta, append_ctas<T, VPT>()) cache_append_kernel(const Geo g, const Cache c, const T *kn, const T *vn, int per_row,
                                                            int *err)
{
    constexpr int N = Vec16<T>::N;
    __shared__ uint32_t red[kCta / 32];
    dependents_may_start();
    dependency_wait();
    if (blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y == 0)
            append_check(g, c, per_row, err);
        return;
    }
    // block x: a touched page (row * per_row + j); block y and group: a head of k or v
    const int lane = threadIdx.x % GROUP, b = blockIdx.x / per_row, j = blockIdx.x - b * per_row;
    const int part = blockIdx.y * (kCta / GROUP) + threadIdx.x / GROUP, which = part >= c.Hkv ? 1 : 0, h = part - which * c.Hkv;
    const bool live = part < 2 * c.Hkv;
    int lo = 0, n = 0, page = -1, t0 = 0;  // the page's slots [lo, lo + n) get tokens t0 ..
    if (live) {
        int nn, start;
        if (places(g, c, b, nn, start)) {
            const int col = (start >> c.bsh) + j, first = max(start, col * c.bs), end = min(start + nn, (col + 1) * c.bs);
            if (first < end) {
                page = c.table[(int64_t)b * c.cols + col];
                lo = first - col * c.bs;
                n = writable(c, page) ? end - first : 0;
                t0 = first - start;
            }
        }
    }
    if (GROUP < kCta ? __all_sync(0xffffffffu, n == 0) : n == 0)
        return;  // uniform over the group
    const int vec_tok = c.D / N;  // vectors per token: a power of two
    const int shift = 31 - __clz(vec_tok);
    const int nvec = n << shift;
    const T *src = (which ? vn : kn) + (n > 0 ? kv_off(g, b, h, t0) : 0);
    const int st = (int)c.st;
    // a thread's vectors lie at one place of tokens GROUP / vec_tok apart
    const T *from = src + (lane >> shift) * g.skv.t + (lane & (vec_tok - 1)) * N;
    uint4 w[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        w[i] = make_uint4(0, 0, 0, 0);
        if (lane + i * GROUP < nvec)
            w[i] = *(const uint4 *)from;
        from += (GROUP >> shift) * g.skv.t;
    }
    float *scales = (which ? c.vs : c.ks) + (int64_t)(n > 0 ? page : 0) * c.Hkv + h;
    const float old = lo > 0 && n > 0 ? *scales : 0.f;
    auto of_group = [&](uint32_t bits) {  // their maximum
        bits = __reduce_max_sync(0xffffffffu, bits);
        if constexpr (GROUP > 32) {
            __syncthreads();
            if ((threadIdx.x & 31) == 0)
                red[threadIdx.x / 32] = bits;
            __syncthreads();
            bits = max(max(red[0], red[1]), max(red[2], red[3]));
        }
        return bits;
    };
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        top = Vec16<T>::top(top, w[i]);
    float amax = __uint_as_float(of_group(Vec16<T>::top_bits(top)));
    if (!(amax < INFINITY)) {  // infinities or NaN (the group's threads alike): of the others
        float fin = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float x[N];
            Vec16<T>::get(w[i], x);
#pragma unroll
            for (int e = 0; e < N; ++e)
                fin = fabsf(x[e]) < INFINITY ? fmaxf(fin, fabsf(x[e])) : fin;
        }
        amax = __uint_as_float(of_group(__float_as_uint(fin)));
    }
    if (n == 0)
        return;
    const float need = e4m3_scale(amax), scale = fmaxf(need, old);
    uint8_t *dst = (which ? c.v : c.k) + (int64_t)page * c.sp + (int64_t)h * c.sh;
    if (lo > 0 && scale != old) {  // the earlier tokens' codes on the larger scale
        const float ratio = __fdiv_rn(old, scale);
        const int per_tok = c.D / 16, sh16 = 31 - __clz(per_tok);
        for (int x = lane; x < lo << sh16; x += GROUP) {
            uint4 *p = (uint4 *)(dst + (x >> sh16) * st + (x & (per_tok - 1)) * 16);
            const uint4 q = *p;
            uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t a, d;
                e4m3x4_to_half(u[i], a, d);
                const float2 fa = __half22float2(*(const __half2 *)&a), fd = __half22float2(*(const __half2 *)&d);
                u[i] = e4m3_pack2(fa.x * ratio, fa.y * ratio) | e4m3_pack2(fd.x * ratio, fd.y * ratio) << 16;
            }
            *p = make_uint4(u[0], u[1], u[2], u[3]);
        }
    }
    const float inv = pow2_inverse(scale);
    if (inv != 0.f) {
        uint8_t *to = dst + (int64_t)(lo + (lane >> shift)) * st + (lane & (vec_tok - 1)) * N;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (lane + i * GROUP < nvec) {
                float f[N];
                Vec16<T>::scaled(w[i], inv, f);
                store_codes<N>(to, f);
            }
            to += (GROUP >> shift) * st;
        }
    } else {  // a scale of the caller's, larger than the new tokens need: divided, off the common path
#pragma unroll 1
        for (int x = lane; x < nvec; x += GROUP) {
            float f[N];
            Vec16<T>::get(*(const uint4 *)(src + (x >> shift) * g.skv.t + (x & (vec_tok - 1)) * N), f);
#pragma unroll
            for (int e = 0; e < N; ++e)
                f[e] = __fdiv_rn(f[e], scale);
            store_codes<N>(dst + (lo + (x >> shift)) * st + (x & (vec_tok - 1)) * N, f);
        }
    }
    if (lane == 0)
        *scales = scale;
}

template <typename T> cudaError_t append_t(const Geo &g, const Cache &c, const void *k, const void *v, int *err, cudaStream_t st)
{
    constexpr int N = Vec16<T>::N;
    const int longest = longest_tokens(g), per_row = (longest + c.bs - 2) / c.bs + 1;
    // few new tokens per row: a warp per head, its values in 4 (fp32: 8)
    // vectors per thread; else a block per head
    constexpr int FEW = sizeof(T) == 2 ? 4 : 8;
    const int vecs = min(longest, c.bs) * c.D / N;
    const bool few = vecs <= 32 * FEW;
    const dim3 grid((unsigned)((int64_t)c.rows * per_row + 1), (unsigned)(few ? (2 * c.Hkv + kCta / 32 - 1) / (kCta / 32) : 2 * c.Hkv));
    const T *kn = (const T *)k, *vn = (const T *)v;
    if (vecs <= 32)
        return launch_dependent(cache_append_kernel<T, 32, 1>, grid, dim3(kCta), 0, st, g, c, kn, vn, per_row, err);
    if (few)
        return launch_dependent(cache_append_kernel<T, 32, FEW>, grid, dim3(kCta), 0, st, g, c, kn, vn, per_row, err);
    if (vecs <= kCta * 4)
        return launch_dependent(cache_append_kernel<T, kCta, 4>, grid, dim3(kCta), 0, st, g, c, kn, vn, per_row, err);
    return launch_dependent(cache_append_kernel<T, kCta, 64 * 128 / N / kCta>, grid, dim3(kCta), 0, st, g, c, kn, vn, per_row, err);
}

}  // namespace

cudaError_t launch_cache_append(const Geo &g, const Cache &c, const void *k, const void *v, int dtype, int *err,
                                cudaStream_t st)
{
    return dtype == NSA_DTYPE_BF16 ? append_t<__nv_bfloat16>(g, c, k, v, err, st) : append_t<float>(g, c, k, v, err, st);
}

}  // namespace nsa
