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
#include <math.h>

#include "cache_common.cuh"
#include "launch.h"

namespace nsa {

namespace {

constexpr int kCta = 128;

// a 16-byte vector of the element type as floats
template <typename T> struct Vec16;
template <> struct Vec16<__nv_bfloat16> {
    static constexpr int N = 8;
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
    static __device__ __forceinline__ void get(const uint4 &w, float (&x)[4])
    {
        x[0] = __uint_as_float(w.x);
        x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z);
        x[3] = __uint_as_float(w.w);
    }
};

// x / s for a scale that is usually a power of two (its reciprocal is then
// exact and a product gives the quotient); a caller's own scale may not be
struct Divide {
    float s, inv;
    bool pow2;
    __device__ __forceinline__ explicit Divide(float scale) : s(scale)
    {
        const uint32_t u = __float_as_uint(scale);
        pow2 = (u & 0x7fffffu) == 0 && (u >> 23) > 1 && (u >> 23) < 253;
        inv = pow2 ? __uint_as_float((254u - (u >> 23)) << 23) : 0.f;
    }
    __device__ __forceinline__ float operator()(float x) const { return pow2 ? x * inv : __fdiv_rn(x, s); }
};

// the new tokens of row b: their count and first position; false where the
// row's length or packed range cannot hold them
__device__ __forceinline__ bool new_tokens(const Geo &g, const Cache &c, int b, int &n, int &start)
{
    const int len = c.lens[b];
    n = seq_len(g, b);
    start = len - n;
    return n >= 0 && n <= g.T && start >= 0 && (int64_t)len <= (int64_t)c.cols * c.bs &&
           (!g.thd || (g.cu[b] >= 0 && g.cu[b + 1] <= g.ntok));
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
        if (!new_tokens(g, c, b, n, start))
            bad = 1;
        else if (n > 0 && start / c.bs + j <= (start + n - 1) / c.bs)
            bad |= !writable(c, c.table[(int64_t)b * c.cols + start / c.bs + j]);
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0)
        *err = bad ? NSA_ERR_BAD_INDEX : NSA_OK;
}

// GROUP threads per (row, touched page, head, k or v); VPT vectors of the
// page's new tokens per thread (VPT * GROUP * N elements cover a page, or
// the call's few new tokens).
template <typename T, int GROUP, int VPT>
__global__ void __launch_bounds__(kCta) cache_append_kernel(const Geo g, const Cache c, const T *kn, const T *vn, int per_row,
                                                            int64_t nunits, int *err)
{
    constexpr int N = Vec16<T>::N;
    __shared__ float red[kCta / 32];
    if (blockIdx.x == gridDim.x - 1) {
        append_check(g, c, per_row, err);
        return;
    }
    const int64_t unit = blockIdx.x * (int64_t)(kCta / GROUP) + threadIdx.x / GROUP;
    const int lane = threadIdx.x % GROUP;
    // unit = ((row * per_row + j) * 2 + which) * Hkv + h
    const bool live = unit < nunits;
    const int h = live ? (int)(unit % c.Hkv) : 0;
    const int64_t u1 = live ? unit / c.Hkv : 0;
    const int which = (int)(u1 & 1);
    const int64_t u2 = u1 >> 1;
    const int j = (int)(u2 % per_row), b = (int)(u2 / per_row);
    int lo = 0, n = 0, page = -1, t0 = 0;  // the page's slots [lo, lo + n) get tokens t0 ..
    if (live) {
        int nn, start;
        if (new_tokens(g, c, b, nn, start)) {
            const int col = start / c.bs + j, first = max(start, col * c.bs), end = min(start + nn, (col + 1) * c.bs);
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
    const T *src = which ? vn : kn;
    uint4 w[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int x = lane + i * GROUP;
        if (x < nvec)
            w[i] = __ldg((const uint4 *)(src + kv_off(g, b, h, t0 + (x >> shift)) + (x & (vec_tok - 1)) * N));
    }
    float *scales = (which ? c.vs : c.ks) + (int64_t)(n > 0 ? page : 0) * c.Hkv + h;
    const float old = lo > 0 && n > 0 ? *scales : 0.f;
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (lane + i * GROUP < nvec) {
            float x[N];
            Vec16<T>::get(w[i], x);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float a = fabsf(x[e]);
                amax = a < INFINITY ? fmaxf(amax, a) : amax;
            }
        }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if constexpr (GROUP > 32) {
        if ((threadIdx.x & 31) == 0)
            red[threadIdx.x / 32] = amax;
        __syncthreads();
        amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    }
    if (n == 0)
        return;
    const float need = e4m3_scale(amax), scale = fmaxf(need, old);
    uint8_t *dst = (which ? c.v : c.k) + (int64_t)page * c.sp + (int64_t)h * c.sh;
    if (lo > 0 && scale != old) {  // the earlier tokens' codes on the larger scale
        const float ratio = __fdiv_rn(old, scale);
        const int per_tok = c.D / 16, sh16 = 31 - __clz(per_tok);
        for (int x = lane; x < lo << sh16; x += GROUP) {
            uint4 *p = (uint4 *)(dst + (int64_t)(x >> sh16) * c.st + (x & (per_tok - 1)) * 16);
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
    const Divide by(scale);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int x = lane + i * GROUP;
        if (x < nvec) {
            float f[N];
            Vec16<T>::get(w[i], f);
            uint32_t u[N / 4];
#pragma unroll
            for (int e = 0; e < N / 4; ++e)
                u[e] = e4m3_pack2(by(f[4 * e]), by(f[4 * e + 1])) | e4m3_pack2(by(f[4 * e + 2]), by(f[4 * e + 3])) << 16;
            uint8_t *p = dst + (int64_t)(lo + (x >> shift)) * c.st + (x & (vec_tok - 1)) * N;
            if constexpr (N == 8)
                *(uint2 *)p = make_uint2(u[0], u[1]);
            else
                *(uint32_t *)p = u[0];
        }
    }
    if (lane == 0)
        *scales = scale;
}

template <typename T> cudaError_t append_t(const Geo &g, const Cache &c, const void *k, const void *v, int *err, cudaStream_t st)
{
    constexpr int N = Vec16<T>::N;
    const int per_row = (g.T + c.bs - 2) / c.bs + 1;
    const int64_t nunits = (int64_t)c.rows * per_row * 2 * c.Hkv;
    // few new tokens per row: a warp per unit, its values in 4 (fp32: 8)
    // vectors per thread; else a block per unit
    constexpr int FEW = sizeof(T) == 2 ? 4 : 8;
    const int vecs = min(g.T, c.bs) * c.D / N;
    const bool few = vecs <= 32 * FEW;
    const int64_t blocks = few ? (nunits + kCta / 32 - 1) / (kCta / 32) : nunits;
    if (blocks + 1 > INT32_MAX)
        return cudaErrorInvalidValue;
    if (few && vecs <= 32)
        cache_append_kernel<T, 32, 1><<<(unsigned)blocks + 1, kCta, 0, st>>>(g, c, (const T *)k, (const T *)v, per_row, nunits, err);
    else if (few)
        cache_append_kernel<T, 32, FEW><<<(unsigned)blocks + 1, kCta, 0, st>>>(g, c, (const T *)k, (const T *)v, per_row, nunits, err);
    else if (vecs <= kCta * 4)
        cache_append_kernel<T, kCta, 4><<<(unsigned)blocks + 1, kCta, 0, st>>>(g, c, (const T *)k, (const T *)v, per_row, nunits, err);
    else
        cache_append_kernel<T, kCta, 64 * 128 / N / kCta>
            <<<(unsigned)blocks + 1, kCta, 0, st>>>(g, c, (const T *)k, (const T *)v, per_row, nunits, err);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const Geo &g, const Cache &c, const void *k, const void *v, int dtype, int *err,
                                cudaStream_t st)
{
    return dtype == NSA_DTYPE_BF16 ? append_t<__nv_bfloat16>(g, c, k, v, err, st) : append_t<float>(g, c, k, v, err, st);
}

}  // namespace nsa
