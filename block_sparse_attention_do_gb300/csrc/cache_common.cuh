// cache_common.cuh -- the paged 8-bit key/value cache on the device: its
// geometry, and the e4m3 conversions that its kernels share.
#pragma once

#include <cuda_fp8.h>

#include "nsa_common.cuh"

namespace nsa {

// Device-side view of an nsa_cache.  A page is one block of bs tokens; the
// codes of (page p, head h, token i of the page) start at p*sp + h*sh + i*st
// bytes (one byte per code), the D codes of a token are contiguous.
struct Cache {
    int pages, Hkv, D, bs, rows, cols;
    int bsh;         // log2 of bs
    int64_t sp, sh, st;
    uint8_t *k, *v;
    float *ks, *vs;  // [pages, Hkv]
    int *table;      // [rows, cols], -1: no page
    int *lens;       // [rows]
    int *ref;        // [pages] (nullptr: the caller keeps no counts)
};

// Workspace of the page operations: header, then three arrays of one int per
// page and two of one int per row.
struct CacheWs {
    int *err;     // nsa_status recorded by the device
    int *npairs;  // pages to copy
    int *p0, *p1, *p2;
    int *r0, *r1;
};

// New tokens and query rows of a kv head of the longest sequence, as far as
// the host knows: the caller's bound may be far above the packed tokens.
inline int longest_tokens(const Geo &g) { return g.thd ? min(g.T, max(g.ntok, 1)) : g.T; }
inline int64_t longest_rows(const Geo &g) { return (int64_t)longest_tokens(g) * g.G; }

// The new tokens (queries; keys and values to append) of sequence b; -1 for a
// packed range that is none or is longer than the problem says: none of its
// rows is read or written.  The offsets may be any ints: they are compared
// before they are subtracted.
__device__ __forceinline__ int new_tokens(const Geo &g, int b)
{
    if (!g.thd)
        return g.T;
    const int from = g.cu[b], to = g.cu[b + 1];
    return from < 0 || to < from || to > g.ntok || to - from > g.T ? -1 : to - from;
}

constexpr float kE4m3Max = 448.f;
constexpr float kScaleFloor = 7.888609052210118e-31f;  // 2^-100: the scale of a block of zeros

// The attention's weights carry their page's value scale, w = p vs; with scales
// within 2^-kNearScale .. 2^kNearScale the sum of p can be had from them, as
// w / vs: a w that has left float's range belongs to a p below 2^-46 of the
// row's largest.  A page outside has its p summed by an exponential of their own.
constexpr float kNearScale = 40.f;

// The cache's kernels run one behind the other in steps of a few microseconds,
// so each is launched as a programmatic dependent: it is set up while the one
// before it ends, and waits here before it reads or writes anything.  What the
// one before may have written is then read by plain loads: to a read-only load
// nothing changes while its kernel runs, and this one runs already.
__device__ __forceinline__ void dependents_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The least power of two s with amax <= 448 s, at least 2^-100 (amax finite,
// >= 0): 448 = 1.75 * 2^8, so with amax = m * 2^e, 1 <= m < 2, s is 2^(e-8)
// for m <= 1.75 and 2^(e-7) above.  A power of two makes x / s exact, so a
// code is x rounded once, and makes a later rescaling exact but for codes
// that fall below e4m3's normal range.
__device__ __forceinline__ float e4m3_scale(float amax)
{
    const uint32_t u = __float_as_uint(fmaxf(amax, kE4m3Max * kScaleFloor));
    const int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)e << 23);
}

// two floats to two codes (lo in the low byte): nearest, ties to even,
// beyond +-448 (infinities too) to +-448; NaN stays NaN
__device__ __forceinline__ uint32_t e4m3_pack2(float lo, float hi)
{
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// four codes to two pairs of halves (lo: bytes 0, 1): exact, e4m3 is a subset
__device__ __forceinline__ void e4m3x4_to_half(uint32_t four, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}

}  // namespace nsa
