// k_cache_tc.cu -- attention of many new tokens (chunks of prompts) over the
// paged 8-bit cache on the tcgen05 tensor cores; bf16 queries, D = 64 or 128.
//
// The formulas are those of k_cache_attn.cu (scales of a page's values in the
// exponent, a row's unit raised only when a weight would pass 2^15, the sum
// taken from the scores alone from a page of far values on).  Here
// the products bound the time: 4 D operations per query row and key, so each
// code is converted once for 256 rows and the conversion leaves the critical
// path to warps of its own:
//   2 + 2 converter warps  keys' and values' codes from global memory (a
//                       tile's loads in flight as soon as the one before is
//                       stored) to halves in shared memory, 128 keys x D,
//                       128-byte swizzled
//   2 issuing warps     S_q = Q_q K^T and O_q += P_q V for the tile q = 0, 1
//                       of 128 rows, in turns: one tile's softmax runs under
//                       the other's products
//   2 x 4 softmax warps a row per thread: maximum, exponentials, P as halves
//                       over S's own columns of tensor memory
// Halves hold e4m3 exactly, bf16 queries scaled by a power of two per row
// exactly (but for elements 2^-29 below the row's largest), and P with 11
// bits, three more than bf16.  Tensor memory is full: S 2 x 128 columns, O 2 x D.
//
// Measured: chunks of up to 2048 tokens of 6 sequences over 2048 .. 8192 keys
// (32 query heads on 8, D = 128; 395 GFLOP, masked keys not counted) 321 us,
// 1.23 PFLOP/s, 64% of the measured bf16 rate.  A tile of 128 keys takes 1.5
// us, where its products take 1.0 and its softmax (256 x 128 exponentials, with
// a maximum, a scaling, a sum and a rounding of each) about as long beside
// them; beginning and ending a unit of 256 rows costs some 10 us.  CTAs that
// keep their tensor memory and take several units in turn did not lower that
// (at 1.65 us a tile), and their inner loop no longer fitted its registers
// (1.75).  The sum of the scores alone reads S from tensor memory once more:
// held in registers for it, S cost every tile (345 us), as did a second copy of
// the loop (350) and the same reads ahead of the maximum (368).
#include <math.h>

#include "cache_common.cuh"
#include "tc_common.cuh"

namespace nsa {

using namespace tc;

namespace {

constexpr int kTileKeys = 128;
constexpr int kTileRows = 256;  // query rows of a CTA: two tiles of 128
constexpr int kSoftmaxWarps = 8, kConvWarps = 4;
constexpr int kThreads = (kSoftmaxWarps + kConvWarps + 4) * 32;  // whole warpgroups: the issuing thread's is the last
// Registers per thread of the softmax, converter and issuing warpgroups: a
// row of S (128) stays in registers from its maximum to its exponentials.
// 256 x 176 + 128 x 104 + 128 x 56 = 65,536, all that the launch has.
constexpr int kRegsSoftmax = 176, kRegsConv = 104, kRegsMma = 56;
constexpr int kStages = 2;      // K and V tiles in shared memory
constexpr int kScaleRing = 4;   // tiles whose page scales are kept: softmax lags the converters by up to 3
constexpr float kNoMax = -1e30f, kTop = 15.f, kUp = 5.f;  // a row's weights grow from 2^kUp to 2^kTop before its unit is raised
constexpr float kTiny = 1.17549435e-38f;    // keeps kNoScore * scale from being a NaN
constexpr uint32_t kNoScore = 0xff800000u;  // -infinity

enum { B_Q, B_KF, B_KE = B_KF + kStages, B_VF = B_KE + kStages, B_VE = B_VF + kStages, B_SF = B_VE + kStages, B_P = B_SF + 2, B_TURN = B_P + 4, B_O = B_TURN + 2, B_COUNT };

struct Params {
    Geo g;
    Cache c;
    const __nv_bfloat16 *q;
    const float *sinks;
    __nv_bfloat16 *o;
    float *lse;
    int *err;
    int tiles;    // row tiles of the longest sequence
    int wait_us;  // bounded-wait limit in microseconds (0: the default)
    int stall;    // self-test: the S-product issuers stay idle (see wait_test)
};

template <int D> struct Layout {
    static constexpr int kHalves = D / 64;                 // 128-byte wide column halves
    static constexpr int kHalf = 128 * 128;                // one half of 128 rows
    static constexpr int kTile = kHalves * kHalf;          // 128 rows x D halves
    static constexpr int q = 0, k = 2 * kTile, v = k + kStages * kTile;
    static constexpr int scales = v + kStages * kTile;     // float4 [kScaleRing][8]: k scale, log2 and reciprocal of the v scale, 1 if the tile has one far from 1
    static constexpr int bars = scales + kScaleRing * 8 * 16;
    static constexpr int misc = bars + B_COUNT * 8;        // wait context, tensor memory address, NaN flag
    static constexpr int total = misc + 32 + 1024;         // and room to align
};

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn)
{
    // accumulator f32, A and B f16
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *(const uint32_t *)&h;
}

// true in one lane of the warp, always the same
__device__ __forceinline__ bool elect_one()
{
    uint32_t y;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(y));
    return y != 0;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// 16-byte chunk c of row r in a tile of 128-byte rows, 128-byte swizzled
__device__ __forceinline__ uint32_t chunk_at(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// D and BS, the tokens of a page, are the cache's.
template <int D, int BS> __global__ void __launch_bounds__(kThreads, 1) cache_chunk_kernel(const Params p)
{
    constexpr int PAGES = kTileKeys / BS;
    using L = Layout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint64_t *bars = (uint64_t *)(sm + L::bars);
    volatile int *ctx = (volatile int *)(sm + L::misc);
    uint32_t *tmem_slot = (uint32_t *)(sm + L::misc + 8);
    volatile int *nan_seen = (volatile int *)(sm + L::misc + 16);
    float4 *scales = (float4 *)(sm + L::scales);
    const Geo &g = p.g;
    const Cache &c = p.c;
    dependents_may_start();
    dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // the unit: 256 query rows (row = token * G + head) of one kv head.  Every
    // sequence's last rows, which attend the most keys, come first
    const int nbg = g.B * g.Hkv, bg = blockIdx.x % nbg, from_end = blockIdx.x / nbg;
    const int b = bg / g.Hkv, kvh = bg % g.Hkv;
    const int nq = new_tokens(g, b), cap = c.cols * c.bs, lens = c.lens[b];
    const int len = min(max(lens, 0), cap);
    if (from_end == 0 && kvh == 0 && threadIdx.x == 0 && (lens != len || nq < 0))
        set_error(p.err, NSA_ERR_BAD_INDEX);
    const int tile = nq > 0 ? (nq * g.G + kTileRows - 1) / kTileRows - 1 - from_end : -1;
    if (tile < 0)
        return;
    const int row0 = tile * kTileRows, nrows = min(kTileRows, nq * g.G - row0);
    const int pos0 = len - nq;
    const int pmin = pos0 + row0 / g.G, pmax = pos0 + (row0 + nrows - 1) / g.G;
    const int key_first = g.window > 0 ? max(0, pmin - g.window + 1) : 0;  // of any row
    const int j0 = key_first / kTileKeys, ntiles = pmax < 0 ? 0 : pmax / kTileKeys - j0 + 1;
    // whether some row attends a part of tile j only
    auto masked = [&](int j) {
        return (j + 1) * kTileKeys - 1 > pmin || (g.window > 0 && j * kTileKeys <= pmax - g.window);
    };

    if (threadIdx.x == 0) {
        ctx[0] = 0;
        ctx[1] = p.wait_us;
        *nan_seen = 0;
        mbar_init(&bars[B_Q], 2 * 128);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars[B_KF + s], kConvWarps / 2 * 32);
            mbar_init(&bars[B_VF + s], kConvWarps / 2 * 32);
            mbar_init(&bars[B_KE + s], 2);
            mbar_init(&bars[B_VE + s], 2);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&bars[B_SF + x], 1);
            mbar_init(&bars[B_P + 2 * x], 128);  // tile x, the first half of a tile's keys
            mbar_init(&bars[B_P + 2 * x + 1], 128);
            mbar_init(&bars[B_TURN + x], 1);
        }
        mbar_init(&bars[B_O], 2);
        fence_barrier_init();
    }
    if (warp == kSoftmaxWarps + kConvWarps) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    constexpr uint32_t TM_S = 0, TM_O = 256;  // S_q at q * 128, O_q at 256 + q * 128

    if (warp < kSoftmaxWarps) {
        // ------------------------------------------------- softmax, epilogue
        setmaxnreg_inc<kRegsSoftmax>();
        const int q = warp >> 2, r = (warp & 3) * 32 + lane, row = row0 + q * 128 + r;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const bool have = q * 128 + r < nrows;
        const int t = row / g.G, h = kvh * g.G + row % g.G;
        const int pos = have ? pos0 + t : -1;
        // the thread's row of Q: to halves, its largest element to [2^14, 2^15)
        float qmul;
        {
            const __nv_bfloat16 *src = p.q + (have ? q_off(g, b, h, t) : 0);
            uint4 x[D / 8];
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                x[i] = have ? ((const uint4 *)src)[i] : make_uint4(0, 0, 0, 0);
            uint32_t top = 0;  // largest magnitude's bits
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t lo = u[e] << 16 & 0x7fffffffu, hi = u[e] & 0x7fff0000u;
                    top = max(top, lo <= 0x7f800000u ? lo : 0u);  // (NaN does not count)
                    top = max(top, hi <= 0x7f800000u ? hi : 0u);
                }
            }
            const int be = (int)(top >> 23);
            const int e2 = be == 0 || be == 255 ? 0 : min(max(14 - (be - 127), -120), 120);
            const float up = __uint_as_float((uint32_t)(127 + e2) << 23);
            qmul = g.scale_l2 * __uint_as_float((uint32_t)(127 - e2) << 23);
            const uint32_t base = smem_u32(sm + L::q + q * L::kTile);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = pack_half(__uint_as_float(u[e] << 16) * up, __uint_as_float(u[e] & 0xffff0000u) * up);
                st_shared_v4(base + (i >> 3) * L::kHalf + chunk_at(r, i & 7), w[0], w[1], w[2], w[3]);
            }
            fence_async_smem();
            mbar_arrive(&bars[B_Q]);
        }
        float m = kNoMax, l = 0.f, N = 0.f;
        bool apart = false;  // (uniform over the CTA) l is in units of 2^N, else of 2^m
        bool ok = true;
        for (int i = 0; i < ntiles; ++i) {
            const int j = j0 + i;
            const bool part = masked(j);
            const int cmax = pos - j * kTileKeys, cmin = g.window > 0 ? cmax - g.window + 1 : 0;  // the row's columns
            if (!mbar_wait_warp(&bars[B_SF + q], i & 1, ctx)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const float4 *sc = scales + (i & (kScaleRing - 1)) * 8;
            const uint32_t s_at = lanes + TM_S + q * 128;
            uint32_t s[128];
            tmem_ld64(s_at, *(uint32_t(*)[64])s);
            tmem_ld64(s_at + 64, *(uint32_t(*)[64])(s + 64));
            tmem_wait_ld();
            if (part) {  // columns that the row does not attend count as nothing
#pragma unroll
                for (int e = 0; e < 128; ++e)
                    s[e] = e <= cmax && e >= cmin ? s[e] : kNoScore;
            }
            // ---- the row's maximum, page by page
            float top = -INFINITY;
            float4 f[PAGES];
#pragma unroll
            for (int n = 0; n < PAGES; ++n)
                f[n] = sc[n];
#pragma unroll
            for (int n = 0; n < PAGES; ++n) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[e] = __uint_as_float(s[n * BS + e]);
#pragma unroll
                for (int e = 4; e < BS; e += 2)
                    y[e / 2 % 4] = max3(y[e / 2 % 4], __uint_as_float(s[n * BS + e]), __uint_as_float(s[n * BS + e + 1]));
                f[n].x = fmaxf(f[n].x * qmul, kTiny);
                top = fmaxf(top, fmaf(fmaxf(max3(y[0], y[1], y[2]), y[3]), f[n].x, f[n].y));
            }
            const bool raise = top > m + kTop;  // (no column attended: top is -infinity)
            if (__any_sync(0xffffffffu, raise || apart || f[0].w != 0.f)) {
                if (apart || f[0].w != 0.f) {  // the sum by the scores alone, here and from here on
                    if (!apart)
                        N = m;
                    apart = true;
#pragma unroll 1
                    for (int pass = 0; pass < 2; ++pass) {  // their maximum, then their sum
                        float y = N;
#pragma unroll 1
                        for (int cc = 0; cc < kTileKeys; cc += 16) {  // (of one page)
                            uint32_t a[16];
                            tmem_ld16(s_at + cc, a);
                            tmem_wait_ld();
                            const float4 page = sc[cc / BS];
                            const float mul = fmaxf(page.x * qmul, kTiny);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float x = fmaf(__uint_as_float(a[e]), mul, pass ? -N : 0.f);
                                // (a page that is not in the pool has no keys)
                                if (page.z != 0.f && cc + e <= cmax && cc + e >= cmin) {
                                    if (pass)
                                        l += ex2(x);
                                    else
                                        y = fmaxf(y, x);
                                }
                            }
                        }
                        l *= pass ? 1.f : ex2(N - y);
                        N = y;
                    }
                }
                const float mn = raise ? top - kUp : m, f = ex2(m - mn);
                m = mn;
                l *= apart ? 1.f : f;
                if (i > 0) {  // (S_q of this tile follows P_q V of the last one: O_q is at rest)
#pragma unroll 1
                    for (int cc = 0; cc < D; cc += 16) {
                        uint32_t a[16];
                        tmem_ld16(lanes + TM_O + q * 128 + cc, a);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            a[e] = __float_as_uint(__uint_as_float(a[e]) * f);
                        tmem_st16(lanes + TM_O + q * 128 + cc, a);
                    }
                    tmem_wait_st();
                }
            }
            // ---- weights: P over the columns of S, handed on by halves
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint32_t w[32];
#pragma unroll
                for (int n = 0; n < (PAGES + 1) / 2; ++n) {
                    constexpr int COLS = BS < 64 ? BS : 64;
                    float4 fn = f[hf * (PAGES / 2) + n];
                    if (PAGES > 4) {  // (eight pages' scales would not fit the registers beside S)
                        fn = sc[hf * (PAGES / 2) + n];
                        fn.x = fmaxf(fn.x * qmul, kTiny);
                    }
                    const float add = fn.y - m;
                    const uint64_t mul2 = f2(fn.x, fn.x), add2 = f2(add, add);
                    uint64_t sum[2];
#pragma unroll
                    for (int e = 0; e < COLS; e += 2) {
                        const int k = hf * 64 + n * COLS + e;
                        float x0, x1;
                        f2_split(f2_fma(f2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), mul2, add2), x0, x1);
                        x0 = ex2(x0);
                        x1 = ex2(x1);
                        sum[e / 2 % 2] = e >= 4 ? f2_add(sum[e / 2 % 2], f2(x0, x1)) : f2(x0, x1);
                        w[(n * COLS + e) >> 1] = pack_half(x0, x1);
                    }
                    float a0, a1;
                    f2_split(f2_add(sum[0], sum[1]), a0, a1);
                    l = fmaf(a0 + a1, apart ? 0.f : fn.z, l);
                }
                tmem_st32(s_at + hf * 32, w);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&bars[B_P + q * 2 + hf]);
            }
        }
        // ---- O / l
        if (ok && ntiles > 0)
            ok = mbar_wait_warp(&bars[B_O], 0, ctx);
        if (!ok)  // a wait gave up: NaN in the rows, which are not finished, whether it is reported or not
            l = __int_as_float(0x7fffffff);
        tc_fence_after();
        float f = 1.f;
        if (apart) {  // O from units of 2^m to those of 2^N, N raised by the sum's exponent: O is then a mean of values
            const int e = l > 0.f && l < INFINITY ? (int)(__float_as_uint(l) >> 23) - 127 : 0;
            N += (float)e;
            l *= __uint_as_float((uint32_t)(127 - e) << 23);
            f = exp2f(fminf(m - N, 127.f));
            m = N;
        }
        if (p.sinks && have) {
            const float sk = p.sinks[h] * 1.4426950408889634f, mn = fmaxf(m, sk);
            const float down = ex2(m - mn);
            f *= down;
            l = l * down + ex2(sk - mn);
            m = mn;
        }
        const bool some = l > 0.f || l != l;
        f = some ? f / l : 0.f;
        // values that were NaN in tiles that some rows attend in part
        // were taken as 0 there: put them back for the rows that attend them
        uint32_t nan_dim[D / 32];
#pragma unroll
        for (int x = 0; x < D / 32; ++x)
            nan_dim[x] = 0;
        if (*nan_seen && have) {
#pragma unroll 1
            for (int key = max(key_first, g.window > 0 ? pos - g.window + 1 : 0); key <= pos; ++key) {
                if (!masked(key / kTileKeys)) {
                    key |= kTileKeys - 1;
                    continue;
                }
                const int page = c.table[(int64_t)b * c.cols + (key / BS)];
                if (page < 0 || page >= c.pages)
                    continue;
                const uint8_t *v = c.v + (int64_t)page * c.sp + (int64_t)kvh * c.sh + (int64_t)(key & (BS - 1)) * c.st;
#pragma unroll
                for (int x = 0; x < D / 4; ++x) {
                    const uint32_t u = ((const uint32_t *)v)[x] & 0x7f7f7f7fu, hit = (u + 0x01010101u) & 0x80808080u;
                    // bits 7, 15, 23, 31 to dimensions 4 x ..
                    nan_dim[x / 8] |= ((hit >> 7 & 1u) | (hit >> 14 & 2u) | (hit >> 21 & 4u) | (hit >> 28 & 8u)) << (x % 8 * 4);
                }
            }
        }
        __nv_bfloat16 *dst = p.o + (have ? o_off(g, b, h, t) : 0);
#pragma unroll
        for (int cc = 0; cc < D; cc += 32) {
            uint32_t a[32];
            if (ntiles > 0) {
                tmem_ld32(lanes + TM_O + q * 128 + cc, a);
                tmem_wait_ld();
            }
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float y0 = nan_dim[cc / 32] >> (2 * e) & 1u ? __uint_as_float(0x7fffffffu) : __uint_as_float(a[2 * e]) * f;
                const float y1 = nan_dim[cc / 32] >> (2 * e + 1) & 1u ? __uint_as_float(0x7fffffffu) : __uint_as_float(a[2 * e + 1]) * f;
                w[e] = some && ntiles > 0 ? pack_bf16(y0, y1) : 0u;
            }
            if (have)
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    *(uint4 *)(dst + cc + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
        }
        if (have)
            p.lse[stat_off(g, b, h, t)] = some ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
    } else if (warp < kSoftmaxWarps + kConvWarps) {
        // ------------------------------------------------------- converters
        // Two warps take a tile's keys, two its values: a warp half of the
        // tile's 64 keys, 16 codes per lane and load, and the next tile's are
        // under way as soon as these are stored.  Lane bits 0-1 (and, with D =
        // 128, 4) name the 16 codes, the others the key, so that the 8 lanes
        // of a shared-memory store phase hold two neighbouring keys, whose
        // swizzled chunks lie in different banks.
        setmaxnreg_dec<kRegsConv>();
        constexpr int KEYS = 64, PER_LOAD = D == 128 ? 4 : 8, LOADS = KEYS / PER_LOAD;
        const int cw = warp - kSoftmaxWarps, half = cw & 1;
        const bool values = cw >= 2;
        const int sub = D == 128 ? (lane & 3) | (lane >> 4 & 1) << 2 : lane & 3, key_in = D == 128 ? lane >> 2 & 3 : lane >> 2;
        constexpr int page_sh = BS == 64 ? 6 : BS == 32 ? 5 : 4, npages = PAGES;
        const int st = (int)c.st;
        const uint8_t *pool = (values ? c.v : c.k) + (int64_t)kvh * c.sh + sub * 16;
        const int last_page = pmax >> page_sh, first_page = key_first >> page_sh;
        bool bad = false;
        // page n of the sequence, -1 where no row attends a key of it
        auto page_id = [&](int n) { return n < first_page || n > last_page ? -1 : c.table[(int64_t)b * c.cols + n]; };
        auto in_pool = [&](int id, int n) {
            if (lane < npages && n >= first_page && n <= last_page && (id < 0 || id >= c.pages)) {
                bad = true;
                return -1;
            }
            return id;
        };
        // lane x holds the id of page x of the tile (of the next one: id_next);
        // the warp's keys lie in up to 4 of them
        auto tile_page = [&](int j) { return (j * kTileKeys >> page_sh) + lane; };
        auto fetch_id = [&](int j) { return lane < npages && j < j0 + ntiles ? page_id(tile_page(j)) : -1; };
        uint4 x[LOADS];
        // the warp's codes of tile j; lane n of `id` holds page n of the tile,
        // and 16 keys lie in one page
        auto load = [&](int j, int id) {
            const int first = j * kTileKeys + half * KEYS;
            const uint8_t *at[KEYS / 16];
            bool there[KEYS / 16], all = first >= key_first && first + KEYS - 1 <= pmax;
#pragma unroll
            for (int n = 0; n < KEYS / 16; ++n) {
                const int page = __shfl_sync(0xffffffffu, id, (half * KEYS + n * 16) >> page_sh);
                there[n] = page >= 0;
                all = all && there[n];
                at[n] = pool + (int64_t)page * c.sp + (((first + n * 16) & (BS - 1)) + key_in) * st;
            }
            if (all) {
#pragma unroll
                for (int y = 0; y < LOADS; ++y)
                    x[y] = *(const uint4 *)(at[y * PER_LOAD / 16] + y % (16 / PER_LOAD) * PER_LOAD * st);
            } else {
#pragma unroll
                for (int y = 0; y < LOADS; ++y) {
                    const int key = first + y * PER_LOAD + key_in;
                    x[y] = there[y * PER_LOAD / 16] && key <= pmax && key >= key_first
                               ? *(const uint4 *)(at[y * PER_LOAD / 16] + y % (16 / PER_LOAD) * PER_LOAD * st)
                               : make_uint4(0, 0, 0, 0);
                }
            }
        };
        uint64_t *full = &bars[values ? B_VF : B_KF], *empty = &bars[values ? B_VE : B_KE];
        uint8_t *tiles = sm + (values ? L::v : L::k) + (sub >> 2) * L::kHalf;
        int id = in_pool(fetch_id(j0), tile_page(j0)), id_next = fetch_id(j0 + 1);
        float ks = 0.f, vs = 1.f;
        auto load_scales = [&]() {
            if (cw == 0 && id >= 0) {
                ks = c.ks[(int64_t)id * c.Hkv + kvh];
                vs = c.vs[(int64_t)id * c.Hkv + kvh];
            }
        };
        load(j0, id);
        load_scales();
        for (int i = 0; i < ntiles; ++i) {
            const int j = j0 + i, s = i % kStages;
            // (a page that is not in the pool gets weight 0)
            if (cw == 0) {
                const float vsc = fmaxf(vs, kScaleFloor), lvs = log2f(vsc);
                const bool far = __any_sync(0xffffffffu, id >= 0 && fabsf(lvs) > kNearScale);
                if (lane < npages)
                    scales[(i & (kScaleRing - 1)) * 8 + lane] = id >= 0 ? make_float4(ks, lvs, 1.f / vsc, far ? 1.f : 0.f) : make_float4(1.f, -INFINITY, 0.f, far ? 1.f : 0.f);
            }
            if (values && masked(j)) {
                // a NaN value must not meet the weight 0 of a row that does
                // not attend it: 0 in its place, and the epilogue told
                bool nan = false;
#pragma unroll
                for (int y = 0; y < LOADS; ++y) {
                    uint32_t *u = (uint32_t *)&x[y];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t hit = ((u[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                        nan |= hit != 0;
                        u[e] &= ~((hit >> 7) * 0xffu);
                    }
                }
                if (nan)
                    *nan_seen = 1;
            }
            if (!mbar_wait_warp(&empty[s], ((i / kStages) & 1) ^ 1, ctx))
                break;
            const uint32_t base = smem_u32(tiles + s * L::kTile);
            const int ch = (sub & 3) * 2;
            id = i + 1 < ntiles ? in_pool(id_next, tile_page(j + 1)) : -1;
#pragma unroll
            for (int y = 0; y < LOADS; ++y) {
                const int r = half * KEYS + y * PER_LOAD + key_in;
                uint32_t w[8];
                e4m3x4_to_half(x[y].x, w[0], w[1]);
                e4m3x4_to_half(x[y].y, w[2], w[3]);
                e4m3x4_to_half(x[y].z, w[4], w[5]);
                e4m3x4_to_half(x[y].w, w[6], w[7]);
                st_shared_v4(base + chunk_at(r, ch), w[0], w[1], w[2], w[3]);
                st_shared_v4(base + chunk_at(r, ch + 1), w[4], w[5], w[6], w[7]);
            }
            // (the issuing warp orders these writes for the tensor cores: a
            // proxy fence of every converter costs more)
            mbar_arrive(&full[s]);
            load(j + 1, id);
            load_scales();
            id_next = fetch_id(j + 2);
        }
        if (bad)
            set_error(p.err, NSA_ERR_BAD_INDEX);
    } else {
        setmaxnreg_dec<kRegsMma>();
        const int q = warp - kSoftmaxWarps - kConvWarps;
        if (q < 2) {
            // ---------------------------------------------------------- MMA
            // One warp per tile of rows (one for both, on a scheduler that
            // also runs softmax and converter warps, issues a product only
            // every 100 cycles or so).  The whole warp walks the loop, so that
            // descriptors stay in uniform registers, and one elected lane issues.
            const uint32_t idS = idesc_f16(128, 128, false), idO = idesc_f16(128, D, true);
            const uint64_t q_d = sdesc_sw128(smem_u32(sm + L::q) + q * L::kTile, 16, 1024), k_d = sdesc_sw128(smem_u32(sm + L::k), 16, 1024),
                           v_d = sdesc_sw128(smem_u32(sm + L::v), L::kHalf, 1024);
            const uint32_t tm_s = tmem + TM_S + q * 128, tm_o = tmem + TM_O + q * 128;
            auto product_s = [&](int s) {
                const uint64_t k_s = k_d + (s * L::kTile >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const int at = ((kk >> 2) * L::kHalf + (kk & 3) * 32) >> 4;
                        mma_bf16(tm_s, q_d + at, k_s + at, idS, kk > 0);
                    }
                    mma_commit(&bars[B_SF + q]);
                    mma_commit(&bars[B_KE + s]);
                }
                __syncwarp();
            };
            // The warps take turns: a turn is P_q V and the next S_q, so that
            // one tile's softmax lies under the other's products (left to
            // themselves the two fall into step: 449 us for 389).
            bool ok = !p.stall && ntiles > 0 && mbar_wait_warp(&bars[B_Q], 0, ctx) && mbar_wait_warp(&bars[B_KF], 0, ctx);
            if (ok) {
                fence_async_smem();  // the converters' writes, for the tensor cores
                tc_fence_after();
                product_s(0);
            }
            for (int i = 0; ok && i < ntiles; ++i) {
                const int s = i % kStages, s1 = (i + 1) % kStages;
                const bool more = i + 1 < ntiles;
                ok = mbar_wait_warp(&bars[B_VF + s], (i / kStages) & 1, ctx) &&
                     (!more || mbar_wait_warp(&bars[B_KF + s1], ((i + 1) / kStages) & 1, ctx)) &&
                     mbar_wait_warp(&bars[B_P + q * 2], i & 1, ctx) &&
                     (q == 1 ? mbar_wait_warp(&bars[B_TURN + 1], i & 1, ctx) : i == 0 || mbar_wait_warp(&bars[B_TURN], (i - 1) & 1, ctx));
                if (!ok)
                    break;
                fence_async_smem();
                tc_fence_after();
                const uint64_t v_s = v_d + (s * L::kTile >> 4);
                auto product_o = [&](int hf) {  // 64 keys
                    if (elect_one()) {
#pragma unroll
                        for (int kk = hf * 4; kk < hf * 4 + 4; ++kk)
                            mma_bf16_ts(tm_o, tm_s + kk * 8, v_s + (kk * 2048 >> 4), idO, i > 0 || kk > 0);
                        if (hf == 1)
                            mma_commit(&bars[B_VE + s]);
                    }
                    __syncwarp();
                };
                product_o(0);  // while the softmax takes the second half
                if (!(ok = mbar_wait_warp(&bars[B_P + q * 2 + 1], i & 1, ctx)))
                    break;
                tc_fence_after();
                product_o(1);
                if (more)  // over P_q, once the product that reads it is done: issued behind it
                    product_s(s1);
                if (lane == 0)
                    mbar_arrive(&bars[B_TURN + 1 - q]);
            }
            // every product completes before tensor memory is freed
            if (elect_one())
                mma_commit(&bars[B_O]);
            __syncwarp();
            volatile int never[2] = {0, ctx[1]};  // own limit, no abort
            mbar_wait(&bars[B_O], 0, never);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (ctx[0] && threadIdx.x == 0)
        set_error(p.err, NSA_ERR_DEVICE_TIMEOUT);
    if (warp == kSoftmaxWarps + kConvWarps) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

// Where this kernel takes over from the list's (k_cache_attn.cu), whose time
// goes by 32-row tiles, all SMs together, while a CTA here takes 256 rows by
// itself.  Measured over 4096 cached tokens, 8 kv heads of 4 query heads: 16
// sequences of 5, 8, 16 and 32 tokens (128 .. 512 tiles of 32 rows) 57, 62, 103
// and 184 us by the list, 66, 66, 66 and 67 here; one of 64, 128 and 256 tokens
// 31, 57 and 95 us there, 62 here; 64 sequences of 8 and 16 (2048 cached, four
// rounds of CTAs) 125 and 230 us there, 139 and 140 here.
bool cache_chunk_supported(const Geo &g, int dtype, bool sel)
{
    const int64_t rows = longest_rows(g), seqs = (int64_t)g.B * g.Hkv;
    const int64_t units = (rows + kTileRows - 1) / kTileRows * seqs, tiles32 = (rows + 31) / 32 * seqs;
    return !sel && dtype == NSA_DTYPE_BF16 && (g.D == 64 || g.D == 128) && units < INT32_MAX && rows > 32 &&
           tiles32 > 150 * ((units + num_sms() - 1) / num_sms());
}

cudaError_t launch_cache_chunk(const Geo &g, const Cache &c, const void *q, const float *sinks, void *o, float *lse, int *err,
                               cudaStream_t st)
{
    Params p;
    p.g = g;
    p.c = c;
    p.q = (const __nv_bfloat16 *)q;
    p.sinks = sinks;
    p.o = (__nv_bfloat16 *)o;
    p.lse = lse;
    p.err = err;
    p.tiles = (int)((longest_rows(g) + kTileRows - 1) / kTileRows);
    p.wait_us = wait_test().wait_us;
    p.stall = wait_test().kernel == WAIT_TEST_FWD;
    void (*const kernels[2][3])(const Params) = {{cache_chunk_kernel<64, 16>, cache_chunk_kernel<64, 32>, cache_chunk_kernel<64, 64>},
                                                 {cache_chunk_kernel<128, 16>, cache_chunk_kernel<128, 32>, cache_chunk_kernel<128, 64>}};
    auto kernel = kernels[g.D == 128][c.bsh - 4];
    const int smem = g.D == 128 ? Layout<128>::total : Layout<64>::total;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    return launch_dependent(kernel, dim3((unsigned)(p.tiles * g.B * g.Hkv)), dim3(kThreads), smem, st, p);
}

}  // namespace nsa
