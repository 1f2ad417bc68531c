// k_weigh_tc.cu -- k_weigh.cu's sums for many query rows (parts of prompts), on the
// tcgen05 tensor cores; bf16 queries, D = 64 or 128.
//
// The products are taken transposed, S^T[key, row] = K q^T with 128 keys as M and
// 128 query rows as N: a thread of the epilogue holds one key, so its sum over all
// query rows stays in a register, a block's keys are added up once per unit, and
// nothing is joined across CTAs.  Codes are e4m3, a subset of bf16: a unit's keys
// are converted once, exactly, into shared memory, and the queries come as they
// are, by TMA, tile after tile of whole tokens (128 / G of them):
//   8 epilogue warps  the unit's keys to bf16, then, in two sets of 128 threads that
//                     take the tiles in turn, exp2(s * f - z) and its sum: f the
//                     key's scale, z the row's LSE from shared memory
//   1 loading warp    a tile's queries by TMA, its LSEs and positions
//   1 issuing warp    the products, two tiles' columns of tensor memory in turn
// Two CTAs share an SM, so that one's start and end lie under the other's products.
//
// What bounds it: the chain of a unit (table, codes, conversion, products, sums),
// of which two CTAs' lie side by side, and with many tiles a unit an exponential
// for each pair beside 2 D operations.  Measured, D = 128, 8 kv heads of 4: parts of
// prompts, 512 tokens behind 6 rows of up to 8192 at random lengths, 106 us (64.6
// GFLOP of products, 0.61 PFLOP/s; k_weigh.cu 1713); 24 tokens each behind 32 rows
// of 16384, 402 us.  A unit's place in the list takes half a microsecond to find
// (a search, divisions), so that a CTA's are looked up 64 at a time, a thread each:
// found one by one by every warp, the latter took 603.  Tensor memory read 16
// columns ahead of the sums instead of 32 in front of them: 118 and 438 (registers);
// two keys a thread, one CTA an SM: 126; products of 64 query rows, four in turn: 123.
#include <math.h>

#include "cache_common.cuh"
#include "launch.h"
#include "tc_common.cuh"
#include "weigh_common.cuh"

namespace nsa {

using namespace tc;

namespace {

constexpr int kKeysTile = 128, kRowsTile = 128;
constexpr int kEpiWarps = 8, kEpi = kEpiWarps * 32, kThreads = kEpi + 64;
constexpr int kStages = 2, kLseRing = 4, kCtas = 2;
constexpr int kNoRow = 1 << 30;  // the token of a row that is not there
constexpr int kUnits = 64;  // units of a CTA that are looked up together

enum { B_K, B_QF, B_QE = B_QF + kStages, B_SF = B_QE + kStages, B_SE = B_SF + 2, B_END = B_SE + 2, B_COUNT };

struct Params {
    WeighArgs a;
    int tq;       // tokens of a tile of query rows
    int wait_us;  // bounded-wait limit in microseconds (0: the default)
    int stall;    // self-test: the issuing warp stays idle (see wait_test)
};

template <int D> struct Layout {
    static constexpr int kHalves = D / 64, kHalf = 128 * 128, kTile = kHalves * kHalf;  // 128 rows x D
    static constexpr int k = 0, q = kTile;
    static constexpr int z = q + kStages * kTile;                // float [kLseRing][128]: -LSE / ln 2
    static constexpr int pos = z + kLseRing * kRowsTile * 4;     // int [kLseRing][128]: positions
    static constexpr int red = pos + kLseRing * kRowsTile * 4;   // float [2][2][8]
    static constexpr int masked = red + 2 * 2 * 8 * 4;           // int [kLseRing]: a row of the tile attends nothing
    static constexpr int bars = masked + kLseRing * 4;
    static constexpr int misc = bars + B_COUNT * 8;              // wait context, tensor memory address
    static constexpr int prefix = misc + 16;
    static constexpr int units = (prefix + (kWeighMaxRows + 1) * 4 + 15) / 16 * 16;
    static constexpr int total = units + kUnits * 32 + 1024;  // and room to align
};

// true in one lane of the warp, always the same
__device__ __forceinline__ bool elect_one()
{
    uint32_t y;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(y));
    return y != 0;
}

__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kEpi) : "memory"); }

// four codes to four bf16 (exact)
__device__ __forceinline__ void e4m3x4_to_bf16(uint32_t four, uint32_t &lo, uint32_t &hi)
{
    uint32_t a, b;
    e4m3x4_to_half(four, a, b);
    const float2 x = __half22float2(*(const __half2 *)&a), y = __half22float2(*(const __half2 *)&b);
    lo = pack_bf16(x.x, x.y);
    hi = pack_bf16(y.x, y.y);
}

// 16-byte chunk c of row r in a tile of 128-byte rows, 128-byte swizzled
__device__ __forceinline__ uint32_t chunk_at(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// A unit: 128 keys of a row's kv head, and the tiles [t0, t1) of query rows that
// some of them are attended by.
struct alignas(16) WeighUnit {
    int b, kvh, nq, pos0, key0, key_last, t0, t1;  // its new tokens, keys key0 .. key_last, tiles of query rows t0 ..< t1
};
static_assert(sizeof(WeighUnit) == 32, "");

__device__ __forceinline__ WeighUnit unit_at(const Params &p, const int *prefix, int item)
{
    const WeighArgs &a = p.a;
    const Geo &g = a.g;
    WeighUnit u;
    u.b = weigh_row(prefix, g, item);
    const int len = weigh_len(a, u.b);
    u.nq = new_tokens(g, u.b);
    u.pos0 = len - u.nq;
    const int tiles = (len + kKeysTile - 1) / kKeysTile, in = item - prefix[u.b] * g.Hkv;
    u.kvh = in / tiles;
    u.key0 = (in - u.kvh * tiles) * kKeysTile;
    u.key_last = min(u.key0 + kKeysTile, len) - 1;
    u.t0 = max(0, u.key0 - u.pos0) / p.tq;
    u.t1 = (u.nq + p.tq - 1) / p.tq;
    if (g.window > 0)  // tiles whose first token's window reaches the last key
        u.t1 = max(u.t0, min(u.t1, (int)(((int64_t)u.key_last + g.window - u.pos0 + p.tq - 1) / p.tq)));
    return u;
}

template <int D> __global__ void __launch_bounds__(kThreads, kCtas) weigh_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const Params p)
{
    using L = Layout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint64_t *bars = (uint64_t *)(sm + L::bars);
    volatile int *ctx = (volatile int *)(sm + L::misc);
    uint32_t *tmem_slot = (uint32_t *)(sm + L::misc + 8);
    float *zs = (float *)(sm + L::z);
    int *ps = (int *)(sm + L::pos), *masked = (int *)(sm + L::masked);
    int *prefix = (int *)(sm + L::prefix);
    WeighUnit *list = (WeighUnit *)(sm + L::units);
    dependents_may_start();
    dependency_wait();
    const WeighArgs &a = p.a;
    const Geo &g = a.g;
    const Cache &c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int total = weigh_prefix<kThreads>(a, kKeysTile, 0, prefix);
    if ((int)blockIdx.x >= total)
        return;
    if (threadIdx.x == 0) {
        ctx[0] = 0;
        ctx[1] = p.wait_us;
        mbar_init(&bars[B_K], kEpi);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars[B_QF + s], 32);
            mbar_init(&bars[B_QE + s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars[B_SF + s], 1);
            mbar_init(&bars[B_SE + s], kEpi / 2);
        }
        mbar_init(&bars[B_END], 1);
        fence_barrier_init();
    }
    if (warp == kEpiWarps + 1) {
        tmem_alloc(tmem_slot, 256);
        tmem_relinquish();
    }
    // Columns of a tile that are computed; those behind its tokens have no LSE and
    // are products with zeros (so are tokens behind the last of a fixed length, which
    // TMA fills; packed, another sequence's lie there, and they are masked).
    const int used = p.tq * g.G, cols = (used + 31) / 32 * 32;
    for (int i = threadIdx.x; i < kStages * L::kHalves * (cols - used) * 8; i += kThreads) {
        const int tile = i / ((cols - used) * 8), at = i % ((cols - used) * 8);
        *(uint4 *)(sm + L::q + tile * L::kHalf + used * 128 + at * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // n: tiles of all units so far; a tile's stage, columns and ring places go by it
    int n = 0, units = 0, turn = 0;
    bool ok = true;
    for (int first = blockIdx.x; first < total; first += kUnits * gridDim.x) {
        const int count = min(kUnits, (total - first + (int)gridDim.x - 1) / (int)gridDim.x);
        if ((int)threadIdx.x < count)
            list[threadIdx.x] = unit_at(p, prefix, first + threadIdx.x * gridDim.x);
        __syncthreads();
        if (warp < kEpiWarps) {
            const int set = warp >> 2, r = (warp & 3) * 32 + lane;  // the thread's key of a unit
            const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
            // a unit's keys: a thread half a key, its codes under way while the unit before is worked on
            constexpr int VEC = D / 32;  // 16-byte loads of half a key
            const int row = threadIdx.x >> 1, half = threadIdx.x & 1;
            uint4 w[VEC];
            int page_row = -1;
            auto find_page = [&](const WeighUnit &u) { page_row = u.key0 + row <= u.key_last && u.t0 < u.t1 ? c.table[(int64_t)u.b * c.cols + ((u.key0 + row) >> c.bsh)] : -1; };
            auto load_key = [&](const WeighUnit &u) {
                const bool in = page_row >= 0 && page_row < c.pages;
                const uint8_t *from = c.k + (int64_t)(in ? page_row : 0) * c.sp + (int64_t)u.kvh * c.sh + (int64_t)((u.key0 + row) & (c.bs - 1)) * c.st + half * (D / 2);
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    w[i] = in ? ((const uint4 *)from)[i] : make_uint4(0, 0, 0, 0);
            };
            auto weight_of = [&](const WeighUnit &u, int key) { return a.weight + ((int64_t)u.b * c.Hkv + u.kvh) * c.cols + (key >> c.bsh); };
            find_page(list[0]);
            load_key(list[0]);
            if (count > 1)
                find_page(list[1]);
            for (int i = 0; i < count; ++i, turn ^= 1) {
                const WeighUnit u = list[i];
                if (ok && u.t0 < u.t1) {
                    const uint32_t base = smem_u32(sm + L::k) + (D == 128 ? half * L::kHalf : 0);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        uint32_t x[8];
                        e4m3x4_to_bf16(w[i].x, x[0], x[1]);
                        e4m3x4_to_bf16(w[i].y, x[2], x[3]);
                        e4m3x4_to_bf16(w[i].z, x[4], x[5]);
                        e4m3x4_to_bf16(w[i].w, x[6], x[7]);
                        const int ch = (D == 128 ? 0 : half * 4) + 2 * i;
                        st_shared_v4(base + chunk_at(row, ch), x[0], x[1], x[2], x[3]);
                        st_shared_v4(base + chunk_at(row, ch + 1), x[4], x[5], x[6], x[7]);
                    }
                    fence_async_smem();
                    mbar_arrive(&bars[B_K]);
                }
                // ---- the thread's key, and what its block had
                const int key = u.key0 + r;
                bool have = key <= u.key_last;
                float f = 0.f;
                if (have) {
                    const int page = c.table[(int64_t)u.b * c.cols + (key >> c.bsh)];
                    if (page < 0 || page >= c.pages) {
                        have = false;
                        set_error(a.err, NSA_ERR_BAD_INDEX);
                    } else
                        f = c.ks[(int64_t)page * c.Hkv + u.kvh] * g.scale_l2;
                }
                const int k0 = u.key0 + (int)threadIdx.x * c.bs;
                const bool writes = threadIdx.x < kKeysTile / c.bs && k0 <= u.key_last;
                const bool adds = writes && a.decay != 0.f && k0 < u.pos0;
                const float old = adds ? *weight_of(u, k0) : 0.f;
                if (i + 1 < count) {
                    load_key(list[i + 1]);
                    if (i + 2 < count)
                        find_page(list[i + 2]);
                }
                const uint64_t ff = f2(f, f);
                uint64_t sum[2] = {0, 0};
                for (int t = u.t0; t < u.t1; ++t, ++n) {
                    if ((n & 1) != set || !ok)
                        continue;
                    if (!(ok = mbar_wait_warp(&bars[B_SF + set], (n >> 1) & 1, ctx)))
                        continue;
                    tc_fence_after();
                    const int pmin = u.pos0 + t * p.tq, pmax = u.pos0 + min(u.nq, (t + 1) * p.tq) - 1;
                    const bool part = pmin < u.key_last || (g.window > 0 && u.key0 <= pmax - g.window) || (g.thd && (t + 1) * p.tq > u.nq) || masked[n & (kLseRing - 1)];
                    const float *z = zs + (n & (kLseRing - 1)) * kRowsTile;
                    const int *at = ps + (n & (kLseRing - 1)) * kRowsTile;
#pragma unroll 1
                    for (int cc = 0; cc < cols; cc += 32) {
                        uint32_t s[32];
                        tmem_ld32(lanes + set * kRowsTile + cc, s);
                        tmem_wait_ld();
                        if (!part) {
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const ulonglong2 zz = *(const ulonglong2 *)&z[cc + e];
                                float x0, x1, x2, x3;
                                f2_split(f2_fma(f2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), ff, zz.x), x0, x1);
                                f2_split(f2_fma(f2(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), ff, zz.y), x2, x3);
                                sum[0] = f2_add(sum[0], f2(ex2(x0), ex2(x1)));
                                sum[1] = f2_add(sum[1], f2(ex2(x2), ex2(x3)));
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                const float2 zz = *(const float2 *)&z[cc + e];
                                const int2 pp = *(const int2 *)&at[cc + e];
                                float x0 = fmaf(__uint_as_float(s[e]), f, zz.x), x1 = fmaf(__uint_as_float(s[e + 1]), f, zz.y);
                                x0 = key <= pp.x && !(g.window > 0 && key <= pp.x - g.window) ? x0 : -INFINITY;
                                x1 = key <= pp.y && !(g.window > 0 && key <= pp.y - g.window) ? x1 : -INFINITY;
                                sum[e / 2 % 2] = f2_add(sum[e / 2 % 2], f2(ex2(x0), ex2(x1)));
                            }
                        }
                    }
                    tc_fence_before();
                    mbar_arrive(&bars[B_SE + set]);
                }
                // ---- a block's keys together: lanes, then warps and sets in order
                float x0, x1, x;
                f2_split(f2_add(sum[0], sum[1]), x0, x1);
                x = !ok ? __int_as_float(0x7fffffff) : have ? x0 + x1 : 0.f;  // (a wait gave up: NaN)
                const int seg = min(c.bs, 32);
                for (int o = seg / 2; o > 0; o >>= 1)
                    x += __shfl_xor_sync(0xffffffffu, x, o);
                float *red = (float *)(sm + L::red) + turn * 16;
                if ((lane & (seg - 1)) == 0)
                    red[set * 8 + r / seg] = x;
                epilogue_sync();  // (and every product of the unit is done: its keys may be overwritten)
                if (writes) {
                    x = 0.f;
                    for (int i = 0; i < c.bs / seg; ++i)
                        x += red[threadIdx.x * (c.bs / seg) + i] + red[8 + threadIdx.x * (c.bs / seg) + i];
                    *weight_of(u, k0) = adds ? fmaf(a.decay, old, x) : x;
                }
            }
        } else if (warp == kEpiWarps) {
            // ------------------------------------------------- a tile's queries
            int tl[4], hh[4];  // of the lane's rows lane, lane + 32 ..: token of the tile (a far one: no row) and head
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = lane + i * 32;
                tl[i] = g.thd ? r / g.G : r % p.tq;
                hh[i] = g.thd ? r - tl[i] * g.G : r / p.tq;
                if (r >= used)
                    tl[i] = kNoRow, hh[i] = 0;
            }
            const int64_t step = g.thd ? g.Hq : 1;  // a token's in the LSEs
            for (int i = 0; i < count && ok; ++i) {
                const WeighUnit u = list[i];
                const int tok0 = g.thd ? g.cu[u.b] : 0;
                const float *from[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    from[i] = a.lse + stat_off(g, u.b, u.kvh * g.G + hh[i], 0);
                float z[4];
                auto fetch = [&](int t) {  // the rows' LSEs
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tok = t * p.tq + tl[i];
                        z[i] = tok < u.nq ? from[i][tok * step] : -INFINITY;
                    }
                };
                if (u.t0 < u.t1)
                    fetch(u.t0);
                for (int t = u.t0; t < u.t1; ++t, ++n) {
                    const int s = n % kStages;
                    if (!(ok = mbar_wait_warp(&bars[B_QE + s], ((n / kStages) & 1) ^ 1, ctx)))
                        break;
                    // (the tile before last's products are issued, so the ring's place four tiles back has been read)
                    bool none = false;  // an LSE of -inf: the query attends nothing, whatever its scores are
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int at = (n & (kLseRing - 1)) * kRowsTile + lane + i * 32, tok = t * p.tq + tl[i];
                        const bool nothing = z[i] == -INFINITY;
                        zs[at] = nothing ? -INFINITY : -z[i] * 1.4426950408889634f;
                        ps[at] = nothing ? -1 : u.pos0 + tok;
                        none |= nothing && tok < u.nq;
                    }
                    none = __any_sync(0xffffffffu, none);
                    if (lane == 0)
                        masked[n & (kLseRing - 1)] = none;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bars[B_QF + s], (uint32_t)(L::kHalves * used * 128));
                        for (int h = 0; h < L::kHalves; ++h) {
                            uint8_t *dst = sm + L::q + s * L::kTile + h * L::kHalf;
                            if (g.thd)
                                tma_load_3d(dst, &tm_q, &bars[B_QF + s], h * 64, u.kvh * g.G, tok0 + t * p.tq);
                            else
                                tma_load_4d(dst, &tm_q, &bars[B_QF + s], h * 64, t * p.tq, u.kvh * g.G, u.b);
                        }
                    } else
                        mbar_arrive(&bars[B_QF + s]);
                    if (t + 1 < u.t1)
                        fetch(t + 1);
                    __syncwarp();
                }
            }
        } else {
            // --------------------------------------------------------- products
            const uint32_t id = idesc_bf16(128, cols, false, false);
            const uint64_t k_d = sdesc_sw128(smem_u32(sm + L::k), 16, 1024), q_d = sdesc_sw128(smem_u32(sm + L::q), 16, 1024);
            for (int i = 0; i < count && ok && !p.stall; ++i) {
                const WeighUnit u = list[i];
                if (u.t0 >= u.t1)
                    continue;
                ok = mbar_wait_warp(&bars[B_K], units & 1, ctx);
                ++units;
                for (int t = u.t0; t < u.t1 && ok; ++t, ++n) {
                    const int s = n % kStages;
                    ok = mbar_wait_warp(&bars[B_QF + s], (n / kStages) & 1, ctx) && mbar_wait_warp(&bars[B_SE + (n & 1)], ((n >> 1) & 1) ^ 1, ctx);
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint64_t q_s = q_d + (s * L::kTile >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const int at = ((kk >> 2) * L::kHalf + (kk & 3) * 32) >> 4;
                            mma_bf16(tmem + (n & 1) * kRowsTile, k_d + at, q_s + at, id, kk > 0);
                        }
                        mma_commit(&bars[B_QE + s]);
                        mma_commit(&bars[B_SF + (n & 1)]);
                    }
                    __syncwarp();
                }
            }
        }
        __syncthreads();  // the list is read
    }
    volatile int never[2] = {0, ctx[1]};  // own limit, no abort
    if (warp == kEpiWarps) {  // no copy is under way when the CTA ends
        for (int i = max(0, n - kStages); i < n; ++i)
            mbar_wait(&bars[B_QF + i % kStages], (i / kStages) & 1, never);
    } else if (warp == kEpiWarps + 1) {  // every product completes before tensor memory is freed
        if (elect_one())
            mma_commit(&bars[B_END]);
        __syncwarp();
        mbar_wait(&bars[B_END], 0, never);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (ctx[0] && threadIdx.x == 0)
        set_error(a.err, NSA_ERR_DEVICE_TIMEOUT);
    if (warp == kEpiWarps + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

template <int D> cudaError_t weigh_tc_t(const CUtensorMap &tm, const Params &p, cudaStream_t st)
{
    cudaError_t e = allow_shared((const void *)weigh_tc_kernel<D>);
    if (e != cudaSuccess)
        return e;
    return launch_dependent(weigh_tc_kernel<D>, dim3((unsigned)(num_sms() * kCtas)), dim3(kThreads), Layout<D>::total, st, tm, p);
}

}  // namespace

// From where k_weigh.cu needs a second pass over the keys on.  Measured, 8 kv heads of
// 4 query heads of 128, that kernel and this one: 32 sequences of 16384 tokens, 64 query
// rows per kv head 246 and 381 us, 80 rows 366 and 402, 96 rows 415 and 402, 192 rows
// 769 and 540; one sequence of 8192, 64 rows 19 and 15, 80 rows 23 and 15, 128 rows 31
// and 15.
bool cache_weigh_tc_supported(const Geo &g, int dtype)
{
    return dtype == NSA_DTYPE_BF16 && (g.D == 64 || g.D == 128) && g.G <= kRowsTile && longest_rows(g) > 64;
}

cudaError_t launch_cache_weigh_tc(const Geo &g, const Cache &c, const void *q, const float *lse, float decay, float *weight, int *err,
                                  cudaStream_t st)
{
    Params p;
    p.a = {g, c, q, lse, weight, decay, err};
    p.tq = min(kRowsTile / g.G, longest_tokens(g));
    p.wait_us = wait_test().wait_us;
    p.stall = wait_test().kernel == WAIT_TEST_FWD;
    CUtensorMap tm;
    if (!make_tmap(&tm, q, g, g.Hq, p.tq, g.G, g.sq))
        return cudaErrorInvalidValue;
    return g.D == 128 ? weigh_tc_t<128>(tm, p, st) : weigh_tc_t<64>(tm, p, st);
}

}  // namespace nsa
