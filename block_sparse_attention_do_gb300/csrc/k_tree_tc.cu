// k_tree_tc.cu -- attention of a tree of drafted tokens over the paged 8-bit cache
// on the tcgen05 tensor cores, for more query rows per kv head than k_tree.cu's
// tiles take; bf16 queries, D = 64 or 128.
//
// The formulas, the roles of the warps and their numbers are k_cache_tc.cu's (two
// tiles of 128 query rows whose products and softmax alternate; converter warps for
// the codes; a row per softmax thread), the mask is k_tree.cu's: a row's line of
// ancestors in shared memory, and 32 columns' bits at a time in tiles with drafts.
// Drafts are few rows over long caches, so the work is shared out differently:
//   - the call's key tiles, of every sequence, kv head and 256 query rows, are one
//     list cut into equal runs, a CTA each; rows whose tiles fall to several CTAs are
//     joined by a second kernel, in the order of the CTAs;
//   - a unit of at most 128 rows has its key tiles taken in turn by both row tiles'
//     pipelines, over the same queries; the two sums are joined in shared memory.
// Weights go to the products as halves there and here, 11 bits, three more than the
// outputs have: these are 1.7e-3 from 64 bits, as they are with weights in 32 bits, and
// 8.5e-4 from those, where a rounding to bf16 falls to the other side.
#include <math.h>

#include "cache_common.cuh"
#include "tc_common.cuh"

namespace nsa {

using namespace tc;

namespace {

constexpr int kTileKeys = 128, kTileRows = 256;
constexpr int kSoftmaxWarps = 8, kConvWarps = 4;
constexpr int kSoftmax = kSoftmaxWarps * 32;
constexpr int kThreads = (kSoftmaxWarps + kConvWarps + 4) * 32;  // whole warpgroups: the issuing warps' is the last
// 256 x 176 + 128 x 104 + 128 x 56 registers = 65,536, all that the launch has
constexpr int kRegsSoftmax = 176, kRegsConv = 104, kRegsMma = 56;
constexpr int kStages = 2;      // K and V tiles in shared memory
constexpr int kScaleRing = 8;   // tiles whose page scales are kept: softmax lags the converters by up to 5
constexpr float kNoMax = -1e30f, kTop = 15.f, kUp = 5.f;  // a row's weights grow from 2^kUp to 2^kTop before its unit is raised
constexpr float kTiny = 1.17549435e-38f;    // keeps kNoScore * scale from being a NaN
constexpr uint32_t kNoScore = 0xff800000u;  // -infinity
constexpr int kAhead = 2;        // tiles of keys and values on their way to L2
constexpr int kMaxSeqs = 1024;  // sequences of a call: the list's prefix sits in shared memory
// The list's entries, half a microsecond each: of a key tile of more than 128 query
// rows, of one of fewer, and what stands for beginning and ending a unit.
constexpr int kWide = 4, kNarrow = 3, kStartCost = 40;
constexpr int kMinRun = 12;      // entries of a run at least
static_assert(kMinRun >= kWide, "every CTA between a unit's first and last has a tile of it");

enum { B_Q, B_KF, B_KE = B_KF + kStages, B_VF = B_KE + kStages, B_VE = B_VF + kStages, B_SF = B_VE + kStages, B_P = B_SF + 2, B_TURN = B_P + 4, B_O = B_TURN + 2, B_OE, B_END = B_OE + 2, B_COUNT };

// The unit that begins in a CTA's run and ends in another's, for the join.
struct Cut {
    int b, kvh, row0, nrows;  // nrows 0: none
    int last;                 // the CTA that has its last key tile
    int pad[3];
};

struct Params {
    Geo g;
    Cache c;
    const __nv_bfloat16 *q;
    const float *sinks;
    const int *parents;  // of the new tokens, [B, T] or [ntok]
    __nv_bfloat16 *o;
    float *lse;
    int *err;
    Cut *cuts;           // [ctas]
    float2 *part_ml;     // [ctas * 2][kTileRows]
    float *part_o;       // [ctas * 2][kTileRows][D]
    int ctas;
    int wait_us;         // bounded-wait limit in microseconds (0: the default)
    int stall;           // self-test: the S-product issuers stay idle (see wait_test)
};

template <int D> struct Layout {
    static constexpr int kHalves = D / 64;                 // 128-byte wide column halves
    static constexpr int kHalf = 128 * 128;                // one half of 128 rows
    static constexpr int kTile = kHalves * kHalf;          // 128 rows x D halves
    static constexpr int q = 0, k = 2 * kTile, v = k + kStages * kTile;  // (q: at a unit's end, float [D][128] of the second sums)
    static constexpr int scales = v + kStages * kTile;     // float4 [kScaleRing][8]: k scale, log2 and reciprocal of the v scale, 1 if the tile has one far from 1
    static constexpr int line = scales + kScaleRing * 8 * 16;           // the rows' lines of ancestors
    static constexpr int parents = line + kTileRows * kTreeWords * 4;
    static constexpr int other = parents + kTreeMax * 4;   // float2 [128]: the second sums' unit and sum
    static constexpr int prefix = other + 128 * 8;
    static constexpr int part = prefix + (kMaxSeqs + 4) * 4;             // the softmax warps' Part
    static constexpr int own = part + 64;                  // int2 [kSoftmax]: a thread's position, and the unit of its sum once that is apart
    static constexpr int bars = own + kSoftmax * 8;
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

__device__ __forceinline__ void prefetch_l2(const void *from, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(bytes) : "memory");
}

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftmax) : "memory"); }

// Which of the 32 columns from draft d0 on (cached tokens: below 0) a row with
// this line of ancestors and `left` cached columns in front of its window attends.
__device__ __forceinline__ uint32_t tree_columns(const uint32_t *line, int d0, int left)
{
    uint32_t cached = 0, drafts = 0;
    if (d0 < 0) {
        cached = d0 <= -32 ? 0xffffffffu : (1u << -d0) - 1u;
        cached &= left >= 32 ? 0u : left > 0 ? 0xffffffffu << left : 0xffffffffu;
    }
    if (d0 > -32 && d0 < kTreeMax)
        drafts = d0 < 0 ? line[0] << -d0 : __funnelshift_r(line[d0 >> 5], line[(d0 >> 5) + 1], d0 & 31);
    return cached | drafts;
}

// A sequence's place in the list: key tiles [j0, j0 + n) (one at least), row tiles.
struct Seq {
    int len, nq, rows, j0, n, tiles, last;  // last: entries a key tile of its last row tile takes (of the others: kWide)
    __device__ __forceinline__ Seq(const Params &p, int b)
    {
        const Cache &c = p.c;
        nq = new_tokens(p.g, b);
        len = min(max(c.lens[b], 0), c.cols * c.bs);
        rows = max(nq, 0) * p.g.G;
        const int64_t first = p.g.window > 0 ? (int64_t)len - nq - p.g.window : 0;  // of the first draft's window
        j0 = first > 0 ? (int)(first / kTileKeys) : 0;
        n = max((len - 1) / kTileKeys - j0 + 1, 1);
        tiles = (rows + kTileRows - 1) / kTileRows;
        last = (rows - 1) % kTileRows < 128 ? kNarrow : kWide;
    }
    __device__ __forceinline__ int unit_cost(int tile) const { return n * (tile == tiles - 1 ? last : kWide) + kStartCost; }
    // entries of one kv head
    __device__ __forceinline__ int cost() const { return rows > 0 ? (tiles - 1) * (kWide * n + kStartCost) + unit_cost(tiles - 1) : 0; }
};

// entries of a run
__device__ __forceinline__ int run_length(int total, int ctas) { return max(kMinRun, (total + ctas - 1) / ctas); }

// What a CTA has of a unit: key tiles [t0, t1) of kv head kvh's row tile.
struct Part {
    int b, kvh, len, nq, pos0, row0, nrows, key_first, j, ntiles;  // j: its first key tile
    int next;             // the list's entry behind it
    int last;             // the CTA that has the unit's last key tile
    bool two, whole, head;  // more than 128 rows; the unit is the CTA's alone; its first key tile is another CTA's
};
__device__ __forceinline__ Part part_at(const Params &p, const int *prefix, int at, int run1, int per)
{
    const Geo &g = p.g;
    Part u;
    int lo = 0, hi = g.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] * g.Hkv <= at)
            lo = mid;
        else
            hi = mid - 1;
    }
    u.b = lo;
    const Seq s(p, lo);
    const int cost = max(s.cost(), 1), in = at - prefix[lo] * g.Hkv;
    u.kvh = in / cost;
    const int tile = min((in - u.kvh * cost) / (kWide * s.n + kStartCost), s.tiles - 1), w = tile == s.tiles - 1 ? s.last : kWide;
    const int begin = prefix[lo] * g.Hkv + u.kvh * cost + tile * (kWide * s.n + kStartCost) + kStartCost, end = begin + s.n * w;
    const int t0 = max(at - begin + w - 1, 0) / w, t1 = (max(min(run1, end) - begin, 0) + w - 1) / w;
    u.len = s.len;
    u.nq = s.nq;
    u.pos0 = s.len - s.nq;
    u.row0 = tile * kTileRows;
    u.nrows = min(kTileRows, s.rows - u.row0);
    u.key_first = g.window > 0 ? max(0, u.pos0 - g.window) : 0;
    u.j = s.j0 + t0;
    u.ntiles = max(t1 - t0, 0);
    u.next = max(at + 1, min(run1, end));
    u.last = (begin + (s.n - 1) * w) / per;
    u.two = w == kWide;
    u.whole = t0 == 0 && t1 == s.n;
    u.head = t0 > 0;
    return u;
}

// whether some row attends a part of key tile j only, as far as the tile's bounds tell
__device__ __forceinline__ bool masked(const Geo &g, int pos0, int len, int j)
{
    return (j + 1) * kTileKeys > pos0 || (g.window > 0 && j * kTileKeys <= len - 1 - g.window);
}

// D and BS, the tokens of a page, are the cache's.
template <int D, int BS> __global__ void __launch_bounds__(kThreads, 1) tree_chunk_kernel(const Params p)
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
    int *prefix = (int *)(sm + L::prefix), *scan = prefix + kMaxSeqs + 1;  // (one more int each)
    const Geo &g = p.g;
    const Cache &c = p.c;
    dependents_may_start();
    dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // ---- the list
    {
        int *sums = (int *)(sm + L::line);  // (not in use yet)
        int base = 0;
        for (int b0 = 0; b0 < g.B; b0 += kThreads) {
            const int b = b0 + (int)threadIdx.x;
            int n = 0;
            if (b < g.B) {
                const Seq s(p, b);
                n = s.cost();
                if (blockIdx.x == 0 && (s.nq < 0 || s.len != c.lens[b]))
                    set_error(p.err, NSA_ERR_BAD_INDEX);
            }
            int incl = n;
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                incl += lane >= o ? y : 0;
            }
            if (lane == 31)
                sums[warp] = incl;
            __syncthreads();
            int before = 0, all = 0;
            for (int k = 0; k < kThreads / 32; ++k) {
                before += k < warp ? sums[k] : 0;
                all += sums[k];
            }
            if (b < g.B)
                prefix[b] = base + before + incl - n;
            base += all;
            __syncthreads();
        }
        if (threadIdx.x == 0) {
            prefix[g.B] = base;
            *scan = base;
        }
    }
    if (threadIdx.x == 0) {
        ctx[0] = 0;
        ctx[1] = p.wait_us;
        *nan_seen = 0;
        mbar_init(&bars[B_Q], kSoftmax);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars[B_KF + s], kConvWarps / 2 * 32);
            mbar_init(&bars[B_VF + s], kConvWarps / 2 * 32);
            mbar_init(&bars[B_KE + s], 2);
            mbar_init(&bars[B_VE + s], 2);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&bars[B_SF + x], 1);
            mbar_init(&bars[B_P + 2 * x], 128);  // pipeline x, the first half of a tile's keys
            mbar_init(&bars[B_P + 2 * x + 1], 128);
            mbar_init(&bars[B_TURN + x], 1);
            mbar_init(&bars[B_OE + x], 128);
        }
        mbar_init(&bars[B_O], 2);
        mbar_init(&bars[B_END], 2);
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
    const int total = *scan * g.Hkv, per = run_length(total, (int)gridDim.x);
    const int run0 = (int)min((int64_t)total, (int64_t)blockIdx.x * per), run1 = (int)min((int64_t)total, (int64_t)(blockIdx.x + 1) * per);
    // a part's tiles are counted on from those before it: stages and phases go by that
    int base = 0, part = 0;

    if (warp < kSoftmaxWarps) {
        // ------------------------------------------------- softmax, epilogue
        setmaxnreg_inc<kRegsSoftmax>();
        const int q = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        uint32_t *line = (uint32_t *)(sm + L::line) + threadIdx.x * kTreeWords;
        int *parents = (int *)(sm + L::parents);
        volatile int *pos = (volatile int *)(sm + L::own) + 2 * threadIdx.x;
        volatile float *N = (volatile float *)(pos + 1);
        bool ok = true;
        int mine = 0;  // the pipeline's tiles so far
        // the part lies in shared memory: what the loop over its tiles does not need takes no registers there
        static_assert(sizeof(Part) <= 64, "");
        Part &u = *(Part *)(sm + L::part);
        if (threadIdx.x == 0)
            p.cuts[blockIdx.x].nrows = 0;
        for (int at = run0; at < run1;) {
            softmax_sync();  // the part before is done with shared memory
            if (threadIdx.x == 0) {
                u = part_at(p, prefix, at, run1, per);
                if (u.ntiles > 0 && !u.whole && !u.head)
                    p.cuts[blockIdx.x] = Cut{u.b, u.kvh, u.row0, u.nrows, u.last, {0, 0, 0}};
            }
            softmax_sync();
            at = u.next;
            const int ntiles = u.ntiles, j_first = u.j, pos0 = u.pos0;
            if (ntiles == 0)
                continue;
            // (no row: tokens and heads of the first)
            auto in_tile_of = [&]() { return (u.two ? q * 128 : 0) + r; };
            auto token_of = [&](int in_tile, int &h) {
                const int row = in_tile < u.nrows ? u.row0 + in_tile : u.row0, t = row / g.G;
                h = u.kvh * g.G + row - t * g.G;
                return t;
            };
            // The queries to halves, each row's largest element to [2^14, 2^15): a row's
            // 16-byte pieces by neighbouring lanes, all loads of a warp's 32 rows under way
            // together (a row by its own thread would take five times as long)
            float qmul;
            {
                constexpr int PIECES = D / 8, ROWS = 32 / PIECES, STEPS = 32 / ROWS;  // of a row; rows of a load; loads
                const int in_tile = in_tile_of();
                int h;
                const int t = token_of(in_tile, h);
                const int64_t mine_at = in_tile < u.nrows ? q_off(g, u.b, h, t) : -1;
                uint4 x[STEPS];
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    const int64_t at_row = __shfl_sync(0xffffffffu, mine_at, i * ROWS + lane / PIECES);
                    x[i] = at_row >= 0 ? *(const uint4 *)(p.q + at_row + lane % PIECES * 8) : make_uint4(0, 0, 0, 0);
                }
                if ((int)threadIdx.x < u.nq)
                    parents[threadIdx.x] = p.parents[tree_at(g, u.b) + threadIdx.x];
                const uint32_t to = smem_u32(sm + L::q + q * L::kTile) + (lane % PIECES >> 3) * L::kHalf;
                qmul = 0.f;
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                    uint32_t top = 0;  // largest magnitude's bits
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t lo = w[e] << 16 & 0x7fffffffu, hi = w[e] & 0x7fff0000u;
                        top = max(top, lo <= 0x7f800000u ? lo : 0u);  // (NaN does not count)
                        top = max(top, hi <= 0x7f800000u ? hi : 0u);
                    }
#pragma unroll
                    for (int o = PIECES / 2; o > 0; o >>= 1)
                        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    const int be = (int)(top >> 23);
                    const int e2 = be == 0 || be == 255 ? 0 : min(max(14 - (be - 127), -120), 120);
                    const float up = __uint_as_float((uint32_t)(127 + e2) << 23);
                    // (row i * ROWS + k's thread is lane i * ROWS + k)
                    const int of_row = __shfl_sync(0xffffffffu, e2, lane % ROWS * PIECES);
                    if (lane / ROWS == i)
                        qmul = g.scale_l2 * __uint_as_float((uint32_t)(127 - of_row) << 23);
                    if (u.two || q == 0) {  // (128 rows: both pipelines read the first tile)
                        uint32_t y[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            y[e] = pack_half(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xffff0000u) * up);
                        st_shared_v4(to + chunk_at((warp & 3) * 32 + i * ROWS + lane / PIECES, lane % PIECES & 7), y[0], y[1], y[2], y[3]);
                    }
                }
                fence_async_smem();
                mbar_arrive(&bars[B_Q]);
                softmax_sync();  // the parents are there
                bool bad = false;
                *pos = pos0 + tree_line(parents, t, g.window, line, bad);
                if (bad)
                    set_error(p.err, NSA_ERR_BAD_INDEX);
            }
            float m = kNoMax, l = 0.f;
            bool apart = false;  // (uniform over the pipeline's threads) l is in units of 2^N, else of 2^m
            bool first = true;
            const int step = u.two ? 1 : 2;
            for (int i = step == 1 ? 0 : q; i < ntiles && ok; i += step) {
                const int j = j_first + i;
                if (!mbar_wait_warp(&bars[B_SF + q], mine & 1, ctx)) {
                    ok = false;
                    break;
                }
                ++mine;
                tc_fence_after();
                const float4 *sc = scales + ((base + i) & (kScaleRing - 1)) * 8;
                const uint32_t s_at = lanes + TM_S + q * 128;
                uint32_t s[128];
                tmem_ld64(s_at, *(uint32_t(*)[64])s);
                tmem_ld64(s_at + 64, *(uint32_t(*)[64])(s + 64));
                tmem_wait_ld();
                if ((j + 1) * kTileKeys > pos0 || g.window > 0) {  // columns that the row does not attend count as nothing
                    const int cmin = g.window > 0 ? *pos - g.window + 1 - j * kTileKeys : 0;  // of the cached columns
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t seen = tree_columns(line, j * kTileKeys + w * 32 - pos0, cmin - w * 32);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            s[w * 32 + e] = seen >> e & 1u ? s[w * 32 + e] : kNoScore;
                    }
                }
                // ---- the row's maximum, page by page
                float top = -INFINITY;
                float far = 0.f;
#pragma unroll
                for (int n = 0; n < PAGES; ++n) {
                    const float4 f = sc[n];
                    far = n == 0 ? f.w : far;
                    float y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[e] = __uint_as_float(s[n * BS + e]);
#pragma unroll
                    for (int e = 4; e < BS; e += 2)
                        y[e / 2 % 4] = max3(y[e / 2 % 4], __uint_as_float(s[n * BS + e]), __uint_as_float(s[n * BS + e + 1]));
                    top = fmaxf(top, fmaf(fmaxf(max3(y[0], y[1], y[2]), y[3]), fmaxf(f.x * qmul, kTiny), f.y));
                }
                const bool raise = top > m + kTop;  // (no column attended: top is -infinity)
                if (__any_sync(0xffffffffu, raise || apart || far != 0.f)) {
                    if (apart || far != 0.f) {  // the sum by the scores alone, here and from here on
                        if (!apart)
                            *N = m;
                        apart = true;
                        const int cmin = g.window > 0 ? *pos - g.window + 1 - j * kTileKeys : 0;
#pragma unroll 1
                        for (int pass = 0; pass < 2; ++pass) {  // their maximum, then their sum
                            float y = *N;
                            const float unit = y;
#pragma unroll 1
                            for (int cc = 0; cc < kTileKeys; cc += 16) {  // (of one page)
                                uint32_t a[16];
                                tmem_ld16(s_at + cc, a);
                                tmem_wait_ld();
                                const float4 page = sc[cc / BS];
                                const float mul = fmaxf(page.x * qmul, kTiny);
                                const uint32_t seen = tree_columns(line, j * kTileKeys + cc - pos0, cmin - cc);
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    const float x = fmaf(__uint_as_float(a[e]), mul, pass ? -unit : 0.f);
                                    // (a page that is not in the pool has no keys)
                                    if (page.z != 0.f && (seen >> e & 1u)) {
                                        if (pass)
                                            l += ex2(x);
                                        else
                                            y = fmaxf(y, x);
                                    }
                                }
                            }
                            l *= pass ? 1.f : ex2(unit - y);
                            *N = y;
                        }
                    }
                    const float mn = raise ? top - kUp : m, down = ex2(m - mn);
                    m = mn;
                    l *= apart ? 1.f : down;
                    if (!first) {  // (S_q of this tile follows P_q V of the last one: O_q is at rest)
#pragma unroll 1
                        for (int cc = 0; cc < D; cc += 16) {
                            uint32_t a[16];
                            tmem_ld16(lanes + TM_O + q * 128 + cc, a);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                a[e] = __float_as_uint(__uint_as_float(a[e]) * down);
                            tmem_st16(lanes + TM_O + q * 128 + cc, a);
                        }
                        tmem_wait_st();
                    }
                }
                first = false;
                // ---- weights: P over the columns of S, handed on by halves
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    uint32_t w[32];
#pragma unroll
                    for (int n = 0; n < (PAGES + 1) / 2; ++n) {
                        constexpr int COLS = BS < 64 ? BS : 64;
                        float4 fn = sc[hf * (PAGES / 2) + n];  // (once more: kept, they would not fit the registers beside S)
                        fn.x = fmaxf(fn.x * qmul, kTiny);
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
            if (ok)
                ok = mbar_wait_warp(&bars[B_O], part & 1, ctx);
            if (!ok)  // a wait gave up: NaN in the rows, which are not finished, whether it is reported or not
                l = __int_as_float(0x7fffffff);
            tc_fence_after();
            float f = first ? 0.f : 1.f;  // (no tile: O_q holds nothing)
            if (apart) {  // O from units of 2^m to those of 2^N, N raised by the sum's exponent: O is then a mean of values
                const int e = l > 0.f && l < INFINITY ? (int)(__float_as_uint(l) >> 23) - 127 : 0;
                const float unit = *N + (float)e;
                l *= __uint_as_float((uint32_t)(127 - e) << 23);
                f = exp2f(fminf(m - unit, 127.f));
                m = unit;
            }
            float *second = (float *)(sm + L::q);  // (every product is done: Q is used up)
            float2 *second_ml = (float2 *)(sm + L::other);
            float f1 = 0.f;
            if (!u.two) {  // the second pipeline's sums go to the first's threads
                if (q == 1) {
                    second_ml[r] = make_float2(m, l);
#pragma unroll
                    for (int cc = 0; cc < D; cc += 32) {
                        uint32_t a[32];
                        tmem_ld32(lanes + TM_O + 128 + cc, a);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            second[(cc + e) * 128 + r] = first ? 0.f : __uint_as_float(a[e]) * f;
                    }
                }
                softmax_sync();
                if (q == 0) {
                    const float2 o1 = second_ml[r];
                    const float mn = fmaxf(m, o1.x), down = ex2(m - mn);
                    f1 = ex2(o1.x - mn);
                    l = l * down + o1.y * f1;
                    f *= down;
                    m = mn;
                }
            }
            if (u.two || q == 0) {
                const int in_tile = in_tile_of();
                const bool have = in_tile < u.nrows;
                int h;
                const int t = token_of(in_tile, h);
                if (u.whole && p.sinks) {
                    const float sk = p.sinks[h] * 1.4426950408889634f, mn = fmaxf(m, sk);
                    const float down = ex2(m - mn);
                    f *= down;
                    f1 *= down;
                    l = l * down + ex2(sk - mn);
                    m = mn;
                }
                const bool some = l > 0.f || l != l;
                if (u.whole) {
                    f = some ? f / l : 0.f;
                    f1 = some ? f1 / l : 0.f;
                }
                // values that were NaN in tiles that some rows attend in part
                // were taken as 0 there: put them back for the rows that attend them
                uint32_t nan_dim[D / 32];
#pragma unroll
                for (int x = 0; x < D / 32; ++x)
                    nan_dim[x] = 0;
                if (*nan_seen && have) {
                    const int key_end = min(u.len, (j_first + ntiles) * kTileKeys);
#pragma unroll 1
                    for (int key = max(u.key_first, j_first * kTileKeys); key < key_end; ++key) {
                        if (!masked(g, pos0, u.len, key / kTileKeys)) {
                            key |= kTileKeys - 1;
                            continue;
                        }
                        const int draft = key - pos0;
                        if (draft >= 0 ? draft >= kTreeMax || !(line[draft >> 5] >> (draft & 31) & 1u) : g.window > 0 && key <= *pos - g.window)
                            continue;
                        const int page = c.table[(int64_t)u.b * c.cols + (key / BS)];
                        if (page < 0 || page >= c.pages)
                            continue;
                        const uint8_t *v = c.v + (int64_t)page * c.sp + (int64_t)u.kvh * c.sh + (int64_t)(key & (BS - 1)) * c.st;
#pragma unroll
                        for (int x = 0; x < D / 4; ++x) {
                            const uint32_t w = ((const uint32_t *)v)[x] & 0x7f7f7f7fu, hit = (w + 0x01010101u) & 0x80808080u;
                            // bits 7, 15, 23, 31 to dimensions 4 x ..
                            nan_dim[x / 8] |= ((hit >> 7 & 1u) | (hit >> 14 & 2u) | (hit >> 21 & 4u) | (hit >> 28 & 8u)) << (x % 8 * 4);
                        }
                    }
                }
                const int64_t slot = (int64_t)blockIdx.x * 2 + (u.head ? 0 : 1);
                __nv_bfloat16 *dst = p.o + o_off(g, u.b, h, t);
                float *part_o = p.part_o + (slot * kTileRows + in_tile) * D;
#pragma unroll
                for (int cc = 0; cc < D; cc += 32) {
                    uint32_t a[32];
                    tmem_ld32(lanes + TM_O + q * 128 + cc, a);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float y = f != 0.f ? __uint_as_float(a[e]) * f : 0.f;
                        if (!u.two && f1 != 0.f)
                            y = fmaf(second[(cc + e) * 128 + r], f1, y);
                        a[e] = nan_dim[cc / 32] >> e & 1u || !ok ? 0x7fffffffu : __float_as_uint(y);
                    }
                    if (have && u.whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            *(uint4 *)(dst + cc + e) = make_uint4(pack_bf16(__uint_as_float(a[e]), __uint_as_float(a[e + 1])), pack_bf16(__uint_as_float(a[e + 2]), __uint_as_float(a[e + 3])),
                                                                  pack_bf16(__uint_as_float(a[e + 4]), __uint_as_float(a[e + 5])), pack_bf16(__uint_as_float(a[e + 6]), __uint_as_float(a[e + 7])));
                    } else if (have) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            st_global_v8(part_o + cc + e, a + e);
                    }
                }
                if (have && u.whole)
                    p.lse[stat_off(g, u.b, h, t)] = some ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
                else if (have)
                    p.part_ml[slot * kTileRows + in_tile] = make_float2(m, l);
            }
            tc_fence_before();
            mbar_arrive(&bars[B_OE + q]);
            base += ntiles;
            ++part;
        }
    } else if (warp < kSoftmaxWarps + kConvWarps) {
        // ------------------------------------------------------- converters
        // Two warps take a tile's keys, two its values, as in k_cache_tc.cu.
        setmaxnreg_dec<kRegsConv>();
        constexpr int KEYS = 64, PER_LOAD = D == 128 ? 4 : 8, LOADS = KEYS / PER_LOAD;
        const int cw = warp - kSoftmaxWarps, half = cw & 1;
        const bool values = cw >= 2;
        const int sub = D == 128 ? (lane & 3) | (lane >> 4 & 1) << 2 : lane & 3, key_in = D == 128 ? lane >> 2 & 3 : lane >> 2;
        constexpr int page_sh = BS == 64 ? 6 : BS == 32 ? 5 : 4, npages = PAGES;
        const int st = (int)c.st;
        uint64_t *full = &bars[values ? B_VF : B_KF], *empty = &bars[values ? B_VE : B_KE];
        uint8_t *tiles = sm + (values ? L::v : L::k) + (sub >> 2) * L::kHalf;
        bool bad = false, ok = true;
        for (int at = run0; at < run1 && ok;) {
            const Part u = part_at(p, prefix, at, run1, per);
            at = u.next;
            if (u.ntiles == 0)
                continue;
            const uint8_t *pool = (values ? c.v : c.k) + (int64_t)u.kvh * c.sh + sub * 16;
            const int pmax = u.len - 1, last_page = pmax >> page_sh, first_page = u.key_first >> page_sh, j_end = u.j + u.ntiles;
            // page n of the sequence, -1 where no row attends a key of it
            auto page_id = [&](int n) { return n < first_page || n > last_page ? -1 : c.table[(int64_t)u.b * c.cols + n]; };
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
            auto fetch_id = [&](int j) { return lane < npages && j < j_end ? page_id(tile_page(j)) : -1; };
            uint4 x[LOADS];
            // the warp's codes of tile j; lane n of `id` holds page n of the tile,
            // and 16 keys lie in one page
            auto load = [&](int j, int id) {
                const int first = j * kTileKeys + half * KEYS;
                const uint8_t *from[KEYS / 16];
                bool there[KEYS / 16], all = first >= u.key_first && first + KEYS - 1 <= pmax;
#pragma unroll
                for (int n = 0; n < KEYS / 16; ++n) {
                    const int page = __shfl_sync(0xffffffffu, id, (half * KEYS + n * 16) >> page_sh);
                    there[n] = page >= 0;
                    all = all && there[n];
                    from[n] = pool + (int64_t)page * c.sp + (((first + n * 16) & (BS - 1)) + key_in) * st;
                }
                if (all) {
#pragma unroll
                    for (int y = 0; y < LOADS; ++y)
                        x[y] = *(const uint4 *)(from[y * PER_LOAD / 16] + y % (16 / PER_LOAD) * PER_LOAD * st);
                } else {
#pragma unroll
                    for (int y = 0; y < LOADS; ++y) {
                        const int key = first + y * PER_LOAD + key_in;
                        x[y] = there[y * PER_LOAD / 16] && key <= pmax && key >= u.key_first
                                   ? *(const uint4 *)(from[y * PER_LOAD / 16] + y % (16 / PER_LOAD) * PER_LOAD * st)
                                   : make_uint4(0, 0, 0, 0);
                    }
                }
            };
            // A warp's registers hold one tile's loads, less than the memory's latency asks for, and
            // unlike prompts' keys these are read once: pages kAhead tiles on are
            // brought to L2, by the warps that take a tile's first half
            auto prefetch = [&](int id) {
                if (half == 0 && lane < npages && id >= 0 && id < c.pages && st == D)
                    prefetch_l2((values ? c.v : c.k) + (int64_t)id * c.sp + (int64_t)u.kvh * c.sh, BS * D);
            };
            int id = in_pool(fetch_id(u.j), tile_page(u.j)), id_next = fetch_id(u.j + 1);
            {
                int far[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    far[i] = fetch_id(u.j + 1 + i);
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    prefetch(far[i]);
            }
            int id_far = fetch_id(u.j + 1 + kAhead);
            float ks = 0.f, vs = 1.f;
            auto load_scales = [&]() {
                if (cw == 0 && id >= 0) {
                    ks = c.ks[(int64_t)id * c.Hkv + u.kvh];
                    vs = c.vs[(int64_t)id * c.Hkv + u.kvh];
                }
            };
            load(u.j, id);
            load_scales();
            for (int i = 0; i < u.ntiles; ++i) {
                const int j = u.j + i, n = base + i, s = n % kStages;
                // (a page that is not in the pool gets weight 0)
                if (cw == 0) {
                    const float vsc = fmaxf(vs, kScaleFloor), lvs = log2f(vsc);
                    const bool far = __any_sync(0xffffffffu, id >= 0 && fabsf(lvs) > kNearScale);
                    if (lane < npages)
                        scales[(n & (kScaleRing - 1)) * 8 + lane] = id >= 0 ? make_float4(ks, lvs, 1.f / vsc, far ? 1.f : 0.f) : make_float4(1.f, -INFINITY, 0.f, far ? 1.f : 0.f);
                }
                if (values && masked(g, u.pos0, u.len, j)) {
                    // a NaN value must not meet the weight 0 of a row that does
                    // not attend it: 0 in its place, and the epilogue told
                    bool nan = false;
#pragma unroll
                    for (int y = 0; y < LOADS; ++y) {
                        uint32_t *w = (uint32_t *)&x[y];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t hit = ((w[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                            nan |= hit != 0;
                            w[e] &= ~((hit >> 7) * 0xffu);
                        }
                    }
                    if (nan)
                        *nan_seen = 1;
                }
                if (!(ok = mbar_wait_warp(&empty[s], ((n / kStages) & 1) ^ 1, ctx)))
                    break;
                const uint32_t to = smem_u32(tiles + s * L::kTile);
                const int ch = (sub & 3) * 2;
                id = i + 1 < u.ntiles ? in_pool(id_next, tile_page(j + 1)) : -1;
#pragma unroll
                for (int y = 0; y < LOADS; ++y) {
                    const int r = half * KEYS + y * PER_LOAD + key_in;
                    uint32_t w[8];
                    e4m3x4_to_half(x[y].x, w[0], w[1]);
                    e4m3x4_to_half(x[y].y, w[2], w[3]);
                    e4m3x4_to_half(x[y].z, w[4], w[5]);
                    e4m3x4_to_half(x[y].w, w[6], w[7]);
                    st_shared_v4(to + chunk_at(r, ch), w[0], w[1], w[2], w[3]);
                    st_shared_v4(to + chunk_at(r, ch + 1), w[4], w[5], w[6], w[7]);
                }
                // (the issuing warp orders these writes for the tensor cores: a
                // proxy fence of every converter costs more)
                mbar_arrive(&full[s]);
                prefetch(id_far);
                id_far = fetch_id(j + 2 + kAhead);
                load(j + 1, id);
                load_scales();
                id_next = fetch_id(j + 2);
            }
            base += u.ntiles;
        }
        if (bad)
            set_error(p.err, NSA_ERR_BAD_INDEX);
    } else {
        setmaxnreg_dec<kRegsMma>();
        const int q = warp - kSoftmaxWarps - kConvWarps;
        if (q < 2) {
            // ---------------------------------------------------------- MMA
            // A warp for each pipeline, as in k_cache_tc.cu.
            const uint32_t idS = idesc_f16(128, 128, false), idO = idesc_f16(128, D, true);
            const uint64_t q0_d = sdesc_sw128(smem_u32(sm + L::q), 16, 1024), k_d = sdesc_sw128(smem_u32(sm + L::k), 16, 1024),
                           v_d = sdesc_sw128(smem_u32(sm + L::v), L::kHalf, 1024);
            const uint32_t tm_s = tmem + TM_S + q * 128, tm_o = tmem + TM_O + q * 128;
            int mine = 0, turns = 0;  // the pipeline's tiles, and the turns it waited for, so far
            bool ok = !p.stall;
            for (int at = run0; at < run1 && ok;) {
                const Part u = part_at(p, prefix, at, run1, per);
                at = u.next;
                if (u.ntiles == 0)
                    continue;
                const uint64_t q_d = q0_d + (u.two ? q * L::kTile >> 4 : 0);
                const int step = u.two ? 1 : 2, i0 = u.two ? 0 : q;
                auto product_s = [&](int s) {
                    const uint64_t k_s = k_d + (s * L::kTile >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const int to = ((kk >> 2) * L::kHalf + (kk & 3) * 32) >> 4;
                            mma_bf16(tm_s, q_d + to, k_s + to, idS, kk > 0);
                        }
                        mma_commit(&bars[B_SF + q]);
                        mma_commit(&bars[B_KE + s]);
                        if (!u.two)  // (the other pipeline does not read this tile)
                            mma_commit(&bars[B_KE + s]);
                    }
                    __syncwarp();
                };
                // The warps take turns: a turn is P_q V and the next S_q, so that
                // one's softmax lies under the other's products.
                ok = mbar_wait_warp(&bars[B_Q], part & 1, ctx) && (part == 0 || mbar_wait_warp(&bars[B_OE + q], (part - 1) & 1, ctx)) &&
                     (i0 >= u.ntiles || mbar_wait_warp(&bars[B_KF + (base + i0) % kStages], ((base + i0) / kStages) & 1, ctx));
                if (ok && i0 < u.ntiles) {
                    fence_async_smem();  // the converters' writes, for the tensor cores
                    tc_fence_after();
                    product_s((base + i0) % kStages);
                }
                for (int i = i0; ok && i < u.ntiles; i += step) {
                    const int n = base + i, s = n % kStages, n1 = n + step, s1 = n1 % kStages;
                    const bool more = i + step < u.ntiles;
                    // the first pipeline's first tile of a part waits for no turn
                    const bool turn = q == 1 || i > 0;
                    ok = mbar_wait_warp(&bars[B_VF + s], (n / kStages) & 1, ctx) &&
                         (!more || mbar_wait_warp(&bars[B_KF + s1], (n1 / kStages) & 1, ctx)) && mbar_wait_warp(&bars[B_P + q * 2], mine & 1, ctx) &&
                         (!turn || mbar_wait_warp(&bars[B_TURN + q], turns & 1, ctx));
                    if (!ok)
                        break;
                    turns += turn;
                    fence_async_smem();
                    tc_fence_after();
                    const uint64_t v_s = v_d + (s * L::kTile >> 4);
                    auto product_o = [&](int hf) {  // 64 keys
                        if (elect_one()) {
#pragma unroll
                            for (int kk = hf * 4; kk < hf * 4 + 4; ++kk)
                                mma_bf16_ts(tm_o, tm_s + kk * 8, v_s + (kk * 2048 >> 4), idO, i > i0 || kk > 0);
                            if (hf == 1) {
                                mma_commit(&bars[B_VE + s]);
                                if (!u.two)
                                    mma_commit(&bars[B_VE + s]);
                            }
                        }
                        __syncwarp();
                    };
                    product_o(0);  // while the softmax takes the second half
                    if (!(ok = mbar_wait_warp(&bars[B_P + q * 2 + 1], mine & 1, ctx)))
                        break;
                    ++mine;
                    tc_fence_after();
                    product_o(1);
                    if (more)  // over P_q, once the product that reads it is done: issued behind it
                        product_s(s1);
                    // the other pipeline's turn, if it has a tile for it: of the first one's k-th tile the second one's
                    // k-th, of that the first one's next
                    const int theirs = u.two ? (q == 0 ? i : i + 1) : i + 1;
                    if (theirs < u.ntiles && lane == 0)
                        mbar_arrive(&bars[B_TURN + 1 - q]);
                    __syncwarp();
                }
                if (ok) {
                    if (elect_one())
                        mma_commit(&bars[B_O]);
                    __syncwarp();
                }
                base += u.ntiles;
                ++part;
            }
            // every product completes before tensor memory is freed
            if (elect_one())
                mma_commit(&bars[B_END]);
            __syncwarp();
            volatile int never[2] = {0, ctx[1]};  // own limit, no abort
            mbar_wait(&bars[B_END], 0, never);
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

// Joins the parts of the units that several CTAs worked on, in the order of the
// CTAs: block (c, slice) for the unit that begins in CTA c's run, a warp for a row.
// (It may start before the kernels in front of the main one have ended: it waits
// before it reads anything.)
constexpr int kJoinWarps = 8;
template <int D> __global__ void __launch_bounds__(kJoinWarps * 32) tree_join_kernel(const Params p)
{
    constexpr int E = D / 32, PARTS = 8;  // parts under way together
    const Geo &g = p.g;
    const int lane = threadIdx.x & 31;
    dependents_may_start();
    dependency_wait();
    const Cut u = p.cuts[blockIdx.x];
    const int first = blockIdx.x, in_tile = (int)blockIdx.y * kJoinWarps + (int)(threadIdx.x >> 5);
    if (in_tile < u.nrows) {
        const int row = u.row0 + in_tile, t = row / g.G, h = u.kvh * g.G + row - t * g.G;
        auto at = [&](int cta) { return ((int64_t)cta * 2 + (cta == first ? 1 : 0)) * kTileRows + in_tile; };
        float top = p.sinks ? p.sinks[h] * 1.4426950408889634f : kNoMax, sum = p.sinks ? 1.f : 0.f, acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = 0.f;
        for (int c0 = first; c0 <= u.last; c0 += PARTS) {
            float2 ml[PARTS];
            float x[PARTS][E];
#pragma unroll
            for (int c = 0; c < PARTS; ++c) {
                ml[c] = make_float2(kNoMax, 0.f);
                if (c0 + c <= u.last) {
                    ml[c] = p.part_ml[at(c0 + c)];
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        x[c][e] = p.part_o[at(c0 + c) * D + e * 32 + lane];
                }
            }
            float mn = top;
#pragma unroll
            for (int c = 0; c < PARTS; ++c)
                mn = fmaxf(mn, ml[c].x);
            const float older = exp2f(top - mn);
            sum *= older;
#pragma unroll
            for (int e = 0; e < E; ++e)
                acc[e] *= older;
#pragma unroll
            for (int c = 0; c < PARTS; ++c)
                if (c0 + c <= u.last) {
                    const float f = exp2f(ml[c].x - mn);
                    sum = fmaf(ml[c].y, f, sum);
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        acc[e] = fmaf(x[c][e], f, acc[e]);
                }
            top = mn;
        }
        const bool some = sum > 0.f || sum != sum;
        const float scale = some ? 1.f / sum : 0.f;
        __nv_bfloat16 *dst = p.o + o_off(g, u.b, h, t);
#pragma unroll
        for (int e = 0; e < E; ++e)
            dst[e * 32 + lane] = __float2bfloat16_rn(acc[e] * scale);
        if (lane == 0)
            p.lse[stat_off(g, u.b, h, t)] = some ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
    }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct WsLayout {
    size_t cuts, ml, o, total;
};
WsLayout ws_layout(const Geo &g)
{
    const size_t slots = (size_t)num_sms() * 2 * kTileRows;
    WsLayout w;
    w.cuts = 256;
    w.ml = w.cuts + up256(sizeof(Cut) * (size_t)num_sms());
    w.o = w.ml + up256(sizeof(float2) * slots);
    w.total = w.o + sizeof(float) * slots * g.D;
    return w;
}

template <int D> cudaError_t tree_chunk_t(const Params &p, cudaStream_t st)
{
    void (*const kernels[3])(const Params) = {tree_chunk_kernel<D, 16>, tree_chunk_kernel<D, 32>, tree_chunk_kernel<D, 64>};
    auto kernel = kernels[p.c.bsh - 4];
    cudaError_t e = allow_shared((const void *)kernel);
    if (e != cudaSuccess || (e = launch_dependent(kernel, dim3((unsigned)p.ctas), dim3(kThreads), Layout<D>::total, st, p)) != cudaSuccess)
        return e;
    return launch_dependent(tree_join_kernel<D>, dim3((unsigned)p.ctas, kTileRows / kJoinWarps), dim3(kJoinWarps * 32), 0, st, p);
}

}  // namespace

// Where this kernel takes over from k_tree.cu's, whose time goes by 32-row tiles of
// every key: about 14 us and 0.075 for a thousand keys of a kv head and tile, against
// 25 and 0.1 for a thousand keys here (D = 128, 8 kv heads of 4 query heads; one
// sequence of 2048 tokens with 24 and 64 drafts 19 and 24 us there, 28 and 33 here; of
// 8192 31 and 53 us there, 31 and 37 here; 4 of 8192 with 12 and 24 drafts 51 and 70
// us there, 49 and 50 here; 8 of 512 with 12 drafts 17 there, 31 here).  The lengths
// are the device's: the table's width stands for them.  Where it is wider than its
// rows, k_tree.cu's clusters are not to be had either (they go by the width too), and
// its list is what there is: in a table of 131,072 tokens, one row of 2048 with 12, 24 and
// 64 drafts 21, 25 and 31 us there, 27, 27 and 31 here; of 8192 27, 35 and 56 there, 31,
// 31 and 37 here; of 32,768 51, 69 and 140 there, 43, 46 and 58 here; 8 rows of 512 and
// of 2048 with 24 drafts 38 and 56 there, 31 and 45 here.  So at most 6 us are lost
// to the width, on few drafts behind short rows.
bool tree_chunk_supported(const Geo &g, const Cache &c, int dtype, bool sel)
{
    const int64_t rows = longest_rows(g), heads = (int64_t)g.B * g.Hkv, keys = (int64_t)c.cols * c.bs;
    const int64_t entries = (keys + kTileKeys - 1) / kTileKeys * kWide + kStartCost;
    return !sel && dtype == NSA_DTYPE_BF16 && (g.D == 64 || g.D == 128) && g.B <= kMaxSeqs &&
           heads * ((rows + kTileRows - 1) / kTileRows) * entries < INT32_MAX && ((rows + 31) / 32 - 1) * heads * keys > 180000;
}

size_t tree_chunk_ws_bytes(const Geo &g) { return ws_layout(g).total; }

cudaError_t launch_tree_chunk(const Geo &g, const Cache &c, const void *q, const int *parents, const float *sinks, void *o, float *lse,
                              char *ws, cudaStream_t st)
{
    const WsLayout w = ws_layout(g);
    Params p;
    p.g = g;
    p.c = c;
    p.q = (const __nv_bfloat16 *)q;
    p.sinks = sinks;
    p.parents = parents;
    p.o = (__nv_bfloat16 *)o;
    p.lse = lse;
    p.err = (int *)ws;
    p.cuts = (Cut *)(ws + w.cuts);
    p.part_ml = (float2 *)(ws + w.ml);
    p.part_o = (float *)(ws + w.o);
    p.ctas = num_sms();
    p.wait_us = wait_test().wait_us;
    p.stall = wait_test().kernel == WAIT_TEST_FWD;
    return g.D == 128 ? tree_chunk_t<128>(p, st) : tree_chunk_t<64>(p, st);
}

}  // namespace nsa
