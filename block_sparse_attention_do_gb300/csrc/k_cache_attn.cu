// k_cache_attn.cu -- attention of new tokens over the paged 8-bit cache, for
// few query rows per kv head: the kernel that decoding runs on.
//
// Per query row r (token t, query head h of kv head g) over the attended
// keys j, code vectors ck_j, cv_j and their pages' scales ks_j, vs_j:
//   x_j = scale * log2(e) * ks_j * <q_r, ck_j>,  w_j = 2^(x_j + log2(vs_j) - M)
//   O = sum w_j cv_j / sum (w_j / vs_j),  LSE = ln 2 * (M + log2 sum (w_j / vs_j))
// The value scale rides in the exponent, so the second product runs on plain
// codes and a page of small values costs O no range.  For the sum it may: where
// a page's scale lies outside 2^-40 .. 2^40 a weight w can underflow although
// w / vs counts (64 values of zero, scale 2^-100, beside others of scale 2^27:
// half the sum).  From a list with such a page on the sum is taken from the
// scores alone, 2^(x_j - log2(vs_j) - N) with a maximum N of their own, in a pass
// over the keys of its own; at the unit's end O is turned to units of 2^N.
//
// What bounds it: the cache's bytes, 2 D per key and kv head, each read once;
// 4 G D operations on them are far below the tensor cores' rate (G = 4: 8
// operations a byte).  So the layout is made for the loads: every warp keeps
// its next steps of 16 tokens under way into a ring of its own in shared
// memory, and no warp waits for another before the end.  Measured, D = 128, 8
// kv heads of 4 query heads: 32 sequences of 128 .. 32768 tokens, 1.08 GB of
// codes, 183 us, 5.9 TB/s (87% of a plain copy's rate); one sequence of 8192,
// 17 MB, 13 us, of which 4 are any launch's.  The products are taken
// transposed, tokens (then head dimensions) as the 16 rows of mma.m16n8k16
// and query rows as its 8 columns:
//   S^T[token, row] = K q^T     A: a thread's 16 code bytes of one token are
//       the pairs of four k-steps, in an order of the head dimension that q's
//       fragments share;
//   O^T[dim, row] = V^T P^T     A: two tokens' code bytes interleaved by byte
//       permutes give the (token, token + 1) pairs that A's columns want; B
//       is the transposed S fragment (one movmatrix per 8x8).
// e4m3 is a subset of half, so codes convert exactly; q is scaled to half's
// range by a power of two per row (bf16: exact but for elements 2^-29 below
// the row's largest; fp32: two halves, 22 bits) and P is rounded to half, 11
// bits (fp32: two halves, 22).  A half is exact to 2^-24 and holds 2^15: the row's
// largest weight is brought to 2^5 .. 2^15 (fp32: 2^13 .. 2^15), so that weights
// down to 2^-19 (fp32, 22 bits: 2^-16, 2^-38 absolute) of it keep their bits.
// Sums are fp32.  A CTA's work is a run of pages of
// the whole call's list of (sequence, kv head, page), cut into equal runs so
// that long and short sequences load every SM alike; rows whose pages fall to
// several CTAs are joined by a second kernel, in a fixed order.
//
// The legacy mma.sync path is enough here: the tensor pipe is a few percent
// busy, and tcgen05 would take the codes through shared memory first.
#include <math.h>

#include <cooperative_groups.h>

#include <atomic>

#include "cache_common.cuh"
#include "launch.h"
#include "tc_common.cuh"

namespace cg = cooperative_groups;

namespace nsa {

namespace {

// Warps of a CTA, CTAs of an SM and steps of a warp under way, by the tiles of
// 8 query rows.  A thread holds O in D / 4 registers a tile: up to two tiles 16
// warps an SM of 128 registers, with four 8 of 255.  16 warps with two steps
// of 4 KB ahead have 128 KB of codes under way on an SM; the memory's rate
// times its latency asks for about 50.
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kList = kThreads;  // pages of a run listed at a time, one per thread
__host__ __device__ constexpr int attn_ctas(int nt) { return nt >= 4 ? 1 : 2; }
__host__ __device__ constexpr int attn_stages(int nt) { return nt >= 4 ? 4 : 3; }
constexpr float kNoMax = -1e30f; // running maximum of a row that has seen no key
constexpr int kMaxRows = 8192;   // sequences of a call without an index (their prefix sits in shared memory)
constexpr int kNoKey = 0x7f000000; // position of the keys of an entry that is left out
// a row's unit M: its weights may grow from 2^up to 2^kTop (half holds 2^16) before
// it is raised; fp32 keeps more small ones, and is raised more often
constexpr float kTop = 15.f;
__host__ __device__ constexpr float attn_up(bool split) { return split ? 13.f : 5.f; }

// Division of 0 <= n < 2^31 by a number that the host knows: with 2^(l-1) < d
// <= 2^l and m = floor(2^(31+l) / d) + 1, m d exceeds 2^(31+l) by at most 2^l,
// so n m / 2^(31+l) has the quotient as its whole part.
struct FastDiv {
    int d;
    uint32_t m, sh;
    FastDiv() = default;
    explicit FastDiv(int d_) : d(d_)
    {
        uint32_t l = 0;
        while (((int64_t)1 << l) < d)
            ++l;
        sh = 31 + l;
        m = (uint32_t)(((uint64_t)1 << sh) / (uint32_t)d + 1);
    }
    __device__ __forceinline__ int div(int n) const { return (int)((uint64_t)(uint32_t)n * m >> sh); }
    __device__ __forceinline__ int divmod(int n, int &rem) const
    {
        const int q = div(n);
        rem = n - q * d;
        return q;
    }
};

struct AttnArgs {
    Geo g;
    Cache c;
    FastDiv by_G, by_Hkv, by_Hq, by_T, by_S, by_tiles, by_ncta, by_quantum;  // of G, .., row_tiles, ncta, quantum
    const void *q;
    const int *idx;      // selection: [.., S], else nullptr
    const float *sinks;  // or nullptr
    void *o;
    float *lse;
    int row_tiles;       // query-row tiles per index row (clustered form without one: per sequence, at most)
    int quantum;         // pages that are not cut
    int start_cost;      // dense: list entries that stand before a unit's pages for what it costs to begin one
    int ncta;            // CTAs of the main kernel
    int units, cs;       // clustered form: its units, and the CTAs of one
    int *err;            // clustered form: the call's error word (may be null)
    int *status;         // [ncta]: what each CTA found
    int *prefix;         // [rows + 1] dense: list entries of one kv head before each sequence
    float *part_o;       // [ncta * 2][rows of a tile][D]
    float2 *part_ml;     // [ncta * 2][rows of a tile]
};

// log2 of the running maximum and the sum: a row's statistics
__device__ __forceinline__ float lse_of(float m, float l) { return l > 0.f || l != l ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY; }

__device__ __forceinline__ uint32_t pack_half(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *(const uint32_t *)&h;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// E (1, 2, 4) consecutive elements of a row as floats
template <int E> __device__ __forceinline__ void load_row(const float *p, float (&x)[E])
{
    if constexpr (E == 4) {
        const float4 v = *(const float4 *)p;
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else if constexpr (E == 2) {
        const float2 v = *(const float2 *)p;
        x[0] = v.x, x[1] = v.y;
    } else
        x[0] = *p;
}
template <int E> __device__ __forceinline__ void load_row(const __nv_bfloat16 *p, float (&x)[E])
{
    if constexpr (E >= 2) {
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const float2 v = __bfloat1622float2(*(const __nv_bfloat162 *)(p + i));
            x[i] = v.x, x[i + 1] = v.y;
        }
    } else
        x[0] = __bfloat162float(*p);
}
// four outputs of a row
__device__ __forceinline__ void store4(float *p, const float4 &x) { *(float4 *)p = x; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float4 &x)
{
    *(uint2 *)p = make_uint2(tc::pack_bf16(x.x, x.y), tc::pack_bf16(x.z, x.w));
}

// BYTES (4, 8, 16) consecutive bytes of shared memory as words
template <int BYTES> __device__ __forceinline__ void load_shared(uint32_t at, uint32_t *w)
{
    if constexpr (BYTES == 16)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
    else if constexpr (BYTES == 8)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
    else
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at) : "memory");
}

// Place, in 16-byte units, of unit u of token t in a step's 16 tokens (D / 16
// units each): exclusive-ors of the token's bits, so that the lanes that read
// together find their fragments in different banks.  Keys are read by two
// neighbouring tokens at a time (rows of 128 bytes would share banks), values
// by every other token of eight.
template <int D> __device__ __forceinline__ int k_at(int t, int u) { return (t * (D / 16) + u) ^ (D == 128 ? (t & 1) << 2 : 0); }
template <int D> __device__ __forceinline__ int v_at(int t, int u)
{
    return (t * (D / 16) + u) ^ (D == 128 ? (t >> 1 & 3) << 1 : D == 64 ? (t >> 1 & 1) << 2 | (t >> 2 & 1) << 1 : (t >> 2 & 1) << 1);
}

// Whether packed token tok is a query of some sequence: then of sequence b,
// its t-th.  Tokens in front of the first offset, or of a range that is none,
// are nobody's.
__device__ __forceinline__ bool query_of(const Geo &g, int tok, int &b, int &t)
{
    b = seq_of_token(g, tok);
    const int n = new_tokens(g, b);
    t = n > 0 ? tok - g.cu[b] : 0;
    return t >= 0 && t < n;
}

// tokens of sequence b in the cache (a length that the table cannot hold is reported by the join)
__device__ __forceinline__ int held_tokens(const AttnArgs &a, int b)
{
    return min(max(a.c.lens[b], 0), a.c.cols * a.c.bs);
}

// The pages of sequence b that any of its query rows attends: [lo, lo + n).
__device__ __forceinline__ int attended_pages(const AttnArgs &a, int b, int &lo)
{
    const int nq = new_tokens(a.g, b), len = held_tokens(a, b);
    lo = 0;
    if (nq <= 0 || len <= 0)
        return 0;
    if (a.g.window > 0) {
        const int64_t first = (int64_t)len - nq - a.g.window + 1;  // the first row's left edge
        lo = first > 0 ? (int)(first >> a.c.bsh) : 0;
    }
    return max(0, ((len - 1) >> a.c.bsh) + 1 - lo);
}

// tiles of R query rows of sequence b (dense)
template <int R> __device__ __forceinline__ int row_tiles_of(const Geo &g, int b)
{
    return (max(new_tokens(g, b), 0) * g.G + R - 1) / R;
}

// A unit of the list: a tile of query rows and the run of list entries that
// belongs to it.
struct UnitRows {
    int b, kvh, row0, nrows;  // rows row0 .. of sequence b (row = token * G + head), nrows of them valid
    int begin, count;         // its pages in the list
    int page_lo;              // dense: first page
};

// The list cut into equal runs, one per CTA, at multiples of the quantum.
struct Runs {
    int total, quantum, per, rem;
    __device__ __forceinline__ Runs(int total_, const AttnArgs &a) : total(total_), quantum(a.quantum)
    {
        per = a.by_ncta.divmod(a.by_quantum.div(total + quantum - 1), rem);
    }
    __device__ __forceinline__ int begin(int cta) const
    {
        return (int)min((int64_t)total, (int64_t)(cta * per + min(cta, rem)) * quantum);
    }
    __device__ __forceinline__ int cta_of(int entry, const AttnArgs &a) const
    {
        const int q = a.by_quantum.div(entry), longer = rem * (per + 1);
        return q < longer ? q / (per + 1) : rem + (q - longer) / max(per, 1);
    }
};

// NT: tiles of 8 query rows; SPLIT: fp32 queries (two halves)
template <int D, int NT, bool SPLIT> struct Smem {
    static constexpr int R = NT * 8;
    static constexpr int KS = D / 16;  // k-steps of S
    uint2 qf[SPLIT ? 2 : 1][KS][NT][32];
    float qmul[R];  // scale * log2(e) * 2^-e of each row
    int pos[R];     // key position of each row's token (-1: no such row)
    int64_t o_at[R], lse_at[R];  // its places in o and lse
    int64_t off[kList];  // of the listed entries: byte offset of the page and head
    int key0[kList];     // first key (kNoKey: left out)
    float4 sc[kList];    // k scale, log2 and reciprocal of the v scale
    float2 ml[kWarps][R];       // each warp's maximum and sum (before the end: of the scores alone, once those are kept apart)
    float2 cta_ml[R];           // the CTA's, for its cluster
    uint32_t nan[kWarps][R * D / 32];  // each warp's outputs that a NaN value reaches
    union {
        float o[kWarps][R][D + 4];                     // its part of O
        uint8_t ring[kWarps][attn_stages(NT)][32 * D];  // its steps under way: 16 tokens' keys, then values
    };
};

// Every length, index entry and page of a call, checked by one block, which
// alone writes the error word (the clustered form's calls are small).
__device__ __noinline__ void attn_check(const AttnArgs &a)
{
    const Geo &g = a.g;
    const Cache &c = a.c;
    const int tid = threadIdx.x, lane = tid & 31;
    int bad = 0;
    auto bad_page = [&](int b, int col) {
        const int page = c.table[(int64_t)b * c.cols + col];
        return page < 0 || page >= c.pages;
    };
    for (int b = tid; b < g.B; b += kThreads)
        bad |= c.lens[b] < 0 || c.lens[b] > c.cols * c.bs || new_tokens(g, b) < 0;
    if (!a.idx)
        for (int b = tid >> 5; b < g.B; b += kWarps) {
            int lo;
            const int n = attended_pages(a, b, lo);
#pragma unroll 8
            for (int col = lo + lane; col < lo + n; col += 32)
                bad |= bad_page(b, col);
        }
    else
#pragma unroll 2
        for (int i = tid; i < g.ntok * g.Hkv * g.S; i += kThreads) {
            const int j = a.idx[i];
            if (j == -1)
                continue;
            int s, h, b, t;
            const int row = a.by_S.divmod(i, s);
            if (g.thd) {
                const int tok = a.by_Hkv.divmod(row, h);
                if (!query_of(g, tok, b, t))
                    continue;  // a token of no sequence
            } else
                b = a.by_Hkv.divmod(a.by_T.divmod(row, t), h);
            const int pos = held_tokens(a, b) - new_tokens(g, b) + t;
            if (j < 0 || j >= c.cols || j * c.bs > pos || bad_page(b, j))
                bad = 1;
            for (int k = i - s; k < i; ++k)
                bad |= a.idx[k] == j;
        }
    bad = __syncthreads_or(bad);
    if (tid == 0)
        *a.err = bad ? NSA_ERR_BAD_INDEX : NSA_OK;
}

// CLUSTER: a unit's pages are cut into equal runs for the CTAs of a cluster,
// which join their sums through one another's shared memory: one launch, for
// calls that are a few microseconds of latencies.
template <typename T, int D, int NT, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, attn_ctas(NT)) cache_attn_kernel(const AttnArgs a)
{
    constexpr bool SPLIT = sizeof(T) == 4;
    constexpr int R = NT * 8, KS = D / 16, MT = D / 16;
    constexpr int KB = D >= 64 ? 16 : 8;       // bytes of a K load
    constexpr int KL = D / 4 / KB;             // K loads per token and thread
    constexpr int VB = D / 8;                  // bytes of a V load: one per token and thread
    constexpr int VW = VB / 4;                 // words
    constexpr int kStages = attn_stages(NT), kStageBytes = 32 * D, CPT = D / 16;
    using SM = Smem<D, NT, SPLIT>;
    extern __shared__ __align__(16) char smem_raw[];
    SM &sm = *(SM *)smem_raw;
    const Geo &g = a.g;
    const Cache &c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gq = lane >> 2, tq = lane & 3;  // the fragment's row group and column pair
    const int cta = blockIdx.x;
    dependents_may_start();
    dependency_wait();
    const bool sel = a.idx != nullptr;
    bool bad = false;

    // ---- the call's list of pages and this CTA's run of it
    __shared__ int part_s[kWarps];
    int *prefix = (int *)(smem_raw + sizeof(SM));  // dense: as a.prefix
    int total;
    const int rank = CLUSTER ? cta & (a.cs - 1) : 0, cunit = CLUSTER ? cta / a.cs : 0;
    if (CLUSTER) {
        if (cunit == a.units) {  // the cluster behind the units'
            if (rank == 0)
                attn_check(a);
            return;
        }
        total = 0;
    } else if (sel)
        total = g.ntok * g.Hkv * a.row_tiles * g.S;
    else {
        int base = 0;
        for (int b0 = 0; b0 < g.B; b0 += kThreads) {
            const int b = b0 + tid;
            int lo, n = b < g.B ? attended_pages(a, b, lo) : 0;
            n = n > 0 ? (n + a.start_cost) * row_tiles_of<R>(g, b) : 0;
            int incl = n;
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                incl += lane >= o ? y : 0;
            }
            if (lane == 31)
                part_s[warp] = incl;
            __syncthreads();
            int before = 0, all = 0;
            for (int k = 0; k < kWarps; ++k) {
                before += k < warp ? part_s[k] : 0;
                all += part_s[k];
            }
            if (b < g.B) {
                prefix[b] = base + before + incl - n;
                if (cta == 0)
                    a.prefix[b] = prefix[b];
            }
            base += all;
            __syncthreads();
        }
        if (tid == 0) {
            prefix[g.B] = base;
            if (cta == 0)
                a.prefix[g.B] = base;
        }
        __syncthreads();
        total = base * g.Hkv;
    }
    // the lane's places in a stage of the warp's ring: where it copies to
    // (16 bytes of each 512, a token's D / 16 units by neighbouring lanes),
    // and where its fragments lie
    const uint32_t ring = tc::smem_u32(sm.ring[warp]);
    const uint32_t to_k = k_at<D>(lane / CPT, lane % CPT) * 16, to_v = 16 * D + v_at<D>(lane / CPT, lane % CPT) * 16;
    const uint32_t from_k = k_at<D>(gq, tq * KB / 16) * 16 + tq * KB % 16;
    const uint32_t from_v = 16 * D + v_at<D>(tq * 2, gq * VB / 16) * 16 + gq * VB % 16;
    const int from_lane = lane / CPT * (int)c.st + lane % CPT * 16;
    const int st = (int)c.st, per_sh = c.bsh - 4, per_mask = (1 << per_sh) - 1;  // steps per page
    const Runs runs(total, a);
    const int run0 = runs.begin(cta), run1 = runs.begin(cta + 1);

    for (int at = run0; CLUSTER || at < run1;) {
        // ---- the unit that holds list entry `at`
        UnitRows u;
        if (sel) {
            const int unit = CLUSTER ? cunit : a.by_S.div(at);
            u.begin = CLUSTER ? 0 : unit * g.S;
            u.count = g.S;
            int rt, t;
            bool query = true;
            const int row = a.by_tiles.divmod(unit, rt);  // of the index
            if (g.thd)
                query = query_of(g, a.by_Hkv.divmod(row, u.kvh), u.b, t);
            else
                u.b = a.by_Hkv.divmod(a.by_T.divmod(row, t), u.kvh);
            u.row0 = t * g.G + rt * R;
            u.nrows = query ? min(R, g.G - rt * R) : 0;  // 0: a token of no sequence
            u.page_lo = 0;
        } else if (CLUSTER) {
            int rt;
            u.b = a.by_Hkv.divmod(a.by_tiles.divmod(cunit, rt), u.kvh);
            u.begin = 0;
            u.count = attended_pages(a, u.b, u.page_lo);
            u.row0 = rt * R;
            u.nrows = min(R, new_tokens(g, u.b) * g.G - u.row0);
        } else {
            int lo = 0, hi = g.B - 1;  // the sequence: prefix[b] * Hkv <= at < prefix[b + 1] * Hkv
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (prefix[mid] * g.Hkv <= at)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            u.b = lo;
            const int n = attended_pages(a, lo, u.page_lo), tiles = row_tiles_of<R>(g, lo);
            const int in = (at - prefix[lo] * g.Hkv) / (n + a.start_cost);  // (kv head, row tile)
            u.begin = prefix[lo] * g.Hkv + in * (n + a.start_cost) + a.start_cost;
            u.count = n;
            u.kvh = tiles == 1 ? in : in / tiles;
            u.row0 = tiles == 1 ? 0 : in % tiles * R;
            u.nrows = min(R, new_tokens(g, lo) * g.G - u.row0);
        }
        int seg1;
        if constexpr (CLUSTER) {
            const int per = (u.count + a.cs - 1) / a.cs;
            at = min(u.count, rank * per);
            seg1 = min(u.count, at + per);
            if (u.nrows <= 0)
                return;  // (the whole cluster)
        } else {
            seg1 = min(run1, u.begin + u.count);
            at = max(at, u.begin);
            if (u.nrows <= 0 || at >= seg1) {
                at = max(at, seg1);
                continue;
            }
        }
        const int len = held_tokens(a, u.b);
        const int pos0 = len - new_tokens(g, u.b);  // position of the sequence's first query token
        const int t_first = a.by_G.div(u.row0), t_last = a.by_G.div(u.row0 + u.nrows - 1);
        const int pmin = pos0 + t_first, pmax = pos0 + t_last;  // of the tile's rows
        const int key_lo = g.window > 0 ? pmin - g.window - 14 : INT32_MIN;  // steps before it lie left of every window

        // One list entry per thread: its block (-1: left out) and page.  Only
        // the ids stand before the first loads of codes; what else an entry
        // needs is fetched behind those.
        const int64_t irow = sel ? index_row(g, u.b, u.kvh, t_first) * g.S : 0;
        auto list_block = [&](int entry) {
            int j = sel ? a.idx[irow + entry - u.begin] : u.page_lo + entry - u.begin;
            if (sel && j != -1 && (j < 0 || j >= c.cols || j * c.bs > pmax || j * c.bs >= len)) {  // no block, or in the future
                bad = true;
                j = -1;
            }
            return j;
        };
        auto list_page = [&](int j) { return j >= 0 ? c.table[(int64_t)u.b * c.cols + j] : -1; };
        auto in_pool = [&](int j, int page) {
            if (j >= 0 && (page < 0 || page >= c.pages)) {
                bad = true;
                page = -1;
            }
            return page;
        };
        // the tile's queries, E elements of a row per lane, then the first
        // page ids: all under way together
        constexpr int E = D / 32, QR = (R + kWarps - 1) / kWarps;
        float qx[QR][E];
        int row_pos[QR];
        int64_t row_o[QR], row_lse[QR];
#pragma unroll
        for (int i = 0; i < QR; ++i) {
            const int r = warp + i * kWarps;
            if (r < u.nrows) {
                int hh;
                const int t = a.by_G.divmod(u.row0 + r, hh), h = u.kvh * g.G + hh;
                load_row<E>((const T *)a.q + q_off(g, u.b, h, t) + lane * E, qx[i]);
                row_pos[i] = pos0 + t;
                row_o[i] = o_off(g, u.b, h, t);
                row_lse[i] = stat_off(g, u.b, h, t);
            } else
#pragma unroll
                for (int e = 0; e < E; ++e)
                    qx[i][e] = 0.f;
        }
        int my_block = -1, my_page = -1;
        if (at + tid < min(seg1, at + kList)) {
            my_block = list_block(at + tid);
            my_page = list_page(my_block);
        }

        // ---- queries into fragments: element (k, n) of B is row n's element
        // k, in the order of the head dimension that the K loads give
        __syncthreads();  // the previous unit is done with shared memory
        for (int i = lane; i < R * D / 32; i += 32)
            sm.nan[warp][i] = 0;
        bool nan_seen = false;
#pragma unroll
        for (int i = 0; i < QR; ++i) {
            const int r = warp + i * kWarps;
            if (r >= R)
                break;
            float amax = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e)
                amax = fmaxf(amax, fabsf(qx[i][e]));
            amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));  // of values >= 0
            // the row's largest element to [2^14, 2^15)
            const int be = (int)(__float_as_uint(amax) >> 23);  // biased exponent (0: none, 255: infinity)
            const int e2 = be == 0 || be == 255 ? 0 : min(max(14 - (be - 127), -120), 120);
            const float up = __uint_as_float((uint32_t)(127 + e2) << 23);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int d = lane * E + e;
                // dimension d sits in load d / (4 KB), thread column d / KB % 4,
                // byte d % KB of the load: word / 4 is a k-step, bytes 0-1 its
                // low and 2-3 its high half
                const int tqd = d / KB % 4, k = d % KB;
                const int step = d / (4 * KB) * (KB / 4) + k / 4, slot = k % 4;
                const float y = qx[i][e] * up;
                const __half hi = __float2half_rn(y);
                ((__half *)&sm.qf[0][step][r / 8][(r % 8) * 4 + tqd])[slot] = hi;
                if constexpr (SPLIT)
                    ((__half *)&sm.qf[SPLIT ? 1 : 0][step][r / 8][(r % 8) * 4 + tqd])[slot] = __float2half_rn(y - __half2float(hi));
            }
            if (lane == 0) {
                sm.qmul[r] = g.scale_l2 * __uint_as_float((uint32_t)(127 - e2) << 23);
                sm.pos[r] = r < u.nrows ? row_pos[i] : -1;
                sm.o_at[r] = row_o[i];
                sm.lse_at[r] = row_lse[i];
            }
        }
        my_page = in_pool(my_block, my_page);

        // S^T = K q^T of a thread's 16 codes of two tokens
        auto scores = [&](const uint32_t (&kw)[2][KL * KB / 4], float (&x)[NT][4]) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[n][i] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t af[4];
                e4m3x4_to_half(kw[0][k], af[0], af[2]);
                e4m3x4_to_half(kw[1][k], af[1], af[3]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint2 bf = sm.qf[0][k][n][lane];
                    mma_f16(x[n], af, bf.x, bf.y);
                    if constexpr (SPLIT) {
                        const uint2 bl = sm.qf[SPLIT ? 1 : 0][k][n][lane];
                        mma_f16(x[n], af, bl.x, bl.y);
                    }
                }
            }
        };
        // over the lanes that share a query row
        auto sum_of_rows = [](float x) {
            x += __shfl_xor_sync(0xffffffffu, x, 4);
            x += __shfl_xor_sync(0xffffffffu, x, 8);
            return x + __shfl_xor_sync(0xffffffffu, x, 16);
        };
        float o[NT][MT][4];
        float m[NT][2], l[NT][2];
        bool apart = false;  // (uniform over the CTA) the sums are in sm.ml
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[n][i] = kNoMax;
                l[n][i] = 0.f;
            }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[n][j][i] = 0.f;

        for (int e0 = at; e0 < seg1; e0 += kList) {
            const int ne = min(kList, seg1 - e0);
            if (e0 > at) {
                my_block = my_page = -1;
                if (tid < ne) {
                    my_block = list_block(e0 + tid);
                    my_page = in_pool(my_block, list_page(my_block));
                }
                __syncthreads();  // the list before is used up
            }
            if (tid < ne) {
                sm.off[tid] = my_page >= 0 ? (int64_t)my_page * c.sp + (int64_t)u.kvh * c.sh : 0;
                sm.key0[tid] = my_page >= 0 ? my_block * c.bs : kNoKey;
            }
            __syncthreads();

            // ---- 16-token steps of the listed pages, the warps in turn
            const int steps = ne << per_sh;
            // the step's first key; a step that no row attends is not read
            auto step_key = [&](int s) { return s < steps ? sm.key0[s >> per_sh] + (s & per_mask) * 16 : kNoKey; };
            auto attended = [&](int key) { return key <= pmax && key >= key_lo; };
            // step s into a stage of the warp's ring, 16 bytes per lane and copy
            auto fetch = [&](int s, int stage) {
                if (attended(step_key(s))) {
                    const int64_t from = sm.off[s >> per_sh] + (s & per_mask) * 16 * st + from_lane;
                    const uint32_t to = ring + stage * kStageBytes;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {  // 512 bytes, 32 / CPT tokens each
                        tc::cp_async_16(to + to_k + i * 512, c.k + from + i * (32 / CPT) * st, 16);
                        tc::cp_async_16(to + (to_v ^ (D == 128 ? (i & 1) << 6 : 0)) + i * 512, c.v + from + i * (32 / CPT) * st, 16);
                    }
                }
                tc::cp_async_commit();
            };
            int stage = 0;
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i)
                fetch(warp + i * kWarps, i);
            bool far = apart;  // a scale of values outside the common range
            if (tid < ne) {
                float ks = 0.f, vs = 1.f;
                if (my_page >= 0) {
                    ks = c.ks[(int64_t)my_page * c.Hkv + u.kvh];
                    vs = fmaxf(c.vs[(int64_t)my_page * c.Hkv + u.kvh], kScaleFloor);
                }
                const float lvs = log2f(vs);
                far = far || fabsf(lvs) > kNearScale;
                sm.sc[tid] = make_float4(ks, lvs, 1.f / vs, 0.f);
            }
            if (sel && warp * 32 < ne) {  // an entry that its row has before is left out: no row attends its keys
                bool twice = false;
                const int s = e0 + tid - u.begin;  // (warp-uniform rounds of 32 of the row's entries)
                for (int k0 = 0; k0 < min(g.S, e0 + warp * 32 + 32 - u.begin); k0 += 32) {
                    const int v = k0 + lane < g.S ? a.idx[irow + k0 + lane] : -1;
                    for (int k = 0; k < min(32, g.S - k0); ++k) {
                        const int w = __shfl_sync(0xffffffffu, v, k);
                        twice |= k0 + k < s && w == my_block;
                    }
                }
                if (tid < ne && my_page >= 0 && twice) {
                    bad = true;
                    sm.key0[tid] = kNoKey;
                }
            }
            far = __syncthreads_or(far);
            if (far) {
                if (!apart)  // the warp's sums so far
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float x = sum_of_rows(l[n][i]);
                            if (gq == 0)
                                sm.ml[warp][n * 8 + tq * 2 + i] = make_float2(m[n][i], x);
                            l[n][i] = 0.f;
                        }
                apart = true;
                if (tid < ne)
                    sm.sc[tid].z = 0.f;  // its weights add nothing to the sum
                __syncthreads();
            }
            for (int s = warp; s < steps; s += kWarps) {
                __syncwarp();  // the stage that is filled now has been read
                fetch(s + (kStages - 1) * kWarps, stage == 0 ? kStages - 1 : stage - 1);
                tc::cp_async_wait<kStages - 1>();
                __syncwarp();
                const uint32_t at = ring + stage * kStageBytes;
                stage = stage == kStages - 1 ? 0 : stage + 1;
                const int key_now = step_key(s);
                if (!attended(key_now))
                    continue;
                uint32_t kw[2][KL * KB / 4], vw[4][VW];
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int i = 0; i < KL; ++i)
                        load_shared<KB>(at + (from_k ^ i * 64) + r * 8 * D, &kw[r][i * (KB / 4)]);
                float x[NT][4];
                scores(kw, x);
                // ---- w = 2^(x + log2 vs - M)
                const float4 sc = sm.sc[s >> per_sh];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float f = sc.x * sm.qmul[n * 8 + tq * 2 + i];
                        x[n][i] = fmaf(x[n][i], f, sc.y);
                        x[n][i + 2] = fmaf(x[n][i + 2], f, sc.y);
                    }
                // keys past a row's own, left of its window, or of an entry that is left out
                const bool part = key_now + 15 > pmin || (g.window > 0 && key_now <= pmax - g.window);
                if (part) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int kk = key_now + gq + (i >> 1) * 8, p = sm.pos[n * 8 + tq * 2 + (i & 1)];
                            if (kk > p || (g.window > 0 && kk <= p - g.window))
                                x[n][i] = -INFINITY;
                        }
                }
                bool raise = false;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        raise |= fmaxf(x[n][i], x[n][i + 2]) > m[n][i] + kTop;
                if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float y = fmaxf(x[n][i], x[n][i + 2]);
                            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
                            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
                            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
                            y = fmaxf(y - attn_up(SPLIT), m[n][i]);
                            const float f = exp2f(m[n][i] - y);
                            m[n][i] = y;
                            l[n][i] *= f;
#pragma unroll
                            for (int j = 0; j < MT; ++j) {
                                o[n][j][i] *= f;
                                o[n][j][i + 2] *= f;
                            }
                        }
                }
                uint32_t pb[SPLIT ? 2 : 1][NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[n][i] = tc::ex2(x[n][i] - m[n][i & 1]);
                        l[n][i & 1] = fmaf(x[n][i], sc.z, l[n][i & 1]);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t hi = pack_half(x[n][2 * i], x[n][2 * i + 1]);
                        pb[0][n][i] = transpose8x8(hi);
                        if constexpr (SPLIT) {
                            const float2 f = __half22float2(*(const __half2 *)&hi);
                            pb[SPLIT ? 1 : 0][n][i] = transpose8x8(pack_half(x[n][2 * i] - f.x, x[n][2 * i + 1] - f.y));
                        }
                    }
                }
                auto load_v = [&]() {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        load_shared<VB>(at + (from_v ^ (i & 1) * D) + (i >> 1) * 8 * D, vw[i]);
                    if (part)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int kk = key_now + tq * 2 + (i & 1) + (i >> 1) * 8;
                            const bool out = kk > pmax || (g.window > 0 && kk <= pmin - g.window);
#pragma unroll
                            for (int w = 0; w < VW; ++w)
                                vw[i][w] = out ? 0u : vw[i][w];
                        }
                };
                load_v();
                // ---- values that a row does not attend must not reach it,
                // whatever they hold (0 * NaN would): tokens that no row
                // attends are taken as zeros, and so is every NaN, which its
                // rows get back when the warps' sums are joined
                if (part) {
                    bool nan = false;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int w = 0; w < VW; ++w)
                            nan |= (((vw[i][w] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
                    if (__any_sync(0xffffffffu, nan)) {
                        const uint8_t *vs = sm.ring[warp][stage == 0 ? kStages - 1 : stage - 1] + 16 * D;
#pragma unroll 1
                        for (int x = lane; x < 16 * D; x += 32) {
                            const int tok = x / D, d = x % D, kk = key_now + tok;
                            uint8_t *code = (uint8_t *)vs + v_at<D>(tok, d / 16) * 16 + d % 16;
                            if ((*code & 0x7f) != 0x7f)
                                continue;
                            *code = 0;
#pragma unroll 1
                            for (int r = 0; r < u.nrows; ++r) {
                                const int p = sm.pos[r];
                                if (kk <= p && !(g.window > 0 && kk <= p - g.window))
                                    atomicOr(&sm.nan[warp][r * (D / 32) + d / 32], 1u << (d % 32));
                            }
                        }
                        nan_seen = true;
                        __syncwarp();
                        load_v();
                    }
                }
                // ---- O^T += V^T P^T
#pragma unroll
                for (int w = 0; w < VW; ++w)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        uint32_t af[4];
                        e4m3x4_to_half(__byte_perm(vw[0][w], vw[1][w], hf ? 0x7362 : 0x5140), af[0], af[1]);
                        e4m3x4_to_half(__byte_perm(vw[2][w], vw[3][w], hf ? 0x7362 : 0x5140), af[2], af[3]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma_f16(o[n][w * 2 + hf], af, pb[0][n][0], pb[0][n][1]);
                            if constexpr (SPLIT)
                                mma_f16(o[n][w * 2 + hf], af, pb[SPLIT ? 1 : 0][n][0], pb[SPLIT ? 1 : 0][n][1]);
                        }
                    }
            }
            tc::cp_async_wait<0>();
            if (far) {  // the list's keys once more, for the sum of the scores alone
#pragma unroll 1
                for (int s = warp; s < steps; s += kWarps) {
                    const int key_now = step_key(s);
                    if (!attended(key_now))
                        continue;
                    const uint8_t *from = c.k + sm.off[s >> per_sh] + (int64_t)((s & per_mask) * 16 + gq) * st + tq * KB;
                    uint32_t kw[2][KL * KB / 4];
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int i = 0; i < KL * KB / 4; i += 2)
                            *(uint2 *)&kw[r][i] = *(const uint2 *)(from + r * 8 * st + i / (KB / 4) * 4 * KB + i % (KB / 4) * 4);
                    float x[NT][4];
                    scores(kw, x);
                    const float ks = sm.sc[s >> per_sh].x;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int r = n * 8 + tq * 2 + i, p = sm.pos[r];
                            const float f = ks * sm.qmul[r];
                            const float2 old = sm.ml[warp][r];
                            float y[2], top = old.x, sum = 0.f;
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int kk = key_now + gq + e * 8;
                                y[e] = kk > p || (g.window > 0 && kk <= p - g.window) ? -INFINITY : x[n][i + 2 * e] * f;
                                top = fmaxf(top, y[e]);
                            }
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                sum += tc::ex2(y[e] - top);
                            sum = sum_of_rows(sum);
                            __syncwarp();  // (every lane has read the old ones)
                            if (gq == 0)
                                sm.ml[warp][r] = make_float2(top, old.y * exp2f(old.x - top) + sum);
                        }
                    __syncwarp();
                }
            }
        }

        // ---- the warps' sums joined in shared memory (over the rings)
        __syncthreads();
        float2 *end_ml = apart ? (float2 *)sm.sc + warp * R : sm.ml[warp];  // (the lists' scales are used up)
        static_assert(sizeof(sm.sc) >= sizeof(sm.ml), "");
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x = sum_of_rows(l[n][i]);
                const int r = n * 8 + tq * 2 + i;
                if (gq == 0)
                    end_ml[r] = make_float2(m[n][i], x);
                if (r < u.nrows) {
#pragma unroll
                    for (int j = 0; j < MT; j += 2)  // dimensions gq * VB + 2 j ..
                        *(float4 *)&sm.o[warp][r][gq * VB + 2 * j] = make_float4(o[n][j][i], o[n][j][i + 2], o[n][j + 1][i], o[n][j + 1][i + 2]);
                }
            }
        if (apart) {  // O to units of 2^N, N raised by the sum's exponent: O is then a mean of values
            __syncwarp();
            for (int r = 0; r < u.nrows; ++r) {
                const float2 alone = sm.ml[warp][r], ml = end_ml[r];
                const int e = alone.y > 0.f && alone.y < INFINITY ? (int)(__float_as_uint(alone.y) >> 23) - 127 : 0;
                const float top = alone.x + (float)e, f = exp2f(fminf(ml.x - top, 127.f));
                __syncwarp();
                for (int d = lane; d < D; d += 32)
                    sm.o[warp][r][d] *= f;
                if (lane == 0)  // (the other sum is 0, or a NaN that its row keeps)
                    sm.ml[warp][r] = make_float2(top, ml.y + alone.y * __uint_as_float((uint32_t)(127 - e) << 23));
            }
            __syncwarp();
        }
        if (nan_seen) {  // (warp-uniform)
            __syncwarp();
            for (int x = lane; x < u.nrows * D; x += 32)
                if (sm.nan[warp][x / 32] >> (x % 32) & 1u)
                    sm.o[warp][x / D][x % D] = __int_as_float(0x7fffffff);
        }
        __syncthreads();
        const bool whole = CLUSTER ? a.cs == 1 : at == u.begin && seg1 == u.begin + u.count;
        // a part: the first of the run in slot 0, its last in slot 1 (a run
        // within one unit has one part)
        const int slot = cta * 2 + (at == run0 ? 0 : 1);
        for (int r = warp; r < u.nrows; r += kWarps) {  // the rows' statistics, lane w holding warp w's
            const float2 ml = lane < kWarps ? sm.ml[lane][r] : make_float2(kNoMax, 0.f);
            float top = ml.x;
#pragma unroll
            for (int i = 4; i > 0; i >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
            float f = exp2f(ml.x - top), sum = ml.y * f;
#pragma unroll
            for (int i = 4; i > 0; i >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, i);
            if (!whole) {
                if (lane == 0) {
                    if constexpr (CLUSTER)
                        sm.cta_ml[r] = make_float2(top, sum);
                    else
                        a.part_ml[slot * R + r] = make_float2(top, sum);
                }
            } else {
                if (a.sinks) {
                    int hh;
                    a.by_G.divmod(u.row0 + r, hh);
                    const int h = u.kvh * g.G + hh;
                    const float sk = a.sinks[h] * 1.4426950408889634f, mn = fmaxf(top, sk), g0 = exp2f(top - mn);
                    sum = sum * g0 + exp2f(sk - mn);
                    f *= g0;
                    top = mn;
                }
                f = sum > 0.f || sum != sum ? f / sum : 0.f;
                if (lane == 0)
                    a.lse[sm.lse_at[r]] = lse_of(top, sum);
            }
            if (lane < kWarps)
                sm.ml[lane][r].x = f;  // from here on the warp's factor
        }
        __syncthreads();
        // (thread x has vector x of each warp's part, and puts the sum, of a
        // cluster's CTA, into the first warp's place, which it alone has read)
        for (int x = tid; x < u.nrows * (D / 4); x += kThreads) {
            const int r = x / (D / 4), d = x % (D / 4) * 4;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 p = *(const float4 *)&sm.o[w][r][d];
                const float f = sm.ml[w][r].x;
                y.x += p.x * f, y.y += p.y * f, y.z += p.z * f, y.w += p.w * f;
            }
            if (whole)
                store4((T *)a.o + sm.o_at[r] + d, y);
            else if constexpr (CLUSTER)
                *(float4 *)&sm.o[0][r][d] = y;
            else
                *(float4 *)&a.part_o[((int64_t)slot * R + r) * D + d] = y;
        }
        if constexpr (CLUSTER) {
            if (whole)
                return;
            cg::cluster_group cl = cg::this_cluster();
            cl.sync();
            // cs threads to an output vector, one for each CTA's sum
            const int k = tid & (a.cs - 1), per = kThreads / a.cs, n = u.nrows * (D / 4);
            for (int x0 = rank * per; x0 < n; x0 += kThreads) {  // (uniform over the block)
                const int x = x0 + tid / a.cs, r = min(x, n - 1) / (D / 4), d = x % (D / 4) * 4;
                const float2 ml = *cl.map_shared_rank(&sm.cta_ml[r], k);
                float4 y = *(const float4 *)cl.map_shared_rank(&sm.o[0][r][d], k);
                float top = ml.x;
                for (int i = 1; i < a.cs; i <<= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
                float sink = 0.f;
                if (a.sinks) {
                    int hh;
                    a.by_G.divmod(u.row0 + r, hh);
                    const float sk = a.sinks[u.kvh * g.G + hh] * 1.4426950408889634f;
                    top = fmaxf(top, sk);
                    sink = exp2f(sk - top);
                }
                float f = exp2f(ml.x - top), sum = ml.y * f;
                y.x *= f, y.y *= f, y.z *= f, y.w *= f;
                for (int i = 1; i < a.cs; i <<= 1) {
                    sum += __shfl_xor_sync(0xffffffffu, sum, i);
                    y.x += __shfl_xor_sync(0xffffffffu, y.x, i);
                    y.y += __shfl_xor_sync(0xffffffffu, y.y, i);
                    y.z += __shfl_xor_sync(0xffffffffu, y.z, i);
                    y.w += __shfl_xor_sync(0xffffffffu, y.w, i);
                }
                sum += sink;
                f = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
                if (k == 0 && x < n) {
                    store4((T *)a.o + sm.o_at[r] + d, make_float4(y.x * f, y.y * f, y.z * f, y.w * f));
                    if (d == 0)
                        a.lse[sm.lse_at[r]] = lse_of(top, sum);
                }
            }
            cl.sync();  // no CTA leaves while another reads its sums
            return;
        }
        at = seg1;
    }
    bad = __syncthreads_or(bad);
    if (tid == 0)
        a.status[cta] = bad ? NSA_ERR_BAD_INDEX : NSA_OK;
}

// Joins the parts of the rows that several CTAs worked on, and writes the
// rows that no CTA saw (no attended page).  A block per query row: first the
// parts' maxima and sums, a thread each, then their vectors, the warps taking
// the parts in turn with several loads in flight; the order of the sums is
// that of CTAs and warps, whatever order they ran in.  The kernel is a
// programmatic dependent of the main one, which lets it start before the
// kernels in front of both may have ended: it waits before it reads anything,
// the lengths and offsets too (a reserve two launches back may still write them).
// kJoinWarps: 8 for few rows of many parts, 2 where the rows alone fill the
// GPU (1920 rows of 2 or 3 parts: 64 threads each have them all under way).
template <typename T, int D, int kJoinWarps>
__global__ void __launch_bounds__(kJoinWarps * 32) cache_join_kernel(const AttnArgs a, int R, int *err)
{
    constexpr int kJoinThreads = kJoinWarps * 32;
    constexpr int E = D / 32;
    const Geo &g = a.g;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    dependents_may_start();
    dependency_wait();
    __shared__ float part[kJoinWarps][D];
    __shared__ float factor[kJoinThreads], red[2][kJoinWarps];
    if (blockIdx.x == 0) {  // the call's error word
        int bad = 0;
        for (int b = tid; b < g.B; b += kJoinThreads) {
            const int len = a.c.lens[b];
            bad |= len < 0 || len > a.c.cols * a.c.bs || new_tokens(g, b) < 0;
        }
        for (int i = tid; i < a.ncta; i += kJoinThreads)
            bad |= a.status[i] != NSA_OK;
        bad = __syncthreads_or(bad);
        if (tid == 0)
            *err = bad ? NSA_ERR_BAD_INDEX : NSA_OK;
        return;
    }
    const bool sel = a.idx != nullptr;
    const int nrow = g.ntok * g.Hq;
    for (int w = blockIdx.x - 1; w < nrow; w += gridDim.x - 1) {
        int h, b, t;
        const int tok = a.by_Hq.divmod(w, h);
        if (g.thd) {
            if (!query_of(g, tok, b, t))
                continue;  // a token of no sequence
        } else
            b = a.by_T.divmod(tok, t);
        int hh;
        const int kvh = a.by_G.divmod(h, hh);
        int count, r, in = 0;
        if (sel) {
            r = hh % R;
            count = g.S;
        } else {
            int lo;
            const int row = t * g.G + hh, tiles = (new_tokens(g, b) * g.G + R - 1) / R;
            r = row % R;
            count = attended_pages(a, b, lo);
            in = (kvh * tiles + row / R) * (count + a.start_cost) + a.start_cost;
        }
        int first = 0, last = -1, begin = 0;  // the CTAs with a part of the row
        if (count > 0) {
            int total;
            if (sel) {
                begin = ((int)index_row(g, b, kvh, t) * a.row_tiles + hh / R) * g.S;
                total = g.ntok * g.Hkv * a.row_tiles * g.S;
            } else {
                begin = a.prefix[b] * g.Hkv + in;
                total = a.prefix[g.B] * g.Hkv;
            }
            const Runs runs(total, a);
            first = runs.cta_of(begin, a);
            last = runs.cta_of(begin + count - 1, a);
            if (first == last && runs.begin(first) <= begin && runs.begin(first + 1) >= begin + count)
                continue;  // one CTA had it all and wrote the result
            begin = runs.begin(first) >= begin ? 0 : 1;  // slot of the first part; later runs start within the row's entries
        }
        const float sk = a.sinks ? a.sinks[h] * 1.4426950408889634f : kNoMax;
        auto part_of = [&](int c) { return (int64_t)(c * 2 + (c == first ? begin : 0)) * R + r; };
        float top = sk, sum = a.sinks ? 1.f : 0.f, acc[E];
#pragma unroll
        for (int i = 0; i < E; ++i)
            acc[i] = 0.f;
        for (int c0 = first; c0 <= last; c0 += kJoinThreads) {  // one round unless a row has more parts than threads
            const int c = c0 + tid, n = min(kJoinThreads, last - c0 + 1);
            const float2 ml = c <= last ? a.part_ml[part_of(c)] : make_float2(kNoMax, 0.f);
            float x[4][E];  // the warp's first vectors, under way with the maxima
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (warp + k * kJoinWarps < n)
#pragma unroll
                    for (int i = 0; i < E; ++i)
                        x[k][i] = a.part_o[part_of(c0 + warp + k * kJoinWarps) * D + i * 32 + lane];
            float m = ml.x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (lane == 0)
                red[0][warp] = m;
            __syncthreads();
            float mn = top;
#pragma unroll
            for (int k = 0; k < kJoinWarps; ++k)
                mn = fmaxf(mn, red[0][k]);
            const float f = exp2f(ml.x - mn), older = exp2f(top - mn);
            factor[tid] = f;
            float s = ml.y * f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0)
                red[1][warp] = s;
            __syncthreads();
            sum *= older;
#pragma unroll
            for (int k = 0; k < kJoinWarps; ++k)
                sum += red[1][k];
            top = mn;
#pragma unroll
            for (int i = 0; i < E; ++i)
                acc[i] *= older;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (warp + k * kJoinWarps < n)
#pragma unroll
                    for (int i = 0; i < E; ++i)
                        acc[i] += x[k][i] * factor[warp + k * kJoinWarps];
#pragma unroll 4
            for (int p = warp + 4 * kJoinWarps; p < n; p += kJoinWarps)
#pragma unroll
                for (int i = 0; i < E; ++i)
                    acc[i] += a.part_o[part_of(c0 + p) * D + i * 32 + lane] * factor[p];
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < E; ++i)
            part[warp][i * 32 + lane] = acc[i];
        __syncthreads();
        const float scale = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
        T *dst = (T *)a.o + o_off(g, b, h, t);
        for (int d = tid; d < D; d += kJoinThreads) {
            float y = 0.f;
#pragma unroll
            for (int k = 0; k < kJoinWarps; ++k)
                y += part[k][d];
            dst[d] = from_f<T>(y * scale);
        }
        if (tid == 0)
            a.lse[stat_off(g, b, h, t)] = lse_of(top, sum);
        __syncthreads();
    }
}

// the tile of query rows: as many tiles of 8 as the rows of a kv head need
int row_tile(const Geo &g, bool sel)
{
    const int64_t rows = sel ? g.G : (int64_t)g.T * g.G;
    return rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
}

// Beginning a unit (its first reads one behind the other, the warps' sums
// joined) takes a CTA 5 to 9 us, the time of about 128 KB of codes: in a batch
// of 32 rows of 128 .. 32768 tokens a CTA that had ten short rows ended at 201
// us, the others at 155.  The list counts that many pages before each unit's.
int start_cost(const Geo &g) { return max(1, 65536 / (g.D * g.bs)); }

int ctas_of(const Geo &g, bool sel) { return num_sms() * attn_ctas(row_tile(g, sel)); }

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// The clustered form: CTAs of a unit (0: the list's form).  One launch and no
// workspace, for calls whose time is latencies: units are cut as far as the
// GPU's CTAs and 128 tokens each go, and are whole where there are many.  The
// cut goes by the table's width, not by lengths, so with several sequences
// (which may be of any length) a CTA's share has to be short: 128 KB of codes;
// one sequence alone, or keys that a window bounds, 640 KB (16 sequences of 5
// tokens behind a window of 4096: 40 us by the list, 35 here); an index's equal
// rows any.  Units cut finer than one round of CTAs cost more (the same call in
// two rounds 42 us, 128 index rows of 16 blocks 31 us for 21).  A token over
// 8192 cached ones (8 kv heads): 14.6 us by the list, of which the join's launch
// and the list's own reads were 5, and 22 us of host time; 13.2 and 15 here.
int cluster_size(const Geo &g, const Cache &c, bool sel)
{
    const int nt = row_tile(g, sel), R = nt * 8, slots = num_sms() * attn_ctas(nt);
    const int64_t units = sel ? (int64_t)g.ntok * g.Hkv * ((g.G + R - 1) / R) : (int64_t)g.B * g.Hkv * ((longest_rows(g) + R - 1) / R);
    const int64_t checks = sel ? (int64_t)g.ntok * g.Hkv * g.S : (int64_t)g.B * c.cols;
    int64_t pages = sel ? g.S : c.cols;
    if (g.window > 0)
        pages = min(pages, ((int64_t)g.window + g.T) / c.bs + 2);
    if (units > 8192 || checks > 8192)
        return 0;
    int cs = 1;
    while (cs < 16 && (units + 1) * cs * 2 <= slots && pages * c.bs > (int64_t)cs * 128)
        cs *= 2;
    const int64_t bytes = (pages + cs - 1) / cs * c.bs * 2 * g.D;
    return sel || bytes <= (g.B == 1 || g.window > 0 ? 640 << 10 : 128 << 10) ? cs : 0;
}

// shared memory above the default, and clusters of 16, allowed once per device
template <typename K> cudaError_t allow(K kernel, int smem, std::atomic<uint64_t> &done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)))
        return e;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
        return e;
    if (dev < 64)
        done.fetch_or((uint64_t)1 << dev, std::memory_order_release);
    return cudaSuccess;
}

template <typename T, int D, int NT> cudaError_t attn_t(const AttnArgs &a, cudaStream_t st)
{
    using SM = Smem<D, NT, sizeof(T) == 4>;
    cudaError_t e;
    if (a.cs > 0) {
        static std::atomic<uint64_t> done{0};
        if ((e = allow(cache_attn_kernel<T, D, NT, true>, (int)sizeof(SM), done)) != cudaSuccess)
            return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)((a.units + (a.err ? 1 : 0)) * a.cs));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = sizeof(SM);
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = a.cs;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, cache_attn_kernel<T, D, NT, true>, a);
    }
    static std::atomic<uint64_t> done{0};
    if ((e = allow(cache_attn_kernel<T, D, NT, false>, (int)(sizeof(SM) + sizeof(int) * (kMaxRows + 1)), done)) != cudaSuccess)
        return e;
    const size_t smem = sizeof(SM) + (a.idx ? 0 : sizeof(int) * (size_t)(a.g.B + 1));
    if ((e = launch_dependent(cache_attn_kernel<T, D, NT, false>, dim3(a.ncta), dim3(kThreads), smem, st, a)) != cudaSuccess)
        return e;
    // index rows that are whole (see launch_cache_attn) leave nothing to join: the error word alone
    const int64_t rows = a.idx && a.quantum == a.g.S ? 0 : (int64_t)a.g.ntok * a.g.Hq, most = (int64_t)num_sms() * 8;
    if (rows <= most)
        return launch_dependent(cache_join_kernel<T, D, 8>, dim3((unsigned)rows + 1), dim3(256), 0, st, a, NT * 8, a.err);
    return launch_dependent(cache_join_kernel<T, D, 2>, dim3((unsigned)(rows < 4 * most ? rows : 4 * most) + 1), dim3(64), 0, st, a, NT * 8, a.err);
}

template <typename T> cudaError_t attn_d(const AttnArgs &a, int nt, cudaStream_t st)
{
#define NSA_NT(D)                                   \
    switch (nt) {                                   \
    case 1: return attn_t<T, D, 1>(a, st);     \
    case 2: return attn_t<T, D, 2>(a, st);     \
    default: return attn_t<T, D, 4>(a, st);    \
    }
    if (a.g.D == 128)
        NSA_NT(128)
    else if (a.g.D == 64)
        NSA_NT(64)
    else
        NSA_NT(32)
#undef NSA_NT
}

struct AttnLayout {
    size_t status, prefix, ml, o, total;
};
AttnLayout attn_layout(const Geo &g, bool sel)
{
    const size_t ncta = ctas_of(g, sel), R = row_tile(g, sel) * 8;
    AttnLayout w;
    w.status = 256;
    w.prefix = w.status + up256(sizeof(int) * ncta);
    w.ml = w.prefix + up256(sizeof(int) * (size_t)(g.B + 1));
    w.o = w.ml + up256(sizeof(float2) * ncta * 2 * R);
    w.total = w.o + up256(sizeof(float) * ncta * 2 * R * g.D);
    return w;
}

}  // namespace

bool cache_attn_clustered(const Geo &g, const Cache &c, bool sel) { return cluster_size(g, c, sel) > 0; }

int cache_attn_max_rows() { return kMaxRows; }

int64_t cache_attn_entries(const Geo &g, const Cache &c, bool sel)
{
    const int R = row_tile(g, sel) * 8;
    return sel ? (int64_t)g.ntok * g.Hkv * g.S * ((g.G + R - 1) / R)
               : (int64_t)g.B * (c.cols + start_cost(g)) * g.Hkv * ((longest_rows(g) + R - 1) / R);
}

size_t cache_attn_ws_bytes(const Geo &g, const Cache &c, bool sel) { return cluster_size(g, c, sel) > 0 ? 256 : attn_layout(g, sel).total; }

cudaError_t launch_cache_attn(const Geo &g, const Cache &c, const void *q, const int *idx, const float *sinks, void *o,
                              float *lse, int dtype, char *ws, cudaStream_t st)
{
    const bool sel = idx != nullptr;
    const AttnLayout w = attn_layout(g, sel);
    AttnArgs a;
    a.g = g;
    a.c = c;
    a.q = q;
    a.idx = idx;
    a.sinks = sinks;
    a.o = o;
    a.lse = lse;
    const int nt = row_tile(g, sel);
    a.row_tiles = (g.G + nt * 8 - 1) / (nt * 8);
    a.ncta = ctas_of(g, sel);
    a.cs = cluster_size(g, c, sel);
    a.err = (int *)ws;
    if (a.cs > 0) {
        if (!sel)
            a.row_tiles = (int)((longest_rows(g) + nt * 8 - 1) / (nt * 8));
        a.units = (sel ? g.ntok : g.B) * g.Hkv * a.row_tiles;
    }
    // a run is cut at multiples of 128 tokens, a step of the CTA's warps; of
    // index rows, whole ones where that leaves the fullest CTA at most a
    // quarter above the average (nothing is to join then)
    a.quantum = 128 / c.bs;
    const int64_t units = (int64_t)g.ntok * g.Hkv * a.row_tiles;
    if (sel && (units + a.ncta - 1) / a.ncta * a.ncta * 4 <= units * 5)
        a.quantum = g.S;
    a.start_cost = start_cost(g);
    a.status = (int *)(ws + w.status);
    a.prefix = (int *)(ws + w.prefix);
    a.part_ml = (float2 *)(ws + w.ml);
    a.part_o = (float *)(ws + w.o);
    a.by_G = FastDiv(g.G);
    a.by_Hkv = FastDiv(g.Hkv);
    a.by_Hq = FastDiv(g.Hq);
    a.by_T = FastDiv(g.T);
    a.by_S = FastDiv(max(g.S, 1));
    a.by_tiles = FastDiv(a.row_tiles);
    a.by_ncta = FastDiv(a.ncta);
    a.by_quantum = FastDiv(a.quantum);
    return dtype == NSA_DTYPE_BF16 ? attn_d<__nv_bfloat16>(a, nt, st) : attn_d<float>(a, nt, st);
}

}  // namespace nsa
