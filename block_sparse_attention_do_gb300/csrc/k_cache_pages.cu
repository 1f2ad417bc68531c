// k_cache_pages.cu -- the pages of the cache: reserving them for rows that
// grow, freeing, sharing between forked rows, copying and compacting.
//
// The pool's whole state is one reference count per page (0: free), the
// page table and the rows' lengths.  "The lowest free pages first" makes the
// choice of pages a function of that state alone, whatever order the threads
// run in.  The metadata of a call is one cluster of 1 to 8 CTAs, by the size of
// pool and lists: the counts are read by all its threads at once, barriers
// stand between the steps, and the calls need no host round trip.  What bounds
// it is the chain of those steps (a few dependent reads each, about 0.6 us, and
// as much for a barrier of several CTAs), not the bytes: 0.26 MB of counts for
// 65,536 pages.  The pages' contents move in a wide launch that is bound by
// memory bandwidth: 300 pages of 131 KB, 79 MB read and written, in 14.3 us
// (profiled), 5.5 TB/s; 11.6 at a plain copy's rate; 18 for the call.  Calls
// measured (of each, 4 us are any launch's): 64 of 72 rows forked in a pool of
// 4096 pages 14 us, 64 rows freed and reserved again in one of 65,536 15 us, a
// pool of 4096 compacted 23 us, whose bytes would take 9.9 at a copy's rate.
// Lists, counts and contents in one launch of all SMs, with barriers between
// them, was slower (copy 39 us).
#include <cooperative_groups.h>

#include "cache_common.cuh"
#include "launch.h"
#include "tc_common.cuh"

namespace cg = cooperative_groups;

namespace nsa {

namespace {

constexpr int kMaxCluster = 8;  // (the portable size)
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

struct Where {
    int rank, ctas;        // CTA of the cluster, and their number
    int warp, warps;       // warp of the cluster, and their number
    int lane;
    int thread, threads;   // of the cluster
};
__device__ __forceinline__ Where where(const cg::cluster_group &cl)
{
    const int rank = (int)cl.block_rank(), ctas = (int)cl.num_blocks();
    return Where{rank, ctas, rank * kWarps + (int)(threadIdx.x >> 5), ctas * kWarps, (int)(threadIdx.x & 31),
                 rank * kThreads + (int)threadIdx.x, ctas * kThreads};
}

// blocks that hold len tokens
__device__ __forceinline__ int blocks_of(int len, const Cache &c) { return (int)(((int64_t)len + c.bs - 1) >> c.bsh); }

// Each warp of the cluster owns one run of pages: count() counts those that
// pred() names, scan() turns the cluster's counts into the number before the
// calling warp's run and the total.
struct Runs {
    int begin, end;
    __device__ __forceinline__ Runs(const Cache &c, const Where &w)
    {
        const int per = ((c.pages + w.warps - 1) / w.warps + 31) & ~31;
        begin = (int)min((int64_t)c.pages, (int64_t)w.warp * per);
        end = min(c.pages, begin + per);
    }
    template <typename P> __device__ __forceinline__ int count(int lane, P pred) const
    {
        int n = 0;
#pragma unroll 8
        for (int p = begin + lane; p < end; p += 32)
            n += pred(p) ? 1 : 0;
        return __reduce_add_sync(0xffffffffu, n);
    }
};

// every warp's count into every CTA's table (the cluster synchronises after)
__device__ __forceinline__ void share_count(const cg::cluster_group &cl, int *counts, const Where &w, int n)
{
    if (w.lane < w.ctas)
        cl.map_shared_rank(counts, w.lane)[w.warp] = n;
}
__device__ __forceinline__ void scan_counts(const int *counts, const Where &w, int &before, int &total)
{
    int b = 0, t = 0;
    for (int i = w.lane; i < w.warps; i += 32) {
        t += counts[i];
        b += i < w.warp ? counts[i] : 0;
    }
    before = __reduce_add_sync(0xffffffffu, b);
    total = __reduce_add_sync(0xffffffffu, t);
}

// Exclusive prefix over i < n of need(i), by one CTA: out[i] (if given), the
// sum returned to every thread.
template <typename F> __device__ int64_t cta_prefix(int n, int *out, F need)
{
    __shared__ int64_t part[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t base = 0;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + threadIdx.x;
        const int64_t x = i < n ? need(i) : 0;
        int64_t incl = x;
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
            incl += lane >= o ? y : 0;
        }
        if (lane == 31)
            part[warp] = incl;
        __syncthreads();
        int64_t before = base, all = base;
        for (int k = 0; k < kWarps; ++k) {
            before += k < warp ? part[k] : 0;
            all += part[k];
        }
        if (out && i < n)
            out[i] = (int)min(before + incl - x, (int64_t)INT32_MAX);
        base = all;
        __syncthreads();
    }
    return base;
}

constexpr int kBatch = 4;  // reads of a thread under way together

// Takes the `total` lowest free pages: order[i] = the i-th, its count 1.
__device__ __forceinline__ void take_free(const Cache &c, const Runs &r, int lane, int before, int total, int *order)
{
    for (int p0 = r.begin + lane; p0 - lane < r.end && before < total; p0 += 32 * kBatch) {
        int count[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            count[u] = p0 + u * 32 < r.end ? __ldcg(c.ref + p0 + u * 32) : 1;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const unsigned m = __ballot_sync(0xffffffffu, count[u] <= 0);
            const int nth = before + __popc(m & ((1u << lane) - 1u));
            if (count[u] <= 0 && nth < total) {
                order[nth] = p0 + u * 32;
                c.ref[p0 + u * 32] = 1;
            }
            before += __popc(m);
        }
    }
}

// Rows' columns in pieces of kPiece, a warp each: for_pieces calls f(i, col0)
// for piece col0 .. of list position i.
constexpr int kPiece = 32 * kBatch;
template <typename F> __device__ __forceinline__ void for_pieces(const Cache &c, const Where &w, int n, F f)
{
    const int per = (c.cols + kPiece - 1) / kPiece;  // (n * per is below rows * columns: an int)
    for (int x = w.warp; x < n * per; x += w.warps) {
        const int i = per == 1 ? x : x / per;
        f(i, (x - i * per) * kPiece);
    }
}
// a piece of row r's table entries, lane by lane (-1 past the table's width)
__device__ __forceinline__ void load_piece(const Cache &c, int r, int col0, int lane, int (&p)[kBatch])
{
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
        const int col = col0 + u * 32 + lane;
        p[u] = col < c.cols ? c.table[(int64_t)r * c.cols + col] : -1;
    }
}

// Gives back a piece of the pages of row r and empties it: true if an entry
// names no page or a page that nobody holds.
__device__ __forceinline__ bool release_piece(const Cache &c, int r, int col0, int lane)
{
    int p[kBatch], was[kBatch];
    load_piece(c, r, col0, lane, p);
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
        was[u] = p[u] >= 0 && p[u] < c.pages ? atomicSub(c.ref + p[u], 1) : p[u] == -1 ? 1 : 0;
    bool bad = false;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
        if (was[u] <= 0) {
            bad = true;
            if (p[u] >= 0 && p[u] < c.pages)
                atomicAdd(c.ref + p[u], 1);
        }
        const int col = col0 + u * 32 + lane;
        if (col < c.cols)
            c.table[(int64_t)r * c.cols + col] = -1;
    }
    return bad;
}

// ---- reserve: row b grows by n_new[b] tokens; all rows or none ------------
// The columns that row b grows into; false where it cannot.
__device__ __forceinline__ bool grown_columns(const Cache &c, const int *n_new, int b, int &have, int &want)
{
    const int len = c.lens[b], n = n_new[b];
    const bool ok = n >= 0 && len >= 0 && (int64_t)len + n <= (int64_t)c.cols * c.bs;
    have = ok ? blocks_of(len, c) : 0;
    want = ok ? blocks_of(len + n, c) : 0;
    return ok;
}

// How many of columns [have, want) of row b hold a page of the row's alone; -1
// where one holds what is no page in use.  (The whole warp.)
__device__ __forceinline__ int held_columns(const Cache &c, int b, int have, int want, int lane)
{
    int held = 0;
    bool none = false;
#pragma unroll 4
    for (int col = have + lane; col < want; col += 32) {
        const int p = c.table[(int64_t)b * c.cols + col];
        if (p != -1) {
            const int count = p >= 0 && p < c.pages ? c.ref[p] : 0;
            held += count == 1;
            none |= count <= 0;
        }
    }
    none = __any_sync(0xffffffffu, none);
    held = __reduce_add_sync(0xffffffffu, held);
    return none ? -1 : held;
}

__global__ void __launch_bounds__(kThreads)
    cache_reserve_kernel(const Cache c, const int *n_new, const CacheWs ws)
{
    dependents_may_start();
    dependency_wait();
    cg::cluster_group cl = cg::this_cluster();
    __shared__ int counts[kMaxCluster * kWarps];
    __shared__ int bad, kept;
    __shared__ int64_t need_all;
    const Where w = where(cl);
    if (threadIdx.x == 0)
        bad = kept = 0;
    cl.sync();  // every CTA of the cluster runs from here on: its shared memory may be written
    // every CTA checks every row and knows the sum; CTA 0 writes the offsets.
    // A row whose length was lowered holds a page in the first column that it
    // grows into: its own is kept, one that it shares is given back for another
    // (the read of a thread's first row is under way with the counts)
    int in_first = -1;
    bool none = false, held = false;
#pragma unroll 4
    for (int b = threadIdx.x; b < c.rows; b += kThreads) {
        int have, want;
        held |= in_first != -1;
        none |= !grown_columns(c, n_new, b, have, want);
        in_first = want > have ? c.table[(int64_t)b * c.cols + have] : -1;
    }
    if (none)
        bad = 1;
    const Runs run(c, w);
    share_count(cl, counts, w, run.count(w.lane, [&](int p) { return c.ref[p] <= 0; }));
    if (held || in_first != -1)
        kept = 1;
    int64_t total;
    if (w.rank == 0) {
        total = cta_prefix(c.rows, ws.r1, [&](int b) {
            int have, want;
            grown_columns(c, n_new, b, have, want);
            return want - have;
        });
        if (threadIdx.x < w.ctas)
            *cl.map_shared_rank(&need_all, threadIdx.x) = total;
    }
    cl.sync();
    total = need_all;
    int before, free;
    scan_counts(counts, w, before, free);
    if (kept && !bad) {  // off the common path: what each row lacks (-1: it cannot grow)
        for (int b = w.warp; b < c.rows; b += w.warps) {
            int have, want;
            grown_columns(c, n_new, b, have, want);
            const int held = held_columns(c, b, have, want, w.lane);
            if (w.lane == 0)
                ws.r0[b] = held < 0 ? -1 : want - have - held;
        }
        cl.sync();
        total = cta_prefix(c.rows, w.rank == 0 ? ws.r1 : nullptr, [&](int b) {
            const int lacks = __ldcg(ws.r0 + b);
            if (lacks < 0)
                bad = 1;
            return max(lacks, 0);
        });
    }
    const bool full = total > free;
    if (w.rank == 0 && threadIdx.x == 0)
        *ws.err = bad ? NSA_ERR_BAD_INDEX : full ? NSA_ERR_CACHE_FULL : NSA_OK;
    if (bad || full)
        return;  // the same in every CTA: nothing has changed
    take_free(c, run, w.lane, before, (int)total, ws.p2);
    cl.sync();
    for (int b = w.warp; b < c.rows; b += w.warps) {
        const int len = c.lens[b], n = n_new[b];
        const int have = blocks_of(len, c), want = blocks_of(len + n, c), off = __ldcg(ws.r1 + b);
        int *row = c.table + (int64_t)b * c.cols;
        if (!kept) {
#pragma unroll 4
            for (int col = have + w.lane; col < want; col += 32)
                row[col] = __ldcg(ws.p2 + off + col - have);
        } else
            for (int col0 = have, nth = off; col0 < want; col0 += 32) {  // the empty columns, and those of shared pages
                const int col = col0 + w.lane, old = col < want ? row[col] : -1;
                const bool lacks = col < want && (old == -1 || c.ref[old] > 1);
                const unsigned m = __ballot_sync(0xffffffffu, lacks);
                const int i = nth + __popc(m & ((1u << w.lane) - 1u));
                if (lacks) {
                    row[col] = __ldcg(ws.p2 + i);
                    ws.p0[i] = old;
                }
                nth += __popc(m);
            }
        __syncwarp();
        if (w.lane == 0)
            c.lens[b] = len + n;
    }
    if (!kept)
        return;
    cl.sync();  // (every row has read the counts)
    for (int i = w.thread; i < (int)total; i += w.threads) {
        const int old = __ldcg(ws.p0 + i);
        if (old >= 0)
            atomicSub(c.ref + old, 1);
    }
}

// Claims: first(x) = the first position of `list` that names x, -1 where `no`
// (if given) names it.  Few names are marked in each CTA's shared memory, by
// every CTA for itself; many in global memory, by the cluster together.
constexpr int kMarks = 2048;
struct Claims {
    int *mark;
    bool shared;
    __device__ Claims(const cg::cluster_group &cl, const Where &w, const int *list, const int *no, int n, int names, int *own, int *global)
        : mark(names <= kMarks ? own : global), shared(names <= kMarks)
    {
        const int step = shared ? kThreads : w.threads, first = shared ? (int)threadIdx.x : w.thread;
        for (int i = first; i < n; i += step) {
            if (list[i] >= 0 && list[i] < names)
                mark[list[i]] = INT32_MAX;
            if (no && no[i] >= 0 && no[i] < names)
                mark[no[i]] = INT32_MAX;
        }
        sync(cl);
        for (int i = first; i < n; i += step) {
            if (list[i] >= 0 && list[i] < names)
                atomicMin(mark + list[i], i);
            if (no && no[i] >= 0 && no[i] < names)
                atomicMin(mark + no[i], -1);
        }
        sync(cl);
    }
    __device__ __forceinline__ void sync(const cg::cluster_group &cl) const
    {
        if (shared)
            __syncthreads();
        else
            cl.sync();
    }
    __device__ __forceinline__ int first(int x) const { return shared ? mark[x] : __ldcg(mark + x); }
};

// ---- free: the listed rows give back their pages ---------------------------
__global__ void __launch_bounds__(kThreads)
    cache_free_kernel(const Cache c, const int *rows, int n, const CacheWs ws)
{
    dependents_may_start();
    dependency_wait();
    cg::cluster_group cl = cg::this_cluster();
    const Where w = where(cl);
    if (w.rank == 0 && threadIdx.x == 0)
        *ws.err = NSA_OK;
    __shared__ int marks[kMarks];
    const Claims claims(cl, w, rows, nullptr, n, c.rows, marks, ws.r0);
    cl.sync();  // (the error word is clear)
    bool bad = false;
    for_pieces(c, w, n, [&](int i, int col0) {
        const int r = rows[i];
        if (r < 0 || r >= c.rows || claims.first(r) != i) {  // no row, or listed before
            bad = true;
            return;
        }
        bad |= release_piece(c, r, col0, w.lane);
        if (col0 == 0 && w.lane == 0)
            c.lens[r] = 0;
    });
    if (bad)
        set_error(ws.err, NSA_ERR_BAD_INDEX);
}

// ---- fork: row dst[i] becomes a continuation of row src[i] -----------------
__global__ void __launch_bounds__(kThreads)
    cache_fork_kernel(const Cache c, const int *src, const int *dst, int n, const CacheWs ws)
{
    dependents_may_start();
    dependency_wait();
    cg::cluster_group cl = cg::this_cluster();
    __shared__ int counts[kMaxCluster * kWarps];
    __shared__ int64_t tails_all;
    const Where w = where(cl);
    if (w.rank == 0 && threadIdx.x == 0) {
        *ws.err = NSA_OK;
        *ws.npairs = 0;
    }
    __shared__ int marks[kMarks];
    const Claims claims(cl, w, dst, src, n, c.rows, marks, ws.r0);
    cl.sync();  // (the error word is clear; every CTA runs: its shared memory may be written)
    bool bad = false;
    for_pieces(c, w, n, [&](int i, int col0) {
        const int s = src[i], d = dst[i];
        if (s < 0 || s >= c.rows || d < 0 || d >= c.rows || claims.first(d) != i) {
            bad = true;
            return;
        }
        const int len = c.lens[s];
        if (len < 0 || len > c.cols * c.bs) {
            bad = true;
            return;
        }
        int p[kBatch], x[kBatch];
        load_piece(c, s, col0, w.lane, p);
        load_piece(c, d, col0, w.lane, x);
        const int used = blocks_of(len, c);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {  // src's pages, and what dst gives up, are pages in use
            const bool needed = col0 + u * 32 + w.lane < used;
            bad |= p[u] >= c.pages || (needed && p[u] < 0) || x[u] < -1 || x[u] >= c.pages;
            p[u] = needed && p[u] >= 0 && p[u] < c.pages ? c.ref[p[u]] : 1;
            x[u] = x[u] >= 0 && x[u] < c.pages ? c.ref[x[u]] : 1;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            bad |= p[u] < 1 || x[u] < 1;
    });
    if (bad)
        set_error(ws.err, NSA_ERR_BAD_INDEX);
    cl.sync();
    if (__ldcg(ws.err) != NSA_OK)
        return;  // the same in every CTA: nothing has changed
    // the destinations' own pages come back first: a tail may reuse them (an
    // error here: more table entries name a page than its count says)
    for_pieces(c, w, n, [&](int i, int col0) {
        int p[kBatch];
        load_piece(c, dst[i], col0, w.lane, p);
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (p[u] >= 0)
                bad |= atomicSub(c.ref + p[u], 1) <= 0;
    });
    cl.sync();  // every thread has read ws.err: it may be written again
    if (bad)
        set_error(ws.err, NSA_ERR_BAD_INDEX);
    const Runs run(c, w);
    share_count(cl, counts, w, run.count(w.lane, [&](int p) { return __ldcg(c.ref + p) <= 0; }));
    if (w.rank == 0) {
        const int64_t t = cta_prefix(n, ws.r1, [&](int i) { return (c.lens[src[i]] & (c.bs - 1)) != 0 ? 1 : 0; });
        if (threadIdx.x < w.ctas)
            *cl.map_shared_rank(&tails_all, threadIdx.x) = t;
    }
    cl.sync();
    const int64_t tails = tails_all;
    int before, free;
    scan_counts(counts, w, before, free);
    // (a thread that reads the word late may find CACHE_FULL there: the same)
    if (tails > free || __ldcg(ws.err) != NSA_OK) {  // undo: nothing has changed
        for_pieces(c, w, n, [&](int i, int col0) {
            int p[kBatch];
            load_piece(c, dst[i], col0, w.lane, p);
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (p[u] >= 0)
                    atomicAdd(c.ref + p[u], 1);
        });
        if (w.rank == 0 && threadIdx.x == 0)
            set_error(ws.err, NSA_ERR_CACHE_FULL);
        return;
    }
    take_free(c, run, w.lane, before, (int)tails, ws.p2);
    cl.sync();
    for_pieces(c, w, n, [&](int i, int col0) {
        const int s = src[i], d = dst[i], len = c.lens[s];
        const int full = len >> c.bsh;
        const bool tail = (len & (c.bs - 1)) != 0;
        const int nth = __ldcg(ws.r1 + i);
        int p[kBatch];
        load_piece(c, s, col0, w.lane, p);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int col = col0 + u * 32 + w.lane;
            int mine = -1;
            if (col < full) {
                mine = p[u];
                atomicAdd(c.ref + mine, 1);
            } else if (col == full && tail) {
                mine = __ldcg(ws.p2 + nth);
                ws.p0[nth] = p[u];
                ws.p1[nth] = mine;
            }
            if (col < c.cols)
                c.table[(int64_t)d * c.cols + col] = mine;
        }
        if (col0 == 0 && w.lane == 0)
            c.lens[d] = len;
    });
    if (w.rank == 0 && threadIdx.x == 0)
        *ws.npairs = (int)tails;
}

// ---- copy: the pairs that may be copied -------------------------------------
// A pair with a page outside the pool, a destination that an earlier pair
// has, or a destination that is any pair's source is left out (-1).
__global__ void __launch_bounds__(kThreads)
    cache_copy_check_kernel(const Cache c, const int *src, const int *dst, int n, const CacheWs ws)
{
    dependents_may_start();
    dependency_wait();
    cg::cluster_group cl = cg::this_cluster();
    const Where w = where(cl);
    if (w.rank == 0 && threadIdx.x == 0) {
        *ws.err = NSA_OK;
        *ws.npairs = n;
    }
    __shared__ int marks[kMarks];
    const Claims claims(cl, w, dst, src, n, c.pages, marks, ws.p2);
    cl.sync();
    bool bad = false;
    for (int i = w.thread; i < n; i += w.threads) {
        const int s = src[i], d = dst[i];
        const bool ok = s >= 0 && s < c.pages && d >= 0 && d < c.pages && claims.first(d) == i;
        ws.p0[i] = ok ? s : -1;
        ws.p1[i] = ok ? d : -1;
        bad |= !ok;
    }
    if (bad)
        set_error(ws.err, NSA_ERR_BAD_INDEX);
}

// ---- compact: live pages to the front of the pool ---------------------------
// With n live pages, the live pages at n and above move, in order, to the
// free pages below n, in order.
__global__ void __launch_bounds__(kThreads) cache_compact_kernel(const Cache c, const CacheWs ws)
{
    dependents_may_start();
    dependency_wait();
    cg::cluster_group cl = cg::this_cluster();
    __shared__ int counts[kMaxCluster * kWarps];
    __shared__ int low;  // live pages below n
    const Where w = where(cl);
    if (w.rank == 0 && threadIdx.x == 0)
        *ws.err = NSA_OK;
    cl.sync();  // every CTA of the cluster runs from here on: its shared memory may be written
    const Runs run(c, w);
    share_count(cl, counts, w, run.count(w.lane, [&](int p) { return c.ref[p] > 0; }));
    cl.sync();
    int before, n;
    scan_counts(counts, w, before, n);
    // the warp whose run holds page n (or, with every page live, the last)
    // knows how many live pages lie below it
    if (n == c.pages) {
        if (threadIdx.x == 0)
            low = n;
    } else if (n >= run.begin && n < run.end) {
        int k = before;
#pragma unroll 4
        for (int p0 = run.begin; p0 < n; p0 += 32) {
            const int p = p0 + w.lane;
            k += __popc(__ballot_sync(0xffffffffu, p < n && c.ref[p] > 0));
        }
        if (w.lane < w.ctas)
            *cl.map_shared_rank(&low, w.lane) = k;
    }
    cl.sync();
    const int moved = n - low;
    int rank = before;
    for (int p0 = run.begin + w.lane; p0 - w.lane < run.end; p0 += 32 * kBatch) {
        int count[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            count[u] = p0 + u * 32 < run.end ? c.ref[p0 + u * 32] : 0;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int p = p0 + u * 32;
            const bool live = count[u] > 0;
            const unsigned m = __ballot_sync(0xffffffffu, live);
            const int r = rank + __popc(m & ((1u << w.lane) - 1u));  // live pages below p
            if (live && p >= n) {
                ws.p0[r - low] = p;
                ws.p2[p] = r - low;
            } else if (!live && p < n && p < run.end)
                ws.p1[p - r] = p;
            rank += __popc(m);
        }
    }
    cl.sync();
    bool bad = false;
    const int64_t entries = (int64_t)c.rows * c.cols;
    for (int64_t i = w.thread; i < entries; i += w.threads) {
        const int p = c.table[i];
        if (p >= n && p < c.pages) {
            // p's place among the moved pages, if it is one of them (a free
            // page's entry of p2 was not written and may hold anything)
            const int k = __ldcg(ws.p2 + p);
            if (k >= 0 && k < moved && __ldcg(ws.p0 + k) == p)
                c.table[i] = __ldcg(ws.p1 + k);
            else
                bad = true;
        } else if (p < -1 || p >= c.pages)
            bad = true;
    }
    for (int k = w.thread; k < moved; k += w.threads) {
        const int s = __ldcg(ws.p0 + k), d = __ldcg(ws.p1 + k);
        c.ref[d] = c.ref[s];
        c.ref[s] = 0;
    }
    if (w.rank == 0 && threadIdx.x == 0)
        *ws.npairs = moved;
    if (bad)
        set_error(ws.err, NSA_ERR_BAD_INDEX);
}

// ---- the pages' contents ------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;                          // 16-byte vectors per thread in flight
constexpr int kChunk = kCopyThreads * kCopyVecs;      // vectors per step of a block

// Pairs p0 -> p1, each in chunks of 16 KB of its keys, then of its values.
__global__ void __launch_bounds__(kCopyThreads) cache_move_kernel(const Cache c, const CacheWs ws)
{
    dependents_may_start();
    dependency_wait();
    const int n = *ws.npairs;
    const int vtok = c.D / 16, sh_tok = 31 - __clz(vtok), sh_head = sh_tok + c.bsh;
    const int nvec = c.Hkv << sh_head;  // vectors of one page's keys
    const int chunks = (nvec + kChunk - 1) / kChunk;
    for (int64_t u = blockIdx.x; u < (int64_t)n * 2 * chunks; u += gridDim.x) {
        const int chunk = (int)(u % chunks);
        const int which = (int)(u / chunks & 1);
        const int64_t pair = u / chunks / 2;
        const int s = ws.p0[pair], d = ws.p1[pair];
        if (s < 0)
            continue;
        uint8_t *base = which ? c.v : c.k;
        uint4 x[kCopyVecs];
        int64_t off[kCopyVecs];
#pragma unroll
        for (int i = 0; i < kCopyVecs; ++i) {
            const int v = chunk * kChunk + i * kCopyThreads + threadIdx.x;
            off[i] = (int64_t)(v >> sh_head) * c.sh + (int64_t)((v >> sh_tok) & (c.bs - 1)) * c.st + (v & (vtok - 1)) * 16;
            if (v < nvec)
                x[i] = *(const uint4 *)(base + (int64_t)s * c.sp + off[i]);
        }
#pragma unroll
        for (int i = 0; i < kCopyVecs; ++i)
            if (chunk * kChunk + i * kCopyThreads + threadIdx.x < nvec)
                *(uint4 *)(base + (int64_t)d * c.sp + off[i]) = x[i];
        if (chunk == 0)
            for (int h = threadIdx.x; h < c.Hkv; h += kCopyThreads) {
                float *f = which ? c.vs : c.ks;
                f[(int64_t)d * c.Hkv + h] = f[(int64_t)s * c.Hkv + h];
            }
    }
}

// One cluster over `work` counts or entries: a CTA for each 512 of them.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), int64_t work, cudaStream_t st, Args... args)
{
    int ctas = 1;
    while (ctas < kMaxCluster && work > 512 * (int64_t)ctas)
        ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, KArgs(args)...);
}

}  // namespace

cudaError_t launch_cache_reserve(const Cache &c, const int *n_new, const CacheWs &ws, cudaStream_t st)
{
    return launch_cluster(cache_reserve_kernel, c.pages, st, c, n_new, ws);
}

cudaError_t launch_cache_free(const Cache &c, const int *rows, int n, const CacheWs &ws, cudaStream_t st)
{
    return launch_cluster(cache_free_kernel, (int64_t)n * c.cols, st, c, rows, n, ws);
}

cudaError_t launch_cache_fork(const Cache &c, const int *src, const int *dst, int n, const CacheWs &ws, cudaStream_t st)
{
    return launch_cluster(cache_fork_kernel, max((int64_t)c.pages, (int64_t)n * c.cols), st, c, src, dst, n, ws);
}

cudaError_t launch_cache_copy_check(const Cache &c, const int *src, const int *dst, int n, const CacheWs &ws,
                                    cudaStream_t st)
{
    return launch_cluster(cache_copy_check_kernel, n, st, c, src, dst, n, ws);
}

cudaError_t launch_cache_compact(const Cache &c, const CacheWs &ws, cudaStream_t st)
{
    return launch_cluster(cache_compact_kernel, max((int64_t)c.pages, (int64_t)c.rows * c.cols), st, c, ws);
}

cudaError_t launch_cache_move(const Cache &c, const CacheWs &ws, int max_pairs, cudaStream_t st)
{
    const int nvec = c.Hkv * c.bs * (c.D / 16);
    const int64_t units = (int64_t)max_pairs * 2 * ((nvec + kChunk - 1) / kChunk);
    const int64_t most = (int64_t)num_sms() * 8;
    return launch_dependent(cache_move_kernel, dim3((unsigned)(units < most ? units : most)), dim3(kCopyThreads), 0, st, c, ws);
}

}  // namespace nsa
