// k_evict.cu -- rows beyond their number of blocks give back those with the
// least accumulated attention weight.
//
// A row of n blocks (the last may be partly filled) keeps `keep`: its first
// `first`, its last `recent` and, of the others, those with the largest sum over
// the kv heads of weight[b, head, block] (heads added in order; equal sums: the
// lower block stays; NaN ranks below everything).  Table, weights and whatever
// the row holds behind its length close up, the length shrinks by the dropped
// blocks' tokens, their pages lose a reference.
//
// A block of threads per row.  The K-th largest sum is found digit by digit (8
// bits a pass, a histogram in shared memory) on the sums' bits in floats' order;
// one ordered pass then moves what stays to the front: a column never moves up,
// so a batch of columns is read before it is written and nothing is copied
// aside.  What bounds it: for many rows the bytes (table, kept and weights, read
// and written once), for few the chain of passes.  Measured: 256 rows of 100 ..
// 65536 tokens in blocks of 32 to 512 blocks, 25 us profiled; 8 rows of up to 8192 to 64
// blocks of 64, 11 us and the launch.  One column a thread and batch, and a shared addition
// for each sum: 2 us more.
#include <math.h>

#include "cache_common.cuh"
#include "launch.h"
#include "tc_common.cuh"

namespace nsa {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kCols = 4;          // columns of a thread in a batch
constexpr int kMaxKeys = 48 * 1024;  // sums kept in shared memory; a wider table's are added up again where they are needed

struct EvictArgs {
    Cache c;
    float *weight;  // [rows, Hkv, cols]
    int *kept;      // [rows, cols], or nullptr
    int keep, first, recent;
    int *err;
    int in_smem;
};

// a float's place in the floats' order, NaN lowest
__device__ __forceinline__ uint32_t order_of(float x)
{
    const uint32_t u = __float_as_uint(x + 0.f);  // (-0 to 0)
    return x != x ? 0u : u >> 31 ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictArgs a)
{
    extern __shared__ uint32_t keys[];
    __shared__ int hist[256];
    __shared__ __align__(8) int counts[2][kCols][kWarps];
    __shared__ int s_digit, s_want;
    dependents_may_start();
    dependency_wait();
    const Cache &c = a.c;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int len = c.lens[b], cols = c.cols;
    int *table = c.table + (int64_t)b * cols, *kept = a.kept ? a.kept + (int64_t)b * cols : nullptr;
    float *weight = a.weight + (int64_t)b * c.Hkv * cols;
    const bool fits = len >= 0 && len <= cols * c.bs;
    const int n = fits ? (int)(((int64_t)len + c.bs - 1) >> c.bsh) : 0;
    bool bad = !fits;
    if (n > a.keep)  // every block of a row that changes has a page in use
#pragma unroll 4
        for (int j = tid; j < n; j += kThreads) {
            const int page = table[j];
            bad |= page < 0 || page >= c.pages || c.ref[page] < 1;
        }
    bad = __syncthreads_or(bad);
    if (bad && tid == 0)
        set_error(a.err, NSA_ERR_BAD_INDEX);
    if (bad || n <= a.keep) {
        if (kept)
            for (int j = tid; j < cols; j += kThreads)
                kept[j] = j;
        return;
    }
    // ---- the candidates [lo, hi) and their keys
    const int lo = a.first, hi = n - a.recent;
    auto add_up = [&](int j) {
        float x = weight[j];
#pragma unroll 4
        for (int h = 1; h < c.Hkv; ++h)
            x += weight[(int64_t)h * cols + j];
        return order_of(x);
    };
    if (a.in_smem) {
#pragma unroll 4
        for (int j = lo + tid; j < hi; j += kThreads)
            keys[j] = add_up(j);
        __syncthreads();
    }
    auto key = [&](int j) { return a.in_smem ? keys[j] : add_up(j); };
    // ---- the K-th largest: digits from the top, `want` of those with the digits so far still to stay
    uint32_t top = 0;
    int want = a.keep - a.first - a.recent;
    const bool none = want == 0;  // no candidate stays
    for (int shift = 24; shift >= 0 && !none; shift -= 8) {
        if (tid < 256)
            hist[tid] = 0;
        __syncthreads();
        for (int j0 = lo; j0 < hi; j0 += kThreads) {  // a warp adds equal digits (most of the first ones are) once
            const int j = j0 + tid;
            const uint32_t k = j < hi ? key(j) : 0;
            const uint32_t digit = j < hi && (shift == 24 || k >> (shift + 8) == top >> (shift + 8)) ? k >> shift & 255u : 256u;
            const uint32_t same = __match_any_sync(0xffffffffu, digit);
            if (digit < 256u && lane == __ffs(same) - 1)
                atomicAdd(&hist[digit], __popc(same));
        }
        __syncthreads();
        if (warp == 0) {  // lane l: digits 255 - 8 l downwards
            int own[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                own[i] = hist[255 - lane * 8 - i];
                sum += own[i];
            }
            int incl = sum;
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                incl += lane >= o ? y : 0;
            }
            int before = incl - sum;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (before < want && before + own[i] >= want) {  // (one lane, one digit)
                    s_digit = 255 - lane * 8 - i;
                    s_want = want - before;
                }
                before += own[i];
            }
        }
        __syncthreads();
        top |= (uint32_t)s_digit << shift;
        want = s_want;
    }
    // ---- what stays closes up, a batch of columns at a time: thread t has columns
    // t, t + kThreads .., and each warp's votes give every column its place
    auto places = [&](const uint32_t (&votes)[kCols], int (*count)[kWarps], int (&nth)[kCols]) {
#pragma unroll
        for (int v = 0; v < kCols; ++v)
            if (lane == 0)
                count[v][warp] = __popc(votes[v]);
        __syncthreads();
        static_assert(kCols * kWarps == 64, "two counts a lane");
        const int2 own = ((const int2 *)count)[lane];
        int incl = own.x + own.y;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            incl += lane >= o ? y : 0;
        }
        const int before = incl - own.x - own.y;
#pragma unroll
        for (int v = 0; v < kCols; ++v) {
            const int at = v * kWarps + warp, x = __shfl_sync(0xffffffffu, before, at / 2), first = __shfl_sync(0xffffffffu, own.x, at / 2);
            nth[v] = x + (at & 1 ? first : 0) + __popc(votes[v] & ((1u << lane) - 1u));
        }
        return __shfl_sync(0xffffffffu, incl, 31);
    };
    bool low = false;       // a page was dropped more often than its count said
    int equal = 0, to = 0;  // candidates equal to `top`, and columns that stay, before the batch
    for (int j0 = 0; j0 < cols; j0 += kThreads * kCols) {
        uint32_t k[kCols], votes[kCols];
        int nth[kCols], dst[kCols], page[kCols], was[kCols];
        bool stays[kCols];
#pragma unroll
        for (int v = 0; v < kCols; ++v) {
            const int j = j0 + v * kThreads + tid;
            const bool cand = j >= lo && j < hi;
            page[v] = j < cols ? table[j] : -1;
            k[v] = cand && !none ? key(j) : 0;
            votes[v] = __ballot_sync(0xffffffffu, cand && !none && k[v] == top);
        }
        const int ties = places(votes, counts[0], nth);
#pragma unroll
        for (int v = 0; v < kCols; ++v) {
            const int j = j0 + v * kThreads + tid;
            const bool cand = j >= lo && j < hi;
            stays[v] = j < cols && (!cand || (!none && (k[v] > top || (k[v] == top && equal + nth[v] < want))));
            votes[v] = __ballot_sync(0xffffffffu, stays[v]);
        }
        const int staying = places(votes, counts[1], dst);
#pragma unroll
        for (int v = 0; v < kCols; ++v) {
            const int j = j0 + v * kThreads + tid;
            dst[v] += to;
            was[v] = j < cols && !stays[v] ? atomicSub(c.ref + page[v], 1) : 1;  // (a page of the pool: checked)
            stays[v] = stays[v] && dst[v] != j;  // (from here on: moves)
            if (kept && j < cols && dst[v] == j)
                kept[j] = j;
        }
        equal += ties;
        to += staying;
        constexpr int kHeads = 4;  // heads whose weights are under way together
        for (int h0 = 0; h0 < c.Hkv; h0 += kHeads) {
            float x[kCols][kHeads];
#pragma unroll
            for (int v = 0; v < kCols; ++v)
#pragma unroll
                for (int h = 0; h < kHeads; ++h)
                    x[v][h] = stays[v] && h0 + h < c.Hkv ? weight[(int64_t)(h0 + h) * cols + j0 + v * kThreads + tid] : 0.f;
            __syncthreads();  // the batch is read
#pragma unroll
            for (int v = 0; v < kCols; ++v)
#pragma unroll
                for (int h = 0; h < kHeads; ++h)
                    if (stays[v] && h0 + h < c.Hkv)
                        weight[(int64_t)(h0 + h) * cols + dst[v]] = x[v][h];
        }
#pragma unroll
        for (int v = 0; v < kCols; ++v)
            if (stays[v]) {
                table[dst[v]] = page[v];
                if (kept)
                    kept[dst[v]] = j0 + v * kThreads + tid;
            }
#pragma unroll
        for (int v = 0; v < kCols; ++v)
            if (was[v] <= 0) {
                atomicAdd(c.ref + page[v], 1);
                low = true;
            }
    }
    __syncthreads();
    for (int j = to + tid; j < cols; j += kThreads) {
        table[j] = -1;
        if (kept)
            kept[j] = -1;
        for (int h = 0; h < c.Hkv; ++h)
            weight[(int64_t)h * cols + j] = 0.f;
    }
    if (low)
        set_error(a.err, NSA_ERR_BAD_INDEX);
    if (tid == 0)
        c.lens[b] = len - (cols - to) * c.bs;
}

}  // namespace

cudaError_t launch_cache_evict(const Cache &c, float *weight, int keep, int first, int recent, int *kept, int *err, cudaStream_t st)
{
    EvictArgs a = {c, weight, kept, keep, first, recent, err, c.cols <= kMaxKeys};
    const size_t smem = a.in_smem ? sizeof(uint32_t) * (size_t)c.cols : 0;
    if (smem > 40 * 1024) {
        cudaError_t e = allow_shared((const void *)evict_kernel);
        if (e != cudaSuccess)
            return e;
    }
    return launch_dependent(evict_kernel, dim3(c.rows), dim3(kThreads), smem, st, a);
}

}  // namespace nsa
