// k_accept.cu -- drafted tokens that were accepted move to consecutive places
// behind what their rows held before; the others are dropped.
//
// Row b ends in n drafts, path[b] names the accepted ones in ascending order
// (-1 behind them): draft path[i] goes to place i behind the row's first
// len - n tokens.  The first of them mostly stay where they are (path[i] = i);
// from the first that moves on, what the cache holds of them (code * scale, in
// 32 bits) is appended by append's own rule, so a page's scale grows only as
// far as the moved values need, and its earlier codes are rounded again then.
// A token never moves up, and the sources of a page's tokens lie in that page
// or behind it: a page is read whole before it is written, pages one after
// another, and nothing is needed to hold what moves.
//
// What bounds it: the chain of dependent reads (length -> path -> table -> codes,
// scales), about as long as the two launches it takes; the bytes are a few KB a
// row.  The first launch, one cluster, checks every row and writes lengths and
// errors; the second has a warp for each row, head and k or v.  Measured, 8 heads
// of 128: 128 rows of 64 drafts, up to 12 accepted, 6 and 13 us profiled; one row of 24,
// 8 accepted, 10 us with the append before it, replayed from a graph.
#include <math.h>

#include <cooperative_groups.h>

#include "cache_common.cuh"
#include "launch.h"
#include "tc_common.cuh"

namespace cg = cooperative_groups;

namespace nsa {

namespace {

constexpr int kPlanThreads = 512, kMoveWarps = 4;

// What the first kernel leaves for the second: where the row's first draft
// that moves goes (-1: none does), and how many drafts are accepted.
__global__ void __launch_bounds__(kPlanThreads)
    accept_plan_kernel(const Cache c, const int *n_new, const int *path, int A, const CacheWs ws)
{
    dependents_may_start();
    dependency_wait();
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), lane = threadIdx.x & 31;
    const int warp = rank * (kPlanThreads / 32) + (int)(threadIdx.x >> 5), warps = (int)cl.num_blocks() * (kPlanThreads / 32);
    if (rank == 0 && threadIdx.x == 0)
        *ws.err = NSA_OK;
    cl.sync();  // (the error word is clear)
    for (int b = warp; b < c.rows; b += warps) {
        const int *p = path + (int64_t)b * A;
        int x = lane < A ? p[lane] : -1;  // (under way with the counts)
        const int n = n_new[b], len = c.lens[b];
        bool bad = n < 0 || len < n || len > c.cols * c.bs;
        const int first = bad ? 0 : len - n;
        int a = 0, lead = 0, end = -1;  // end: the entry before the lanes'
        for (int i0 = 0; i0 < A; i0 += 32) {
            const int i = i0 + lane;
            if (i0 > 0)
                x = i < A ? p[i] : -1;
            const int up = __shfl_up_sync(0xffffffffu, x, 1), before = lane > 0 ? up : end;
            end = __shfl_sync(0xffffffffu, x, 31);
            // a prefix of drafts, ascending; -1 from its end on
            bad |= x < -1 || x >= max(n, 0) || (x >= 0 && before >= x) || (x >= 0 && i > 0 && before < 0);
            a += __popc(__ballot_sync(0xffffffffu, x >= 0));
            lead += __popc(__ballot_sync(0xffffffffu, x == i));  // (ascending: then all before stay too)
        }
        bad = __any_sync(0xffffffffu, bad);
        // the pages that tokens move from and to: in the pool, and the row's own
        if (!bad)
            for (int i0 = lead; i0 < a; i0 += 32) {
                const int i = i0 + lane;
                if (i < a) {
                    const int from = c.table[(int64_t)b * c.cols + ((first + p[i]) >> c.bsh)], to = c.table[(int64_t)b * c.cols + ((first + i) >> c.bsh)];
                    bad |= from < 0 || from >= c.pages || to < 0 || to >= c.pages || (c.ref && c.ref[to] != 1);
                }
            }
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) {
            if (bad)
                set_error(ws.err, NSA_ERR_BAD_INDEX);
            else
                c.lens[b] = first + a;
            ws.r0[b] = bad || lead == a ? -1 : lead;
            ws.r1[b] = a;
        }
    }
}

// A warp: row, head, k or v.  Codes go 16 bytes to a lane, D / 16 lanes to a
// token; a page's moved tokens stay in registers between maximum and rounding.
template <int D> __global__ void __launch_bounds__(kMoveWarps * 32) accept_move_kernel(const Cache c, const int *path, int A, const CacheWs ws)
{
    constexpr int L = D / 16, TOK = 32 / L, VEC = 64 / TOK;  // lanes of a token, tokens of a load, loads of a page
    dependents_may_start();
    dependency_wait();
    const int lane = threadIdx.x & 31, parts = 2 * c.Hkv, per = (parts + kMoveWarps - 1) / kMoveWarps;
    const int b = blockIdx.x / per, part = (blockIdx.x - b * per) * kMoveWarps + (threadIdx.x >> 5);
    const int lead = ws.r0[b], a = ws.r1[b];
    if (lead < 0 || part >= parts)
        return;
    const bool values = part >= c.Hkv;
    const int h = values ? part - c.Hkv : part, first = c.lens[b] - a;
    uint8_t *pool = (values ? c.v : c.k) + (int64_t)h * c.sh;
    float *scales = (values ? c.vs : c.ks) + h;
    const int *table = c.table + (int64_t)b * c.cols, *p = path + (int64_t)b * A;
    const int tok = lane / L, off = lane % L * 16;
    for (int i0 = lead; i0 < a;) {
        const int slot0 = (first + i0) & (c.bs - 1), n = min(a - i0, c.bs - slot0);  // the page's slots [slot0, slot0 + n)
        const int page = table[(first + i0) >> c.bsh];
        uint4 w[VEC];
        float ss[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            if (v * TOK >= n)
                break;
            w[v] = make_uint4(0, 0, 0, 0);
            ss[v] = 0.f;
            if (v * TOK + tok < n) {
                const int at = first + p[i0 + v * TOK + tok], from = table[at >> c.bsh];
                w[v] = *(const uint4 *)(pool + (int64_t)from * c.sp + (int64_t)(at & (c.bs - 1)) * c.st + off);
                ss[v] = scales[(int64_t)from * c.Hkv];
            }
        }
        const float old = slot0 > 0 ? scales[(int64_t)page * c.Hkv] : 0.f;
        float amax = 0.f;  // of the finite values
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            if (v * TOK >= n)  // (uniform over the warp)
                break;
            const uint32_t u[4] = {w[v].x, w[v].y, w[v].z, w[v].w};
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const uint32_t m = u[e / 4] >> (e % 4 * 8) & 0x7fu;  // a code's magnitude orders as its bits do
                top = max(top, m == 0x7fu ? 0u : m);
            }
            uint32_t lo, hi;
            e4m3x4_to_half(top, lo, hi);
            const float x = __half22float2(*(const __half2 *)&lo).x * ss[v];
            if (x < INFINITY) {
                amax = fmaxf(amax, x);
                continue;
            }
            // a product beyond float's range counts in no maximum: the largest of the others (as in append)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                e4m3x4_to_half(u[i], lo, hi);
                const float2 f = __half22float2(*(const __half2 *)&lo), g = __half22float2(*(const __half2 *)&hi);
                for (float y : {f.x, f.y, g.x, g.y}) {
                    y = fabsf(y * ss[v]);
                    amax = y < INFINITY ? fmaxf(amax, y) : amax;
                }
            }
        }
        amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
        const float scale = fmaxf(e4m3_scale(amax), old);
        uint8_t *dst = pool + (int64_t)page * c.sp;
        __syncwarp();  // (every lane has its codes: the page may be written)
        auto rounded = [&](uint4 x, float mul, float div) {  // four words of codes times mul / div
            uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t lo, hi;
                e4m3x4_to_half(u[i], lo, hi);
                const float2 f = __half22float2(*(const __half2 *)&lo), g = __half22float2(*(const __half2 *)&hi);
                u[i] = e4m3_pack2(__fdiv_rn(f.x * mul, div), __fdiv_rn(f.y * mul, div)) |
                       e4m3_pack2(__fdiv_rn(g.x * mul, div), __fdiv_rn(g.y * mul, div)) << 16;
            }
            return make_uint4(u[0], u[1], u[2], u[3]);
        };
        if (slot0 > 0 && scale != old) {  // the earlier tokens' codes on the larger scale
            const float ratio = __fdiv_rn(old, scale);
            constexpr int BATCH = 4;
            for (int s0 = tok; s0 < slot0; s0 += BATCH * TOK) {  // their loads under way together
                uint4 x[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i)
                    if (s0 + i * TOK < slot0)
                        x[i] = *(const uint4 *)(dst + (int64_t)(s0 + i * TOK) * c.st + off);
#pragma unroll
                for (int i = 0; i < BATCH; ++i)
                    if (s0 + i * TOK < slot0)
                        *(uint4 *)(dst + (int64_t)(s0 + i * TOK) * c.st + off) = rounded(x[i], ratio, 1.f);
            }
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            if (v * TOK >= n)
                break;
            if (v * TOK + tok < n)
                *(uint4 *)(dst + (int64_t)(slot0 + v * TOK + tok) * c.st + off) = rounded(w[v], ss[v], scale);
        }
        __syncwarp();
        if (lane == 0)
            scales[(int64_t)page * c.Hkv] = scale;
        i0 += n;
    }
}

}  // namespace

cudaError_t launch_cache_accept(const Cache &c, const int *n_new, const int *path, int A, const CacheWs &ws, cudaStream_t st)
{
    int ctas = 1;  // a warp for each row, as far as the portable cluster goes
    while (ctas < 8 && c.rows > ctas * (kPlanThreads / 32))
        ctas *= 2;
    cudaError_t e = launch_cluster(accept_plan_kernel, ctas, kPlanThreads, st, c, n_new, path, A, ws);
    if (e != cudaSuccess)
        return e;
    const dim3 grid((unsigned)((int64_t)c.rows * ((2 * c.Hkv + kMoveWarps - 1) / kMoveWarps))), block(kMoveWarps * 32);
    auto kernel = c.D == 128 ? accept_move_kernel<128> : c.D == 64 ? accept_move_kernel<64> : accept_move_kernel<32>;
    return launch_dependent(kernel, grid, block, 0, st, c, path, A, ws);
}

}  // namespace nsa
