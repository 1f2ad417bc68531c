// k_cache_attn.cu -- attention of new tokens over the paged 8-bit cache, for
// few query rows per kv head: the kernel that decoding runs on.
//
// Per query row r (token t, query head h of kv head g) over the attended
// keys j, code vectors ck_j, cv_j and their pages' scales ks_j, vs_j:
//   x_j = scale * log2(e) * ks_j * <q_r, ck_j>,  w_j = 2^(x_j + log2(vs_j) - M)
//   O = sum w_j cv_j / sum (w_j / vs_j),  LSE = ln 2 * (M + log2 sum (w_j / vs_j))
// The value scale rides in the exponent, so the second product runs on plain
// codes and a page of small values costs no range.
//
// What bounds it: the cache's bytes, 2 D per key and kv head, each read once;
// 4 G D operations on them are far below the tensor cores' rate (G = 4: 4
// operations a byte).  So the layout is made for the loads: codes go from
// global memory straight into the registers of the matrix instruction that
// consumes them.  The products are taken transposed, tokens (then head
// dimensions) as the 16 rows of mma.m16n8k16 and query rows as its 8 columns:
//   S^T[token, row] = K q^T     A: a thread's 16 code bytes of one token are
//       the pairs of four k-steps, in an order of the head dimension that q's
//       fragments share;
//   O^T[dim, row] = V^T P^T     A: two tokens' code bytes interleaved by byte
//       permutes give the (token, token + 1) pairs that A's columns want; B
//       is the transposed S fragment (one movmatrix per 8x8).
// e4m3 is a subset of half, so codes convert exactly; q is scaled to half's
// range by a power of two per row (bf16: exact but for elements 2^-29 below
// the row's largest; fp32: two halves, 22 bits) and P is rounded to half, 11
// bits (fp32: two halves).  Sums are fp32.  A CTA's work is a run of pages of
// the whole call's list of (sequence, kv head, page), cut into equal runs so
// that long and short sequences load every SM alike; rows whose pages fall to
// several CTAs are joined by a second kernel, in a fixed order.
//
// The legacy mma.sync path is enough here: the tensor pipe is a few percent
// busy, and tcgen05 would take the codes through shared memory first.
#include <math.h>

#include "cache_common.cuh"
#include "launch.h"
#include "tc_common.cuh"

namespace nsa {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kList = 256;       // pages of a run listed in shared memory at a time
constexpr float kNoMax = -1e30f; // running maximum of a row that has seen no key
constexpr float kLazy = 10.f;    // w may reach 2^10 before its row's maximum is raised (half holds 2^15)

struct AttnArgs {
    Geo g;
    Cache c;
    const void *q;
    const int *idx;      // selection: [.., S], else nullptr
    const float *sinks;  // or nullptr
    void *o;
    float *lse;
    int row_tiles;       // selection: query-row tiles per index row
    int quantum;         // pages that are not cut
    int ncta;            // CTAs of the main kernel
    int *status;         // [ncta]: what each CTA found
    int *prefix;         // [rows + 1] dense: list entries (pages x row tiles) of one kv head before each sequence
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

// BYTES (4, 8, 16) consecutive bytes as words
template <int BYTES> __device__ __forceinline__ void load_bytes(const uint8_t *p, uint32_t *w)
{
    if constexpr (BYTES == 16) {
        const uint4 x = __ldcs((const uint4 *)p);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else if constexpr (BYTES == 8) {
        const uint2 x = __ldcs((const uint2 *)p);
        w[0] = x.x, w[1] = x.y;
    } else
        w[0] = __ldcs((const uint32_t *)p);
}

// query tokens of sequence b; -1 for a packed range that is not one, or is
// longer than the problem says (none of its rows is read or written)
__device__ __forceinline__ int query_tokens(const Geo &g, int b)
{
    const int n = seq_len(g, b);
    return g.thd && (n < 0 || n > g.T || g.cu[b] < 0 || g.cu[b + 1] > g.ntok) ? -1 : n;
}

// The pages of sequence b that any of its query rows attends: [lo, lo + n).
__device__ __forceinline__ int attended_pages(const AttnArgs &a, int b, int &lo)
{
    const int nq = query_tokens(a.g, b), len = (int)min((int64_t)a.c.lens[b], (int64_t)a.c.cols * a.c.bs);
    lo = 0;
    if (nq <= 0 || len <= 0)
        return 0;
    if (a.g.window > 0) {
        const int64_t first = (int64_t)a.c.lens[b] - nq - a.g.window + 1;  // the first row's left edge
        lo = first > 0 ? (int)(first / a.c.bs) : 0;
    }
    return max(0, (len - 1) / a.c.bs + 1 - lo);
}

// tiles of R query rows of sequence b (dense)
template <int R> __device__ __forceinline__ int row_tiles_of(const Geo &g, int b)
{
    return (max(query_tokens(g, b), 0) * g.G + R - 1) / R;
}

// A unit of the list: a tile of query rows and the run of list entries that
// belongs to it.
struct UnitRows {
    int b, kvh, row0, nrows;  // rows row0 .. of sequence b (row = token * G + head), nrows of them valid
    int64_t begin, count;     // its entries in the list
    int page_lo;              // dense: first page
};

// NT: tiles of 8 query rows; SPLIT: fp32 queries (two halves)
template <int D, int NT, bool SPLIT> struct Smem {
    static constexpr int R = NT * 8;
    static constexpr int KS = D / 16;  // k-steps of S
    uint2 qf[SPLIT ? 2 : 1][KS][NT][32];
    float qmul[R];  // scale * log2(e) * 2^-e of each row
    int pos[R];     // key position of each row's token (-1: no such row)
    int page[kList], key0[kList];
    float ks[kList], lv[kList], iv[kList];
    int sidx[256];
    float m[kWarps][R], l[kWarps][R];
    float o[kWarps / 2][R][D + 4];
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, NT >= 4 ? 1 : 2) cache_attn_kernel(const AttnArgs a)
{
    constexpr bool SPLIT = sizeof(T) == 4;
    constexpr int R = NT * 8, KS = D / 16, MT = D / 16;
    constexpr int KB = D >= 64 ? 16 : 8;       // bytes of a K load
    constexpr int KL = D / 4 / KB;             // K loads per token and thread
    constexpr int VB = D / 8;                  // bytes of a V load: one per token and thread
    constexpr int VW = VB / 4;                 // words
    using SM = Smem<D, NT, SPLIT>;
    extern __shared__ __align__(16) char smem_raw[];
    SM &sm = *(SM *)smem_raw;
    const Geo &g = a.g;
    const Cache &c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gq = lane >> 2, tq = lane & 3;  // the fragment's row group and column pair
    const int cta = blockIdx.x;
    const bool sel = a.idx != nullptr;
    bool bad = false;

    // ---- the call's list of pages and this CTA's run of it
    __shared__ int part_s[kWarps];
    int *prefix = (int *)(smem_raw + sizeof(SM));  // dense: as a.prefix
    int64_t total;
    if (sel)
        total = (int64_t)g.ntok * g.Hkv * a.row_tiles * g.S;
    else {
        int64_t base = 0;
        for (int b0 = 0; b0 < g.B; b0 += kThreads) {
            const int b = b0 + tid;
            int lo, n = b < g.B ? attended_pages(a, b, lo) : 0;
            n *= n > 0 ? row_tiles_of<R>(g, b) : 0;
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
                prefix[b] = (int)base + before + incl - n;
                if (cta == 0)
                    a.prefix[b] = prefix[b];
            }
            base += all;
            __syncthreads();
        }
        if (tid == 0) {
            prefix[g.B] = (int)base;
            if (cta == 0)
                a.prefix[g.B] = (int)base;
        }
        __syncthreads();
        total = base * g.Hkv;
    }
    const int64_t nq = (total + a.quantum - 1) / a.quantum;
    const int64_t run0 = nq * cta / a.ncta * a.quantum;
    const int64_t run1 = min(total, nq * (cta + 1) / a.ncta * a.quantum);

    for (int64_t at = run0; at < run1;) {
        // ---- the unit that holds list entry `at`
        UnitRows u;
        if (sel) {
            const int64_t unit = at / g.S;
            u.begin = unit * g.S;
            u.count = g.S;
            const int rt = (int)(unit % a.row_tiles);
            const int64_t row = unit / a.row_tiles;  // index row
            int t;
            if (g.thd) {
                const int tok = (int)(row / g.Hkv);
                u.kvh = (int)(row % g.Hkv);
                u.b = seq_of_token(g, tok);
                t = tok - g.cu[u.b];
            } else {
                t = (int)(row % g.T);
                const int bg = (int)(row / g.T);
                u.b = bg / g.Hkv;
                u.kvh = bg % g.Hkv;
            }
            u.row0 = t * g.G + rt * R;
            u.nrows = t < query_tokens(g, u.b) ? min(R, g.G - rt * R) : 0;  // 0: a token of no sequence
            u.page_lo = 0;
        } else {
            const int64_t per = g.Hkv;
            int lo = 0, hi = g.B - 1;  // the sequence: prefix[b] * per <= at < prefix[b + 1] * per
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if ((int64_t)prefix[mid] * per <= at)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            u.b = lo;
            const int n = attended_pages(a, lo, u.page_lo), tiles = row_tiles_of<R>(g, lo);
            const int64_t in = (at - (int64_t)prefix[lo] * per) / n;  // (kv head, row tile)
            u.begin = (int64_t)prefix[lo] * per + in * n;
            u.count = n;
            u.kvh = (int)(in / tiles);
            u.row0 = (int)(in % tiles) * R;
            u.nrows = min(R, query_tokens(g, lo) * g.G - u.row0);
        }
        const int64_t seg1 = min(run1, u.begin + u.count);
        if (u.nrows <= 0) {
            at = seg1;
            continue;
        }
        const int len = min((int64_t)max(c.lens[u.b], 0), (int64_t)c.cols * c.bs);
        const int pos0 = c.lens[u.b] - seq_len(g, u.b);  // position of the sequence's first query token
        if (c.lens[u.b] < 0 || c.lens[u.b] > len)
            bad = true;

        // ---- queries into fragments: element (k, n) of B is row n's element
        // k, in the order of the head dimension that the K loads give
        __syncthreads();  // the previous unit is done with shared memory
        for (int r = warp; r < R; r += kWarps) {
            const bool have = r < u.nrows;
            const int row = u.row0 + r, t = row / g.G, h = u.kvh * g.G + row % g.G;
            constexpr int E = D / 32;
            float x[E];
            float amax = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                x[e] = have ? to_f<T>(((const T *)a.q)[q_off(g, u.b, h, t) + e * 32 + lane]) : 0.f;
                amax = fmaxf(amax, fabsf(x[e]));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            // the row's largest element to [2^14, 2^15)
            const int be = (int)(__float_as_uint(amax) >> 23);  // biased exponent (0: none, 255: infinity)
            const int e2 = be == 0 || be == 255 ? 0 : min(max(14 - (be - 127), -120), 120);
            const float up = __uint_as_float((uint32_t)(127 + e2) << 23);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int d = e * 32 + lane;
                // dimension d sits in load i, thread column tqd, byte k of the
                // load: word k / 4 is a k-step, bytes 0-1 its low and 2-3 its high half
                const int i = d / (4 * KB), tqd = d / KB % 4, k = d % KB;
                const int step = i * (KB / 4) + k / 4, slot = k % 4;
                const float y = x[e] * up;
                const __half hi = __float2half_rn(y);
                __half *f = (__half *)&sm.qf[0][step][r / 8][(r % 8) * 4 + tqd];
                f[slot] = hi;
                if constexpr (SPLIT) {
                    __half *f2 = (__half *)&sm.qf[SPLIT ? 1 : 0][step][r / 8][(r % 8) * 4 + tqd];
                    f2[slot] = __float2half_rn(y - __half2float(hi));
                }
            }
            if (lane == 0) {
                sm.qmul[r] = g.scale_l2 * __uint_as_float((uint32_t)(127 - e2) << 23);
                sm.pos[r] = have ? pos0 + t : -1;
            }
        }
        __syncthreads();

        float o[NT][MT][4];
        float m[NT][2], l[NT][2], qm[NT][2];
        int pos[NT][2];
        int pmin = INT32_MAX, pmax = -1;  // of the tile's rows
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[n][i] = kNoMax;
                l[n][i] = 0.f;
                qm[n][i] = sm.qmul[n * 8 + tq * 2 + i];
                pos[n][i] = sm.pos[n * 8 + tq * 2 + i];
            }
        for (int r = 0; r < u.nrows; ++r) {
            pmin = min(pmin, sm.pos[r]);
            pmax = max(pmax, sm.pos[r]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[n][j][i] = 0.f;

        for (int64_t e0 = at; e0 < seg1; e0 += kList) {
            const int ne = (int)min((int64_t)kList, seg1 - e0);
            // ---- the run's next pages
            __syncthreads();
            if (sel) {
                const int64_t irow = index_row(g, u.b, u.kvh, u.row0 / g.G);
                for (int s = tid; s < g.S; s += kThreads)
                    sm.sidx[s] = a.idx[irow * g.S + s];
                __syncthreads();
            }
            for (int i = tid; i < ne; i += kThreads) {
                const int s = (int)(e0 + i - u.begin);
                int j = sel ? sm.sidx[s] : u.page_lo + s, page = -1;
                if (sel && j >= 0) {
                    bool twice = false;
                    for (int k = 0; k < s; ++k)
                        twice |= sm.sidx[k] == j;
                    if (twice || (int64_t)j * c.bs > pmax || (int64_t)j * c.bs >= len) {  // repeated or in the future
                        bad = true;
                        j = -1;
                    }
                } else if (sel && j != -1) {
                    bad = true;
                    j = -1;
                }
                float ks = 0.f, vs = 1.f;
                if (j >= 0) {
                    page = c.table[(int64_t)u.b * c.cols + j];
                    if (page < 0 || page >= c.pages) {
                        bad = true;
                        page = -1;
                    } else {
                        ks = c.ks[(int64_t)page * c.Hkv + u.kvh];
                        vs = fmaxf(c.vs[(int64_t)page * c.Hkv + u.kvh], kScaleFloor);
                    }
                }
                sm.page[i] = page;
                sm.key0[i] = j * c.bs;
                sm.ks[i] = ks;
                sm.lv[i] = log2f(vs);
                sm.iv[i] = 1.f / vs;
            }
            __syncthreads();

            // ---- 16-token steps of the listed pages, the warps in turn
            const int per = c.bs / 16, steps = ne * per;
            const int64_t head_off = (int64_t)u.kvh * c.sh;
            uint32_t kw[2][KL * KB / 4], vw[4][VW];
            auto step_page = [&](int s, int &page, int &key) {
                const int e = s / per;
                page = sm.page[e];
                key = sm.key0[e] + s % per * 16;
                // a step that no row attends is not read
                return page >= 0 && key < len && key <= pmax && !(g.window > 0 && key + 15 <= pmin - g.window);
            };
            auto next_step = [&](int s, int &page, int &key) {
                while (s < steps && !step_page(s, page, key))
                    s += kWarps;
                return s;
            };
            auto load_k = [&](int page, int key) {
                const uint8_t *p = c.k + (int64_t)page * c.sp + head_off + (int64_t)(key % c.bs) * c.st;
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int i = 0; i < KL; ++i)
                        load_bytes<KB>(p + (gq + r * 8) * c.st + i * 4 * KB + tq * KB, &kw[r][i * (KB / 4)]);
            };
            auto load_v = [&](int page, int key) {
                const uint8_t *p = c.v + (int64_t)page * c.sp + head_off + (int64_t)(key % c.bs) * c.st;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    load_bytes<VB>(p + (tq * 2 + (i & 1) + (i >> 1) * 8) * c.st + gq * VB, vw[i]);
            };
            int page, key;
            int s = next_step(warp, page, key);
            if (s < steps) {
                load_k(page, key);
                load_v(page, key);
            }
            while (s < steps) {
                const int e = s / per;
                const float ks = sm.ks[e], lv = sm.lv[e], iv = sm.iv[e];
                const int key_now = key;
                const int s_next = next_step(s + kWarps, page, key);
                // ---- S^T = K q^T
                float sc[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sc[n][i] = 0.f;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const uint32_t af[4] = {e4m3_to_half2(kw[0][k] & 0xffffu), e4m3_to_half2(kw[1][k] & 0xffffu),
                                            e4m3_to_half2(kw[0][k] >> 16), e4m3_to_half2(kw[1][k] >> 16)};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint2 bf = sm.qf[0][k][n][lane];
                        mma_f16(sc[n], af, bf.x, bf.y);
                        if constexpr (SPLIT) {
                            const uint2 bl = sm.qf[SPLIT ? 1 : 0][k][n][lane];
                            mma_f16(sc[n], af, bl.x, bl.y);
                        }
                    }
                }
                if (s_next < steps)
                    load_k(page, key);  // in flight over the softmax and the second product
                // ---- w = 2^(x + log2 vs - M)
                const bool part = key_now + 15 > pmin || key_now + 16 > len || (g.window > 0 && key_now <= pmax - g.window);
                bool raise = false;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float x = sc[n][i] * (ks * qm[n][i & 1]) + lv;
                        if (part) {
                            const int kk = key_now + gq + (i >> 1) * 8, p = pos[n][i & 1];
                            if (kk > p || kk >= len || (g.window > 0 && kk <= p - g.window))
                                x = -INFINITY;
                        }
                        sc[n][i] = x;
                        raise |= x > m[n][i & 1] + kLazy;
                    }
                if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float x = fmaxf(sc[n][i], sc[n][i + 2]);
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                            const float mn = fmaxf(m[n][i], x);
                            const float f = exp2f(m[n][i] - mn);
                            m[n][i] = mn;
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
                        sc[n][i] = tc::ex2(sc[n][i] - m[n][i & 1]);
                        l[n][i & 1] += sc[n][i] * iv;
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t hi = pack_half(sc[n][2 * i], sc[n][2 * i + 1]);
                        pb[0][n][i] = transpose8x8(hi);
                        if constexpr (SPLIT) {
                            const float2 f = __half22float2(*(const __half2 *)&hi);
                            pb[SPLIT ? 1 : 0][n][i] = transpose8x8(pack_half(sc[n][2 * i] - f.x, sc[n][2 * i + 1] - f.y));
                        }
                    }
                }
                // ---- values that a row does not attend must not reach it, whatever they hold
                unsigned nan_words = 0;  // bit (i * VW + w): word w of token i holds a NaN
                if (part) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int kk = key_now + tq * 2 + (i & 1) + (i >> 1) * 8;
                        const bool out = kk > pmax || kk >= len || (g.window > 0 && kk <= pmin - g.window);
#pragma unroll
                        for (int w = 0; w < VW; ++w) {
                            if (out)
                                vw[i][w] = 0u;
                            const uint32_t x = vw[i][w] & 0x7f7f7f7fu;
                            if ((x + 0x01010101u) & 0x80808080u)
                                nan_words |= 1u << (i * VW + w);
                        }
                    }
                }
                const bool any_nan = part && __any_sync(0xffffffffu, nan_words != 0);
                if (any_nan) {
                    // a NaN value: it goes, whole, to the rows that attend its
                    // token and to no other (0 * NaN would reach them all)
#pragma unroll 1
                    for (int from = 0; from < 4; ++from)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int w = 0; w < VW; ++w) {
                                const uint32_t x = __shfl_sync(0xffffffffu, vw[i][w], (lane & ~3) | from);
                                const int kk = key_now + from * 2 + (i & 1) + (i >> 1) * 8;
#pragma unroll
                                for (int y = 0; y < 4; ++y)
                                    if (((x >> (8 * y)) & 0x7fu) == 0x7fu) {
                                        // byte 4 w + y of the thread's dimensions: tile (4w + y) / 2, half y % 2
#pragma unroll
                                        for (int n = 0; n < NT; ++n)
#pragma unroll
                                            for (int h = 0; h < 2; ++h)
                                                if (kk <= pos[n][h] && !(g.window > 0 && kk <= pos[n][h] - g.window))
                                                    o[n][(4 * w + y) / 2][(y % 2) * 2 + h] = __int_as_float(0x7fffffff);
                                    }
                            }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int w = 0; w < VW; ++w)
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                if (((vw[i][w] >> (8 * y)) & 0x7fu) == 0x7fu)
                                    vw[i][w] &= ~(0xffu << (8 * y));
                }
                // ---- O^T += V^T P^T
#pragma unroll
                for (int w = 0; w < VW; ++w)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const uint32_t lo2 = __byte_perm(vw[0][w], vw[1][w], hf ? 0x7362 : 0x5140);
                        const uint32_t hi2 = __byte_perm(vw[2][w], vw[3][w], hf ? 0x7362 : 0x5140);
                        const uint32_t af[4] = {e4m3_to_half2(lo2 & 0xffffu), e4m3_to_half2(lo2 >> 16),
                                                e4m3_to_half2(hi2 & 0xffffu), e4m3_to_half2(hi2 >> 16)};
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma_f16(o[n][w * 2 + hf], af, pb[0][n][0], pb[0][n][1]);
                            if constexpr (SPLIT)
                                mma_f16(o[n][w * 2 + hf], af, pb[SPLIT ? 1 : 0][n][0], pb[SPLIT ? 1 : 0][n][1]);
                        }
                    }
                if (s_next < steps)
                    load_v(page, key);
                s = s_next;
            }
        }

        // ---- the warps' sums joined: statistics, then O in two rounds of
        // half the warps (shared memory for 4)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x = l[n][i];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                if (gq == 0) {
                    sm.m[warp][n * 8 + tq * 2 + i] = m[n][i];
                    sm.l[warp][n * 8 + tq * 2 + i] = x;
                }
            }
        __syncthreads();
        constexpr int PER = R * D / kThreads > 0 ? R * D / kThreads : 1;  // outputs per thread
        float acc[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i)
            acc[i] = 0.f;
#pragma unroll
        for (int round = 0; round < 2; ++round) {
            if (warp / (kWarps / 2) == round) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = n * 8 + tq * 2 + i;
                        float top = kNoMax;
#pragma unroll
                        for (int w = 0; w < kWarps; ++w)
                            top = fmaxf(top, sm.m[w][r]);
                        const float f = exp2f(m[n][i] - top);
#pragma unroll
                        for (int j = 0; j < MT; ++j) {
                            sm.o[warp % (kWarps / 2)][r][gq * VB + 2 * j] = o[n][j][i] * f;
                            sm.o[warp % (kWarps / 2)][r][gq * VB + 2 * j + 1] = o[n][j][i + 2] * f;
                        }
                    }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int x = i * kThreads + tid;
                if (x < R * D)
#pragma unroll
                    for (int w = 0; w < kWarps / 2; ++w)
                        acc[i] += sm.o[w][x / D][x % D];
            }
            __syncthreads();
        }
        const bool whole = at == u.begin && seg1 == u.begin + u.count;
        // a part: the first of the run in slot 0, its last in slot 1 (a run
        // within one unit has one part)
        const int64_t slot = (int64_t)cta * 2 + (at == run0 ? 0 : 1);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int x = i * kThreads + tid, r = x / D, d = x % D;
            if (x >= R * D || r >= u.nrows)
                continue;
            float top = kNoMax, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                top = fmaxf(top, sm.m[w][r]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                sum += sm.l[w][r] * exp2f(sm.m[w][r] - top);
            if (!whole) {
                a.part_o[(slot * R + r) * D + d] = acc[i];
                if (d == 0)
                    a.part_ml[slot * R + r] = make_float2(top, sum);
                continue;
            }
            const int row = u.row0 + r, t = row / g.G, h = u.kvh * g.G + row % g.G;
            float f = 1.f;
            if (a.sinks) {
                const float sk = a.sinks[h] * 1.4426950408889634f, mn = fmaxf(top, sk);
                f = exp2f(top - mn);
                sum = sum * f + exp2f(sk - mn);
                top = mn;
            }
            const float y = sum > 0.f || sum != sum ? acc[i] * f / sum : 0.f;
            ((T *)a.o)[o_off(g, u.b, h, t) + d] = from_f<T>(y);
            if (d == 0)
                a.lse[stat_off(g, u.b, h, t)] = lse_of(top, sum);
        }
        at = seg1;
    }
    bad = __syncthreads_or(bad);
    if (tid == 0)
        a.status[cta] = bad ? NSA_ERR_BAD_INDEX : NSA_OK;
}

// Joins the parts of the rows that several CTAs worked on, and writes the
// rows that no CTA saw (no attended page).  A warp per query row; the parts
// are taken in the order of the CTAs.
template <typename T, int D> __global__ void __launch_bounds__(256) cache_join_kernel(const AttnArgs a, int R, int *err)
{
    const Geo &g = a.g;
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == gridDim.x - 1) {  // the call's error word
        int bad = 0;
        for (int i = threadIdx.x; i < a.ncta; i += 256)
            bad |= a.status[i] != NSA_OK;
        for (int b = threadIdx.x; b < g.B; b += 256) {
            const int len = a.c.lens[b];
            bad |= len < 0 || (int64_t)len > (int64_t)a.c.cols * a.c.bs || query_tokens(g, b) < 0;
        }
        bad = __syncthreads_or(bad);
        if (threadIdx.x == 0)
            *err = bad ? NSA_ERR_BAD_INDEX : NSA_OK;
        return;
    }
    const bool sel = a.idx != nullptr;
    const int64_t nrow = (int64_t)g.ntok * g.Hq;
    for (int64_t w = blockIdx.x * 8 + threadIdx.x / 32; w < nrow; w += (int64_t)(gridDim.x - 1) * 8) {
        const int h = (int)(w % g.Hq);
        const int tok = (int)(w / g.Hq);
        int b, t;
        if (g.thd) {
            b = seq_of_token(g, tok);
            t = tok - g.cu[b];
            if (t >= query_tokens(g, b))
                continue;
        } else {
            b = tok / g.T;
            t = tok % g.T;
        }
        const int kvh = h / g.G, hh = h % g.G;
        int64_t begin, count, total;
        int r;
        if (sel) {
            const int64_t unit = index_row(g, b, kvh, t) * a.row_tiles + hh / R;
            r = hh % R;
            begin = unit * g.S;
            count = g.S;
            total = (int64_t)g.ntok * g.Hkv * a.row_tiles * g.S;
        } else {
            const int row = t * g.G + hh;
            r = row % R;
            int lo;
            const int tiles = (query_tokens(g, b) * g.G + R - 1) / R;
            count = attended_pages(a, b, lo);
            begin = (int64_t)a.prefix[b] * g.Hkv + ((int64_t)kvh * tiles + row / R) * count;
            total = (int64_t)a.prefix[g.B] * g.Hkv;
        }
        const int64_t nq = (total + a.quantum - 1) / a.quantum;
        float top = kNoMax, sum = 0.f, acc[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            acc[i] = 0.f;
        if (count > 0) {
            // the first CTA whose run reaches past `begin`
            auto run_at = [&](int64_t x) { return nq * x / a.ncta * a.quantum; };
            int64_t cta = begin / a.quantum * a.ncta / max(nq, (int64_t)1);
            while (cta > 0 && run_at(cta) > begin)
                --cta;
            while (min(run_at(cta + 1), total) <= begin)
                ++cta;
            if (run_at(cta) <= begin && run_at(cta + 1) >= begin + count)
                continue;  // one CTA had it all and wrote the result
            const int64_t first = cta;
            int64_t last = first;
            for (; last < a.ncta && run_at(last) < begin + count; ++last)
                if (run_at(last + 1) > run_at(last)) {
                    const int64_t slot = last * 2 + (run_at(last) >= begin ? 0 : 1);
                    top = fmaxf(top, a.part_ml[slot * R + r].x);
                }
            for (cta = first; cta < last; ++cta)
                if (run_at(cta + 1) > run_at(cta)) {
                    const int64_t slot = cta * 2 + (run_at(cta) >= begin ? 0 : 1);
                    const float2 ml = a.part_ml[slot * R + r];
                    const float f = exp2f(ml.x - top);
                    sum += ml.y * f;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i)
                        acc[i] += a.part_o[(slot * R + r) * D + i * 32 + lane] * f;
                }
        }
        if (a.sinks) {
            const float sk = a.sinks[h] * 1.4426950408889634f, mn = fmaxf(top, sk);
            const float f = exp2f(top - mn);
            sum = sum * f + exp2f(sk - mn);
            top = mn;
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
                acc[i] *= f;
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const float y = sum > 0.f || sum != sum ? acc[i] / sum : 0.f;
            ((T *)a.o)[o_off(g, b, h, t) + i * 32 + lane] = from_f<T>(y);
        }
        if (lane == 0)
            a.lse[stat_off(g, b, h, t)] = lse_of(top, sum);
    }
}

// the tile of query rows: as many tiles of 8 as the rows of a kv head need
int row_tile(const Geo &g, bool sel)
{
    const int64_t rows = sel ? g.G : (int64_t)g.T * g.G;
    return rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
}

int ctas_of(const Geo &g, bool sel) { return num_sms() * (row_tile(g, sel) >= 4 ? 1 : 2); }

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

template <typename T, int D, int NT> cudaError_t attn_t(AttnArgs a, int *err, cudaStream_t st)
{
    using SM = Smem<D, NT, sizeof(T) == 4>;
    const size_t smem = sizeof(SM) + (a.idx ? 0 : sizeof(int) * (size_t)(a.g.B + 1));
    cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess)
        return e;
    cache_attn_kernel<T, D, NT><<<a.ncta, kThreads, smem, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    const int64_t rows = (int64_t)a.g.ntok * a.g.Hq;
    const int64_t blocks = (rows + 7) / 8, most = (int64_t)num_sms() * 8;
    cache_join_kernel<T, D><<<(unsigned)(blocks < most ? blocks : most) + 1, 256, 0, st>>>(a, NT * 8, err);
    return cudaGetLastError();
}

template <typename T> cudaError_t attn_d(const AttnArgs &a, int nt, int *err, cudaStream_t st)
{
#define NSA_NT(D)                                   \
    switch (nt) {                                   \
    case 1: return attn_t<T, D, 1>(a, err, st);     \
    case 2: return attn_t<T, D, 2>(a, err, st);     \
    default: return attn_t<T, D, 4>(a, err, st);    \
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

size_t cache_attn_ws_bytes(const Geo &g, bool sel) { return attn_layout(g, sel).total; }

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
    // a run is cut at multiples of 128 tokens, a step of the CTA's 8 warps;
    // with many index rows at the rows themselves (nothing to join then)
    a.quantum = 128 / c.bs;
    if (sel && (int64_t)g.ntok * g.Hkv * a.row_tiles >= 4 * (int64_t)a.ncta)
        a.quantum = g.S;
    a.status = (int *)(ws + w.status);
    a.prefix = (int *)(ws + w.prefix);
    a.part_ml = (float2 *)(ws + w.ml);
    a.part_o = (float *)(ws + w.o);
    int *err = (int *)ws;
    return dtype == NSA_DTYPE_BF16 ? attn_d<__nv_bfloat16>(a, nt, err, st) : attn_d<float>(a, nt, err, st);
}

}  // namespace nsa
