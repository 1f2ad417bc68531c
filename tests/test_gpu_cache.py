"""The paged 8-bit cache on the GPU against plain 64-bit implementations:
attention over it, appending to it, and its pages."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_do_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
U32 = 2.0 ** -24  # half a step of fp32, relative


# ------------------------------------------------------------ plain forms

def e4m3_round(x):
    """x (float64 array) to the nearest e4m3 value, ties to even, clamped to +-448."""
    a = np.minimum(np.abs(x), 448.0)
    step = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.copysign(np.minimum(np.rint(a / step) * step, 448.0), x)


def scale_for(x):
    """Least power of two s with max|x| <= 448 s over the finite x, at least 2^-100."""
    f = x[np.isfinite(x)]
    amax = np.abs(f).max() if f.size else 0.0
    s = 2.0 ** -100
    if amax > 448.0 * s:
        s = 2.0 ** math.floor(math.log2(amax / 448.0))
        while amax > 448.0 * s:
            s *= 2.0
        while amax <= 448.0 * (s / 2.0):
            s /= 2.0
    return s


class Plain:
    """The cache in numpy, float64 code values; the operators by their definition."""

    def __init__(self, cache):
        self.k, self.v = (x.cpu().float().double().numpy().copy() for x in (cache.k, cache.v))
        self.ks, self.vs = (x.cpu().double().numpy().copy() for x in (cache.k_scale, cache.v_scale))
        self.table, self.lens = cache.page_table.cpu().numpy().copy(), cache.seq_lens.cpu().numpy().copy()
        self.ref = cache.refcount.cpu().numpy().copy()
        self.bs, self.Hkv = self.k.shape[2], self.k.shape[1]

    def blocks(self, n):
        return -(-int(n) // self.bs)

    def free_ids(self):
        return [p for p in range(len(self.ref)) if self.ref[p] <= 0]

    def reserve(self, n_new):
        need = [self.blocks(a + n) - self.blocks(a) for a, n in zip(self.lens, n_new)]
        free = self.free_ids()
        if sum(need) > len(free):
            return 7
        at = 0
        for b, n in enumerate(n_new):
            have = self.blocks(self.lens[b])
            for c in range(have, have + need[b]):
                self.table[b, c] = free[at]
                self.ref[free[at]] = 1
                at += 1
            self.lens[b] += n
        return 0

    def release(self, r):
        for c in range(self.table.shape[1]):
            if self.table[r, c] >= 0:
                self.ref[self.table[r, c]] -= 1
                self.table[r, c] = -1
        self.lens[r] = 0

    def copy_page(self, s, d):
        for x in (self.k, self.v, self.ks, self.vs):
            x[d] = x[s]

    def fork(self, src, dst):
        saved = self.table.copy(), self.lens.copy(), self.ref.copy()
        for d in dst:
            self.release(d)
        free = self.free_ids()
        tails = sum(1 for s in src if self.lens[s] % self.bs)
        if tails > len(free):
            self.table, self.lens, self.ref = saved
            return 7
        at = 0
        for s, d in zip(src, dst):
            full = self.lens[s] // self.bs
            self.table[d, :full] = self.table[s, :full]
            for p in self.table[s, :full]:
                self.ref[p] += 1
            if self.lens[s] % self.bs:
                p = free[at]
                at += 1
                self.copy_page(self.table[s, full], p)
                self.table[d, full] = p
                self.ref[p] = 1
            self.lens[d] = self.lens[s]
        return 0

    def compact(self):
        n = int((self.ref > 0).sum())
        src = [p for p in range(n, len(self.ref)) if self.ref[p] > 0]
        dst = [p for p in range(n) if self.ref[p] <= 0]
        to = {s: d for s, d in zip(src, dst)}
        for s, d in zip(src, dst):
            self.copy_page(s, d)
            self.ref[d], self.ref[s] = self.ref[s], 0
        for i, p in np.ndenumerate(self.table):
            if p in to:
                self.table[i] = to[p]

    def append(self, b, kn, vn):
        """kn, vn [n, Hkv, D] (float64 of the given dtype's values): row b's last n positions."""
        n = len(kn)
        start = self.lens[b] - n
        for codes, scales, new in ((self.k, self.ks, kn), (self.v, self.vs, vn)):
            for col in range(start // self.bs, self.blocks(self.lens[b]) if n else 0):
                p, lo, hi = self.table[b, col], max(start, col * self.bs), min(self.lens[b], (col + 1) * self.bs)
                for h in range(self.Hkv):
                    x = new[lo - start:hi - start, h]
                    s = scale_for(x)
                    at = lo - col * self.bs
                    if at:
                        s = max(s, scales[p, h])
                        if s != scales[p, h]:
                            codes[p, h, :at] = e4m3_round(codes[p, h, :at] * (scales[p, h] / s))
                    codes[p, h, at:at + hi - lo] = e4m3_round(x / s)
                    scales[p, h] = s

    def keys(self, b, h):
        n = int(self.lens[b])
        pg = self.table[b, :self.blocks(n)]
        flat = lambda c, s: (c[pg, h] * s[pg, h][:, None, None]).reshape(-1, c.shape[-1])[:n]  # noqa: E731
        return flat(self.k, self.ks), flat(self.v, self.vs)

    def attend(self, b, q, scale, idx=None, window=0, sinks=None):
        """q [n, Hq, D] of row b: (o, lse, tolerance factors) in 64 bits.
        tol[t, h]: see check_attend."""
        n, Hq, D = q.shape
        o, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
        vmax, serr, nkeys = np.zeros((n, Hq)), np.zeros((n, Hq)), np.zeros((n, Hq))
        for h in range(Hq):
            g = h // (Hq // self.Hkv)
            K, V = self.keys(b, g)
            for t in range(n):
                pos = int(self.lens[b]) - n + t
                j = np.arange(0, max(pos + 1, 0))
                if window:
                    j = j[j > pos - window]
                if idx is not None:
                    j = j[np.isin(j // self.bs, idx[t, g][idx[t, g] >= 0])]
                z = K[j] @ q[t, h] * scale
                if sinks is not None:
                    z = np.append(z, sinks[h])
                if z.size == 0:
                    continue
                m = z.max()
                lse[t, h] = m + math.log(np.exp(z - m).sum()) if np.isfinite(m) else m
                w = np.exp(z - lse[t, h])[:len(j)]
                if len(j):
                    o[t, h] = w @ V[j]
                    vmax[t, h] = np.nanmax(np.abs(V[j]))
                    serr[t, h] = np.nanmax(np.abs(K[j]) @ np.abs(q[t, h])) * scale
                nkeys[t, h] = len(j)
        return o, lse, (vmax, serr, nkeys)


def check_attend(got_o, got_lse, o, lse, fac, dtype, D):
    """Per row: a score is off by at most d = (D + 8) roundings of its sum of
    magnitudes (fp32 sums; fp32 queries are held to 2^-22, 4 roundings) plus
    the exponential's 2^-21 (its own error 2^-22, the scales' product and the
    logarithm of the value scale); weights then by 2 d relative (numerator and
    denominator), their rounding to half 2^-11 (fp32: two halves, 2^-21), the
    sums by (keys + 16) roundings, all times the largest value attended; and
    the output's own rounding, half a step.  LSE: d, the sum's roundings, and
    its own scale."""
    vmax, serr, n = fac
    d = (D + 8) * U32 * serr + 2.0 ** -21
    half = 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -21
    out = torch.finfo(dtype).eps / 2
    tol = out * np.abs(o) * (1 + 2.0 ** -7) + ((2 * d + half + 2 * (n + 16) * U32) * vmax)[..., None]
    nan = np.isnan(o)
    assert np.array_equal(np.isnan(got_o), nan)
    err = np.where(nan, 0.0, np.abs(got_o - o) - tol)
    assert err.max(initial=0) <= 0, (err.max(), np.unravel_index(err.argmax(), err.shape))
    fine = np.isfinite(lse)
    assert np.array_equal(np.isnan(got_lse), np.isnan(lse))
    assert np.array_equal(got_lse[~fine & ~np.isnan(lse)], lse[~fine & ~np.isnan(lse)])
    ltol = d + (n + 16) * U32 + 8 * U32 * (np.abs(lse) + 64)
    off = np.abs(got_lse[fine] - lse[fine])
    assert (off <= ltol[fine]).all(), off.max()


# ------------------------------------------------------------------ making

def filled(lens, Hkv, D, bs, seed, spare=5, cols=None, garbage=True, scale_spread=3, layout="dense"):
    """A cache whose rows hold lens tokens in shuffled pages; every slot that
    holds no token is NaN."""
    g = np.random.default_rng(seed)
    used = [-(-n // bs) for n in lens]
    cols = cols or max(max(used), 1)
    npool = sum(used) + spare
    order = g.permutation(npool)
    vals = lambda: e4m3_round(g.normal(size=(npool, Hkv, bs, D)) * 100)  # noqa: E731
    k, v = vals(), vals()
    table, at = np.full((len(lens), cols), -1, np.int32), 0
    live = np.zeros((npool, bs), bool)
    ref = np.zeros(npool, np.int32)
    for b, n in enumerate(lens):
        table[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
        for c in range(used[b]):
            live[table[b, c], :min(bs, n - c * bs)] = True
            ref[table[b, c]] = 1
    if garbage:
        k[~live.repeat(Hkv, 0).reshape(npool, Hkv, bs)] = np.nan
        v[~live.repeat(Hkv, 0).reshape(npool, Hkv, bs)] = np.nan
    mk = lambda x: torch.tensor(x, dtype=torch.float32).to(torch.float8_e4m3fn).to(DEV)  # noqa: E731
    sc = lambda: torch.tensor(2.0 ** g.integers(-8, -8 + scale_spread, (npool, Hkv)) * g.choice([1.0, 1.25], (npool, Hkv)), dtype=torch.float32, device=DEV)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    kk, vv = mk(k), mk(v)
    if layout == "token":  # [page, token, head, D]
        turn = lambda x: x.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(torch.float8_e4m3fn)  # noqa: E731
        kk, vv = turn(kk), turn(vv)
    elif layout == "both":  # k and v of a page side by side
        both = torch.stack([kk.view(torch.uint8), vv.view(torch.uint8)], 1).view(torch.float8_e4m3fn)
        kk, vv = both[:, 0], both[:, 1]
    return api.KVCache(kk, vv, sc(), sc(), i32(table), i32(np.array(lens)), i32(ref))


def index_rows(lens, new, Hkv, S, bs, g):
    """Own block, earlier ones at random, -1: [tokens, Hkv, S]; every fourth row all -1."""
    rows = []
    for n, q in zip(lens, new):
        for t in range(q):
            pos = n - q + t
            for h in range(Hkv):
                own = pos // bs
                r = [-1] * S
                if pos >= 0 and len(rows) % 4 != 3:
                    pick = g.permutation(own)[:S - 1] if own > 0 else []
                    r = ([own] + list(pick) + [-1] * S)[:S]
                    r = list(g.permutation(r))
                rows.append(r)
    return np.array(rows, np.int32).reshape(-1, Hkv, S)


def attend_case(lens, new, Hq, Hkv, D, bs, dtype, ragged=False, S=0, window=0, sinks=False, seed=0, layout="dense",
                cache=None, scale=None, edit=None, cols=None):
    g = np.random.default_rng(seed + 1)
    cache = cache or filled(lens, Hkv, D, bs, seed, layout=layout, cols=cols)
    if edit is not None:
        edit(cache)
    total = sum(new)
    q = torch.tensor(g.normal(size=(total, Hq, D)), dtype=torch.float32).to(dtype)
    idx = index_rows(lens, new, Hkv, S, bs, g) if S else None
    sk = torch.tensor(g.normal(size=Hq) * 2, dtype=torch.float32) if sinks else None
    kw = dict(window=window or None, sinks=sk.to(DEV) if sinks else None, scale=scale)
    if ragged:
        cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
        o, lse = api.cache_fwd(q.to(DEV), cache, cu_seqlens=cu, max_seqlen=max(new),
                               block_idx=torch.tensor(idx, device=DEV) if S else None, **kw)
    else:
        B, T = len(lens), new[0]
        qb = q.view(B, T, Hq, D).transpose(1, 2).contiguous().to(DEV)
        ib = torch.tensor(idx, device=DEV).view(B, T, Hkv, S).transpose(1, 2).contiguous() if S else None
        o, lse = api.cache_fwd(qb, cache, block_idx=ib, **kw)
        o, lse = o.transpose(1, 2).reshape(total, Hq, D), lse.transpose(1, 2).reshape(total, Hq)
    plain, at = Plain(cache), 0
    for b, n in enumerate(new):
        sl = slice(at, at + n)
        want = plain.attend(b, q[sl].double().numpy(), scale or 1 / math.sqrt(D), idx[sl] if S else None, window,
                            sk.double().numpy() if sinks else None)
        check_attend(o[sl].double().cpu().numpy(), lse[sl].double().cpu().numpy(), *want, dtype, D)
        at += n


BF, F32 = torch.bfloat16, torch.float32


# --------------------------------------------------------------- attention

@pytest.mark.parametrize("Hq,Hkv,D,bs", [(4, 1, 128, 64), (16, 1, 128, 64), (6, 2, 64, 32), (2, 1, 32, 16), (5, 5, 64, 16),
                                         (24, 1, 32, 64), (40, 1, 128, 32), (3, 1, 128, 16), (34, 2, 64, 64)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_one_token(Hq, Hkv, D, bs, dtype):
    attend_case([1, bs - 1, bs, bs + 1, 3 * bs + 5, 700], [1] * 6, Hq, Hkv, D, bs, dtype)


@pytest.mark.parametrize("kw", [dict(window=1), dict(window=37), dict(window=64), dict(window=5000), dict(sinks=True),
                                dict(window=50, sinks=True), dict(S=1), dict(S=5), dict(S=16), dict(scale=0.3)])
@pytest.mark.parametrize("dtype,Hq,Hkv,D,bs,T", [(BF, 8, 2, 128, 64, 1), (BF, 6, 2, 64, 32, 3), (F32, 2, 1, 32, 16, 7),
                                                 (BF, 24, 2, 128, 32, 2), (F32, 16, 1, 128, 64, 1)])
def test_attend_masks(kw, dtype, Hq, Hkv, D, bs, T):
    attend_case([2, 0, 200, 65, 130, T], [T] * 6, Hq, Hkv, D, bs, dtype, **kw)


@pytest.mark.parametrize("dtype,Hq,Hkv,D,bs", [(BF, 8, 2, 128, 64), (F32, 6, 2, 64, 32), (BF, 4, 4, 32, 16),
                                               (BF, 16, 1, 64, 64), (BF, 4, 1, 128, 16), (BF, 12, 1, 128, 32)])
@pytest.mark.parametrize("kw", [dict(), dict(window=40), dict(S=4), dict(sinks=True)])
def test_attend_packed_chunks(dtype, Hq, Hkv, D, bs, kw):
    attend_case([300, 17, 0, 129, 64, 70], [130, 17, 0, 1, 64, 33], Hq, Hkv, D, bs, dtype, ragged=True, **kw)


@pytest.mark.parametrize("layout", ["token", "both"])
@pytest.mark.parametrize("T", [1, 40])
def test_attend_strided_pools(layout, T):
    attend_case([200, 70, 333], [T] * 3, 8, 2, 128, 64, BF, layout=layout)


def test_attend_many_rows_of_the_table():
    g = np.random.default_rng(3)
    lens = [int(n) for n in g.integers(0, 90, 700)]
    attend_case(lens, [1] * 700, 2, 1, 32, 16, BF)


def test_attend_long_and_short_together():
    attend_case([20000, 3, 64, 1], [1] * 4, 4, 1, 128, 64, BF)
    attend_case([9000, 3], [2, 2], 4, 1, 64, 32, F32, window=4000)


def test_attend_more_queries_than_keys():
    attend_case([2, 0, 5], [6] * 3, 4, 2, 64, 16, BF)
    attend_case([2, 0, 5], [6] * 3, 4, 2, 64, 16, BF, sinks=True)


@pytest.mark.parametrize("T", [1, 5, 40])
@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64)])
def test_a_nan_reaches_only_rows_that_attend_it(dtype, D, T):
    def edit(cache):
        for t, h, d in ((150, 0, 3), (199, 1, 30), (199, 0, D - 1), (198, 0, 7)):  # among the last tokens: some rows see them
            p = int(cache.page_table[0, t // 64])
            cache.v.view(torch.uint8)[p, h, t % 64, d] = 0xff
    attend_case([200, 90], [T] * 2, 8, 2, D, 64, dtype, edit=edit)

    def edit_k(cache):
        p = int(cache.page_table[0, 3])
        cache.k.view(torch.uint8)[p, 1, 7, 0] = 0x7f
    attend_case([200, 90], [T] * 2, 8, 2, D, 64, dtype, edit=edit_k)


def test_attend_scales_far_apart():
    def edit(cache):
        cache.v_scale[::2] = 2.0 ** -60
        cache.v_scale[1::3] = 2.0 ** 40
        cache.k_scale[::3] *= 2.0 ** -20
    attend_case([500], [1], 8, 2, 128, 64, BF, edit=edit)
    attend_case([500], [70], 8, 2, 128, 64, BF, edit=edit)


def test_attend_zero_scale_and_large_scores():
    def edit(cache):
        cache.v_scale[0] = 0.0
        cache.v.view(torch.uint8)[0] = 0
        cache.k_scale *= 30.0
    attend_case([300, 64], [1, 1], 4, 1, 64, 16, F32, edit=edit)
    attend_case([300, 64], [33, 33], 4, 1, 128, 64, BF, edit=edit)


def test_attend_offsets_beyond_32_bits():
    """Pages whose first byte lies past 2^32."""
    Hkv, D, bs = 8, 128, 64
    npool = (1 << 32) // (Hkv * D * bs) + 64
    cache = api.make_cache(npool, Hkv, D, bs, 2, 8)
    few = filled([200, 300], Hkv, D, bs, 5, spare=0, cols=8)
    n = few.k.shape[0]
    for a, b in ((cache.k, few.k), (cache.v, few.v)):
        a.view(torch.uint8)[npool - n:] = b.view(torch.uint8)
    for a, b in ((cache.k_scale, few.k_scale), (cache.v_scale, few.v_scale), (cache.refcount, few.refcount)):
        a[npool - n:] = b
    cache.page_table.copy_(torch.where(few.page_table >= 0, few.page_table + (npool - n), -1))
    cache.seq_lens.copy_(few.seq_lens)
    q = torch.randn(2, 16, 3, D, device=DEV).to(BF)
    for kw in (dict(), dict(block_idx=torch.zeros(2, Hkv, 3, 1, dtype=torch.int32, device=DEV))):
        for a, b in zip(api.cache_fwd(q, cache, **kw), api.cache_fwd(q, few, **kw)):
            assert torch.equal(a, b)
    # an appended token and copied pages land there too
    one = torch.ones(2, dtype=torch.int32, device=DEV)
    cache.seq_lens += one
    few.seq_lens += one
    kn, vn = (torch.randn(2, Hkv, 1, D, device=DEV).to(BF) for _ in range(2))
    api.cache_append(cache, kn, vn)
    api.cache_append(few, kn, vn)
    assert torch.equal(cache.k[npool - n:].view(torch.uint8), few.k.view(torch.uint8))
    assert torch.equal(cache.v_scale[npool - n:], few.v_scale)
    src = torch.arange(npool - n, npool, dtype=torch.int32, device=DEV)
    dst = torch.arange(n, dtype=torch.int32, device=DEV)
    api.cache_copy(cache, src, dst)
    assert torch.equal(cache.k[:n].view(torch.uint8), few.k.view(torch.uint8))
    assert torch.equal(cache.v[:n].view(torch.uint8), few.v.view(torch.uint8))


def test_rows_behind_the_last_sequence_are_left():
    cache = filled([100, 50], 2, 64, 32, 1)
    cu = torch.tensor([0, 3, 40], dtype=torch.int32, device=DEV)
    q = torch.randn(48, 4, 64, device=DEV).to(BF)
    idx = torch.zeros(48, 2, 1, dtype=torch.int32, device=DEV)
    for kw in (dict(), dict(block_idx=idx)):
        p = api.problem(2, 4, 2, 37, 64, 32, 1, BF, layout=api.LAYOUT_THD, total_tokens=48)
        o, lse = torch.full((48, 4, 64), 7.0, device=DEV).to(BF), torch.full((48, 4), 7.0, device=DEV)
        n = api.lib().nsa_cache_fwd_workspace_size(p, cache.ref, int("block_idx" in kw))
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        s = api.lib().nsa_cache_fwd(p, cache.ref, 0, cu.data_ptr(), idx.data_ptr() if kw else None, None, q.data_ptr(),
                                    o.data_ptr(), lse.data_ptr(), ws.data_ptr(), n, api._stream())
        assert s == 0 and api.get_error(ws) == 0
        assert (o[40:] == 7).all() and (lse[40:] == 7).all() and (lse[:40] != 7).all()
        a, b = api.cache_fwd(q[:40].contiguous(), cache, cu_seqlens=cu, max_seqlen=37,
                             block_idx=idx[:40].contiguous() if kw else None)
        assert torch.equal(a, o[:40]) and torch.equal(b, lse[:40])


def with_errors(q, cache, **kw):
    big = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    out = api.cache_fwd(q, cache, ws=big, **kw)
    return out, api.get_error(big)


def test_bad_table_entries_are_reported_and_left_out():
    """Entries outside the pool (the kernel checks each before it reads):
    their tokens are absent, as if the row did not attend them."""
    cache = filled([256, 100], 2, 64, 64, 2)
    q = torch.randn(2, 4, 1, 64, device=DEV).to(BF)
    idx = torch.tensor([0, 2, 3], dtype=torch.int32, device=DEV).expand(2, 2, 1, 3).clone()
    idx[1] = torch.tensor([0, 1, -1])
    (want, wl), e = with_errors(q, cache, block_idx=idx)
    assert e == api.NSA_OK
    for bad in (-1, -7, cache.k.shape[0], 2 ** 31 - 1):
        cache.page_table[0, 1] = bad
        (o, lse), e = with_errors(q, cache)
        assert e == 3
        tol = 2 ** -8 * want[0].abs().float() + 2 ** -9 * 448 * 2.0 ** -5  # the same sums in another order
        assert ((o[0].float() - want[0].float()).abs() <= tol).all() and (lse[0] - wl[0]).abs().max() < 1e-4


def test_bad_index_entries_and_lengths_are_reported():
    cache = filled([256, 100], 2, 64, 64, 2)
    q = torch.randn(2, 4, 1, 64, device=DEV).to(BF)
    good = torch.tensor([0, 1, -1], dtype=torch.int32, device=DEV).expand(2, 2, 1, 3).clone()
    (want, _), e = with_errors(q, cache, block_idx=good)
    assert e == api.NSA_OK
    for entry in (0, 2 ** 31 - 1, 77, -2):  # repeated, in the future, not an entry
        idx = good.clone()
        idx[1, 0, 0, 2] = entry
        (o, _), e = with_errors(q, cache, block_idx=idx)
        assert e == 3 and torch.equal(o, want)
    lens = cache.seq_lens.clone()
    for n in (-1, 4 * 64 + 1, 2 ** 31 - 1):
        cache.seq_lens[1] = n
        assert with_errors(q, cache)[1] == 3
    cache.seq_lens.copy_(lens)
    assert with_errors(q, cache)[1] == api.NSA_OK


def test_a_window_beyond_every_key_is_none():
    cache = filled([300, 64], 2, 64, 32, 2)
    for T in (1, 40):
        q = torch.randn(2, 8, T, 64, device=DEV).to(BF)
        want = api.cache_fwd(q, cache)
        for window in (320, 5000, 2 ** 31 - 1):
            assert all(torch.equal(a, b) for a, b in zip(want, api.cache_fwd(q, cache, window=window)))


def test_loose_bounds_and_empty_calls():
    """max_seqlen far above the longest run; no token at all."""
    cache = filled([300, 64, 9], 2, 64, 32, 2)
    cu = torch.tensor([0, 3, 3, 5], dtype=torch.int32, device=DEV)
    q = torch.randn(5, 8, 64, device=DEV).to(BF)
    want = api.cache_fwd(q, cache, cu_seqlens=cu, max_seqlen=3)
    for bound in (4, 1000, 1 << 20):
        o, lse = api.cache_fwd(q, cache, cu_seqlens=cu, max_seqlen=bound)
        assert (o.float() - want[0].float()).abs().max() <= 2 ** -7 * want[0].float().abs().max() and (lse - want[1]).abs().max() < 1e-4
    none = torch.zeros(4, dtype=torch.int32, device=DEV)
    o, lse = api.cache_fwd(q[:0], cache, cu_seqlens=none, max_seqlen=1)
    assert o.shape == (0, 8, 64) and lse.shape == (0, 8)
    before = cache.k.view(torch.uint8).clone()
    api.cache_append(cache, q[:0, :2], q[:0, :2], cu_seqlens=none, max_seqlen=1)
    x = torch.randn(5, 2, 64, device=DEV).to(BF)
    api.cache_append(cache, x, x, cu_seqlens=none, max_seqlen=7)  # rows that belong to no sequence
    assert api.get_error(cache.ws) == 0 and torch.equal(before, cache.k.view(torch.uint8))
    free = torch.tensor([9], dtype=torch.int32, device=DEV)
    api.cache_free(cache, free)  # no such row; then a call that finds nothing
    api.cache_append(cache, q[:0, :2], q[:0, :2], cu_seqlens=none, max_seqlen=1)
    assert api.get_error(cache.ws) == 0
    p = api.problem(3, 8, 2, 1, 64, 32, 1, BF, layout=api.LAYOUT_THD, total_tokens=0)
    ws = torch.full((1 << 22,), 0xff, dtype=torch.uint8, device=DEV)
    for idx in (None, cu.data_ptr()):
        assert api.lib().nsa_cache_fwd(p, cache.ref, 0, none.data_ptr(), idx, None, q.data_ptr(), o.data_ptr() or q.data_ptr(),
                                       lse.data_ptr() or q.data_ptr(), ws.data_ptr(), ws.numel(), api._stream()) == 0
        assert api.get_error(ws) == 0


def test_packed_offsets_that_are_none_are_reported():
    """Runs longer than the bound, backward, or past the tensor: their rows are neither read nor written."""
    cache = filled([300, 64], 2, 64, 32, 2)
    q = torch.randn(6, 8, 64, device=DEV).to(BF)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    for offsets, bound in (([0, 4, 6], 3), ([0, 5, 3], 6), ([0, 2, 60], 60), ([-3, 2, 6], 6)):
        cu = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        api.cache_fwd(q, cache, cu_seqlens=cu, max_seqlen=bound, ws=ws)
        assert api.get_error(ws) == 3, offsets
        before = cache.k.view(torch.uint8).clone()
        bad = 0 if offsets[1] - offsets[0] > bound or offsets[0] < 0 else 1
        api.cache_append(cache, q[:, :2].contiguous(), q[:, :2].contiguous(), cu_seqlens=cu, max_seqlen=bound)
        assert api.get_error(cache.ws) == 3, offsets
        held = cache.page_table[bad]
        assert torch.equal(before[held[held >= 0].long()], cache.k.view(torch.uint8)[held[held >= 0].long()])
    long = torch.tensor([0, 500, 400], dtype=torch.int32, device=DEV)  # a chunk's
    many = torch.randn(600, 16, 64, device=DEV).to(BF)
    wide = filled([500, 600], 8, 64, 32, 2)
    assert form_of(lambda: api.cache_fwd(many, wide, cu_seqlens=long, max_seqlen=500, ws=ws)) == "cache_chunk"
    assert api.get_error(ws) == 3


def packed_call(q, cache, offsets, bound, idx=None, **kw):
    """nsa_cache_fwd on packed queries, outputs set to 7 before: (o, lse, error, form)."""
    total, Hq, D = q.shape
    o, lse = torch.full_like(q, 7.0), torch.full((total, Hq), 7.0, device=DEV)
    p = api.problem(len(offsets) - 1, Hq, cache.struct.Hkv, bound, D, cache.struct.block_size, 1 if idx is None else idx.shape[-1],
                    q.dtype, layout=api.LAYOUT_THD, total_tokens=total)
    n = api.lib().nsa_cache_fwd_workspace_size(p, cache.ref, int(idx is not None))
    ws, cu = torch.empty(n, dtype=torch.uint8, device=DEV), i32(*offsets)
    sinks = kw.get("sinks")
    form = form_of(lambda: api._check(api.lib().nsa_cache_fwd(
        p, cache.ref, kw.get("window", 0), cu.data_ptr(), None if idx is None else idx.data_ptr(),
        None if sinks is None else sinks.data_ptr(), q.data_ptr(), o.data_ptr(), lse.data_ptr(), ws.data_ptr(), n, api._stream()), "fwd"))
    return o, lse, api.get_error(ws), form


def check_packed(q, cache, offsets, o, lse, idx=None):
    """The runs that are one against the plain form; every other row untouched."""
    total, Hq, D = q.shape
    mine = np.zeros(total, bool)
    for b, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        if 0 <= lo <= hi <= total:
            mine[lo:hi] = True
            want = Plain(cache).attend(b, q[lo:hi].double().cpu().numpy(), 1 / math.sqrt(D), None if idx is None else idx[lo:hi].cpu().numpy())
            check_attend(o[lo:hi].double().cpu().numpy(), lse[lo:hi].double().cpu().numpy(), *want, q.dtype, D)
    other = torch.tensor(~mine, device=DEV)
    assert (o[other] == 7).all() and (lse[other] == 7).all()


@pytest.mark.parametrize("front,error", [(True, 0), (False, 3)])
@pytest.mark.parametrize("form,dtype,Hq,Hkv,D,bs,lens,runs,S,cols", [
    ("cache_attn_cluster", BF, 8, 2, 64, 32, [100, 70], (5, 9, 14), 3, None),
    ("cache_attn_cluster", F32, 8, 2, 64, 32, [100, 70], (5, 9, 14), 0, None),
    ("cache_attn", BF, 8, 2, 64, 32, [300, 200], (37, 60, 165), 40, None),  # index rows cut, and joined
    ("cache_attn", F32, 40, 2, 32, 16, [300, 200], (37, 60, 125), 40, None),
    ("cache_attn", F32, 8, 2, 64, 32, [300, 200], (37, 60, 125), 0, 600),
    ("cache_chunk", BF, 16, 8, 64, 32, [500, 400], (15, 300, 600), 0, None)])
def test_tokens_in_front_of_the_first_offset_are_left(form, dtype, Hq, Hkv, D, bs, lens, runs, S, cols, front, error):
    """Offsets that begin behind the first token ([5, 9, 14]), and a first run that goes backward ([9, 5, 14]):
    the tokens before belong to no sequence, and none of their rows is read or written."""
    a, b, c = runs
    offsets, total = [a, b, c] if front else [b, a, c], c + 6
    cache = filled(lens, Hkv, D, bs, 4, cols=cols)
    g = np.random.default_rng(4)
    q = torch.tensor(g.normal(size=(total, Hq, D)), dtype=torch.float32).to(dtype).to(DEV)
    idx = None
    if S:
        idx = torch.zeros(total, Hkv, S, dtype=torch.int32, device=DEV)
        new = [max(0, y - x) for x, y in zip(offsets, offsets[1:])]
        at = a if front else offsets[1]
        idx[at:at + sum(new)] = torch.tensor(index_rows(lens, new, Hkv, S, bs, g), device=DEV)
    o, lse, e, took = packed_call(q, cache, offsets, c, idx)
    assert took == form and e == error
    check_packed(q, cache, offsets, o, lse, idx)


@pytest.mark.parametrize("offsets", [[2 ** 31 - 1, -2 ** 31, 4], [2 ** 31 - 1, -2 ** 31 + 300, 400], [-2 ** 31, 2 ** 31 - 1, 5],
                                     [2, 2 ** 31 - 1, 2 ** 31 - 1]])
@pytest.mark.parametrize("total,Hq,Hkv,S", [(12, 8, 2, 0), (12, 8, 2, 3), (600, 16, 8, 0)])
def test_offsets_whose_difference_leaves_the_ints_are_reported(offsets, total, Hq, Hkv, S):
    """Runs from one end of the ints to the other, some of them 1 or 300 tokens long by a difference that wraps round."""
    cache = filled([400, 300], Hkv, 64, 32, 4)
    q = torch.randn(total, Hq, 64, device=DEV).to(BF)
    idx = torch.zeros(total, Hkv, S, dtype=torch.int32, device=DEV) if S else None
    o, lse, e, _ = packed_call(q, cache, offsets, total, idx)
    assert e == 3 and (o == 7).all() and (lse == 7).all()
    before = [x.clone() for x in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale)]
    new = torch.randn(total, Hkv, 64, device=DEV).to(BF)
    api.cache_append(cache, new, new, cu_seqlens=i32(*offsets), max_seqlen=total)
    assert api.get_error(cache.ws) == 3
    for a, b in zip(before, (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("form,dtype,Hq,Hkv,D,T,cols", [("cache_attn_cluster", BF, 8, 2, 128, 1, None), ("cache_attn_cluster", F32, 6, 2, 64, 5, None),
                                                        ("cache_attn", BF, 8, 2, 128, 3, 900), ("cache_attn", F32, 24, 2, 32, 2, 2000),
                                                        ("cache_chunk", BF, 16, 8, 64, 150, None), ("cache_chunk", BF, 16, 8, 128, 150, None)])
def test_strided_queries_give_the_same(form, dtype, Hq, Hkv, D, T, cols):
    """Queries as a model's projection leaves them: token before head, a slice of one tensor of queries, keys and values."""
    cache = filled([400, 170, 0, 151], Hkv, D, 32, 7, cols=cols)
    wide = torch.randn(4, T, Hq + 2 * Hkv, D, device=DEV).to(dtype)
    q = wide[:, :, :Hq].transpose(1, 2)
    sinks = torch.randn(Hq, device=DEV)
    for kw in (dict(), dict(window=60, sinks=sinks)):
        got = []
        assert form_of(lambda: got.append(api.cache_fwd(q, cache, **kw))) == form or kw
        want = api.cache_fwd(q.contiguous(), cache, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got[0], want))
    if T < 40:
        idx = torch.zeros(4, Hkv, T, 2, dtype=torch.int32, device=DEV)
        idx[..., 1] = -1
        assert all(torch.equal(a, b) for a, b in zip(api.cache_fwd(q, cache, block_idx=idx), api.cache_fwd(q.contiguous(), cache, block_idx=idx)))
    packed = wide.view(4 * T, Hq + 2 * Hkv, D)[:, :Hq]
    cu = i32(*[T * i for i in range(5)])
    a, b = (api.cache_fwd(x, cache, cu_seqlens=cu, max_seqlen=T) for x in (packed, packed.contiguous()))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_calls_keep_their_own_word():
    """A chunk's and a list's call in graphs, replayed on two streams at once: each graph has its workspace."""
    cache = filled([700, 300, 40], 8, 64, 32, 6, cols=900)
    q = torch.randn(3, 16, 150, 64, device=DEV).to(BF)
    one = q[:, :, :1].contiguous()
    want = [api.cache_fwd(x, cache) for x in (q, one)]
    torch.cuda.synchronize()
    graphs, outs, words = [], [], []
    for x, form in ((q, "cache_chunk"), (one, "cache_attn")):
        assert form_of(lambda: api.cache_fwd(x, cache)) == form
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(api.cache_fwd(x, cache))
        graphs.append(g)
        words.append(cache.fwd_ws)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert [api.get_error(w) for w in words] == [0, 0]
        for a, b in zip(want, outs):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    page = cache.page_table[0, 2].clone()
    cache.page_table[0, 2] = -5
    for g in graphs:
        g.replay()
    assert [api.get_error(w) for w in words] == [3, 3]
    cache.page_table[0, 2] = page


def test_the_most_rows_of_a_call():
    g = np.random.default_rng(9)
    takes("cache_attn", [int(n) for n in g.integers(0, 40, 8192)], [1] * 8192, 2, 1, 32, 16, F32)


def test_calls_on_two_streams_and_in_graphs():
    cache = filled([3000, 100, 0, 64], 2, 128, 64, 4)
    qs = [torch.randn(4, 8, T, 128, device=DEV).to(BF) for T in (1, 1, 3, 50)]
    want = [api.cache_fwd(q, cache) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(api.cache_fwd(q, cache))
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        got = [api.cache_fwd(q, cache, stream=s) for q, s in zip(qs, streams)]
        torch.cuda.synchronize()
        for a, b, c in zip(want, outs, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b)) and all(torch.equal(x, y) for x, y in zip(a, c))


# --------------------------------------- each of the attention's three forms

def form_of(call):
    """The name under which the call's kernel was launched: the form it took."""
    api.trace_enable(64)
    try:
        call()
        torch.cuda.synchronize()
        return [name for name, _ in api.trace_records()][-1]
    finally:
        api.trace_enable(0)


def takes(form, *a, **kw):
    assert form_of(lambda: attend_case(*a, **kw)) == form


MASKS = [dict(), dict(window=1), dict(window=37), dict(window=200), dict(sinks=True), dict(window=70, sinks=True)]


@pytest.mark.parametrize("kw", MASKS)
@pytest.mark.parametrize("Hq,Hkv,D,bs", [(16, 8, 128, 64), (8, 8, 64, 16), (24, 8, 128, 32), (40, 8, 64, 64), (16, 8, 128, 16),
                                         (16, 8, 64, 32)])
def test_chunk_form(kw, Hq, Hkv, D, bs):
    T = -(-256 // (Hq // Hkv))  # 256 rows and, of the last sequence, some more
    lens, new = [T + 130, 40, 0, 3 * T, T + 1], [T, 40, 0, 1, T + 1]
    takes("cache_chunk", lens, new, Hq, Hkv, D, bs, BF, ragged=True, **kw)


@pytest.mark.parametrize("layout", ["dense", "token", "both"])
def test_chunk_form_fixed_length(layout):
    """Rows before the first key, one tile of rows and a part of another, strided pools."""
    takes("cache_chunk", [100, 500, 3, 150], [150] * 4, 16, 8, 128, 64, BF, layout=layout)
    takes("cache_chunk", [100, 500, 3, 150], [150] * 4, 16, 8, 64, 16, BF, layout=layout, sinks=True, window=90)


def test_chunk_form_long():
    takes("cache_chunk", [1500, 700], [600, 700], 16, 2, 128, 64, BF, ragged=True)


@pytest.mark.parametrize("D,bs", [(128, 64), (64, 16)])
def test_chunk_form_nan_values(D, bs):
    """NaN among the chunk's own tokens (some rows see them) and among earlier
    ones (every row does; with the window the early rows alone), values and a key."""
    def edit(cache):
        for t, h, d in ((150, 0, 3), (199, 1, 30), (199, 0, D - 1), (130, 7, 0), (20, 3, 11)):
            p = int(cache.page_table[0, t // bs])
            cache.v.view(torch.uint8)[p, h, t % bs, d] = 0xff
        p = int(cache.page_table[1, 180 // bs])
        cache.k.view(torch.uint8)[p, 2, 180 % bs, 5] = 0x7f
    for kw in (dict(), dict(window=60)):
        takes("cache_chunk", [200, 230, 90, 160], [130, 130, 90, 160], 16, 8, D, bs, BF, ragged=True, edit=edit, **kw)


def test_chunk_form_scales_and_bad_pages():
    def edit(cache):
        cache.v_scale[::2] = 2.0 ** -60
        cache.v_scale[1::3] = 2.0 ** 40
        cache.k_scale[::3] *= 2.0 ** -20
        cache.k_scale[1::5] = 0.0
    takes("cache_chunk", [300, 700], [300, 200], 16, 8, 128, 64, BF, ragged=True, edit=edit)
    cache = filled([700, 400], 8, 128, 64, 3)
    q = torch.randn(2, 16, 400, 128, device=DEV).to(BF)
    cu = torch.tensor([0, 400, 800], dtype=torch.int32, device=DEV)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    packed = q.transpose(1, 2).reshape(800, 16, 128).contiguous()
    for bad in (-1, -9, cache.k.shape[0], 2 ** 31 - 1):
        cache.page_table[0, 2] = bad
        o, lse = api.cache_fwd(packed, cache, cu_seqlens=cu, max_seqlen=400, ws=ws)
        assert api.get_error(ws) == 3
        # the page's tokens are absent: the same rows with those keys out of every row's scores
        plain = Plain(cache)
        plain.table = plain.table.copy()
        plain.table[0, 2] = 0
        for t in (0, 250, 399):
            K, V = plain.keys(0, 3)
            keep = np.ones(301 + t, bool)
            keep[128:192] = False
            z = K[:301 + t][keep] @ packed[t, 7].double().cpu().numpy() / math.sqrt(128)
            w = np.exp(z - z.max())
            want = w @ V[:301 + t][keep] / w.sum()
            tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -10 + 2.0 ** -14) * np.abs(V[:301 + t][keep]).max()
            assert (np.abs(o[t, 7].double().cpu().numpy() - want) <= tol).all()
    cache.page_table[0, 2] = 0
    lens = cache.seq_lens.clone()
    for n in (-1, 11 * 64 + 1, 2 ** 31 - 1):
        cache.seq_lens[1] = n
        api.cache_fwd(packed, cache, cu_seqlens=cu, max_seqlen=400, ws=ws)
        assert api.get_error(ws) == 3
    cache.seq_lens.copy_(lens)
    api.cache_fwd(packed, cache, cu_seqlens=cu, max_seqlen=400, ws=ws)
    assert api.get_error(ws) == 0


def far_values(*scales):
    """Pages in turn: zeros (the scale that append gives them), then values of each scale."""
    def edit(cache):
        n = len(scales) + 1
        cache.v_scale[::n] = 2.0 ** -100
        cache.v.view(torch.uint8)[::n] = 0
        for i, s in enumerate(scales):
            cache.v_scale[i + 1::n] = s
    return edit


SPREAD = (2.0 ** 27, 2.0 ** 60, 1.0, 2.0 ** -60, 2.0 ** 100, 2.0 ** -90)


@pytest.mark.parametrize("scales,kw", [((2.0 ** 27,), dict()), ((2.0 ** 60,), dict(sinks=True)), ((2.0 ** 41, 2.0 ** -41), dict(window=200)),
                                       ((1.0,), dict()), (SPREAD, dict(S=9)), (SPREAD, dict())])
@pytest.mark.parametrize("form,dtype,G,D,bs", [
    ("cache_attn_cluster", BF, 4, 128, 64), ("cache_attn_cluster", F32, 12, 64, 32), ("cache_attn_cluster", BF, 20, 32, 16),
    ("cache_attn", BF, 4, 128, 16), ("cache_attn", F32, 3, 128, 64), ("cache_attn", BF, 12, 128, 64), ("cache_attn", F32, 20, 64, 32)])
def test_values_of_zero_beside_large_ones(scales, kw, form, dtype, G, D, bs):
    """Every page counts in the denominator, however far apart its values' scale lies (a page of zeros beside one of
    large values, ordinary scores): O and LSE by each form of the attention."""
    if form == "cache_attn_cluster":
        lens, cols = [900, 65, 300], None
    else:
        g = np.random.default_rng(3)
        lens = [int(n) for n in g.integers(1, 250, 110 if "S" not in kw else 460)]
        cols = 9000 * 128 // (bs * D) if "window" not in kw else 4000 * 128 // (bs * D)
    kw = dict(kw, window=3500) if form == "cache_attn" and "window" in kw else kw  # (many keys in reach: the list form)
    takes(form, lens, [1] * len(lens), 2 * G, 2, D, bs, dtype, cols=cols, edit=far_values(*scales), **kw)


@pytest.mark.parametrize("scales,kw", [((2.0 ** 27,), dict()), ((2.0 ** 60,), dict(window=70, sinks=True)), (SPREAD, dict()),
                                       (SPREAD, dict(window=150))])
@pytest.mark.parametrize("D,bs", [(128, 64), (128, 16), (64, 32)])
def test_chunk_form_values_of_zero_beside_large_ones(scales, kw, D, bs):
    takes("cache_chunk", [700, 300, 40], [260, 300, 40], 16, 8, D, bs, BF, ragged=True, edit=far_values(*scales), **kw)


@pytest.mark.parametrize("form,dtype,D,bs,lens,T", [
    ("cache_attn_cluster", BF, 32, 16, [16, 15], 1), ("cache_attn_cluster", F32, 32, 16, [16, 15], 1),
    ("cache_attn_cluster", F32, 64, 32, [16, 9], 1), ("cache_attn", F32, 32, 16, [16] * 90, 1), ("cache_attn", BF, 32, 16, [16] * 90, 1),
    ("cache_chunk", BF, 64, 32, [300, 300], 300)])
def test_small_weights_beside_a_large_one_keep_their_bits(form, dtype, D, bs, lens, T):
    """One key takes nearly the whole weight and has a value of zero (a sink among the keys); what is left is the others,
    all of one weight: the output is held to their relative roundings.  (The weight's place between two halves of step
    2^-24 is the worst: 45.5 of them, or in 32 bits 1420.5.)"""
    gap = 24 - math.log2(45.5 if dtype == BF else 1420.5)
    Hkv, G = (8, 2) if form == "cache_chunk" else (2, 4)
    cache = filled(lens, Hkv, D, bs, 5, garbage=False, cols=1000 * 64 // bs if form == "cache_attn" else None)
    cache.k.view(torch.uint8).zero_()
    cache.v.view(torch.uint8).fill_(0x38)  # 1.0
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(1.0)
    for b in range(len(lens)):
        p = int(cache.page_table[b, 0])
        cache.k.view(torch.uint8)[p, :, 0, 0] = 0x38
        cache.v.view(torch.uint8)[p, :, 0] = 0
    B = len(lens)
    q = torch.zeros(B, Hkv * G, T, D)
    q[..., 0] = 16.0
    scale = gap * math.log(2) / 16
    out = []
    assert form_of(lambda: out.append(api.cache_fwd(q.to(dtype).to(DEV), cache, scale=scale))) == form
    o, lse = (x.double().cpu().numpy() for x in out[0])
    s32 = float(torch.tensor(scale, dtype=torch.float32).double())
    keys = np.maximum(np.array(lens)[:, None] - T + 1 + np.arange(T)[None], 0)  # [B, T]
    small = (keys - 1) * math.exp(-16 * s32)
    want = (small / (1 + small))[:, None, :, None]
    # the score: two roundings of the scale and one of the product; the exponential 2^-21; the weight's 11 or 22 bits;
    # the sums' roundings; the output's own
    rel = 2 * (3 * U32 * gap + 2.0 ** -21) + (2.0 ** -11 if dtype == BF else 2.0 ** -21) + 2 * (max(lens) + 16) * U32
    rel += torch.finfo(dtype).eps / 2
    assert (np.abs(o - want) <= rel * (1 + 2.0 ** -7) * want).all(), np.abs(o / np.maximum(want, 1e-30) - 1).max()
    assert (np.abs(lse - (16 * s32 + np.log1p(small))[:, None]) <= (gap + 4) * 8 * U32).all()


def test_chunk_form_leaves_rows_behind_the_last_sequence():
    cache = filled([400, 300], 8, 64, 32, 1)
    cu = torch.tensor([0, 300, 600], dtype=torch.int32, device=DEV)
    q = torch.randn(620, 16, 64, device=DEV).to(BF)
    p = api.problem(2, 16, 8, 300, 64, 32, 1, BF, layout=api.LAYOUT_THD, total_tokens=620)
    o, lse = torch.full((620, 16, 64), 7.0, device=DEV).to(BF), torch.full((620, 16), 7.0, device=DEV)
    call = lambda: api._check(api.lib().nsa_cache_fwd(p, cache.ref, 0, cu.data_ptr(), None, None, q.data_ptr(), o.data_ptr(), lse.data_ptr(), None, 0, api._stream()), "fwd")  # noqa: E731
    assert form_of(call) == "cache_chunk"
    assert (o[600:] == 7).all() and (lse[600:] == 7).all() and (lse[:600] != 7).all()


@pytest.mark.parametrize("kw", MASKS + [dict(S=27), dict(S=130)])
@pytest.mark.parametrize("dtype,Hq,Hkv,D,bs,T", [(BF, 8, 2, 128, 64, 1), (F32, 6, 2, 64, 32, 2), (BF, 32, 2, 128, 16, 1),
                                                 (F32, 2, 1, 32, 16, 7), (BF, 20, 1, 64, 64, 1), (F32, 16, 1, 128, 64, 1)])
def test_list_form(kw, dtype, Hq, Hkv, D, bs, T):
    g = np.random.default_rng(5)
    B = 320 // Hkv
    lens = [int(n) for n in g.integers(0, 300, B)]
    cols = None if "S" in kw else 1100 * 128 // (bs * D)  # a table wide enough for long sequences
    if kw.get("window", 0) or cols is None:
        attend_case(lens, [T] * B, Hq, Hkv, D, bs, dtype, cols=cols, **kw)
    else:
        takes("cache_attn", lens, [T] * B, Hq, Hkv, D, bs, dtype, cols=cols, **kw)


def test_list_form_window():
    g = np.random.default_rng(8)
    takes("cache_attn", [int(n) for n in g.integers(0, 5000, 40)], [2] * 40, 16, 8, 128, 64, BF, window=3500)


@pytest.mark.parametrize("kw", [dict(window=1), dict(window=37), dict(window=200), dict(window=70, sinks=True)])
@pytest.mark.parametrize("dtype,Hq,Hkv,D,bs,T", [(BF, 8, 2, 128, 64, 1), (F32, 6, 2, 64, 32, 2), (BF, 32, 2, 128, 16, 1),
                                                 (F32, 2, 1, 32, 16, 7), (BF, 20, 1, 64, 64, 1), (F32, 16, 1, 128, 64, 1)])
def test_list_form_short_windows(kw, dtype, Hq, Hkv, D, bs, T):
    """Windows of any length take the list where the table has many entries."""
    g = np.random.default_rng(5)
    B = 320 // Hkv
    takes("cache_attn", [int(n) for n in g.integers(0, 300, B)], [T] * B, Hq, Hkv, D, bs, dtype, cols=8200 // B + 1, **kw)


@pytest.mark.parametrize("S,rows", [(27, 320), (130, 320), (28, 304), (130, 304)])
@pytest.mark.parametrize("dtype,G,D,bs", [(BF, 4, 128, 64), (F32, 3, 64, 32), (BF, 16, 128, 16), (BF, 20, 64, 64), (F32, 2, 32, 16)])
def test_list_form_index(S, rows, dtype, G, D, bs):
    """Index rows cut at 128 tokens and joined (320 of them over 304 or 152 CTAs), and whole ones, with nothing to join (304)."""
    g = np.random.default_rng(6)
    takes("cache_attn", [int(n) for n in g.integers(0, 300, rows // 2)], [1] * (rows // 2), 2 * G, 2, D, bs, dtype, S=S)


@pytest.mark.parametrize("T", [1, 4])
def test_list_form_nan_values(T):
    def edit(cache):
        for b in (0, 17, 100):
            t = int(cache.seq_lens[b]) - 1
            p = int(cache.page_table[b, t // 32])
            cache.v.view(torch.uint8)[p, 1, t % 32, 5] = 0x7f
    g = np.random.default_rng(6)
    takes("cache_attn", [int(n) for n in g.integers(4, 200, 160)], [T] * 160, 8, 2, 64, 32, BF, edit=edit, cols=40)


@pytest.mark.parametrize("kw", MASKS + [dict(S=1), dict(S=5), dict(S=40)])
@pytest.mark.parametrize("B,Hkv", [(1, 1), (2, 2), (5, 4), (12, 8), (50, 8)])
def test_cluster_form(kw, B, Hkv):
    """One CTA a unit (12 x 8, and 50 x 8 in several rounds) up to 16 (one unit alone)."""
    g = np.random.default_rng(7)
    lens = [int(n) for n in g.integers(0, 700 if B < 50 else 200, B)]
    for dtype, G, D, bs, T in ((BF, 4, 128, 64, 1), (F32, 3, 64, 16, 4), (BF, 20, 32, 32, 1)):
        T = 1 if "S" in kw else T  # (a unit for each token there)
        kw = dict(S=15) if B == 50 and kw.get("S") == 40 else kw  # (8192 entries at most)
        takes("cache_attn_cluster", lens, [T] * B, Hkv * G, Hkv, D, bs, dtype, **kw)


def test_one_long_sequence_takes_the_cluster_form_and_a_longer_one_the_list():
    takes("cache_attn_cluster", [9000], [1], 4, 2, 128, 64, BF)
    takes("cache_attn", [66000], [1], 4, 1, 128, 64, BF)


# ------------------------------------------------------------------ append

def same_pool(cache, plain):
    for a, b in ((cache.k, plain.k), (cache.v, plain.v)):
        x = a.cpu().float().double().numpy()
        assert np.array_equal(np.isnan(x), np.isnan(b)) and np.array_equal(x[~np.isnan(b)], b[~np.isnan(b)])
    assert np.array_equal(cache.k_scale.cpu().double().numpy(), plain.ks)
    assert np.array_equal(cache.v_scale.cpu().double().numpy(), plain.vs)


def same_meta(cache, plain):
    assert np.array_equal(cache.page_table.cpu().numpy(), plain.table)
    assert np.array_equal(cache.seq_lens.cpu().numpy(), plain.lens)
    assert np.array_equal(cache.refcount.cpu().numpy(), plain.ref)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hkv,D,bs", [(2, 128, 64), (3, 64, 32), (1, 32, 16), (2, 128, 16), (1, 64, 64)])
@pytest.mark.parametrize("T", [1, 2, 9, 64, 150])
def test_append_fixed_length(dtype, Hkv, D, bs, T):
    g = np.random.default_rng(T)
    before = [0, 1, bs - 1, bs, 77]
    cache = filled([n + T for n in before], Hkv, D, bs, 7)
    for which in (cache.k_scale, cache.v_scale):  # powers of two, some of which have to grow
        which.copy_(torch.exp2(torch.randint(-12, -4, which.shape, device=DEV).float()))
    plain = Plain(cache)
    kn, vn = (torch.tensor(g.normal(size=(5, Hkv, T, D)) * 10.0 ** g.integers(-3, 3, (5, Hkv, 1, 1)), dtype=torch.float32).to(dtype) for _ in range(2))
    api.cache_append(cache, kn.to(DEV), vn.to(DEV))
    assert api.get_error(cache.ws) == 0
    for b in range(5):
        plain.append(b, *(x[b].transpose(0, 1).double().numpy() for x in (kn, vn)))
    same_pool(cache, plain)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_packed_and_strided(dtype):
    g = np.random.default_rng(9)
    Hkv, D, bs = 2, 64, 32
    before, new = [0, 5, 31, 64, 12], [70, 0, 1, 40, 200]
    cache = filled([a + n for a, n in zip(before, new)], Hkv, D, bs, 8, layout="token")
    plain = Plain(cache)
    total = sum(new) + 6  # rows behind the last sequence
    qkv = torch.tensor(g.normal(size=(total, 3 * Hkv, D)), dtype=torch.float32).to(dtype).to(DEV)  # k and v inside a packed tensor
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
    api.cache_append(cache, qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:], cu_seqlens=cu, max_seqlen=200)
    assert api.get_error(cache.ws) == 0
    x = qkv.double().cpu().numpy()
    for b in range(5):
        rows = x[int(cu[b]):int(cu[b + 1])]
        plain.append(b, rows[:, Hkv:2 * Hkv], rows[:, 2 * Hkv:])
    same_pool(cache, plain)


@pytest.mark.parametrize("offsets,error", [([5, 9, 9, 150], 0), ([9, 5, 40, 60], 3)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_from_behind_the_first_token(dtype, offsets, error):
    """Packed offsets that begin behind the first token, and a first run that goes backward: no row of nobody's is taken."""
    cache = filled([60, 50, 200], 2, 64, 32, 3, garbage=False)
    plain = Plain(cache)
    g = np.random.default_rng(3)
    k, v = (torch.tensor(g.normal(size=(156, 2, 64)), dtype=torch.float32).to(dtype) for _ in range(2))
    api.cache_append(cache, k.to(DEV), v.to(DEV), cu_seqlens=i32(*offsets), max_seqlen=150)
    assert api.get_error(cache.ws) == error
    for b, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        if lo < hi:
            plain.append(b, k[lo:hi].double().numpy(), v[lo:hi].double().numpy())
    same_pool(cache, plain)


def test_append_special_values():
    cache = filled([66, 64], 1, 32, 64, 1, garbage=False)
    cache.k_scale.fill_(2.0 ** -7)
    plain = Plain(cache)
    kn = torch.zeros(2, 1, 2, 32)
    kn[0, 0, 0, :8] = torch.tensor([math.inf, -math.inf, math.nan, 448.0, -449.0, 1e-30, 0.0, -0.0])
    kn[0, 0, 1, :4] = torch.tensor([3.4e38, -3.4e38, 2.0 ** -126, 2.0 ** -149])
    vn = torch.zeros(2, 1, 2, 32)  # a block of zeros
    vn[1, 0, 0, 0] = 1e-38
    api.cache_append(cache, kn.to(DEV), vn.to(DEV))
    with np.errstate(invalid="ignore"):
        for b in range(2):
            plain.append(b, *(x[b].transpose(0, 1).double().numpy() for x in (kn, vn)))
    same_pool(cache, plain)


def test_append_ties_and_boundaries():
    """Every e4m3 value, every midpoint of two neighbours, and fp32's neighbours of those."""
    vals = torch.arange(0, 0x7f, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double().numpy()
    mids = (vals[1:] + vals[:-1]) / 2
    x = np.concatenate([vals, mids, np.nextafter(mids.astype(np.float32), np.float32(1e9)), np.nextafter(mids.astype(np.float32), np.float32(0))])
    x = np.resize(np.concatenate([x, -x]), (17 * 64,)).reshape(17, 64)
    cache = filled([17], 1, 64, 64, 1)
    plain = Plain(cache)
    t = torch.tensor(x, dtype=torch.float32).view(1, 1, 17, 64)
    api.cache_append(cache, t.to(DEV), (t * 2.0 ** -20).to(DEV))
    plain.append(0, t[0].transpose(0, 1).double().numpy(), (t[0] * 2.0 ** -20).transpose(0, 1).double().numpy())
    assert plain.ks[plain.table[0, 0], 0] == 1.0
    same_pool(cache, plain)


def test_append_leaves_shared_and_foreign_pages():
    cache = filled([10, 20], 1, 32, 16, 3, garbage=False)
    before = [x.clone() for x in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale)]
    x = torch.randn(2, 1, 4, 32, device=DEV)
    cache.refcount[cache.page_table[0, 0]] = 2
    cache.page_table[1, 1] = cache.k.shape[0]
    api.cache_append(cache, x, x)
    assert api.get_error(cache.ws) == 3
    for a, b in zip(before, (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale)):
        assert torch.equal(a, b)
    cache.seq_lens.copy_(torch.tensor([3, 33], dtype=torch.int32))  # fewer tokens than are new; beyond the table
    api.cache_append(cache, x, x)
    assert api.get_error(cache.ws) == 3
    for a, b in zip(before, (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------- pages

def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("pool,rows,cols,Hkv,D,bs,seed", [(64, 8, 12, 2, 64, 16, 0), (300, 12, 40, 1, 32, 16, 1),
                                                          (5000, 40, 150, 1, 32, 16, 2), (33, 5, 9, 3, 128, 64, 3)])
def test_page_operations_at_random(pool, rows, cols, Hkv, D, bs, seed):
    g = np.random.default_rng(seed)
    cache = api.make_cache(pool, Hkv, D, bs, rows, cols)
    for x in (cache.k, cache.v):
        x.view(torch.uint8).copy_(torch.randint(0, 0x7f, x.shape, device=DEV, dtype=torch.uint8))
    cache.k_scale.copy_(torch.rand_like(cache.k_scale) + 0.5)
    cache.v_scale.copy_(torch.rand_like(cache.v_scale) + 0.5)
    plain = Plain(cache)
    for step in range(60):
        op = g.choice(["reserve", "reserve", "free", "fork", "copy", "compact"])
        if op == "reserve":
            room = cols * bs - plain.lens
            n = np.minimum(g.integers(0, max(2, 3 * pool * bs // rows // 4), rows) * (g.random(rows) < 0.5), room)
            api.cache_reserve(cache, i32(*n))
            want = plain.reserve(n)
        elif op == "free":
            r = g.permutation(rows)[:g.integers(0, rows // 2 + 1)]
            api.cache_free(cache, i32(*r))
            for x in r:
                plain.release(x)
            want = 0
        elif op == "fork":
            r = list(g.permutation(rows))
            n = int(g.integers(1, rows // 2 + 1))
            dst = r[:n]
            src = list(g.choice(r[n:], n))
            api.cache_fork(cache, i32(*src), i32(*dst))
            want = plain.fork(src, dst)
        elif op == "copy":
            r = g.permutation(pool)
            n = int(g.integers(0, pool // 2))
            free = [p for p in r if plain.ref[p] <= 0][:n]
            src = g.choice([p for p in r if p not in set(free)] or [0], len(free))
            free = [] if (len(src) and src[0] in free) else free
            src = src[:len(free)]
            api.cache_copy(cache, i32(*src), i32(*free))
            for s, d in zip(src, free):
                plain.copy_page(s, d)
            want = 0
        else:
            api.cache_compact(cache)
            plain.compact()
            want = 0
        assert api.get_error(cache.ws) == want, op
        same_meta(cache, plain)
        same_pool(cache, plain)


def test_page_lists_are_checked():
    cache = filled([40, 20, 0, 33], 1, 32, 16, 3, garbage=False)
    plain = Plain(cache)

    def unchanged(call, *a):
        call(cache, *a)
        assert api.get_error(cache.ws) == 3
        same_meta(cache, plain)
        same_pool(cache, plain)

    unchanged(api.cache_fork, i32(0, 1), i32(2, 2))      # one row forked into twice
    unchanged(api.cache_fork, i32(0, 1), i32(1, 2))      # a source that is also a destination
    unchanged(api.cache_fork, i32(0, 4), i32(2, 3))      # no such row
    unchanged(api.cache_fork, i32(0, 0), i32(2, -1))
    unchanged(api.cache_reserve, i32(0, -1, 0, 0))
    unchanged(api.cache_reserve, i32(0, 0, 2 ** 31 - 1, 0))
    unchanged(api.cache_reserve, i32(9, 0, 0, 0))        # 49 tokens: beyond the 3 columns of the table
    n = cache.k.shape[0]
    api.cache_copy(cache, i32(0, 1, 2, n, 4), i32(5, 5, 1, 6, -1))  # repeated, a source, outside: the first alone is copied
    assert api.get_error(cache.ws) == 3
    plain.copy_page(0, 5)
    same_pool(cache, plain)
    api.cache_free(cache, i32(1, 1, 9, -1))
    assert api.get_error(cache.ws) == 3
    plain.release(1)
    same_meta(cache, plain)
    api.cache_free(cache, i32())
    assert api.get_error(cache.ws) == 0
    same_meta(cache, plain)


@pytest.mark.parametrize("pool,rows,cols,bs", [(60, 6, 9, 16), (3000, 300, 9, 32), (9000, 70, 110, 16), (9000, 1300, 8, 16)])
def test_lowered_lengths_keep_their_pages(pool, rows, cols, bs):
    """Drafted tokens that were rejected: the caller lowers a row's length, and the row grows into the pages that it
    holds.  No page is lost: a page is in use exactly as often as the table names it."""
    g = np.random.default_rng(pool)
    cache = api.make_cache(pool, 1, 32, bs, rows, cols)
    table, lens = np.full((rows, cols), -1, np.int64), np.zeros(rows, np.int64)
    for step in range(25):
        grow = np.minimum(g.integers(0, 4 * bs if step % 3 else 9, rows), cols * bs - lens)
        api.cache_reserve(cache, i32(*grow))
        count = np.bincount(table[table >= 0], minlength=pool)
        free = iter(np.flatnonzero(count == 0))
        # a page that several rows hold is no row's to grow into
        missing = [(b, c) for b in range(rows) for c in range(-(-lens[b] // bs), -(-(lens[b] + grow[b]) // bs))
                   if table[b, c] < 0 or count[table[b, c]] > 1]
        if len(missing) > (count == 0).sum():
            assert api.get_error(cache.ws) == 7
        else:
            assert api.get_error(cache.ws) == 0
            for b, c in missing:
                table[b, c] = next(free)
            lens += grow
        if step % 6 == 2:
            order = np.argsort(lens)
            src, dst = order[-3:], order[:3]
            api.cache_fork(cache, i32(*src), i32(*dst))
            tails = sum(int(n % bs > 0) for n in lens[src])
            held = table.copy()
            held[dst] = -1
            free = iter(np.flatnonzero(np.bincount(held[held >= 0], minlength=pool) == 0).tolist() + [-1] * 3)
            ids = [next(free) if lens[s] % bs else -1 for s in src]
            if tails and min(i for s, i in zip(src, ids) if lens[s] % bs) < 0:
                assert api.get_error(cache.ws) == 7
            else:
                assert api.get_error(cache.ws) == 0
                table = held
                for s, d, i in zip(src, dst, ids):
                    full = lens[s] // bs
                    table[d, :full] = table[s, :full]
                    if lens[s] % bs:
                        table[d, full] = i
                    lens[d] = lens[s]
        if step % 8 == 7:
            gone = g.permutation(rows)[:rows // 3]
            api.cache_free(cache, i32(*gone))
            table[gone], lens[gone] = -1, 0
        assert np.array_equal(cache.page_table.cpu().numpy(), table) and np.array_equal(cache.seq_lens.cpu().numpy(), lens)
        assert np.array_equal(cache.refcount.cpu().numpy(), np.bincount(table[table >= 0], minlength=pool))
        lens = np.maximum(lens - g.integers(0, 2 * bs, rows) * (g.random(rows) < 0.7), 0)
        cache.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    row = int(lens.argmin())
    held = cache.page_table[row].clone()
    col = int(-(-lens[row] // bs))
    for entry in (-2, pool, 2 ** 31 - 1, next(p for p in range(pool) if p not in set(table[table >= 0].tolist()))):
        cache.page_table[row, col] = entry
        before = [x.clone() for x in (cache.page_table, cache.seq_lens, cache.refcount)]
        api.cache_reserve(cache, i32(*[bs if b == row else 0 for b in range(rows)]))
        assert api.get_error(cache.ws) == 3
        for a, b in zip(before, (cache.page_table, cache.seq_lens, cache.refcount)):
            assert torch.equal(a, b)
    cache.page_table[row] = held


@pytest.mark.parametrize("spare", [0, 5])
def test_a_fork_over_miscounted_pages_changes_nothing(spare):
    """The destinations' entries name a page more often than its count says: found only when they are given back."""
    for entries, count in (((0, 0), 1), ((0, 1, 0), 2), ((2, 2, 2), 2)):
        cache = filled([40, 48, 48, 48], 1, 32, 16, 3, spare=spare, garbage=False)
        for row in (2, 3):
            for col, e in enumerate(entries):
                cache.page_table[row, col] = cache.page_table[2, e].clone()
        cache.refcount[cache.page_table[2, entries[0]].long()] = count
        plain = Plain(cache)
        api.cache_fork(cache, i32(0, 1), i32(2, 3))
        assert api.get_error(cache.ws) == 3
        same_meta(cache, plain)
        same_pool(cache, plain)


def test_a_full_pool_changes_nothing():
    cache = filled([40, 20, 0, 33], 1, 32, 16, 3, spare=1, cols=8, garbage=False)
    plain = Plain(cache)
    api.cache_reserve(cache, i32(0, 10, 30, 0))
    assert api.get_error(cache.ws) == 7
    same_meta(cache, plain)
    api.cache_fork(cache, i32(0, 3), i32(2, 1))
    assert plain.fork([0, 3], [2, 1]) == 0  # row 1's own pages make the room
    assert api.get_error(cache.ws) == 0
    same_meta(cache, plain)
    same_pool(cache, plain)
    api.cache_reserve(cache, i32(1, 0, 0, 0))
    assert plain.reserve([1, 0, 0, 0]) == 0 and api.get_error(cache.ws) == 0
    same_meta(cache, plain)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("dtype,Hq,Hkv,D,bs", [(BF, 8, 2, 128, 64), (F32, 4, 2, 32, 16)])
def test_serving_steps(dtype, Hq, Hkv, D, bs, graph):
    """Prompts go in, rows are forked, every row takes single tokens (as one
    captured step too), some leave, the pool is compacted, others enter."""
    g = np.random.default_rng(11)
    rows = 6
    cache = api.make_cache(60, Hkv, D, bs, rows, 10)
    plain = Plain(cache)

    def fresh(n, H):
        return torch.tensor(g.normal(size=(n, H, D)), dtype=torch.float32).to(dtype)

    def check(b, q, o, lse):
        want = plain.attend(b, q.double().numpy(), 1 / math.sqrt(D))
        check_attend(o.double().cpu().numpy(), lse.double().cpu().numpy(), *want, dtype, D)

    def prompts(new):
        api.cache_reserve(cache, i32(*new))
        assert plain.reserve(new) == 0
        cu = i32(*np.concatenate([[0], np.cumsum(new)]))
        q, k, v = fresh(sum(new), Hq), fresh(sum(new), Hkv), fresh(sum(new), Hkv)
        api.cache_append(cache, k.to(DEV), v.to(DEV), cu_seqlens=cu, max_seqlen=max(new))
        o, lse = api.cache_fwd(q.to(DEV), cache, cu_seqlens=cu, max_seqlen=max(new))
        at = 0
        for b, n in enumerate(new):
            plain.append(b, k[at:at + n].double().numpy(), v[at:at + n].double().numpy())
            check(b, q[at:at + n], o[at:at + n], lse[at:at + n])
            at += n

    one = i32(*[1] * rows)
    hold = [torch.zeros(rows, H, 1, D, dtype=dtype, device=DEV) for H in (Hq, Hkv, Hkv)]

    def step():
        api.cache_reserve(cache, one)
        api.cache_append(cache, hold[1], hold[2])
        return api.cache_fwd(hold[0], cache)

    prompts([bs + 3, 0, 5, 0, 2 * bs, 0])
    api.cache_fork(cache, i32(0, 2, 4), i32(1, 3, 5))
    assert plain.fork([0, 2, 4], [1, 3, 5]) == 0
    captured = None
    if graph:
        saved = [x.clone() for x in (cache.page_table, cache.seq_lens, cache.refcount)]
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            got = step()
        for a, b in zip((cache.page_table, cache.seq_lens, cache.refcount), saved):
            a.copy_(b)
    for i in range(2 * bs // 8 + 3):
        x = [fresh(rows, H) for H in (Hq, Hkv, Hkv)]
        for a, b in zip(hold, x):
            a.copy_(b[:, :, None])
        if captured is not None:
            captured.replay()
        else:
            got = step()
        assert plain.reserve([1] * rows) == 0
        for b in range(rows):
            plain.append(b, x[1][b:b + 1].double().numpy(), x[2][b:b + 1].double().numpy())
        same_meta(cache, plain)
        for b in range(rows):
            check(b, x[0][b:b + 1], got[0][b].transpose(0, 1), got[1][b].transpose(0, 1))
        if i == 4:
            api.cache_free(cache, i32(0, 4))
            for r in (0, 4):
                plain.release(r)
            api.cache_compact(cache)
            plain.compact()
            prompts([7, 0, 0, 0, bs + 1, 0])
            same_pool(cache, plain)
    same_pool(cache, plain)


@pytest.mark.parametrize("graph", [False, True])
def test_serving_steps_of_the_list_form(graph):
    """Page operations that write lengths, append, and the attention's two kernels directly behind them: rows leave, are
    forked and grow in one step after another, with nothing between the launches."""
    g = np.random.default_rng(12)
    rows, cols, Hq, Hkv, D, bs, dtype = 40, 40, 8, 2, 128, 64, BF
    cache = api.make_cache(300, Hkv, D, bs, rows, cols)
    plain = Plain(cache)
    new = [int(n) for n in g.integers(0, 200, rows)]
    api.cache_reserve(cache, i32(*new))
    assert plain.reserve(new) == 0
    k, v = (torch.tensor(g.normal(size=(sum(new), Hkv, D)), dtype=torch.float32).to(dtype) for _ in range(2))
    cu = np.concatenate([[0], np.cumsum(new)])
    api.cache_append(cache, k.to(DEV), v.to(DEV), cu_seqlens=i32(*cu), max_seqlen=max(new))
    for b in range(rows):
        plain.append(b, *(x[cu[b]:cu[b + 1]].double().numpy() for x in (k, v)))
    free, src, dst = i32(3, 20, 39), i32(0, 1, 5), i32(10, 11, 3)
    grow = i32(*[int(n) for n in g.integers(0, 2, rows)])
    q, kn, vn = (torch.tensor(g.normal(size=(rows, H, 1, D)), dtype=torch.float32).to(dtype).to(DEV) for H in (Hq, Hkv, Hkv))
    turn = i32(*[1] * rows)

    def step():
        api.cache_reserve(cache, grow)
        api.cache_free(cache, free)
        api.cache_fork(cache, src, dst)
        a = api.cache_fwd(q, cache)
        api.cache_reserve(cache, turn)
        api.cache_append(cache, kn, vn)
        return a, api.cache_fwd(q, cache)

    assert form_of(lambda: api.cache_fwd(q, cache)) == "cache_attn"
    run = step
    if graph:
        saved = [x.clone() for x in (cache.page_table, cache.seq_lens, cache.refcount)]
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            got = step()
        for a, b in zip((cache.page_table, cache.seq_lens, cache.refcount), saved):
            a.copy_(b)

        def run():
            captured.replay()
            return got
    # the rows that grow here attend values that no append wrote: the same on both sides
    for i in range(12):
        outs = run()
        assert plain.reserve(grow.tolist()) == 0
        for r in free.tolist():
            plain.release(r)
        assert plain.fork(src.tolist(), dst.tolist()) == 0
        before = [x.copy() for x in (plain.lens, plain.table)]
        pool = [x.copy() for x in (plain.k, plain.v, plain.ks, plain.vs)]
        assert plain.reserve(turn.tolist()) == 0
        for b in range(rows):
            plain.append(b, kn[b, :, 0].double().cpu().numpy()[None], vn[b, :, 0].double().cpu().numpy()[None])
        same_meta(cache, plain)
        same_pool(cache, plain)
        after = [plain.lens, plain.table, plain.k, plain.v, plain.ks, plain.vs]
        for (o, lse), state in ((outs[0], before + pool), (outs[1], after)):
            plain.lens, plain.table, plain.k, plain.v, plain.ks, plain.vs = state
            for b in range(0, rows, 1 if i in (0, 11) else 7):
                want = plain.attend(b, q[b].transpose(0, 1).double().cpu().numpy(), 1 / math.sqrt(D))
                check_attend(o[b].transpose(0, 1).double().cpu().numpy(), lse[b].transpose(0, 1).double().cpu().numpy(), *want, dtype, D)
        plain.lens, plain.table, plain.k, plain.v, plain.ks, plain.vs = after
