"""Blocks' attention weight (nsa_cache_weigh) and their eviction
(nsa_cache_evict) on the GPU, against plain forms in 64 bits."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_do_gb300 import api
from test_gpu_cache import Plain, filled

pytestmark = pytest.mark.gpu
DEV = "cuda"
U32 = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(np.array(x), dtype=torch.int32, device=DEV)


def plain_weigh(plain, b, q, lse, weight, decay, scale, window):
    """Row b's weights [Hkv, cols] after its queries q [n, Hq, D], and how far fp32 may be from them: a weight's exponent is
    off by (D + 8) roundings of its score's sum of magnitudes (fp32 queries are held to 2^-22), those of itself, the
    LSE and their factors, and 2^-21 (exponential, scale); the sum by its terms' number of roundings."""
    n, Hq, D = q.shape
    out, tol = weight.astype(np.float64).copy(), np.zeros_like(weight, dtype=np.float64)
    length, bs, Hkv = int(plain.lens[b]), plain.bs, plain.Hkv
    if n == 0:
        return out, tol
    P, nb = length - n, plain.blocks(length)
    for g in range(Hkv):
        K, _ = plain.keys(b, g)
        new, err = np.zeros(nb * bs), np.zeros(nb * bs)
        for h in range(g * Hq // Hkv, (g + 1) * Hq // Hkv):
            for t in range(n):
                pos = P + t
                if lse[t, h] == -np.inf:
                    continue
                j = np.arange(max(0, pos - window + 1) if window else 0, max(pos + 1, 0))
                x = K[j] @ q[t, h] * scale
                p = np.exp(x - lse[t, h])
                d = (D + 8) * U32 * (np.abs(K[j]) @ np.abs(q[t, h])) * scale + 8 * U32 * (np.abs(x) + abs(lse[t, h])) + 2.0 ** -21
                new[j] += p
                err[j] += p * 2 * d
        terms = bs * n * Hq // Hkv
        s, e = new.reshape(nb, bs).sum(1), err.reshape(nb, bs).sum(1) + new.reshape(nb, bs).sum(1) * (terms + 8) * U32
        old = np.where(np.arange(nb) * bs >= P, 0.0, decay * out[g, :nb]) if decay else 0.0
        out[g, :nb] = old + s
        tol[g, :nb] = e + 4 * U32 * np.abs(out[g, :nb])
    return out, tol


def weigh_case(lens, new, Hq, Hkv, D, bs, dtype, ragged=False, window=0, decay=1.0, sinks=False, seed=0, cols=None, layout="dense",
               scale=None, edit=None, ws=False):
    g = np.random.default_rng(seed + 1)
    cache = filled(lens, Hkv, D, bs, seed, cols=cols, layout=layout)
    if edit is not None:
        edit(cache)
    total = sum(new)
    q = torch.tensor(g.normal(size=(total, Hq, D)), dtype=torch.float32).to(dtype)
    weight = torch.tensor(g.random((len(lens), Hkv, cache.page_table.shape[1])), dtype=torch.float32, device=DEV)
    if decay == 0:
        weight.fill_(math.nan)
    before = weight.clone()
    sk = torch.tensor(g.normal(size=Hq), dtype=torch.float32, device=DEV) if sinks else None
    kw = dict(window=window or None, scale=scale)
    if ragged:
        kw.update(cu_seqlens=i32(np.concatenate([[0], np.cumsum(new)])), max_seqlen=max(new))
        x = q.to(DEV)
    else:
        x = q.view(len(lens), new[0], Hq, D).transpose(1, 2).contiguous().to(DEV)
    _, lse = api.cache_fwd(x, cache, sinks=sk, **kw)
    word = torch.full((256,), 255, dtype=torch.uint8, device=DEV) if ws else None
    api.cache_weigh(x, lse, cache, weight, decay=decay, ws=word, **kw)
    if ws:
        assert api.get_error(word) == 0
    flat = lse if ragged else lse.transpose(1, 2).reshape(total, Hq)
    plain, at = Plain(cache), 0
    for b, n in enumerate(new):
        want, tol = plain_weigh(plain, b, q[at:at + n].double().numpy(), flat[at:at + n].double().cpu().numpy(),
                                before[b].double().cpu().numpy(), decay, scale or 1 / math.sqrt(D), window)
        got = weight[b].double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(want))
        off = np.abs(np.where(np.isnan(want), 0, got - want)) - tol
        assert off.max() <= 0, (b, off.max(), np.unravel_index(off.argmax(), off.shape))
        if n and not sinks and not window and np.isfinite(got[:, :plain.blocks(lens[b])]).all() and decay == 0:
            seen = min(n, int(plain.lens[b])) * Hq // Hkv  # every query that attends something gives 1 in all
            assert np.allclose(got[:, :plain.blocks(lens[b])].sum(1), seen, rtol=1e-4)
        at += n


@pytest.mark.parametrize("Hq,Hkv,D,bs", [(4, 1, 128, 64), (16, 1, 128, 64), (6, 2, 64, 32), (2, 1, 32, 16), (5, 5, 64, 16),
                                         (40, 1, 128, 32), (3, 1, 128, 16), (130, 2, 64, 64)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 5])
def test_weigh(Hq, Hkv, D, bs, dtype, T):
    weigh_case([T, bs - 1, bs, bs + 1, 3 * bs + 5, 700], [T] * 6, Hq, Hkv, D, bs, dtype, decay=0.0 if T == 5 else 0.75)


@pytest.mark.parametrize("kw", [dict(window=1), dict(window=37), dict(window=5000), dict(sinks=True), dict(scale=0.3), dict(decay=0.0),
                                dict(ws=True), dict(layout="token"), dict(layout="both"), dict(cols=100)])
@pytest.mark.parametrize("dtype,Hq,Hkv,D,bs,T", [(BF, 8, 2, 128, 64, 1), (BF, 6, 2, 64, 32, 3), (F32, 2, 1, 32, 16, 70), (BF, 24, 2, 128, 32, 20)])
def test_weigh_options(kw, dtype, Hq, Hkv, D, bs, T):
    weigh_case([T + 1, 0 if T == 1 else T, 200, 65 + T, 130, T], [T] * 6, Hq, Hkv, D, bs, dtype, **kw)


@pytest.mark.parametrize("dtype,Hq,Hkv,D,bs", [(BF, 8, 2, 128, 64), (F32, 6, 2, 64, 32), (BF, 4, 4, 32, 16), (BF, 12, 1, 128, 32)])
@pytest.mark.parametrize("kw", [dict(), dict(window=40), dict(decay=0.0)])
def test_weigh_packed_chunks(dtype, Hq, Hkv, D, bs, kw):
    weigh_case([300, 17, 0, 129, 64, 70], [130, 17, 0, 1, 64, 33], Hq, Hkv, D, bs, dtype, ragged=True, **kw)


def test_weigh_long_chunks():
    weigh_case([1200, 700], [600, 333], 8, 2, 128, 64, BF, ragged=True, decay=0.0)
    weigh_case([1200, 700], [600, 333], 4, 2, 64, 16, BF, ragged=True)


def test_weigh_more_queries_than_keys():
    weigh_case([2, 0, 5], [6] * 3, 4, 2, 64, 16, BF)
    weigh_case([2, 0, 5], [6] * 3, 4, 2, 64, 16, F32, decay=0.0)


def test_weigh_long_rows():
    weigh_case([9000, 3, 5000], [1] * 3, 4, 1, 128, 64, BF)


def test_weigh_rows_that_attend_nothing_and_garbage_behind_the_length():
    """An LSE of -infinity gives nothing, whatever the scores are; NaN codes behind a row's end (filled's) count as no keys."""
    cache = filled([40, 40], 1, 64, 16, 3)
    q = torch.randn(2, 4, 1, 64, device=DEV)
    _, lse = api.cache_fwd(q, cache)
    weight = torch.zeros(2, 1, 3, device=DEV)
    lse[0] = -math.inf
    api.cache_weigh(q, lse, cache, weight)
    assert (weight[0] == 0).all() and abs(weight[1].sum().item() - 4) < 1e-4


@pytest.mark.parametrize("dtype,Hq,D,T", [(BF, 4, 128, 1), (F32, 4, 64, 1), (BF, 4, 64, 6), (BF, 12, 32, 9), (F32, 6, 128, 5),
                                          (BF, 8, 128, 40), (BF, 6, 64, 70)])
def test_weigh_padded_queries_attend_nothing_whatever_they_hold(dtype, Hq, D, T):
    """An LSE of -infinity leaves its query out: NaN and infinities in it, and NaN keys that only such queries attend, reach no
    weight."""
    cache = filled([300, 90, 600], 2, D, 64, 3)
    q = torch.randn(3, Hq, T, D, device=DEV).to(dtype)
    _, lse = api.cache_fwd(q, cache)
    pad = torch.zeros(3, T, dtype=torch.bool, device=DEV)
    pad[0, :T // 2] = True
    pad[1] = True
    lse.masked_fill_(pad[:, None], -math.inf)
    zero, bad = q.clone(), q.clone()
    zero.masked_fill_(pad[:, None, :, None], 0.0)
    bad.masked_fill_(pad[:, None, :, None], math.nan)
    bad[1, :, :, 0] = math.inf
    want, got = (torch.zeros(3, 2, cache.page_table.shape[1], device=DEV) for _ in range(2))
    api.cache_weigh(zero, lse, cache, want)
    cache.k.view(torch.uint8)[cache.page_table[1, :1].long(), :, 3] = 0x7f
    api.cache_weigh(bad, lse, cache, got)
    assert (want[1] == 0).all() and torch.isfinite(want).all() and abs(want[2].sum().item() - Hq * T) < 1e-3 * Hq * T
    assert torch.equal(got, want)


@pytest.mark.parametrize("T", [5, 24, 40, 100])
def test_weigh_reads_nothing_behind_the_tokens(T):
    """Queries that are a slice of longer ones: NaN behind the slice reaches no weight."""
    cache = filled([300, 90, 600], 2, 128, 64, 3)
    whole = torch.full((3, 8, 128, 128), math.nan, device=DEV, dtype=BF)
    whole[:, :, :T] = torch.randn(3, 8, T, 128, device=DEV).to(BF)
    q = whole[:, :, :T]
    _, lse = api.cache_fwd(q.contiguous(), cache)
    want, got = (torch.zeros(3, 2, cache.page_table.shape[1], device=DEV) for _ in range(2))
    api.cache_weigh(q.contiguous(), lse, cache, want)
    api.cache_weigh(q, lse, cache, got)
    assert torch.equal(got, want) and abs(want[2].sum().item() - 8 * T) < 8e-3 * T


def test_weigh_bad_pages_and_lengths_are_reported():
    for edit in ("pool", "none", "long", "negative"):
        cache = filled([100, 90], 2, 64, 32, 1)
        q = torch.randn(2, 4, 1, 64, device=DEV).to(BF)
        _, lse = api.cache_fwd(q, cache)
        weight = torch.zeros(2, 2, cache.page_table.shape[1], device=DEV)
        good = weight.clone()
        api.cache_weigh(q, lse, cache, good)
        if edit == "pool":
            cache.page_table[0, 1] = 4096
        elif edit == "none":
            cache.page_table[0, 1] = -7
        else:
            cache.seq_lens[0] = 10 ** 6 if edit == "long" else -5
        word = torch.zeros(256, dtype=torch.uint8, device=DEV)
        api.cache_weigh(q, lse, cache, weight, ws=word)
        assert api.get_error(word) == 3 and api.get_error(word) == 0, edit
        assert torch.equal(weight[1], good[1])
        if edit in ("pool", "none"):
            assert (weight[0, :, 1] == 0).all() and torch.equal(weight[0, :, [0, 2, 3]], good[0, :, [0, 2, 3]])
    # packed offsets that are none: reported, and the row's weights stay
    cache = filled([100, 90], 2, 64, 32, 1)
    q = torch.randn(10, 4, 64, device=DEV).to(BF)
    weight = torch.full((2, 2, cache.page_table.shape[1]), 3.0, device=DEV)
    word = torch.zeros(256, dtype=torch.uint8, device=DEV)
    api.cache_weigh(q, torch.zeros(10, 4, device=DEV), cache, weight, cu_seqlens=i32([0, 20, 10]), max_seqlen=10, ws=word)
    assert api.get_error(word) == 3 and (weight == 3).all()


def test_weigh_accumulates_over_steps_in_a_graph():
    cache = filled([200, 90], 2, 64, 32, 1)
    qs = [torch.randn(2, 4, 1, 64, device=DEV).to(BF) for _ in range(3)]
    q, weight = qs[0].clone(), torch.zeros(2, 2, cache.page_table.shape[1], device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, lse = api.cache_fwd(q, cache)
        api.cache_weigh(q, lse, cache, weight, decay=0.5)
    weight.zero_()
    want = weight.clone()
    for x in qs:
        q.copy_(x)
        graph.replay()
        _, lse = api.cache_fwd(x, cache)
        api.cache_weigh(x, lse, cache, want, decay=0.5)
    torch.cuda.synchronize()
    assert torch.equal(weight, want)


def test_weigh_many_rows_and_mixed_lengths():
    """More list entries than CTAs, rows of every length, none among them."""
    g = np.random.default_rng(3)
    lens = [int(x) for x in g.integers(0, 400, 90)]
    weigh_case(lens, [1] * 90, 4, 2, 64, 16, BF)
    new = [int(min(n, x)) for n, x in zip(lens, g.integers(0, 60, 90))]
    weigh_case(lens, new, 8, 2, 64, 32, BF, ragged=True, decay=0.5)


@pytest.mark.parametrize("Hq,Hkv,D,bs", [(8, 2, 128, 64), (3, 1, 64, 16), (24, 2, 128, 32), (128, 1, 64, 64), (7, 7, 128, 16), (66, 2, 64, 64)])
@pytest.mark.parametrize("kw", [dict(ragged=True), dict(ragged=True, window=70), dict(ragged=True, window=1, decay=0.25), dict(sinks=True)])
def test_weigh_on_the_tensor_cores(Hq, Hkv, D, bs, kw):
    ragged = kw.get("ragged")
    lens, new = ([400, 260, 0, 129, 130, 70], [200, 3, 0, 129, 1, 65]) if ragged else ([330, 129, 400], [129] * 3)
    weigh_case(lens, new, Hq, Hkv, D, bs, BF, **kw)


def test_weigh_forms_are_the_ones_meant():
    def name(T, dtype, D, Hq=8):
        cache = filled([300, 300], 2, D, 64, 1)
        q, weight = torch.zeros(2, Hq, T, D, dtype=dtype, device=DEV), torch.zeros(2, 2, 5, device=DEV)
        api.trace_enable(8)
        api.trace_reset()
        api.cache_weigh(q, torch.zeros(2, Hq, T, device=DEV), cache, weight)
        got = [n for n, _ in api.trace_records()]
        api.trace_enable(0)
        return got

    assert name(1, BF, 128) == name(16, BF, 64) == name(100, F32, 128) == name(100, BF, 32) == ["cache_weigh"]
    assert name(17, BF, 128) == name(100, BF, 64) == ["cache_weigh_tc"] and name(100, BF, 64, 258) == ["cache_weigh"]


def test_weigh_strided_queries_on_the_tensor_cores():
    cache = filled([300, 200], 2, 64, 32, 1)
    x = torch.randn(2, 90, 10, 64, device=DEV).to(BF)
    q = x[:, :, 1:9].transpose(1, 2)
    _, lse = api.cache_fwd(q, cache)
    a, b = (torch.zeros(2, 2, cache.page_table.shape[1], device=DEV) for _ in range(2))
    api.cache_weigh(q, lse, cache, a)
    api.cache_weigh(q.contiguous(), lse, cache, b)
    assert torch.equal(a, b)
    assert torch.allclose(a.sum(2), torch.full((2, 2), 90.0 * 4, device=DEV), rtol=1e-4)


def test_weigh_nan_outside_what_is_attended():
    """Queries of other sequences and of none (NaN), and NaN codes behind the rows' ends, reach no weight; a NaN key that
    is attended reaches its block alone."""
    cache = filled([300, 200], 2, 128, 64, 1)
    q = torch.randn(200, 8, 128, device=DEV).to(BF)
    q[:10] = math.nan
    q[110:120] = math.nan
    q[190:] = math.nan
    cu = i32([10, 110, 190])
    q2 = q.clone()
    q2[110:120] = 1.0
    _, lse = api.cache_fwd(q2, cache, cu_seqlens=cu, max_seqlen=100)
    weight = torch.zeros(2, 2, cache.page_table.shape[1], device=DEV)
    api.cache_weigh(q2, lse, cache, weight, cu_seqlens=cu, max_seqlen=100)
    assert torch.isfinite(weight).all()
    page = int(cache.page_table[0, 1])
    cache.k.view(torch.uint8)[page, 0, 7, 3] = 0x7f
    other = torch.zeros_like(weight)
    api.cache_weigh(q2, lse, cache, other, cu_seqlens=cu, max_seqlen=100)
    assert torch.isnan(other[0, 0, 1])
    other[0, 0, 1] = weight[0, 0, 1]
    assert torch.equal(other, weight)


def test_weigh_waits_that_give_up():
    """The bounded waits of the tensor-core form: reported, NaN in the weights, and the next call is whole again."""
    cache = filled([300, 200], 2, 128, 64, 1)
    q = torch.randn(2, 8, 100, 128, device=DEV).to(BF)
    _, lse = api.cache_fwd(q, cache)
    good, weight = (torch.zeros(2, 2, cache.page_table.shape[1], device=DEV) for _ in range(2))
    api.cache_weigh(q, lse, cache, good)
    word = torch.zeros(256, dtype=torch.uint8, device=DEV)
    api.debug_stall(1, 20000)
    try:
        api.cache_weigh(q, lse, cache, weight, ws=word)
        assert api.get_error(word) == 4
        assert torch.isnan(weight[0, :, :5]).all() and torch.isnan(weight[1, :, :4]).all()
    finally:
        api.debug_stall(0, 0)
    weight.zero_()
    api.cache_weigh(q, lse, cache, weight, ws=word)
    assert api.get_error(word) == 0 and torch.equal(weight, good)


@pytest.mark.parametrize("dtype,D,T", [(BF, 128, 1), (BF, 64, 12), (F32, 64, 30), (BF, 32, 40), (BF, 128, 40), (BF, 64, 100)])
def test_weigh_a_scale_that_is_nan_is_a_key_that_is(dtype, D, T):
    """NaN in the weights of the page's head, in each form, and in no other."""
    cache = filled([300, 200], 2, D, 32, 1)
    q = torch.randn(2, 8, T, D, device=DEV).to(dtype)
    _, lse = api.cache_fwd(q, cache)
    want, got = (torch.zeros(2, 2, cache.page_table.shape[1], device=DEV) for _ in range(2))
    api.cache_weigh(q, lse, cache, want)
    cache.k_scale[int(cache.page_table[0, 2]), 1] = math.nan
    api.cache_weigh(q, lse, cache, got)
    assert torch.isnan(got[0, 1, 2]) and torch.isfinite(want).all()
    got[0, 1, 2] = want[0, 1, 2]
    assert torch.equal(got, want)


@pytest.mark.parametrize("T", [1, 100])
def test_weigh_reports_without_a_word_of_the_callers(T):
    """Pages that are none, and bounded waits that gave up, through the handle's word; each call has its own."""
    cache = filled([300, 200], 2, 128, 64, 1)
    q = torch.randn(2, 8, T, 128, device=DEV).to(BF)
    _, lse = api.cache_fwd(q, cache)
    weight = torch.zeros(2, 2, cache.page_table.shape[1], device=DEV)
    api.cache_weigh(q, lse, cache, weight)
    first = cache.weigh_ws
    assert api.get_error(first) == 0
    page = int(cache.page_table[1, 0])
    cache.page_table[1, 0] = 4096
    api.cache_weigh(q, lse, cache, weight)
    second = cache.weigh_ws
    cache.page_table[1, 0] = page
    api.cache_weigh(q, lse, cache, weight)
    assert api.get_error(cache.weigh_ws) == 0 and api.get_error(second) == 3 and api.get_error(first) == 0
    word = torch.full((256,), 255, dtype=torch.uint8, device=DEV)
    api.cache_weigh(q, lse, cache, weight, ws=word)
    assert cache.weigh_ws is word and api.get_error(word) == 0
    api.cache_weigh(q[:, :, :0], lse[:, :, :0], cache, weight)
    assert cache.weigh_ws is not word and api.get_error(cache.weigh_ws) == 0
    if T > 16:
        api.debug_stall(1, 20000)
        try:
            api.cache_weigh(q, lse, cache, weight)
            assert api.get_error(cache.weigh_ws) == 4
        finally:
            api.debug_stall(0, 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.cache_weigh(q, lse, cache, weight)
    held = cache.weigh_ws
    for bad in (True, False, True):
        cache.page_table[1, 0] = 4096 if bad else page
        graph.replay()
        torch.cuda.synchronize()
        assert api.get_error(held) == (3 if bad else 0)


# ------------------------------------------------------------------- evict

def plain_evict(cache, weight, keep, first, recent):
    """(table, lens, ref, weight, kept) by the definition, a row at a time."""
    table, lens, ref = (x.cpu().numpy().copy() for x in (cache.page_table, cache.seq_lens, cache.refcount))
    w, bs, cols = weight.cpu().numpy().copy(), cache.k.shape[2], table.shape[1]
    kept = np.tile(np.arange(cols), (len(lens), 1))
    for b in range(len(lens)):
        n = -(-int(lens[b]) // bs)
        if n <= keep:
            continue
        score = w[b, 0].copy()
        for h in range(1, w.shape[1]):
            score = score + w[b, h]  # in 32 bits, head by head
        rank = sorted(range(first, n - recent), key=lambda j: (np.isnan(score[j]), -score[j] if not np.isnan(score[j]) else 0, j))
        out = set(rank[keep - first - recent:])
        stay = [j for j in range(cols) if j not in out]
        for j in out:
            ref[table[b, j]] -= 1
        pad = cols - len(stay)
        table[b] = np.concatenate([table[b][stay], [-1] * pad])
        kept[b] = np.concatenate([stay, [-1] * pad])
        w[b] = np.concatenate([w[b][:, stay], np.zeros((w.shape[1], pad))], 1)
        lens[b] -= len(out) * bs
    return table, lens, ref, w, kept


def evict_case(lens, Hkv, bs, keep, first, recent, seed=0, cols=None, make=None, with_kept=True, edit=None):
    g = np.random.default_rng(seed)
    cache = filled(lens, Hkv, 32, bs, seed, cols=cols)
    if edit is not None:
        edit(cache)
    w = g.random((len(lens), Hkv, cache.page_table.shape[1])) if make is None else make(g, (len(lens), Hkv, cache.page_table.shape[1]))
    weight = torch.tensor(w, dtype=torch.float32, device=DEV)
    want = plain_evict(cache, weight, keep, first, recent)
    kept = torch.full(tuple(cache.page_table.shape), -9, dtype=torch.int32, device=DEV) if with_kept else None
    codes = cache.k.view(torch.uint8).clone()
    api.cache_evict(cache, weight, keep, first=first, recent=recent, kept=kept)
    assert api.get_error(cache.ws) == 0
    assert np.array_equal(cache.page_table.cpu().numpy(), want[0]) and np.array_equal(cache.seq_lens.cpu().numpy(), want[1])
    assert np.array_equal(cache.refcount.cpu().numpy(), want[2])
    assert np.array_equal(weight.cpu().numpy(), want[3], equal_nan=True)
    if with_kept:
        assert np.array_equal(kept.cpu().numpy(), want[4])
    assert torch.equal(codes, cache.k.view(torch.uint8))
    return cache


@pytest.mark.parametrize("keep,first,recent", [(1, 0, 1), (2, 0, 1), (4, 2, 2), (5, 1, 1), (7, 0, 7), (8, 4, 1), (20, 1, 4), (300, 3, 9)])
@pytest.mark.parametrize("Hkv,bs", [(1, 64), (2, 32), (9, 16), (17, 16)])
def test_evict(keep, first, recent, Hkv, bs):
    lens = [0, 1, bs, keep * bs, keep * bs + 1, (keep + 1) * bs, (keep + 3) * bs - 5, 20 * bs, 21 * bs + 3]
    evict_case(lens, Hkv, bs, keep, first, recent, seed=keep)


def test_evict_wide_rows_and_a_table_wider_than_the_rows():
    evict_case([16 * 5000 - 3, 16 * 700, 16 * 513], 2, 16, 512, 4, 8, cols=5003)
    evict_case([16 * 1000] * 3, 1, 16, 999, 0, 1)
    evict_case([16 * 1000] * 3, 1, 16, 1, 0, 1, with_kept=False)


def test_evict_a_table_beyond_shared_memory():
    evict_case([16 * 50000 - 3, 16 * 300], 1, 16, 256, 4, 8, cols=50000)


@pytest.mark.parametrize("make", [lambda g, s: np.zeros(s), lambda g, s: np.floor(g.random(s) * 3), lambda g, s: -g.random(s),
                                  lambda g, s: np.where(g.random(s) < 0.3, np.nan, g.random(s)),
                                  lambda g, s: np.where(g.random(s) < 0.3, np.inf, g.random(s)),
                                  lambda g, s: np.exp2(g.integers(-149, 127, s).astype(float)) * g.choice([-1, 1], s),
                                  lambda g, s: np.full(s, np.nan), lambda g, s: np.where(g.random(s) < 0.5, 0.0, -0.0)])
def test_evict_ties_and_odd_weights(make):
    for Hkv in (1, 3):
        evict_case([16 * 600 - 3, 16 * 40, 16 * 77 + 1], Hkv, 16, 33, 2, 3, make=make)


def test_evict_shared_pages_and_pages_behind_the_length():
    """Forked rows share pages: each gives up its own reference; a row whose length was lowered keeps the pages behind,
    in the columns behind its new length, and grows into them again."""
    cache = api.make_cache(64, 1, 32, 16, 4, 12)
    api.cache_reserve(cache, i32([16 * 9, 0, 0, 16 * 5]))
    api.cache_fork(cache, i32([0, 0]), i32([1, 2]))
    cache.seq_lens[3] -= 40  # 5 blocks held, 40 tokens: 3 used
    weight = torch.rand(4, 1, 12, device=DEV)
    want = plain_evict(cache, weight, 2, 1, 1)
    api.cache_evict(cache, weight, 2, first=1, recent=1)
    assert api.get_error(cache.ws) == 0
    for got, ref in zip((cache.page_table, cache.seq_lens, cache.refcount), want):
        assert np.array_equal(got.cpu().numpy(), ref)
    assert int((cache.page_table[3] >= 0).sum()) == 4
    held = cache.page_table[3, :4].clone()
    free = int((cache.refcount == 0).sum())
    api.cache_reserve(cache, i32([0, 0, 0, 32]))
    assert api.get_error(cache.ws) == 0
    assert torch.equal(cache.page_table[3, :4], held) and int((cache.refcount == 0).sum()) == free
    for r in range(4):
        api.cache_free(cache, i32([r]))
    assert (cache.refcount == 0).all()


def test_evict_bad_rows_are_left_and_reported():
    for edit in ("pool", "none", "unused", "long", "negative"):
        cache = filled([16 * 9, 16 * 9], 2, 32, 16, 1)
        if edit == "pool":
            cache.page_table[0, 3] = 999
        elif edit == "none":
            cache.page_table[0, 3] = -1
        elif edit == "unused":
            cache.refcount[cache.page_table[0, 3].long()] = 0
        else:
            cache.seq_lens[0] = 10 ** 6 if edit == "long" else -3
        before, lens = cache.page_table.clone(), cache.seq_lens.clone()
        weight, kept = torch.rand(2, 2, 9, device=DEV), torch.zeros(2, 9, dtype=torch.int32, device=DEV)
        old = weight.clone()
        api.cache_evict(cache, weight, 4, kept=kept)
        assert api.get_error(cache.ws) == 3, edit
        assert torch.equal(cache.page_table[0], before[0]) and cache.seq_lens[0] == lens[0] and torch.equal(weight[0], old[0])
        assert kept[0].tolist() == list(range(9)) and cache.seq_lens[1] == 64


def test_evict_counts_too_low_are_reported():
    """A page that two rows name and whose count is 1: both rows close up, the count ends at 0, not below, and that is
    reported; counts that are right are not."""
    for count in (1, 2):
        cache = filled([16 * 9, 16 * 9], 2, 32, 16, 1)
        page = int(cache.page_table[0, 3])
        spare = int(cache.page_table[1, 3])
        cache.page_table[1, 3] = page
        cache.refcount[spare] = 0
        cache.refcount[page] = count
        weight = torch.rand(2, 2, 9, device=DEV)
        weight[:, :, 3] = 0.0
        api.cache_evict(cache, weight, 8)
        # (one row may meet the count that the other has taken: it is then left, and the page is its own again in no table)
        left = [b for b in range(2) if int(cache.seq_lens[b]) == 16 * 9]
        assert api.get_error(cache.ws) == (3 if count == 1 else 0)
        assert len(left) == 0 if count == 2 else len(left) <= 1
        assert int(cache.refcount[page]) == 0 and int(cache.refcount.min()) == 0
        for b in range(2):
            assert (page in cache.page_table[b].tolist()) == (b in left)


def test_evict_in_a_graph_and_repeats():
    cache = filled([16 * 40, 16 * 30], 2, 32, 16, 1)
    table, lens, ref = cache.page_table.clone(), cache.seq_lens.clone(), cache.refcount.clone()
    weight = torch.rand(2, 2, 40, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.cache_evict(cache, weight, 12, first=1, recent=2)
    for _ in range(3):
        for x, y in ((cache.page_table, table), (cache.seq_lens, lens), (cache.refcount, ref)):
            x.copy_(y)
        weight.copy_(torch.rand(2, 2, 40, device=DEV))
        want = plain_evict(cache, weight, 12, 1, 2)
        graph.replay()
        torch.cuda.synchronize()
        for got, x in zip((cache.page_table, cache.seq_lens, cache.refcount, weight), want):
            assert np.array_equal(got.cpu().numpy(), x)
        graph.replay()  # nothing is left to do
        torch.cuda.synchronize()
        assert np.array_equal(cache.page_table.cpu().numpy(), want[0])


def test_a_bounded_row_as_a_server_keeps_it():
    """Prompt, then token after token: rotate at the true position, append, attend, weigh, evict; the pages in use stay
    bounded, and each step's attention is that of what the row still holds."""
    Hq, Hkv, D, bs, B, keep = 4, 2, 64, 16, 2, 5
    cache = api.make_cache(40, Hkv, D, bs, B, 12)
    f, w = (torch.tensor(10000.0 ** (-np.arange(0, D, 2) / D), dtype=torch.float32, device=DEV), torch.ones(D, device=DEV))
    weight = torch.zeros(B, Hkv, 12, device=DEV)
    held = [[], []]  # token numbers that each row should hold
    done = 0
    for step in range(60):
        n = 70 if step == 0 else 1
        api.cache_reserve(cache, i32([n] * B))
        assert api.get_error(cache.ws) == 0
        q, k, v = (torch.randn(B, H, n, D, device=DEV).to(BF) for H in (Hq, Hkv, Hkv))
        pos = i32([list(range(done, done + n))] * B)
        zq, zk = api.norm_rope_fwd(q, k, w, w, f, pos=pos)
        api.cache_append(cache, zk, v)
        o, lse = api.cache_fwd(zq, cache)
        before = weight.double().cpu().numpy()
        api.cache_weigh(zq, lse, cache, weight)
        plain = Plain(cache)
        for b in range(B):
            held[b] += list(range(done, done + n))
            assert len(held[b]) == plain.lens[b]
            want, tol = plain_weigh(plain, b, zq[b].transpose(0, 1).double().cpu().numpy(), lse[b].T.double().cpu().numpy(), before[b], 1.0,
                                    1 / math.sqrt(D), 0)
            assert (np.abs(weight[b].double().cpu().numpy() - want) <= tol).all()
        kept = torch.empty(B, 12, dtype=torch.int32, device=DEV)
        api.cache_evict(cache, weight, keep, first=1, recent=2, kept=kept)
        assert api.get_error(cache.ws) == 0
        for b in range(B):
            n_now = -(-int(cache.seq_lens[b]) // bs)
            assert n_now <= keep
            held[b] = [t for c in kept[b, :n_now].tolist() for t in held[b][c * bs:(c + 1) * bs]]
            assert len(held[b]) == int(cache.seq_lens[b]) and held[b][:bs] == list(range(bs)) and held[b][-1] == done + n - 1
        assert int((cache.refcount > 0).sum()) == sum(-(-int(x) // bs) for x in cache.seq_lens)
        done += n


def at_once(*calls, times=3000):
    """Each call of the C entries over and over in threads and streams of its own; the states that were not 0."""
    import threading
    got = set()
    start = threading.Barrier(2 * len(calls))
    streams = [torch.cuda.Stream() for _ in range(2 * len(calls))]
    torch.cuda.synchronize()

    def run(make, stream):
        call, args = make(stream)
        torch.cuda.synchronize()
        start.wait()
        for _ in range(times):
            s = call(*args)
            if s:
                got.add(s)

    threads = [threading.Thread(target=run, args=(calls[i // 2], stream)) for i, stream in enumerate(streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return got


def test_calls_of_several_threads_with_other_amounts_of_shared_memory():
    """What a kernel is allowed is the process's: a call that needs little takes nothing from one that needs much."""
    held = []

    def weigher(rows):
        def make(stream):
            cache = filled([20] * rows, 1, 128, 64, 1)
            q = torch.zeros(rows, 1, 1, 128, device=DEV)
            lse, weight = torch.zeros(rows, 1, 1, device=DEV), torch.zeros(rows, 1, cache.page_table.shape[1], device=DEV)
            held.append((cache, q, lse, weight))
            p = cache.problem(q, 1, None, None, None, False, True)[1]
            return api.lib().nsa_cache_weigh, (p, cache.ref, 0, None, q.data_ptr(), lse.data_ptr(), 1.0, weight.data_ptr(), None, 0, stream.cuda_stream)
        return make

    def evicter(cols):
        def make(stream):
            cache = filled([20], 1, 32, 16, 1, cols=cols)
            weight = torch.zeros(1, 1, cols, device=DEV)
            held.append((cache, weight))
            return api.lib().nsa_cache_evict, (cache.ref, weight.data_ptr(), 8, 0, 1, None, cache.ws.data_ptr(), cache.ws.numel(), stream.cuda_stream)
        return make

    assert at_once(weigher(1), weigher(2048)) == set()
    assert at_once(evicter(11000), evicter(48000)) == set()


@pytest.mark.parametrize("D,bs,dtype,Hq", [(64, 16, F32, 2), (64, 16, BF, 2), (128, 64, BF, 8)])
def test_training_calls_of_several_threads_with_other_amounts_of_shared_memory(D, bs, dtype, Hq):
    """The same of the kernels whose shared memory goes by the longest sequence's blocks: forward and backward."""
    held = []

    def step(T, backward):
        def make(stream):
            q, o, dq = (torch.zeros(1, Hq, T, D, dtype=dtype, device=DEV) for _ in range(3))
            k, dk, dv = (torch.zeros(1, 1, T, D, dtype=dtype, device=DEV) for _ in range(3))
            idx = torch.zeros(1, 1, T, 1, dtype=torch.int32, device=DEV)
            lse = torch.zeros(1, Hq, T, device=DEV)
            p = api.problem_from(q, k, bs, 1)
            n = api.bwd_workspace_size(p) if backward else api.fwd_workspace_size(p)
            ws = torch.empty(n, dtype=torch.uint8, device=DEV)
            held.append((q, o, dq, k, dk, dv, idx, lse, p, ws))
            at = [x.data_ptr() for x in (q, k, k, o, o, lse, idx, dq, dk, dv)]
            if backward:
                return api.lib().nsa_sel_bwd, (p, *at, ws.data_ptr(), n, stream.cuda_stream)
            return api.lib().nsa_sel_fwd, (p, at[0], at[1], at[2], at[6], at[3], at[5], ws.data_ptr(), n, stream.cuda_stream)
        return make

    for backward in (False, True):
        assert at_once(step(64, backward), step(8192, backward), times=400) == set(), backward
