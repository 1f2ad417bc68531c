"""Trees of drafted tokens over the paged 8-bit cache (nsa_cache_tree_fwd) and
the drafts that are accepted (nsa_cache_accept), against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_do_gb300 import api
from test_gpu_cache import Plain, check_attend, filled, index_rows

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(np.array(x), dtype=torch.int32, device=DEV)


def random_parents(n, wide, g):
    return [int(g.integers(max(-1, t - wide), t)) for t in range(n)]


def line_of(parents, t):
    """The draft, its parent, and so on."""
    out = []
    while t >= 0:
        out.append(t)
        t = parents[t]
    return out


def tree_attend(plain, b, q, parents, scale, idx=None, window=0, sinks=None):
    """As Plain.attend, for the tree's mask."""
    n, Hq, D = q.shape
    o, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    vmax, serr, nkeys = np.zeros((n, Hq)), np.zeros((n, Hq)), np.zeros((n, Hq))
    P = int(plain.lens[b]) - n
    for h in range(Hq):
        g = h // (Hq // plain.Hkv)
        K, V = plain.keys(b, g)
        for t in range(n):
            line = line_of(parents, t)
            depth = len(line) - 1
            lo = max(0, P + depth - window + 1) if window else 0
            j = list(range(min(lo, P), P)) + sorted(P + a for i, a in enumerate(line) if not window or i < window)
            j = np.array([x for x in j if x >= 0], dtype=int)
            if idx is not None:
                j = j[np.isin(j // plain.bs, idx[t, g][idx[t, g] >= 0])]
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


def tree_case(lens, new, Hq, Hkv, D, bs, dtype, ragged=False, S=0, window=0, sinks=False, seed=0, wide=3, layout="dense",
              cols=None, edit=None, parents=None, tmax=None):
    g = np.random.default_rng(seed + 1)
    cache = filled(lens, Hkv, D, bs, seed, layout=layout, cols=cols)
    parents = parents or [random_parents(n, wide, g) for n in new]
    if edit is not None:
        edit(cache)
    total = sum(new)
    q = torch.tensor(g.normal(size=(total, Hq, D)), dtype=torch.float32).to(dtype)
    idx = index_rows(lens, new, Hkv, S, bs, g) if S else None
    sk = torch.tensor(g.normal(size=Hq) * 2, dtype=torch.float32) if sinks else None
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
    kw = dict(window=window or None, sinks=sk.to(DEV) if sinks else None, ws=ws)
    if ragged:
        o, lse = api.cache_tree_fwd(q.to(DEV), cache, i32(sum(parents, [])), cu_seqlens=i32(np.concatenate([[0], np.cumsum(new)])),
                                    max_seqlen=tmax or max(new), block_idx=torch.tensor(idx, device=DEV) if S else None, **kw)
    else:
        B, T = len(lens), new[0]
        qb = q.view(B, T, Hq, D).transpose(1, 2).contiguous().to(DEV)
        ib = torch.tensor(idx, device=DEV).view(B, T, Hkv, S).transpose(1, 2).contiguous() if S else None
        o, lse = api.cache_tree_fwd(qb, cache, i32(parents), block_idx=ib, **kw)
        o, lse = o.transpose(1, 2).reshape(total, Hq, D), lse.transpose(1, 2).reshape(total, Hq)
    assert api.get_error(ws) == 0
    plain, at = Plain(cache), 0
    for b, n in enumerate(new):
        sl = slice(at, at + n)
        want = tree_attend(plain, b, q[sl].double().numpy(), parents[b], 1 / math.sqrt(D), idx[sl] if S else None, window,
                           sk.double().numpy() if sinks else None)
        check_attend(o[sl].double().cpu().numpy(), lse[sl].double().cpu().numpy(), *want, dtype, D)
        at += n


# ------------------------------------------------------------------- trees

@pytest.mark.parametrize("Hq,Hkv,D,bs", [(4, 1, 128, 64), (16, 1, 128, 64), (6, 2, 64, 32), (2, 1, 32, 16), (5, 5, 64, 16), (40, 1, 128, 32)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 7])
def test_small_trees(Hq, Hkv, D, bs, dtype, T):
    tree_case([T, T + 1, bs, bs + T, 3 * bs + 5, 300], [T] * 6, Hq, Hkv, D, bs, dtype)


@pytest.mark.parametrize("kw", [dict(window=1), dict(window=5), dict(window=37), dict(window=5000), dict(sinks=True),
                                dict(window=3, sinks=True), dict(S=1), dict(S=5), dict(S=16)])
@pytest.mark.parametrize("dtype,Hq,Hkv,D,bs,T", [(BF, 8, 2, 128, 64, 21), (BF, 6, 2, 64, 32, 13), (F32, 2, 1, 32, 16, 40),
                                                 (BF, 24, 2, 128, 32, 9), (F32, 16, 1, 128, 64, 5)])
def test_tree_masks(kw, dtype, Hq, Hkv, D, bs, T):
    tree_case([T, 200, 65 + T, 130], [T] * 4, Hq, Hkv, D, bs, dtype, wide=4, **kw)


@pytest.mark.parametrize("wide", [1, 2, 30])
@pytest.mark.parametrize("kw", [dict(), dict(window=9), dict(sinks=True)])
def test_the_chunk_form(wide, kw):
    """Enough rows for the tensor-core kernel, drafts over two tiles of keys."""
    new = [90, 1, 0, 64, 128, 33] * 4
    lens = [90, 300, 5, 64 + 100, 128 + 250, 33 + 95] * 4
    for D, bs in ((128, 64), (64, 16), (128, 32)):
        tree_case(lens, new, 16, 2, D, bs, BF, ragged=True, wide=wide, **kw)


@pytest.mark.parametrize("D,bs,Hq,Hkv,lens,new", [
    (128, 64, 8, 1, [5000], [12]), (128, 64, 8, 2, [3000, 40, 1500], [12, 9, 30]), (64, 16, 4, 1, [2000, 9, 700], [20, 9, 32]),
    (128, 32, 16, 2, [2500, 2500], [15, 17]), (64, 64, 6, 2, [1, 900, 130, 129, 128, 4000], [1, 100, 130, 129, 30, 43]),
    (128, 16, 12, 1, [300] * 9, [64] * 9)])
@pytest.mark.parametrize("kw", [dict(), dict(window=300), dict(sinks=True)])
def test_units_cut_over_many_ctas(D, bs, Hq, Hkv, lens, new, kw):
    """Few sequences, so that their key tiles are spread over the GPU and joined: at most 128 query rows (both pipelines
    take the same rows' tiles in turn), 129 to 256, and more.  (A wide table brings small calls to the tensor cores.)"""
    tree_case(lens, new, Hq, Hkv, D, bs, BF, ragged=True, cols=200000 // bs, **kw)


def test_more_drafts_than_cached_tokens_in_the_chunk_form():
    tree_case([40, 0, 70, 33], [60, 50, 70, 64], 8, 2, 64, 16, BF, ragged=True, wide=2, cols=3000)
    tree_case([40, 0, 70, 33], [60, 50, 70, 64], 8, 2, 128, 64, BF, ragged=True, sinks=True, window=20, cols=1000)


def test_scales_far_apart_in_the_chunk_form():
    """Pages whose value scales lie 2^-100 .. 2^27 apart (zeros beside large values): the sum from the scores alone, in
    units, parts and pipelines that are joined."""
    def edit(cache):
        n = cache.v_scale.shape[0]
        cache.v_scale[:] = torch.exp2(torch.tensor([[-100.0, 27.0, 0.0, -60.0][i % 4] for i in range(n)], device=DEV))[:, None]
        zero = [i for i in range(n) if i % 4 == 0]
        cache.v.view(torch.uint8)[zero] = 0

    for lens, new, Hq in (([2000, 1500], [9, 11], 8), ([900], [70], 8), ([128 * 7], [40], 4)):
        tree_case(lens, new, Hq, 1, 128, 64, BF, ragged=True, edit=edit, cols=3000)
        tree_case(lens, new, Hq, 1, 64, 16, BF, ragged=True, edit=edit, sinks=True, cols=12000)


def test_bad_pages_in_the_chunk_form_are_left_out():
    cache = filled([900, 700], 2, 128, 64, 5, cols=1000)
    q = torch.randn(2, 16, 20, 128, device=DEV).to(BF)
    par = i32([[-1] + list(range(19))] * 2)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
    good = api.cache_tree_fwd(q, cache, par, ws=ws)
    assert api.get_error(ws) == 0
    for entry in (9999, -1, -7):
        old = int(cache.page_table[0, 3])
        cache.page_table[0, 3] = entry
        o, lse = api.cache_tree_fwd(q, cache, par, ws=ws)
        assert api.get_error(ws) == 3
        assert torch.equal(o[1], good[0][1]) and torch.isfinite(o).all() and not torch.equal(o[0], good[0][0])
        cache.page_table[0, 3] = old
    cache.seq_lens[0] = 10 ** 6
    api.cache_tree_fwd(q, cache, par, ws=ws)
    assert api.get_error(ws) == 3


def test_waits_that_give_up():
    """The bounded waits of the tensor-core form: reported, NaN in the rows, and the next call is whole again."""
    for lens, T in (([900, 700], 20), ([300] * 24, 90)):
        cache = filled(lens, 2, 128, 64, 5, cols=1000)
        q = torch.randn(len(lens), 16, T, 128, device=DEV).to(BF)
        par = i32([[-1] + list(range(T - 1))] * len(lens))
        ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
        good = api.cache_tree_fwd(q, cache, par, ws=ws)
        api.debug_stall(1, 20000)
        try:
            o, lse = api.cache_tree_fwd(q, cache, par, ws=ws)
            assert api.get_error(ws) == 4
            assert torch.isnan(o).all() and torch.isnan(lse).all()
        finally:
            api.debug_stall(0, 0)
        o, lse = api.cache_tree_fwd(q, cache, par, ws=ws)
        assert api.get_error(ws) == 0 and torch.equal(o, good[0]) and torch.equal(lse, good[1])


def test_the_most_drafts():
    for dtype, D, n in ((BF, 128, 1), (F32, 32, 1), (BF, 64, 6)):
        tree_case([256 + 77] * n, [256] * n, 8, 2, D, 16, dtype, wide=256)
        tree_case([256] * n, [256] * n, 8, 2, D, 32, dtype, wide=1, window=20)  # a chain


def test_forms_are_the_ones_meant():
    """Each form runs (by the launches' names) on the sizes that the tests above give it."""
    def name(lens, new, Hq, Hkv, D, bs, dtype, cols=None):
        cache = filled(lens, Hkv, D, bs, 1, cols=cols)
        q = torch.zeros(len(lens), Hq, new, D, dtype=dtype, device=DEV)
        api.trace_enable(8)
        api.trace_reset()
        api.cache_tree_fwd(q, cache, i32([[-1] * new] * len(lens)))
        got = [n for n, _ in api.trace_records()]
        api.trace_enable(0)
        return got

    assert name([70, 300], 7, 4, 1, 128, 64, BF) == ["cache_tree_cluster"]
    assert name([70, 300], 7, 4, 1, 128, 64, BF, cols=2000) == ["cache_tree"]
    assert name([300] * 24, 90, 16, 2, 128, 64, BF) == ["cache_tree_chunk"]
    assert name([300], 12, 8, 1, 128, 64, BF) == ["cache_tree_cluster"] and name([300], 12, 8, 1, 128, 64, BF, cols=3125) == ["cache_tree_chunk"]
    assert name([300] * 4, 50, 8, 2, 64, 16, BF, cols=3000) == name([300] * 2, 20, 16, 2, 128, 64, BF, cols=1000) == ["cache_tree_chunk"]


@pytest.mark.parametrize("kw", [dict(), dict(window=30), dict(S=4)])
def test_the_list_form(kw):
    """A wide table: the list's form; long and short rows together."""
    tree_case([300, 3, 70, 1200], [3] * 4, 6, 2, 64, 32, BF, cols=3000, **kw)
    tree_case([300, 13, 70, 500], [13, 13, 1, 40], 4, 1, 128, 64, F32, cols=2000, ragged=True, **kw)


def test_a_chain_is_the_plain_call():
    """Bit by bit, where both run in the same form."""
    for lens, T, Hq, Hkv, D, bs, dtype, cols in (([300, 20], 8, 8, 2, 128, 64, BF, None), ([300, 20], 8, 8, 2, 128, 64, BF, 2000),
                                                 ([200, 40], 30, 4, 2, 32, 16, F32, None), ([200, 40], 30, 4, 2, 32, 16, BF, 2000)):
        cache = filled(lens, Hkv, D, bs, 3, cols=cols)
        q = torch.randn(len(lens), Hq, T, D, device=DEV).to(dtype)
        for window in (None, 11):
            a = api.cache_fwd(q, cache, window=window)
            b = api.cache_tree_fwd(q, cache, i32([list(range(-1, T - 1))] * len(lens)), window=window)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), (T, window)


def test_strided_pools_and_queries():
    for layout in ("token", "both"):
        tree_case([200, 70, 333], [11] * 3, 8, 2, 128, 64, BF, layout=layout)
    cache = filled([90, 300], 2, 64, 32, 1)
    x = torch.randn(2, 9, 10, 64, device=DEV).to(BF)
    par = i32([random_parents(9, 3, np.random.default_rng(i)) for i in range(2)])
    got = api.cache_tree_fwd(x[:, :, 1:9].transpose(1, 2), cache, par)
    want = api.cache_tree_fwd(x[:, :, 1:9].transpose(1, 2).contiguous(), cache, par)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T,n,cols", [(6, 3, None), (6, 3, 2000), (60, 24, None)])
def test_nan_in_other_branches_stays_there(T, n, cols):
    """A draft whose value and key are NaN reaches its descendants and itself, and nobody else."""
    lens = [100 + 3 * i for i in range(n)]

    def edit(cache):
        for b in range(n):
            at = lens[b] - T + 2  # draft 2
            page = int(cache.page_table[b, at // 64])
            cache.v.view(torch.uint8)[page, :, at % 64, 5] = 0x7f
            cache.v.view(torch.uint8)[page, :, at % 64, 77] = 0xff

    parents = [[-1, 0, 0, 1, 2, 1] + [3 + t % 3 for t in range(T - 6)]] * n
    tree_case(lens, [T] * n, 16 if T > 6 else 4, 2, 128, 64, BF, parents=parents, edit=edit, cols=cols)


def test_bad_parents_are_reported_and_taken_as_roots():
    for lens, T, cols in (([100, 90], 6, None), ([100, 90], 6, 2000), ([200] * 24, 60, None)):
        cache = filled(lens, 2, 128, 64, 5, cols=cols)
        B = len(lens)
        q = torch.randn(B, 16, T, 128, device=DEV).to(BF)
        good = [[-1] + [t - 1 - t % 2 for t in range(1, T)] for _ in range(B)]
        for t, x in ((3, 3), (4, T + 7), (2, -2), (5, 2 ** 31 - 1), (0, -2 ** 31)):
            bad = [list(p) for p in good]
            bad[1][t] = x
            root = [list(p) for p in good]
            root[1][t] = -1
            ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
            got = api.cache_tree_fwd(q, cache, i32(bad), ws=ws)
            assert api.get_error(ws) == 3, (T, t, x)
            want = api.cache_tree_fwd(q, cache, i32(root), ws=ws)
            assert api.get_error(ws) == 0
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("n,T,cols,form", [(2, 6, None, "cache_tree_cluster"), (2, 6, 2000, "cache_tree_chunk"), (24, 60, None, "cache_tree_cluster"),
                                           (2, 3, 2000, "cache_tree")])
def test_trees_report_without_a_workspace_of_the_callers(n, T, cols, form):
    """Parents that are none, in each form, through the handle; and nothing where all is well."""
    cache = filled([200] * n, 2, 128, 64, 5, cols=cols)
    q = torch.randn(n, 16, T, 128, device=DEV).to(BF)
    par = i32([list(range(-1, T - 1))] * n)
    api.trace_enable(8)
    api.trace_reset()
    want = api.cache_tree_fwd(q, cache, par)
    names = [x for x, _ in api.trace_records()]
    api.trace_enable(0)
    assert names == [form] and api.get_error(cache.fwd_ws) == 0
    bad = par.clone()
    bad[1, 0] = 7
    got = api.cache_tree_fwd(q, cache, bad)
    assert api.get_error(cache.fwd_ws) == 3
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.cache_tree_fwd(q, cache, par)
    held = cache.fwd_ws
    for x in (7, -1, 7):
        par[1, 0] = x
        graph.replay()
        torch.cuda.synchronize()
        assert api.get_error(held) == (3 if x == 7 else 0)
    api.cache_tree_fwd(q[:, :, :0], cache, par[:, :0].contiguous())
    assert api.get_error(cache.fwd_ws) == 0 and cache.fwd_ws is not held


def test_packed_offsets_that_are_none():
    """Tokens in front of the first offset and behind the last stay as they were; a run that is none is reported."""
    cache = filled([100, 90, 80], 2, 64, 32, 5)
    q = torch.randn(40, 8, 64, device=DEV).to(BF)
    par = i32([-1] * 40)
    for offs in ([5, 12, 12, 30], [0, 10, 7, 20], [3, 50, 60, 70], [-4, 5, 9, 12]):
        ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
        o, lse = api.cache_tree_fwd(q, cache, par, cu_seqlens=i32(offs), max_seqlen=20, ws=ws)
        bad = any(b < a or a < 0 or b > 40 or b - a > 20 for a, b in zip(offs, offs[1:]))
        assert api.get_error(ws) == (3 if bad else 0), offs
        for b, (x, y) in enumerate(zip(offs, offs[1:])):
            if 0 <= x < y <= 40 and y - x <= 20:
                assert torch.isfinite(o[x:y]).all() and torch.isfinite(lse[x:y]).all()


def test_rows_without_drafts_and_empty_calls():
    cache = filled([100, 90], 2, 64, 32, 5)
    o, lse = api.cache_tree_fwd(torch.empty(0, 8, 64, dtype=BF, device=DEV), cache, i32([]).view(0), cu_seqlens=i32([0, 0, 0]), max_seqlen=1)
    assert o.numel() == 0 and lse.numel() == 0
    with pytest.raises(api.NsaError):
        api.cache_tree_fwd(torch.zeros(2, 8, 257, 64, dtype=BF, device=DEV), cache, i32([[-1] * 257] * 2))
    with pytest.raises(api.NsaError):
        api.cache_tree_fwd(torch.zeros(2, 8, 4, 64, dtype=BF, device=DEV), cache, i32([[-1] * 4]))


def test_tree_in_a_graph_and_on_a_stream():
    cache = filled([400, 333, 90], 2, 128, 64, 2)
    T = 12
    trees = [i32([random_parents(T, 3, np.random.default_rng(10 * i + b)) for b in range(3)]) for i in range(3)]
    qs = [torch.randn(3, 8, T, 128, device=DEV).to(BF) for _ in range(3)]
    want = [api.cache_tree_fwd(q, cache, p) for q, p in zip(qs, trees)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = api.cache_tree_fwd(qs[0], cache, trees[0], stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0][0])
    q, p = qs[0].clone(), trees[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = api.cache_tree_fwd(q, cache, p)
    for i in range(3):
        q.copy_(qs[i])
        p.copy_(trees[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


# ------------------------------------------------------------------ accept

def state(cache):
    return [x.view(torch.uint8).clone() if x.dtype == torch.float8_e4m3fn else x.clone()
            for x in (cache.k, cache.v, cache.k_scale, cache.v_scale, cache.page_table, cache.seq_lens, cache.refcount)]


def plain_accept(plain, b, n, path):
    P, m = int(plain.lens[b]) - n, 0
    while m < len(path) and path[m] == m:
        m += 1
    held = []
    for codes, scales in ((plain.k, plain.ks), (plain.v, plain.vs)):
        rows = []
        for t in path[m:]:
            page, slot = plain.table[b, (P + t) // plain.bs], (P + t) % plain.bs
            # (a code times its scale, rounded to 32 bits)
            rows.append((codes[page, :, slot].astype(np.float32) * scales[page].astype(np.float32)[:, None]).astype(np.float64))
        held.append(np.array(rows))
    plain.lens[b] = P + len(path)
    if m < len(path):
        plain.append(b, held[0], held[1])


def same(cache, plain):
    code = lambda x: torch.nan_to_num(x.cpu().float(), nan=1e9).numpy()  # noqa: E731
    want = lambda x: np.where(np.isnan(x), 1e9, x)  # noqa: E731
    assert np.array_equal(code(cache.k), want(plain.k)) and np.array_equal(code(cache.v), want(plain.v))
    assert np.array_equal(cache.k_scale.cpu().double().numpy(), plain.ks) and np.array_equal(cache.v_scale.cpu().double().numpy(), plain.vs)
    assert np.array_equal(cache.seq_lens.cpu().numpy(), plain.lens) and np.array_equal(cache.page_table.cpu().numpy(), plain.table)
    assert np.array_equal(cache.refcount.cpu().numpy(), plain.ref)


def accept_case(lens, new, paths, Hkv, D, bs, seed=0, A=None, layout="dense", spread=3, edit=None, pow2=True):
    cache = filled(lens, Hkv, D, bs, seed, layout=layout, scale_spread=spread)
    if pow2:  # append's scales
        for s in (cache.k_scale, cache.v_scale):
            s.copy_(torch.exp2(torch.floor(torch.log2(s))))
    if edit is not None:
        edit(cache)
    plain = Plain(cache)
    A = A or max(1, max(len(p) for p in paths))
    api.cache_accept(cache, i32(new), i32([list(p) + [-1] * (A - len(p)) for p in paths]))
    assert api.get_error(cache.ws) == 0
    for b, (n, p) in enumerate(zip(new, paths)):
        plain_accept(plain, b, n, list(p))
    same(cache, plain)


@pytest.mark.parametrize("Hkv,D,bs", [(2, 128, 64), (3, 64, 32), (1, 32, 16), (8, 128, 16), (9, 64, 64)])
@pytest.mark.parametrize("layout", ["dense", "token", "both"])
def test_accept(Hkv, D, bs, layout):
    lens = [10, bs, bs + 7, 3 * bs + 9, 7, 64 + bs - 1]
    new = [8, 8, 8, 8, 7, 60]
    paths = [(), (0, 1, 2), (1, 4, 5), (0, 3, 7), (6,), (0, 1, 5, 6, 9, 30, 31, 44, 59)]
    accept_case(lens, new, paths, Hkv, D, bs, layout=layout, spread=6)


def test_accept_at_random():
    g = np.random.default_rng(0)
    for seed in range(6):
        bs = int(g.choice([16, 32, 64]))
        new = [int(x) for x in g.integers(0, 100, 20)]
        lens = [n + int(x) for n, x in zip(new, g.integers(0, 150, 20))]
        paths = [sorted(g.permutation(n)[:int(g.integers(0, n + 1))].tolist()) for n in new]
        accept_case(lens, new, paths, 2, int(g.choice([32, 64, 128])), bs, seed, spread=10, A=100)


def test_accept_a_whole_tree_and_long_paths():
    accept_case([600, 300], [512, 256], [list(range(0, 512, 2)), list(range(1, 256))], 2, 64, 16)
    accept_case([600], [512], [list(range(512))], 2, 64, 16)  # nothing moves


def test_accept_scales_that_are_no_powers_of_two():
    accept_case([100, 90], [40, 50], [(3, 9, 30), (0, 7, 8, 9, 40)], 2, 128, 16, pow2=False, spread=8)


def test_accept_nan_and_zero_codes():
    def edit(cache):
        cache.k.view(torch.uint8)[:, 0, 3] = 0x7f
        cache.v.view(torch.uint8)[:, 1, 5] = 0
        cache.v.view(torch.uint8)[:, 0] = 0x80  # -0
    accept_case([100, 90], [40, 50], [(3, 9, 30, 35), (0, 7, 8, 9, 40)], 2, 64, 16, edit=edit)


@pytest.mark.parametrize("D,bs", [(32, 16), (64, 32), (128, 64)])
@pytest.mark.parametrize("slot", [0, 4])
def test_accept_values_beyond_floats_range(D, bs, slot):
    """A code times its scale that passes float's range counts in no maximum, as in append, where an infinity counts in none;
    the finite values beside it in the same 16 codes do, and what they are divided by is theirs."""
    head = bs + slot

    def edit(cache):
        for at in (head + bs + 3, head + bs + 6):  # 256 * 2^120, 3 * 2^120 and smaller ones in every 16 codes
            page, i = int(cache.page_table[0, at // bs]), at % bs
            cache.k_scale[page] = 2.0 ** 120
            code = cache.k.view(torch.uint8)[page, :, i]
            code.fill_(0x20)
            code[:, ::16], code[:, 5::16], code[:, 7::16] = 0x78, 0x44, 0xf8
        cache.v.view(torch.uint8)[page, :, i, :16] = 0x7f  # NaN alone
    with np.errstate(over="ignore"):
        accept_case([head + bs + 9, 40], [bs + 9, 5], [(bs + 3, bs + 6), (1,)], 2, D, bs, edit=edit)


def test_accept_takes_what_an_append_of_the_values_gives():
    """The rule itself, through the library's append: the accepted drafts' values, appended to a row that never had the
    others, give the same codes and scales."""
    Hkv, D, bs, P, n, path = 2, 128, 16, 21, 30, [0, 1, 5, 9, 10, 22]
    a = api.make_cache(8, Hkv, D, bs, 1, 6)
    one = torch.ones(1, dtype=torch.int32, device=DEV)
    x = torch.randn(1, Hkv, P + n, D, device=DEV) * torch.linspace(0.1, 9, P + n, device=DEV)[:, None]
    api.cache_reserve(a, one * P)
    api.cache_append(a, x[:, :, :P], x[:, :, :P])
    api.cache_reserve(a, one * n)
    api.cache_append(a, x[:, :, P:], x[:, :, P:])
    held = []
    for t in path[2:]:
        page, slot = int(a.page_table[0, (P + t) // bs]), (P + t) % bs
        held.append(a.k[page, :, slot].float() * a.k_scale[page][:, None])
    values = torch.stack(held, 1)[None]  # [1, Hkv, 4, D]
    other = api.KVCache(a.k.view(torch.uint8).clone().view(a.k.dtype), a.v.view(torch.uint8).clone().view(a.k.dtype), a.k_scale.clone(),
                        a.v_scale.clone(), a.page_table.clone(), a.seq_lens.clone(), a.refcount.clone())
    other.seq_lens.fill_(P + 2)
    api.cache_reserve(other, one * 4)
    api.cache_append(other, values.contiguous(), values.contiguous())
    api.cache_accept(a, one * n, i32([path]))
    assert api.get_error(a.ws) == 0 and a.seq_lens.tolist() == other.seq_lens.tolist() == [P + 6]
    assert torch.equal(a.k.view(torch.uint8), other.k.view(torch.uint8)) and torch.equal(a.k_scale, other.k_scale)


@pytest.mark.parametrize("n,path", [(8, [3, 3]), (8, [5, 2]), (8, [8]), (8, [-2]), (8, [1, -1, 4]), (-1, []), (200, [1]), (0, [0]),
                                    (8, [2 ** 31 - 1])])
def test_accept_bad_rows_are_left_and_reported(n, path):
    cache = filled([100, 90, 70], 2, 64, 32, 1)
    before = state(cache)
    rows = [[0, 2, -1, -1], (path + [-1] * 4)[:4], [-1] * 4]
    api.cache_accept(cache, i32([8, n, 8]), i32(rows))
    assert api.get_error(cache.ws) == 3
    assert cache.seq_lens.tolist() == [94, 90, 62]
    pages = cache.page_table[1, :3].long()
    assert torch.equal(cache.k.view(torch.uint8)[pages], before[0][pages]) and torch.equal(cache.v_scale[pages], before[3][pages])


def test_accept_bad_pages_are_left_and_reported():
    for edit in ("pool", "none", "shared", "lens"):
        cache = filled([100, 90], 2, 64, 32, 1)
        col = (100 - 20) // 32
        if edit == "pool":
            cache.page_table[0, 3] = 10000  # the source's
        elif edit == "none":
            cache.page_table[0, col] = -1
        elif edit == "shared":
            cache.refcount[cache.page_table[0, col].long()] = 2
        else:
            cache.seq_lens[0] = 10 ** 6
        before = state(cache)
        api.cache_accept(cache, i32([20, 5]), i32([[1, 18], [0, -1]]))
        assert api.get_error(cache.ws) == 3, edit
        after = state(cache)
        assert torch.equal(after[5][0], before[5][0]) and after[5][1] == 86
        after[5][1] = before[5][1]
        assert all(torch.equal(x, y) for x, y in zip(before, after)), edit
    # without counts, a shared page is the caller's affair
    cache = filled([100, 90], 2, 64, 32, 1)
    own = api.KVCache(cache.k, cache.v, cache.k_scale, cache.v_scale, cache.page_table, cache.seq_lens)
    api.cache_accept(own, i32([20, 5]), i32([[1, 18], [0, -1]]))
    assert api.get_error(own.ws) == 0 and own.seq_lens.tolist() == [82, 86]


def test_accept_in_a_graph():
    cache = filled([100, 90], 2, 64, 32, 1)
    want = filled([100, 90], 2, 64, 32, 1)
    n, path = i32([20, 30]), i32([[-1] * 4] * 2)
    graph = torch.cuda.CUDAGraph()
    lens = cache.seq_lens.clone()
    with torch.cuda.graph(graph):
        api.cache_accept(cache, n, path)
    cache.seq_lens.copy_(lens)
    for p in ([[2, 5, 6, 7], [0, 1, 29, -1]], [[0, 3, -1, -1], [-1] * 4]):
        path.copy_(i32(p))
        cache.seq_lens.copy_(lens)
        want.seq_lens.copy_(lens)
        graph.replay()
        api.cache_accept(want, n, i32(p))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(state(cache), state(want)))


def test_steps_with_drafts_as_a_server_takes_them():
    """Reserve, rotate, append, attend by tree, accept, again and again, against a plain cache that gets the accepted
    tokens' held values only; the next step reserves into the pages that the dropped drafts left."""
    g = np.random.default_rng(5)
    Hq, Hkv, D, bs, B, T = 8, 2, 64, 16, 3, 9
    cache = api.make_cache(60, Hkv, D, bs, B, 12)
    f, w = (torch.tensor(10000.0 ** (-np.arange(0, D, 2) / D), dtype=torch.float32, device=DEV), torch.ones(D, device=DEV))
    counts = np.zeros(B, int)
    for step in range(6):
        n = T if step else 20
        parents = [random_parents(n, 3, g) for _ in range(B)] if step else [list(range(-1, n - 1))] * B
        depth = [[len(line_of(p, t)) - 1 for t in range(n)] for p in parents]
        pos = i32([[counts[b] + d for d in depth[b]] for b in range(B)])
        q, k, v = (torch.randn(B, H, n, D, device=DEV).to(BF) for H in (Hq, Hkv, Hkv))
        n_new = i32([n] * B)
        api.cache_reserve(cache, n_new)
        assert api.get_error(cache.ws) == 0
        zq, zk = api.norm_rope_fwd(q, k, w, w, f, pos=pos)
        api.cache_append(cache, zk, v)
        o, lse = api.cache_tree_fwd(zq, cache, i32(parents))
        plain = Plain(cache)
        for b in range(B):
            want = tree_attend(plain, b, zq[b].transpose(0, 1).double().cpu().numpy(), parents[b], 1 / math.sqrt(D))
            check_attend(o[b].transpose(0, 1).double().cpu().numpy(), lse[b].T.double().cpu().numpy(), *want, BF, D)
        if step:
            ends = [int(g.integers(-1, n)) for _ in range(B)]
            paths = [sorted(line_of(p, e)) for p, e in zip(parents, ends)]
        else:
            paths = [list(range(n))] * B
        api.cache_accept(cache, n_new, i32([list(p) + [-1] * (n - len(p)) for p in paths]))
        assert api.get_error(cache.ws) == 0
        for b in range(B):
            plain_accept(plain, b, n, paths[b])
            counts[b] += len(paths[b])
        same(cache, plain)
        assert cache.seq_lens.tolist() == counts.tolist()
