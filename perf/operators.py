"""Serving from a paged key/value cache held in 8 bits: the calls that are timed, and what they compute.

Operators (``case["op"]``):

* ``attend``: attention of new query tokens over the cache: the whole cache (with an optional sliding window and
  attention sinks) or, with ``S`` > 0, the ``S`` blocks that each index row selects;
* ``append``: new tokens' keys and values rounded to 8 bits with one scale per block and head, written into their pages;
* ``copy`` / ``fork`` / ``turnover`` / ``compact``: the pages themselves: copied one by one, shared by a forked sequence
  (its last, partly filled page copied), freed and reserved again as sequences leave and enter, and moved to the front
  of the pool.

The cache: codes ``k``, ``v`` [pages, Hkv, block, D] in e4m3, one fp32 scale per page and head, a page table
[rows, max_pages], the rows' lengths (new tokens included) and the pages' reference counts.  A page is one block.

With ``own`` false the plain form below runs: elementary torch operations in 32 bits.  With ``own`` true the same inputs
go through the library's entry points.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
SCALE_FLOOR = 2.0 ** -100  # the scale of a block of zeros
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def attend(name, B, Hq, Hkv, D, bs, lo, hi, T=1, ragged=False, S=0, window=0, sinks=False, dtype="bf16", mix=0):
    """B sequences of lo .. hi cached tokens, their last T (ragged: up to T) the queries."""
    return dict(name=name, op="attend", B=B, Hq=Hq, Hkv=Hkv, D=D, bs=bs, lo=lo, hi=hi, T=T, ragged=ragged, S=S,
                window=window, sinks=sinks, dtype=dtype, mix=mix)


def append(name, B, Hkv, D, bs, lo, hi, T=1, ragged=False, dtype="bf16", mix=0):
    """T (ragged: up to T) new tokens behind lo .. hi cached ones, for each of B sequences."""
    return dict(name=name, op="append", B=B, Hkv=Hkv, D=D, bs=bs, lo=lo, hi=hi, T=T, ragged=ragged, dtype=dtype, mix=mix)


def pages(name, op, Hkv, D, bs, pool, B, lo, hi, n, mix=0):
    """A pool of `pool` pages that B rows of lo .. hi tokens use; the call is about n pages (copy) or n rows."""
    return dict(name=name, op=op, Hkv=Hkv, D=D, bs=bs, pool=pool, B=B, lo=lo, hi=hi, n=n, mix=mix)


def listed():
    return [
        # one user's next token: 32 query heads over 8 kv heads, the whole cache read; latency counts
        attend("attend one token", 1, 32, 8, 128, 64, 8192, 8192),
        # a served batch at its next token, lengths as they come; the cache's bytes are the work
        attend("attend batch", 32, 32, 8, 128, 64, 128, 32768, mix=1),
        # the same step of a block-selecting model: 16 selected blocks of 64 keys per token and kv head
        attend("attend selected", 128, 32, 2, 128, 64, 1024, 8192, S=16, mix=2),
        # a few drafted tokens checked at once, sliding window and sinks, an odd group of heads
        attend("attend drafted", 16, 24, 8, 128, 64, 700, 8192, T=5, window=4096, sinks=True, mix=3),
        # the small shape in 32 bits: head dimension 64, blocks of 32
        attend("attend small fp32", 8, 6, 2, 64, 32, 17, 1024, dtype="fp32", mix=4),
        # prompts taken in chunks of up to 2048 tokens behind what is cached: the products are the work
        attend("attend chunk", 6, 32, 8, 128, 64, 2048, 8192, T=2048, ragged=True, mix=5),
        # the served batch's new token goes into its pages
        append("append one token", 64, 8, 128, 64, 0, 8192, mix=6),
        # prompts of odd lengths go in at once
        append("append prompts", 8, 8, 128, 64, 0, 500, T=8192, ragged=True, mix=7),
        # pages copied for sequences that part
        pages("copy pages", "copy", 8, 128, 64, 2048, 16, 64, 4096, 300, mix=8),
        # several samples continue each prompt: pages shared, the last one copied
        pages("fork rows", "fork", 8, 128, 64, 4096, 72, 100, 4096, 64, mix=9),
        # finished sequences leave, new prompts take their rows: metadata of a large pool alone
        pages("turn rows over", "turnover", 1, 32, 16, 65536, 256, 16, 4096, 64, mix=10),
        # the pool is compacted, half its pages free in between
        pages("compact pool", "compact", 2, 128, 64, 4096, 128, 100, 4096, 64, mix=11),
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, even over their logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attend"] * 5 + ["append"] * 2 + ["copy", "fork", "turnover", "compact"])
    mix = rng.randrange(1 << 20)
    Hkv, G, D, bs = rng.choice([(8, 4, 128, 64), (2, 16, 128, 64), (8, 3, 128, 64), (4, 8, 64, 64), (2, 3, 64, 32),
                                (1, 2, 32, 16), (5, 1, 64, 16), (1, 32, 128, 32), (2, 12, 128, 16)])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "attend":
        kind = rng.choice(["token", "token", "few", "selected", "chunk"])
        hi = spread(rng, 1, 8192)
        lo = rng.choice([1, max(1, hi // 2), hi])
        B = spread(rng, 1, max(1, min(64, (1 << 22) // (Hkv * hi))))
        T = {"token": 1, "few": rng.randint(2, 8), "selected": rng.choice([1, 1, 3]), "chunk": spread(rng, 9, 1024)}[kind]
        B = B if kind != "chunk" else min(B, 4)
        S = rng.randint(1, 16) if kind == "selected" else 0
        window = spread(rng, 1, 4096) if S == 0 and rng.random() < 0.25 else 0
        c = attend("", B, Hkv * G, Hkv, D, bs, lo, hi, T=T, ragged=kind == "chunk" or rng.random() < 0.2, S=S,
                   window=window, sinks=S == 0 and rng.random() < 0.25, dtype=dtype, mix=mix)
    elif op == "append":
        T = rng.choice([1, spread(rng, 2, 4096)])
        c = append("", spread(rng, 1, 64 if T == 1 else 8), Hkv, D, bs, 0, spread(rng, 1, 4096), T=T,
                   ragged=T > 1 and rng.random() < 0.7, dtype=dtype, mix=mix)
    else:
        pool = spread(rng, 256, 4096 if op != "turnover" else 65536)
        B = rng.randint(4, 64)
        hi = max(1, pool * bs // (2 * B))
        lo = rng.randint(1, hi)
        n = rng.randint(1, pool // 3) if op == "copy" else rng.randint(1, B // 2)
        c = pages("", op, Hkv, D, bs, pool, B, lo, hi, n, mix=mix)
    del c["name"]
    return c


def shape_of(case):
    """What the case alone settles: the rows' lengths (new tokens included) and new tokens."""
    r = random.Random(case["mix"])
    B = case["B"]
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(B)]
    T = case.get("T", 0)
    new = [r.randint(0, T) if case.get("ragged") else T for _ in range(B)]
    if case["op"] == "append":
        lens = [a + n for a, n in zip(lens, new)]
    elif case.get("ragged"):
        new = [min(n, a) for n, a in zip(new, lens)]
        if sum(new) == 0:
            new[0] = 1
    if case["op"] == "append" and sum(new) == 0:
        lens[0], new[0] = lens[0] + 1, 1
    return lens, new


def blocks(n, bs):
    return -(-n // bs)


def rows_of(case):
    """The rows that a fork, a turnover or a compaction is about."""
    r = random.Random(case["mix"] + 1)
    order = list(range(case["B"]))
    r.shuffle(order)
    return order[:case["n"]], order[case["n"]:]


def work(case):
    lens, new = shape_of(case)
    bs, Hkv, D, op = case["bs"], case["Hkv"], case["D"], case["op"]
    page = 2 * Hkv * (bs * D + 4)  # keys, values, scales
    if op == "attend":
        es, Hq, S, W = (2 if case["dtype"] == "bf16" else 4), case["Hq"], case["S"], case["window"]
        pairs = tokens = 0
        for n, q in zip(lens, new):
            at = range(max(0, n - q), n)
            if S:
                a = sum(min(S - 1, p // bs) * bs + p % bs + 1 for p in at)
                pairs, tokens = pairs + a, tokens + min(a, n)
            else:
                pairs += sum(min(p + 1, W) if W else p + 1 for p in at)
                tokens += (min(n, W + q - 1) if W else n) if q else 0
        nq = sum(new) * Hq
        return {"bytes": 2 * tokens * Hkv * D + 8 * Hkv * blocks(tokens, bs) + nq * (2 * D * es + 4)
                + 4 * sum(new) * Hkv * S + 4 * blocks(tokens, bs), "flops": 4 * D * Hq * pairs}
    if op == "append":
        es = 2 if case["dtype"] == "bf16" else 4
        touched = sum(blocks(n, bs) - (n - q) // bs for n, q in zip(lens, new) if q)
        return {"bytes": 2 * sum(new) * Hkv * D * (es + 1) + 8 * touched * Hkv + 4 * touched, "flops": 0}
    used = [blocks(n, bs) for n in lens]
    rows, rest = rows_of(case)
    if op == "copy":
        return {"bytes": case["n"] * (2 * page + 8), "flops": 0}
    if op == "fork":
        src = [rest[i % len(rest)] for i in range(case["n"])]
        tails = sum(1 for s in src if lens[s] % bs)
        return {"bytes": tails * 2 * page + 4 * case["pool"] + 16 * sum(used[s] for s in src), "flops": 0}
    if op == "turnover":
        return {"bytes": 4 * case["pool"] + 16 * sum(used[r] for r in rows), "flops": 0}
    live = sum(used[r] for r in rest)
    moved = live * (case["pool"] - live) // case["pool"]  # of a random placement, on average
    return {"bytes": moved * 2 * page + 8 * case["pool"] + 8 * live, "flops": 0}


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    cpu = random.Random(seed)
    dev, op, bs, Hkv, D, B = "cuda", case["op"], case["bs"], case["Hkv"], case["D"], case["B"]
    lens, new = shape_of(case)
    used = [blocks(n, bs) for n in lens]
    npool = case.get("pool") or sum(used) + max(4, sum(used) // 16)
    cols = max(max(used), 1)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731

    order = list(range(npool))  # the rows' pages lie anywhere in the pool
    cpu.shuffle(order)
    rows, rest = rows_of(case) if op in ("fork", "turnover", "compact") else ([], [])
    table, at = [[-1] * cols for _ in range(B)], 0
    held = [0 if op in ("fork", "compact") and b in set(rows) else used[b] for b in range(B)]
    for b in range(B):
        table[b][:held[b]] = order[at:at + held[b]]
        at += held[b]
    lens_now = [n if h else 0 for n, h in zip(lens, held)]

    shape = (npool, Hkv, bs, D)
    k = (torch.randn(shape, generator=g, device=dev) * 100).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    v = (torch.randn(shape, generator=g, device=dev) * 100).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    scale = lambda: torch.exp2(torch.randint(-8, -5, (npool, Hkv), generator=g, device=dev).float())  # noqa: E731
    ks, vs = scale(), scale()

    refs = [0] * npool
    for b in range(B):
        for p in table[b][:held[b]]:
            refs[p] = 1
    # table, lengths and counts side by side, so that one copy brings them all back
    n_table, n_lens = blocks(B * cols, 4) * 4, blocks(B, 4) * 4
    meta = torch.zeros(n_table + n_lens + npool, dtype=torch.int32, device=dev)
    s = dict(case=case, meta=meta, k=k, v=v, k_scale=ks, v_scale=vs, page_table=meta[:B * cols].view(B, cols),
             seq_lens=meta[n_table:n_table + B], refcount=meta[n_table + n_lens:])
    s["page_table"].copy_(ints(table))
    s["seq_lens"].copy_(ints(lens_now))
    s["refcount"].copy_(ints(refs))

    if op in ("attend", "append"):
        for b in range(B if op == "attend" else 0):  # behind a row's last token lie another's leavings: NaN among them
            if lens[b] % bs:
                page = table[b][used[b] - 1]
                k.view(torch.uint8)[page, :, lens[b] % bs:] = 0x7f
                v.view(torch.uint8)[page, :, lens[b] % bs:] = 0x7f
        dt, T = TYPES[case["dtype"]], case["T"]
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s["cu"] = ints(cu) if case["ragged"] else None
        s["max_new"] = max(new)
        dims = lambda H: (cu[-1], H, D) if case["ragged"] else (B, H, T, D)  # noqa: E731
        mk = lambda H: torch.randn(dims(H), generator=g, device=dev).to(dt)  # noqa: E731
        if op == "append":
            s["kn"], s["vn"] = mk(Hkv), mk(Hkv)
        else:
            s["q"] = mk(case["Hq"])
            s["sinks"] = torch.randn(case["Hq"], generator=g, device=dev) if case["sinks"] else None
            s["idx"] = None
            if case["S"]:  # the own block, then earlier ones at random, then -1
                S = case["S"]
                pos = torch.cat([torch.arange(n - q, n, device=dev) for n, q in zip(lens, new)])
                own_block = pos.div(bs, rounding_mode="floor").view(-1, 1, 1)
                noise = torch.rand(len(pos), Hkv, max(cols, S), generator=g, device=dev)
                noise = torch.where(torch.arange(noise.shape[-1], device=dev) < own_block, noise, 2.0)
                val, pick = noise.sort(-1)
                idx = torch.where(val < 1.5, pick, -1)[..., :S - 1]
                idx = torch.cat([own_block.expand(-1, Hkv, 1), idx], -1)
                idx = torch.where(own_block < 0, -1, idx).to(torch.int32)
                s["idx"] = idx.contiguous() if case["ragged"] else idx.view(B, T, Hkv, S).transpose(1, 2).contiguous()
    elif op == "copy":
        pick = cpu.sample(range(npool), 2 * case["n"]) if 2 * case["n"] <= npool else order[:2 * (npool // 2)]
        half = len(pick) // 2
        s["src"], s["dst"] = ints(pick[:half]), ints(pick[half:])
    else:
        s["rows"] = ints(rows)
        if op == "fork":
            s["src"] = ints([rest[i % len(rest)] for i in range(len(rows))])
        elif op == "turnover":
            s["grow"] = ints([lens[b] if b in set(rows) else 0 for b in range(B)])
        else:
            s["found"] = meta.clone()
    return s


# -------------------------------------------------------------- the passes

def run(s):
    op = s["case"]["op"]
    if own:
        return run_own(s, op)
    return {"attend": plain_attend, "append": plain_append, "copy": plain_copy, "fork": plain_fork,
            "turnover": plain_turnover, "compact": plain_compact}[op](s)


def run_own(s, op):
    from block_sparse_attention_do_gb300 import api

    if "cache" not in s:  # the handle that a serving program makes once
        s["cache"] = api.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["page_table"], s["seq_lens"], s["refcount"])
    cache, case = s["cache"], s["case"]
    if op == "attend":
        return api.cache_fwd(s["q"], cache, block_idx=s["idx"], cu_seqlens=s["cu"], max_seqlen=s["max_new"],
                             window=case["window"] or None, sinks=s["sinks"])
    if op == "append":
        api.cache_append(cache, s["kn"], s["vn"], cu_seqlens=s["cu"], max_seqlen=s["max_new"])
    elif op == "copy":
        api.cache_copy(cache, s["src"], s["dst"])
    elif op == "fork":
        api.cache_fork(cache, s["src"], s["rows"])
    elif op == "turnover":
        api.cache_free(cache, s["rows"])
        api.cache_reserve(cache, s["grow"])
    else:
        s["meta"].copy_(s["found"])  # the pool as it was found, so that every pass moves the same pages
        api.cache_compact(cache)
    return outputs(s, op)


def outputs(s, op):
    pool = (s["k"], s["v"], s["k_scale"], s["v_scale"])
    meta = (s["page_table"], s["seq_lens"], s["refcount"])
    return {"append": (s["k"], s["k_scale"], s["v"], s["v_scale"]), "copy": pool, "fork": pool + meta, "turnover": meta, "compact": pool + meta}[op]


def token_rows(s):
    """(sequence, place among its new tokens) of each packed token."""
    cu = s["cu"].long()
    tok = torch.arange(s["q"].shape[0] if "q" in s else s["kn"].shape[0], device=cu.device)
    b = torch.searchsorted(cu, tok, right=True) - 1
    return b, tok - cu[b]


def values(codes, *at):
    """The codes at an index, in 32 bits."""
    return codes.view(torch.uint8)[at].view(codes.dtype).float()


def plain_attend(s):
    case, q, cu = s["case"], s["q"], s["cu"]
    Hkv, D, bs, S, W = case["Hkv"], case["D"], case["bs"], case["S"], case["window"]
    table, lens = s["page_table"].long(), s["seq_lens"].long()
    B, T = table.shape[0], s["max_new"]
    dev = q.device
    if cu is not None:  # packed tokens to rows of one length
        b, t = token_rows(s)
        qp = torch.zeros(B, T, q.shape[1], D, device=dev)
        qp[b, t] = q.float()
        qp, n_new = qp.transpose(1, 2), (cu[1:] - cu[:-1]).long()
    else:
        qp, n_new = q.float(), torch.full((B,), T, device=dev)
    Hq = qp.shape[1]
    G = Hq // Hkv
    qp = qp.reshape(B, Hkv, G, T, D)
    pos = (lens - n_new)[:, None] + torch.arange(T, device=dev)  # [B, T]
    scale = 1.0 / math.sqrt(D)
    if S:
        idx = s["idx"].long()
        if cu is not None:
            packed, idx = idx, torch.full((B, T, Hkv, S), -1, device=dev)
            idx[b, t] = packed
            idx = idx.transpose(1, 2)  # [B, Hkv, T, S]
        page = table[torch.arange(B, device=dev)[:, None, None, None], idx.clamp(min=0)].clamp(min=0)
        head = torch.arange(Hkv, device=dev)[None, :, None, None]
        key = idx[..., None] * bs + torch.arange(bs, device=dev)
        seen = (idx[..., None] >= 0) & (key <= pos[:, None, :, None, None]) & (key < lens[:, None, None, None, None])
        kk = values(s["k"], page, head) * s["k_scale"][page, head][..., None, None]  # [B, Hkv, T, S, bs, D]
        vv = values(s["v"], page, head) * s["v_scale"][page, head][..., None, None]
        vv = torch.where(seen[..., None], vv, 0.0).flatten(3, 4)
        seen = seen.flatten(3, 4)[:, :, None]
        x = torch.einsum("bhgtd,bhtkd->bhgtk", qp, kk.flatten(3, 4)) * scale
    else:
        page = table.clamp(min=0)
        kk = (values(s["k"], page) * s["k_scale"][page][..., None, None]).transpose(1, 2).flatten(2, 3)  # [B, Hkv, L, D]
        vv = (values(s["v"], page) * s["v_scale"][page][..., None, None]).transpose(1, 2).flatten(2, 3)
        key = torch.arange(kk.shape[2], device=dev)
        here = key < lens[:, None]
        seen = here[:, None] & (key <= pos[..., None])
        if W:
            seen = seen & (key > pos[..., None] - W)
        vv = torch.where(here[:, None, :, None], vv, 0.0)
        seen = seen[:, None, None]  # [B, 1, 1, T, L]
        x = torch.matmul(qp.flatten(2, 3), kk.transpose(2, 3)).view(B, Hkv, G, T, -1) * scale
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(1, Hkv, G, 1, 1)
        m = torch.maximum(m, sink)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        total = total + torch.exp(sink - m)
    lse = torch.log(total) + m
    p = p / torch.where(total == 0, 1.0, total)
    o = torch.einsum("bhgtk,bhtkd->bhgtd", p, vv) if S else torch.matmul(p.flatten(2, 3), vv).view(B, Hkv, G, T, D)
    o, lse = o.reshape(B, Hq, T, D), lse.reshape(B, Hq, T)
    if cu is not None:
        o, lse = o.transpose(1, 2)[b, t], lse.transpose(1, 2)[b, t]
    return o.to(q.dtype), lse


def pow2_scale(amax):
    """The least power of two s with amax <= 448 s (at least SCALE_FLOOR): 448 = 0.875 * 2^9."""
    mant, exp = torch.frexp(amax.clamp(min=E4M3_MAX * SCALE_FLOOR))
    return ((exp - 9 + (mant > 0.875).int() + 127) << 23).view(torch.float32)


def to_e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def plain_append(s):
    case, cu, bs = s["case"], s["cu"], s["case"]["bs"]
    table, lens = s["page_table"].long(), s["seq_lens"].long()
    B, dev = table.shape[0], table.device
    if cu is not None:
        b, t = token_rows(s)
        n_new = (cu[1:] - cu[:-1]).long()
    else:
        T = s["kn"].shape[2]
        b = torch.arange(B, device=dev).repeat_interleave(T)
        t, n_new = torch.arange(T, device=dev).repeat(B), torch.full((B,), T, device=dev)
    start = lens - n_new
    pos = start[b] + t
    page, slot = table[b, pos.div(bs, rounding_mode="floor")], pos % bs
    # a row's first page may hold earlier tokens, whose scale and codes count
    first = table[torch.arange(B, device=dev), start.div(bs, rounding_mode="floor").clamp(max=table.shape[1] - 1)]
    kept = ((start % bs > 0) & (n_new > 0))[:, None]
    kept_page = first.clamp(min=0)
    older = (torch.arange(bs, device=dev) < (start % bs)[:, None])[:, None, :, None] & kept[..., None, None]
    return plain_write(s, "k", s["kn"], page, slot, kept, kept_page, older) + plain_write(
        s, "v", s["vn"], page, slot, kept, kept_page, older)


def plain_write(s, which, new, page, slot, kept, kept_page, older):
    codes, scales = s[which], s[which + "_scale"]
    new = new.float() if s["cu"] is not None else new.transpose(1, 2).flatten(0, 1).float()  # [tokens, Hkv, D]
    size = torch.where(torch.isfinite(new), new.abs(), 0.0).amax(-1)
    amax = torch.zeros_like(scales).index_reduce_(0, page, size, "amax")
    touched = torch.zeros(scales.shape[0], 1, dtype=torch.bool, device=new.device).index_fill_(0, page, True)
    old = torch.zeros_like(scales).index_reduce_(0, kept_page, torch.where(kept, scales[kept_page], 0.0), "amax")
    scale = torch.where(touched, torch.maximum(pow2_scale(amax), old), scales)
    # earlier codes of a partly filled page, rounded again where its scale grew
    was = codes.view(torch.uint8)[kept_page]
    again = to_e4m3(was.view(codes.dtype).float() * (scales[kept_page] / scale[kept_page])[..., None, None])
    bits = torch.where(older, again.view(torch.uint8), was)
    some = kept[:, 0]
    codes.view(torch.uint8)[kept_page[some]] = bits[some]
    scales.copy_(scale)
    head = torch.arange(new.shape[1], device=new.device)
    codes.view(torch.uint8)[page[:, None], head, slot[:, None]] = to_e4m3(new / scale[page][..., None]).view(torch.uint8)
    return codes, scales


def copy_pages(s, src, dst):
    for_bytes = lambda x: x.view(torch.uint8)  # noqa: E731
    for_bytes(s["k"])[dst] = for_bytes(s["k"])[src]
    for_bytes(s["v"])[dst] = for_bytes(s["v"])[src]
    s["k_scale"][dst] = s["k_scale"][src]
    s["v_scale"][dst] = s["v_scale"][src]


def plain_copy(s):
    copy_pages(s, s["src"].long(), s["dst"].long())
    return outputs(s, "copy")


def release(s, rows):
    held = s["page_table"][rows].long().flatten()
    s["refcount"].index_add_(0, held.clamp(min=0), -(held >= 0).int())
    s["page_table"][rows] = -1
    s["seq_lens"][rows] = 0


def plain_fork(s):
    bs, src, dst = s["case"]["bs"], s["src"].long(), s["rows"].long()
    release(s, dst)
    table, lens, refs = s["page_table"], s["seq_lens"], s["refcount"]
    n, cols = len(src), table.shape[1]
    theirs = table[src].long()
    full, tail = lens[src].long().div(bs, rounding_mode="floor"), lens[src].long() % bs > 0
    shared = torch.arange(cols, device=table.device) < full[:, None]
    free = refs == 0
    by_id = torch.argsort(free.int(), descending=True, stable=True)  # free pages, lowest first
    fresh = by_id[(torch.cumsum(tail.long(), 0) - 1).clamp(min=0)]
    at = full.clamp(max=cols - 1)[:, None]
    last = theirs.gather(1, at)[:, 0]
    copy_pages(s, last.clamp(min=0), torch.where(tail, fresh, last.clamp(min=0)))
    is_tail = tail[:, None] & (torch.arange(cols, device=table.device) == full[:, None])
    mine = torch.where(shared, theirs, torch.where(is_tail, fresh[:, None], -1))
    refs.index_add_(0, mine.clamp(min=0).flatten(), (mine >= 0).int().flatten())
    table[dst] = mine.int()
    lens[dst] = lens[src]
    return outputs(s, "fork")


def plain_turnover(s):
    bs = s["case"]["bs"]
    release(s, s["rows"].long())
    table, lens, refs = s["page_table"], s["seq_lens"], s["refcount"]
    have, want = (lens.long() + bs - 1).div(bs, rounding_mode="floor"), (lens + s["grow"]).long()
    want = (want + bs - 1).div(bs, rounding_mode="floor")
    need = want - have
    col = torch.arange(table.shape[1], device=table.device)
    fresh = (col >= have[:, None]) & (col < want[:, None])
    free = refs == 0
    by_id = torch.argsort(free.int(), descending=True, stable=True)
    nth = (torch.cumsum(need, 0) - need)[:, None] + col - have[:, None]
    fits = need.sum() <= free.sum()
    table.copy_(torch.where(fresh & fits, by_id[nth.clamp(0, len(refs) - 1)], table.long()).int())
    refs.add_((free & fits & (torch.cumsum(free.long(), 0) <= need.sum())).int())
    lens.add_(torch.where(fits, s["grow"], 0))
    return outputs(s, "turnover")


def plain_compact(s):
    s["meta"].copy_(s["found"])
    refs, table = s["refcount"], s["page_table"]
    page = torch.arange(len(refs), device=refs.device)
    live = refs > 0
    front = page < live.sum()
    src, dst = torch.nonzero(live & ~front)[:, 0], torch.nonzero(~live & front)[:, 0]
    copy_pages(s, src, dst)
    refs[dst] = refs[src]
    refs[src] = 0
    page[src] = dst
    table.copy_(torch.where(table >= 0, page[table.clamp(min=0).long()].int(), table))
    return outputs(s, "compact")


# ----------------------------------------------- 64 bits, by the definition

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return exact_attend(case, s)
    if case["op"] == "append":
        return exact_append(case, s)
    return exact_pages(case, s)


def exact_attend(case, s):
    lens, new = shape_of(case)
    Hq, Hkv, D, bs, T, S, W = (case[x] for x in ("Hq", "Hkv", "D", "bs", "T", "S", "window"))
    table, q = s["page_table"].tolist(), s["q"].double()
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:-1], -math.inf, dtype=torch.float64, device="cuda")
    if S and sum(new) * Hkv > 4096:
        return None
    idx = s["idx"].tolist() if S else None
    base = 0
    for b in range(len(lens)):
        pg = torch.tensor(table[b][:blocks(lens[b], bs)], device="cuda", dtype=torch.long)
        for h in range(Hkv if new[b] else 0):
            deq = lambda c, f: (s[c].view(torch.uint8)[pg, h].view(s[c].dtype).double() * s[f][pg, h].double()[:, None, None]).reshape(-1, D)[:lens[b]]  # noqa: E731
            K, V = deq("k", "k_scale"), deq("v", "v_scale")
            heads = slice(h * Hq // Hkv, (h + 1) * Hq // Hkv)
            Q = q[base:base + new[b], heads].transpose(0, 1) if case["ragged"] else q[b, heads]
            pos = torch.arange(lens[b] - new[b], lens[b], device="cuda")[:, None]
            key = torch.arange(lens[b], device="cuda")[None]
            keep = key <= pos
            if W:
                keep &= key > pos - W
            if S:
                rows = [idx[base + t][h] if case["ragged"] else idx[b][h][t] for t in range(new[b])]
                chosen = torch.zeros(new[b], blocks(lens[b], bs), dtype=torch.bool)
                for t, row in enumerate(rows):
                    chosen[t, [j for j in row if j >= 0]] = True
                keep &= chosen.cuda().repeat_interleave(bs, 1)[:, :lens[b]]
            x = torch.where(keep, Q @ K.T / math.sqrt(D), -math.inf)
            if s["sinks"] is not None:
                x = torch.cat([x, s["sinks"][heads].double()[:, None, None].expand(-1, new[b], 1)], -1)
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(z == -math.inf, 0.0, z)[..., None])
            y = p[..., :lens[b]] @ V
            if case["ragged"]:
                o[base:base + new[b], heads], lse[base:base + new[b], heads] = y.transpose(0, 1), z.T
            else:
                o[b, heads], lse[b, heads] = y, z
        base += new[b]
    return o, lse


def exact_round(x):
    """x (64 bits) to the nearest e4m3 value, ties to the even one: a step of 2^-3 of the leading power, 2^-9 at least."""
    lead = torch.frexp(x.abs().clamp(min=2.0 ** -6, max=512.0))[1] - 1
    step = torch.exp2((lead - 3).double())
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact_append(case, s):
    lens, new = shape_of(case)
    bs, out, table = case["bs"], [], s["page_table"].tolist()
    if sum(new) // bs + len(new) > 6000:
        return None
    for c, f, n in (("k", "k_scale", "kn"), ("v", "v_scale", "vn")):
        codes, scale, fresh = s[c].double(), s[f].double(), s[n].double()
        base = 0
        for b in range(len(lens)):
            rows = fresh[base:base + new[b]] if case["ragged"] else fresh[b].transpose(0, 1)  # [tokens, Hkv, D]
            at, first = lens[b] - new[b], lens[b] - new[b]
            while at < lens[b]:
                p, lo = table[b][at // bs], at % bs
                m = min(bs - lo, lens[b] - at)
                x = rows[at - first:at - first + m].transpose(0, 1)  # [Hkv, m, D]
                need = torch.exp2(torch.ceil(torch.log2((x.abs().amax((1, 2)) / E4M3_MAX).clamp(min=SCALE_FLOOR))))
                to = torch.maximum(need, scale[p]) if lo else need
                codes[p, :, :lo] = exact_round(codes[p, :, :lo] * (scale[p] / to)[:, None, None])
                codes[p, :, lo:lo + m] = exact_round(x / to[:, None, None])
                scale[p] = to
                at += m
            base += new[b]
        out += [codes, scale]
    return tuple(out)


def exact_pages(case, s):
    """Pages hold what was written, whole: the copies by the definition, one page after another."""
    op, bs = case["op"], case["bs"]
    if op == "turnover":
        return None
    k, v, ks, vs = (s[x].double() for x in ("k", "v", "k_scale", "v_scale"))
    move = []
    if op == "copy":
        move = list(zip(s["src"].tolist(), s["dst"].tolist()))
    else:
        refs, table, lens = s["refcount"].tolist(), s["page_table"].tolist(), s["seq_lens"].tolist()
        if op == "fork":  # the forked rows start out empty
            free = (p for p, r in enumerate(refs) if r == 0)
            for a in s["src"].tolist():
                if lens[a] % bs:
                    move.append((table[a][lens[a] // bs], next(free)))
        else:
            n = sum(1 for r in refs if r)
            move = list(zip([p for p in range(n, len(refs)) if refs[p]], [p for p in range(n) if not refs[p]]))
    for a, b in move:
        for x in (k, v, ks, vs):
            x[b] = x[a]
    out = (k, v, ks, vs)
    return out if op == "copy" else out + (None, None, None)
