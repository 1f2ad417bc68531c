"""The paged 8-bit cache's entry points refuse bad calls on the host, before
any launch (no GPU needed)."""
import ctypes as C
import glob
import os
import re

import pytest
import torch

from block_sparse_attention_do_gb300 import api, build

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6
P = 256  # a plausible device address: the calls below fail before anything reads it


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.lib()


def cache(**kw):
    base = dict(num_pages=100, Hkv=2, D=128, block_size=64, rows=3, max_pages=10, k=P, v=P, k_scale=P, v_scale=P,
                page_table=P, seq_lens=P, refcount=P)
    stride = kw.pop("stride", None)
    base.update(kw)
    c = api.CacheStruct(**base)
    if stride:
        c.stride[:] = stride
    return c


def problem(**kw):
    base = dict(B=3, Hq=4, Hkv=2, T=1, D=128, block_size=64, S=4, dtype=torch.bfloat16)
    base.update(kw)
    return api.problem(**base)


BIG = 1 << 30
META = dict(page_table=None), dict(seq_lens=None), dict(page_table=258), dict(seq_lens=257)
DATA = (dict(k=None), dict(v=None), dict(k=264), dict(v=P + 8), dict(k_scale=None), dict(v_scale=258),
        dict(stride=(1 << 40, 16, 16)), dict(stride=(64, 24, 16)), dict(stride=(64, 0, 16)), dict(stride=(-64, 16, 16)))
SHAPES = (dict(num_pages=0), dict(Hkv=0), dict(rows=0), dict(max_pages=-1))
LIMITS = (dict(D=96), dict(D=256), dict(block_size=48), dict(block_size=128), dict(max_pages=1 << 26),
          dict(rows=1 << 16, max_pages=1 << 16), dict(num_pages=1 << 30))


def test_struct_layout_matches_the_header(lib):
    assert C.sizeof(api.CacheStruct) == 6 * 4 + 3 * 8 + 7 * 8
    assert api.CacheStruct.stride.offset == 24 and api.CacheStruct.refcount.offset == 96


def test_status_string(lib):
    assert lib.nsa_status_string(7) == b"NSA_ERR_CACHE_FULL"


def test_workspace_sizes(lib):
    def up(n):
        return -(-n // 256) * 256

    assert lib.nsa_cache_workspace_size(cache()) == 256 + 3 * up(400) + 2 * up(12)
    for kw in SHAPES + LIMITS + (dict(stride=(64, 24, 16)),):
        assert lib.nsa_cache_workspace_size(cache(**kw)) == 0, kw
    assert lib.nsa_cache_fwd_workspace_size(problem(), cache(), 0) >= 256
    assert lib.nsa_cache_fwd_workspace_size(problem(), cache(k=None, page_table=None), 1) >= 256
    for kw in (dict(B=2), dict(Hq=3), dict(D=64), dict(block_size=32), dict(T=0)):
        assert lib.nsa_cache_fwd_workspace_size(problem(**kw), cache(), 0) == 0, kw
    assert lib.nsa_cache_fwd_workspace_size(problem(S=0), cache(), 1) == 0
    assert lib.nsa_cache_fwd_workspace_size(None, cache(), 0) == 0
    assert lib.nsa_cache_fwd_workspace_size(problem(), None, 0) == 0


def calls(lib):
    return {
        "reserve": lambda c, n=P, ws=P, size=BIG: lib.nsa_cache_reserve(c, n, ws, size, None),
        "free": lambda c, n=3, rows=P, ws=P, size=BIG: lib.nsa_cache_free(c, rows, n, ws, size, None),
        "fork": lambda c, n=2, src=P, dst=P, ws=P, size=BIG: lib.nsa_cache_fork(c, src, dst, n, ws, size, None),
        "copy": lambda c, n=2, src=P, dst=P, ws=P, size=BIG: lib.nsa_cache_copy(c, src, dst, n, ws, size, None),
        "compact": lambda c, ws=P, size=BIG: lib.nsa_cache_compact(c, ws, size, None),
    }


@pytest.mark.parametrize("name", ["reserve", "free", "fork", "copy", "compact"])
def test_page_operations_refuse(lib, name):
    call = calls(lib)[name]
    assert call(None) == INVALID
    for kw in SHAPES:
        assert call(cache(**kw)) == INVALID, kw
    for kw in LIMITS:
        assert call(cache(**kw)) == UNSUPPORTED, kw
    for kw in () if name == "copy" else META + (dict(refcount=None),):
        assert call(cache(**kw)) == INVALID, kw
    for kw in DATA if name in ("fork", "copy", "compact") else ():
        assert call(cache(**kw)) == INVALID, kw
    assert call(cache(refcount=258)) == INVALID
    need = lib.nsa_cache_workspace_size(cache())
    for ws, size in ((None, BIG), (P + 16, BIG), (P, need - 1)):
        assert call(cache(), ws=ws, size=size) == WORKSPACE


def test_page_lists_refuse(lib):
    c = calls(lib)
    assert c["reserve"](cache(), n=None) == INVALID and c["reserve"](cache(), n=P + 2) == INVALID
    for n in (-1, 4):
        assert c["free"](cache(), n=n) == INVALID and c["fork"](cache(), n=n) == INVALID
    assert c["copy"](cache(), n=101) == INVALID and c["copy"](cache(), n=-1) == INVALID
    assert c["free"](cache(), rows=None) == INVALID
    for name in ("fork", "copy"):
        for kw in (dict(src=None), dict(dst=None), dict(src=P + 1), dict(dst=P + 2)):
            assert c[name](cache(), **kw) == INVALID


def test_append_refuses(lib):
    def call(p, c, cu=None, k=P, v=P, ws=P, size=256):
        return lib.nsa_cache_append(p, c, cu, k, v, ws, size, None)

    assert call(None, cache()) == INVALID and call(problem(), None) == INVALID
    for kw in SHAPES + META + DATA:
        assert call(problem(), cache(**kw)) == INVALID, kw
    for kw in LIMITS:
        assert call(problem(), cache(**kw)) == UNSUPPORTED, kw
    for kw in (dict(B=4), dict(Hkv=1), dict(D=64), dict(block_size=16), dict(T=0), dict(Hq=3)):
        assert call(problem(**kw), cache()) == INVALID, kw
    assert call(problem(D=96), cache()) == UNSUPPORTED
    assert call(problem(), cache(), k=None) == INVALID and call(problem(), cache(), v=P + 8) == INVALID
    assert call(problem(), cache(), cu=P) == INVALID  # packed offsets with a fixed-length problem
    thd = problem(layout=api.LAYOUT_THD, total_tokens=5)
    assert call(thd, cache()) == INVALID              # and none with a packed one
    assert call(problem(), cache(), size=255) == WORKSPACE and call(problem(), cache(), ws=None) == WORKSPACE
    bad = problem()
    bad.kv_stride[:] = (128, 64, 3)
    assert call(bad, cache()) == INVALID


def test_attention_refuses(lib):
    def call(p, c, window=0, cu=None, idx=None, sinks=None, q=P, o=P, lse=P, ws=P, size=BIG):
        return lib.nsa_cache_fwd(p, c, window, cu, idx, sinks, q, o, lse, ws, size, None)

    assert call(None, cache()) == INVALID and call(problem(), None) == INVALID
    for kw in SHAPES + META + DATA:
        assert call(problem(), cache(**kw)) == INVALID, kw
    for kw in (dict(B=4), dict(Hkv=1), dict(D=64), dict(block_size=16), dict(T=0), dict(Hq=3)):
        assert call(problem(**kw), cache()) == INVALID, kw
    for kw in (dict(q=None), dict(o=None), dict(lse=None), dict(q=P + 8), dict(o=P + 4), dict(lse=P + 2), dict(idx=P + 1),
               dict(sinks=P + 2), dict(window=-1), dict(idx=P, window=3), dict(idx=P, sinks=P), dict(cu=P)):
        assert call(problem(), cache(), **kw) == INVALID, kw
    assert call(problem(layout=api.LAYOUT_THD, total_tokens=5), cache()) == INVALID
    assert call(problem(S=0), cache(), idx=P) == INVALID
    assert call(problem(S=257), cache(), idx=P) == UNSUPPORTED
    assert call(problem(B=8193), cache(rows=8193)) == UNSUPPORTED
    assert call(problem(T=1 << 28), cache()) == UNSUPPORTED
    need = lib.nsa_cache_fwd_workspace_size(problem(), cache(), 0)
    assert call(problem(), cache(), size=need - 1) == WORKSPACE
    assert call(problem(), cache(), ws=P + 64) == WORKSPACE


def test_tensors_are_checked():
    """The Python layer's checks of shapes and types (CPU tensors: nothing is launched)."""
    k = torch.zeros(8, 2, 16, 32, dtype=torch.uint8).view(torch.float8_e4m3fn)
    sc = torch.ones(8, 2)
    table, lens, refs = (torch.zeros(s, dtype=torch.int32) for s in ((3, 4), (3,), (8,)))
    good = dict(k=k, v=k.clone(), k_scale=sc, v_scale=sc.clone(), page_table=table, seq_lens=lens, refcount=refs)
    assert api.KVCache(**good).struct.max_pages == 4
    assert api.KVCache(**{**good, "refcount": None}).struct.refcount is None
    for kw in (dict(k=k.view(torch.uint8)), dict(v=k[:7]), dict(k=k[0]), dict(k_scale=sc[:, :1]), dict(v_scale=sc.double()),
               dict(k_scale=sc.t().contiguous().t()), dict(page_table=table.long()), dict(page_table=table[0]),
               dict(seq_lens=lens[:2]), dict(refcount=refs[:7]), dict(page_table=table.t()),
               dict(k=k.transpose(2, 3), v=k.transpose(2, 3))):
        with pytest.raises(api.NsaError):
            api.KVCache(**{**good, **kw})


def test_positions_stay_within_an_int(lib):
    """Positions reach from -T to the table's last key."""
    thd = dict(layout=api.LAYOUT_THD, total_tokens=5)
    for T, code in ((2 ** 31 - 1, 0), (2 ** 31 - 640 - 64, 0), (2 ** 31 - 640 - 66, 1)):
        assert (lib.nsa_cache_fwd_workspace_size(problem(T=T, **thd), cache(), 0) > 0) == bool(code), T
    p = problem(T=2 ** 31 - 1, **thd)
    assert lib.nsa_cache_fwd(p, cache(), 0, P, None, None, P, P, P, P, BIG, None) == UNSUPPORTED
    assert lib.nsa_cache_append(p, cache(), P, P, P, P, BIG, None) == UNSUPPORTED


def test_kernels_wait_before_they_read():
    """Every kernel of the cache may start while the launches before it still run (a reserve that writes lengths, an
    append that writes pages): nothing of a call's arguments is read in front of its wait for them."""
    csrc = os.path.join(os.path.dirname(api.__file__), "csrc")
    seen = 0
    for path in glob.glob(os.path.join(csrc, "k_cache_*.cu")):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for part in text.split("__global__")[1:]:
            name = re.search(r"\b(cache_\w+)\(", part).group(1)
            body = part[part.index("\n{"):part.index("\n}")]
            assert "dependency_wait();" in body, name
            before = body[:body.index("dependency_wait();")]
            assert not re.search(r"\b(lens|cu|table|ref|ks|vs|status|idx|sinks|n_new|rows|src|dst|part_\w+|p[012]|npairs|err)\b|"
                                 r"\b\w+(_tokens|_pages|_of|_off|_len)\(", before), (name, before)
            seen += 1
    assert seen == 10
