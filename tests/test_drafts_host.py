"""Trees of drafts, acceptance, blocks' weights and eviction: the entry points
refuse bad calls on the host, before any launch (no GPU needed)."""
import os
import re

import pytest
import torch

from block_sparse_attention_do_gb300 import api, build
from test_cache_host import DATA, LIMITS, META, SHAPES, cache, problem

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6
P = 256
BIG = 1 << 30


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.lib()


def test_tree_refuses(lib):
    def call(p, c, window=0, cu=None, par=P, idx=None, sinks=None, q=P, o=P, lse=P, ws=P, size=BIG):
        return lib.nsa_cache_tree_fwd(p, c, window, cu, par, idx, sinks, q, o, lse, ws, size, None)

    assert call(None, cache()) == INVALID and call(problem(), None) == INVALID
    for kw in SHAPES + META + DATA:
        assert call(problem(), cache(**kw)) == INVALID, kw
    for kw in LIMITS:
        assert call(problem(), cache(**kw)) == UNSUPPORTED, kw
    for kw in (dict(par=None), dict(par=P + 2), dict(q=None), dict(o=P + 4), dict(lse=P + 2), dict(idx=P + 1), dict(window=-1),
               dict(idx=P, window=3), dict(idx=P, sinks=P), dict(cu=P)):
        assert call(problem(), cache(), **kw) == INVALID, kw
    assert call(problem(T=257), cache()) == UNSUPPORTED
    assert call(problem(T=257, layout=api.LAYOUT_THD, total_tokens=5), cache(), cu=P) == UNSUPPORTED
    assert call(problem(layout=api.LAYOUT_THD, total_tokens=5), cache()) == INVALID
    need = lib.nsa_cache_tree_fwd_workspace_size(problem(), cache(), 0)
    assert need >= 256 and lib.nsa_cache_tree_fwd_workspace_size(problem(T=257), cache(), 0) == 0
    assert lib.nsa_cache_tree_fwd_workspace_size(None, cache(), 0) == lib.nsa_cache_tree_fwd_workspace_size(problem(D=64), cache(), 0) == 0
    assert call(problem(), cache(), size=need - 1) == WORKSPACE and call(problem(), cache(), ws=P + 64) == WORKSPACE


def test_accept_refuses(lib):
    def call(c, n=P, path=P, A=4, ws=P, size=BIG):
        return lib.nsa_cache_accept(c, n, path, A, ws, size, None)

    assert call(None) == INVALID
    for kw in SHAPES + META + DATA + (dict(refcount=258),):
        assert call(cache(**kw)) == INVALID, kw
    for kw in LIMITS:
        assert call(cache(**kw)) == UNSUPPORTED, kw
    for kw in (dict(n=None), dict(n=P + 2), dict(path=None), dict(path=P + 1), dict(A=0), dict(A=-3)):
        assert call(cache(), **kw) == INVALID, kw
    need = lib.nsa_cache_workspace_size(cache())
    for ws, size in ((None, BIG), (P + 16, BIG), (P, need - 1)):
        assert call(cache(), ws=ws, size=size) == WORKSPACE


def test_weigh_refuses(lib):
    def call(p, c, window=0, cu=None, q=P, lse=P, decay=1.0, weight=P, ws=P, size=256):
        return lib.nsa_cache_weigh(p, c, window, cu, q, lse, decay, weight, ws, size, None)

    assert call(None, cache()) == INVALID and call(problem(), None) == INVALID
    for kw in SHAPES + META + DATA:
        assert call(problem(), cache(**kw)) == INVALID, kw
    for kw in LIMITS:
        assert call(problem(), cache(**kw)) == UNSUPPORTED, kw
    for kw in (dict(window=-1), dict(cu=P), dict(q=None), dict(q=P + 8), dict(lse=None), dict(lse=P + 2), dict(weight=None),
               dict(weight=P + 1), dict(decay=-0.5), dict(decay=1.5), dict(decay=float("nan"))):
        assert call(problem(), cache(), **kw) == INVALID, kw
    for ws, size in ((P + 16, 256), (P, 255)):
        assert call(problem(), cache(), ws=ws, size=size) == WORKSPACE


def test_evict_refuses(lib):
    def call(c, weight=P, keep=8, first=1, recent=2, kept=P, ws=P, size=256):
        return lib.nsa_cache_evict(c, weight, keep, first, recent, kept, ws, size, None)

    assert call(None) == INVALID
    for kw in SHAPES + META + (dict(refcount=None), dict(refcount=257)):
        assert call(cache(**kw)) == INVALID, kw
    for kw in LIMITS:
        assert call(cache(**kw)) == UNSUPPORTED, kw
    for kw in (dict(weight=None), dict(weight=P + 2), dict(kept=P + 1), dict(keep=0), dict(keep=2), dict(first=-1), dict(recent=0),
               dict(keep=2 ** 31 - 1, first=2 ** 31 - 1, recent=1)):
        assert call(cache(), **kw) == INVALID, kw
    for ws, size in ((None, 256), (P + 16, 256), (P, 255)):
        assert call(cache(), ws=ws, size=size) == WORKSPACE


def test_kernels_wait_before_they_read():
    """As test_cache_host's check, for the kernels beside the cache's own."""
    csrc = os.path.join(os.path.dirname(api.__file__), "csrc")
    seen = 0
    for name in ("k_accept.cu", "k_weigh.cu", "k_weigh_tc.cu", "k_tree_tc.cu", "k_evict.cu", "k_norm_rope.cu"):
        text = re.sub(r"//[^\n]*|L::\w+", "", open(os.path.join(csrc, name)).read())  # (places in shared memory are no reads)
        for part in text.split("__global__")[1:]:
            body = part[part.index("\n{"):part.index("\n}")]
            before = body[:body.index("dependency_wait();")]
            assert not re.search(r"\b(lens|cu|table|ref|ks|vs|weight|kept|path|n_new|pos|freq|qw|kw|part|err|lse)\b(?!\[)|"
                                 r"\b\w+(_tokens|_of|_off|_at)\(", before), (name, before)
            seen += 1
    assert seen >= 10


def test_tensors_are_checked():
    """The Python layer's checks of shapes and types (CPU tensors: nothing is launched)."""
    k = torch.zeros(8, 2, 16, 32, dtype=torch.uint8).view(torch.float8_e4m3fn)
    sc = torch.ones(8, 2)
    table, lens, refs = (torch.zeros(s, dtype=torch.int32) for s in ((3, 4), (3,), (8,)))
    c = api.KVCache(k, k.clone(), sc, sc.clone(), table, lens, refs)
    for w in (torch.zeros(3, 2, 5), torch.zeros(3, 2, 4).double(), torch.zeros(3, 4, 2).transpose(1, 2)):
        with pytest.raises(api.NsaError):
            api._weights(c, w)
    api._weights(c, torch.zeros(3, 2, 4))


# what a kernel's arguments point to, and the helpers that read it
_GLOBAL = re.compile(r"\b(lens|cu|table|ref|ks|vs|weight|kept|path|n_new|pos|freq|qw|kw|part|part_\w+|cuts|err|lse|parents|sinks|idx|q|k|qr|kr|r0|r1)\b"
                     r"|\b\w+(_tokens|_of|_off|_at|_len|_prefix)\(")


def _early_reads(source):
    """{kernel: what it reads in front of its wait} of a file's kernels; shared memory's declarations and places in it are none."""
    text = re.sub(r"//[^\n]*|L::\w+|[^\n]*__shared__[^\n]*;", "", source)
    found = {}
    for part in text.split("__global__")[1:]:
        name = re.search(r"\b(\w+_kernel)\(", part).group(1)
        body = part[part.index("\n{"):part.index("\n}")]
        assert "dependency_wait();" in body, name
        found[name] = [m.group(0) for m in _GLOBAL.finditer(body[:body.index("dependency_wait();")])]
    return found


def test_no_kernel_reads_in_front_of_its_wait():
    """The kernels beside the cache's own may start while the launches before them still run.  The check finds a read that is
    spliced in front of the wait, however it is written."""
    csrc = os.path.join(os.path.dirname(api.__file__), "csrc")
    seen = set()
    for name in ("k_accept.cu", "k_weigh.cu", "k_weigh_tc.cu", "k_tree_tc.cu", "k_evict.cu", "k_norm_rope.cu"):
        source = open(os.path.join(csrc, name)).read()
        kernels = _early_reads(source)
        assert not any(kernels.values()), (name, kernels)
        seen |= set(kernels)
        for read in ("int x = a.c.lens[0];", "int x = g.cu[b + 1];", "int x = a.pos[tok];", "int x = c.table[(int64_t)b * c.cols];", "float x = *lse;",
                     "int x = new_tokens(g, b);", "*err = 0;", "int x = p.parents[t];", "uint4 x = *(const uint4 *)(a.q + 1);", "int x = ws.r0[b];",
                     "int x = ref[0];", "float x = part[i];"):
            spliced = source.replace("dependency_wait();", read + "\n    dependency_wait();")
            planted = _early_reads(spliced)
            assert set(planted) == set(kernels) and all(planted.values()), (name, read, planted)
    assert len(seen) == 11, seen
