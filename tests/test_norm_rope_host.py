"""The norm and rotation entry points refuse bad calls on the host, before any
launch (no GPU needed)."""
import ctypes as C

import pytest
import torch

from block_sparse_attention_do_gb300 import api, build

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6
P = 256  # a plausible device address: the calls below fail before anything reads it
BIG = 1 << 30


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.lib()


def problem(**kw):
    base = dict(B=2, Hq=4, Hkv=2, T=8, D=128, block_size=64, S=1, dtype=torch.bfloat16)
    base.update(kw)
    return api.problem(**base)


def rope(rotary=128, interleaved=0, eps=1e-6, **strides):
    n = api.NormRopeStruct(rotary, interleaved, eps, 0)
    for name, s in strides.items():
        getattr(n, name)[:] = s
    return n


def fwd(lib, p=None, n=None, cu=None, q=P, k=P, qw=P, kw=P, f=P, pos=P, qr=P, kr=P):
    return lib.nsa_norm_rope_fwd(p or problem(), n or rope(), cu, q, k, qw, kw, f, pos, qr, kr, None)


def bwd(lib, p=None, n=None, cu=None, q=P, k=P, dqr=P, dkr=P, qw=P, kw=P, f=P, pos=P, dq=P, dk=P, dqw=P, dkw=P, ws=P, size=BIG):
    return lib.nsa_norm_rope_bwd(p or problem(), n or rope(), cu, q, k, dqr, dkr, qw, kw, f, pos, dq, dk, dqw, dkw, ws, size, None)


def test_struct_layout_matches_the_header():
    assert C.sizeof(api.NormRopeStruct) == 4 * 4 + 6 * 8 and api.NormRopeStruct.qr_stride.offset == 16


@pytest.mark.parametrize("call", [fwd, bwd])
def test_refusals(lib, call):
    assert lib.nsa_norm_rope_fwd(None, rope(), None, P, P, P, P, P, P, P, P, None) == INVALID
    assert lib.nsa_norm_rope_fwd(problem(), None, None, P, P, P, P, P, P, P, P, None) == INVALID
    for kw in (dict(B=0), dict(T=0), dict(Hq=3), dict(Hkv=0)):
        assert call(lib, problem(**kw)) == INVALID, kw
    assert call(lib, problem(D=96)) == UNSUPPORTED
    assert call(lib, problem(layout=api.LAYOUT_THD, total_tokens=5)) == INVALID  # packed, without offsets
    assert call(lib, cu=P) == INVALID                                            # offsets of a fixed-length problem
    for n in (rope(-2), rope(130), rope(15), rope(interleaved=2), rope(eps=0.0), rope(eps=-1.0), rope(eps=float("nan")),
              rope(eps=float("inf")), rope(qr_stride=(128, 64, 3)), rope(kr_stride=(-128, 64, 8)), rope(kr_stride=(0, 64, 8))):
        assert call(lib, n=n) == INVALID
    for r in (8, 20, 126):
        assert call(lib, n=rope(r)) == UNSUPPORTED
    for kw in (dict(q=None), dict(k=None), dict(q=P + 8), dict(k=P + 2), dict(qw=P + 2), dict(kw=P + 1), dict(f=None), dict(f=P + 2),
               dict(pos=P + 2)):
        assert call(lib, **kw) == INVALID, kw
    bad = problem()
    bad.q_stride[:] = (128, 64, 3)
    assert call(lib, bad) == INVALID


def test_outputs_and_workspace(lib):
    for kw in (dict(qr=None), dict(kr=None), dict(qr=P + 8), dict(kr=P + 4)):
        assert fwd(lib, **kw) == INVALID, kw
    for kw in (dict(dqr=None), dict(dkr=P + 8), dict(dq=None), dict(dk=P + 8), dict(dqw=P + 2), dict(dkw=P + 1)):
        assert bwd(lib, **kw) == INVALID, kw
    need = lib.nsa_norm_rope_bwd_workspace_size(problem())
    assert need > 0 and need % 256 == 0
    for ws, size in ((None, BIG), (P + 16, BIG), (P, 1024)):
        assert bwd(lib, ws=ws, size=size) == WORKSPACE
    assert lib.nsa_norm_rope_bwd_workspace_size(problem(D=96)) == 0 and lib.nsa_norm_rope_bwd_workspace_size(None) == 0
    assert lib.nsa_norm_rope_bwd_workspace_size(problem(layout=api.LAYOUT_THD, total_tokens=5)) > 0


def test_tensors_are_checked():
    """The Python layer refuses CPU tensors (there is no CPU path)."""
    q, k = torch.zeros(1, 4, 8, 64), torch.zeros(1, 2, 8, 64)
    with pytest.raises(api.NsaError):
        api._norm_rope(q, k, q, k, None, None, True, None, None, None, None, 1e-6, False, None)


def test_expanded_tensors_are_refused():
    """All strides 0 declare a dense tensor: one row expanded to many (a gradient that is the same for every token) would be
    read far behind its end."""
    row = torch.zeros(32)
    with pytest.raises(api.NsaError):
        api._row_strides(row.expand(2, 3, 4, 32), False)
    with pytest.raises(ValueError):
        api._bht_strides(row.expand(2, 3, 4, 32), False)
    with pytest.raises(ValueError):
        api._bht_strides(row.expand(5, 3, 32), True)
    # of one dimension alone: a stride of 0 beside others that are not, refused by the call
    p = api.problem(2, 3, 3, 4, 32, 64, 1, torch.float32)
    for x in (torch.zeros(2, 3, 1, 32).expand(2, 3, 4, 32), torch.zeros(1, 3, 4, 32).expand(2, 3, 4, 32)):
        p.q_stride[:] = api._row_strides(x, False)
        assert api.lib().nsa_norm_rope_bwd_workspace_size(p) == 0
    # tensors of one row, and dense ones, as before
    assert any(api._row_strides(row.expand(1, 1, 1, 32), False)) and api._row_strides(torch.zeros(2, 3, 4, 32), False) == (384, 128, 32)
    api._bht_strides(row.expand(1, 1, 1, 32), False)
    assert api._bht_strides(torch.zeros(5, 3, 32), True) == (0, 32, 96)


def test_an_expanded_cache_is_refused():
    k = torch.zeros(32, dtype=torch.uint8).view(torch.float8_e4m3fn).expand(8, 2, 16, 32)
    sc, (table, lens, refs) = torch.ones(8, 2), (torch.zeros(s, dtype=torch.int32) for s in ((3, 4), (3,), (8,)))
    with pytest.raises(api.NsaError):
        api.KVCache(k, k, sc, sc.clone(), table, lens, refs)
