"""Argument checks of the rotating append, the key bounds and the block-sparse
decode: every refusal comes back before anything is launched (no GPU here)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_141_gb300 import build
    build.build()
    from paged_kv_cache_141_gb300 import binding
    binding.lib()
    return binding


OK, ODD = ctypes.c_void_p(256), ctypes.c_void_p(264)


def rope(pk, **kw):
    a = dict(out=OK, q=OK, qs=4096, k=OK, ks=1024, v=OK, vs=1024, kc=OK, vc=OK, cs=OK, maxpos=64, R=128, pos=OK,
             axes=1, fa=None, adj=0, qw=None, kw=None, eps=1e-6, slots=OK, T=4, Hq=32, Hkv=8, D=128, B=16, nb=10,
             dt=pk.PA_BF16, ct=pk.PA_BF16, ksc=1.0, vsc=1.0)
    a.update(kw)
    return pk.lib().pa_rope_and_cache(*a.values(), None, None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(R=0), dict(R=144), dict(R=-16), dict(axes=0), dict(adj=2), dict(maxpos=-1),
    dict(dt=4), dict(ct=-1), dict(qs=4097), dict(ks=1020), dict(vs=4), dict(axes=2), dict(axes=3, fa=b"\3" * 64),
    dict(out=None), dict(q=None), dict(k=None), dict(v=None), dict(kc=None), dict(vc=None), dict(cs=None),
    dict(pos=None), dict(slots=None), dict(out=ODD), dict(q=ODD), dict(v=ODD), dict(kc=ODD), dict(cs=ODD),
    dict(qw=ODD), dict(kw=ODD), dict(pos=ctypes.c_void_p(260)), dict(slots=ctypes.c_void_p(260)),
    dict(qw=OK, eps=-1.0), dict(kw=OK, eps=float("nan")), dict(ct=3, ksc=0.0), dict(ct=3, vsc=float("inf"))])
def test_rope_invalid(pk, kw):
    assert rope(pk, **kw) == pk.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(D=96, R=96), dict(R=40), dict(R=8), dict(B=1025), dict(axes=5, fa=b"\0" * 64),
                                dict(dt=3, ct=3), dict(ct=1), dict(dt=0, ct=2)])
def test_rope_unsupported(pk, kw):
    assert rope(pk, **kw) == pk.PA_ERR_UNSUPPORTED


def test_no_work_is_no_launch(pk):
    assert rope(pk, T=0, out=None, q=None, k=None, v=None, kc=None, vc=None, cs=None, pos=None, slots=None) == pk.PA_OK
    assert rope(pk, T=0, axes=3, fa=b"\2" * 64) == pk.PA_OK
    assert bounds(pk, S=0, kb=None, kc=None, bt=None, cl=None) == pk.PA_OK
    assert bounds(pk, new=OK, maxnew=0) == pk.PA_OK
    assert sparse(pk, S=0, out=None, kb=None, ws=None) == pk.PA_OK


def bounds(pk, **kw):
    a = dict(kb=OK, kc=OK, bt=OK, mb=8, cl=OK, new=None, maxnew=1, S=2, Hkv=8, D=128, B=16, nb=10, maxlen=100,
             ct=pk.PA_BF16, bd=pk.PA_BF16)
    a.update(kw)
    return pk.lib().pa_key_bounds(*a.values(), None, None)


@pytest.mark.parametrize("kw", [dict(S=-1), dict(maxnew=2), dict(maxnew=0), dict(new=OK, maxnew=-1), dict(mb=0),
                                dict(kb=None), dict(kc=None), dict(bt=None), dict(cl=None), dict(kb=ODD), dict(kc=ODD),
                                dict(bt=ctypes.c_void_p(258)), dict(new=ctypes.c_void_p(258)), dict(bd=7)])
def test_bounds_invalid(pk, kw):
    assert bounds(pk, **kw) == pk.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(D=80), dict(B=2000), dict(bd=1), dict(ct=3, bd=0), dict(ct=3, bd=3),
                                dict(maxlen=2 ** 31 - 1)])
def test_bounds_unsupported(pk, kw):
    assert bounds(pk, **kw) == pk.PA_ERR_UNSUPPORTED


def sparse(pk, **kw):
    a = dict(out=OK, q=OK, kc=OK, vc=OK, kb=OK, bt=OK, mb=8, cl=OK, S=2, Hq=32, Hkv=8, D=128, B=16, nb=10, maxlen=100,
             scale=0.1, K=4, first=1, recent=1, sel=None, dt=pk.PA_BF16, ct=pk.PA_BF16, ks=1.0, vs=1.0, ws=OK,
             wsb=1 << 40)
    a.update(kw)
    return pk.lib().pa_sparse_decode(*a.values(), None, None)


@pytest.mark.parametrize("kw", [dict(S=-1), dict(Hq=30), dict(K=0), dict(first=-1), dict(recent=0),
                                dict(first=3, recent=2), dict(first=2 ** 31 - 1, recent=2 ** 31 - 1, K=2 ** 31 - 1),
                                dict(scale=0.0), dict(scale=-0.5), dict(scale=float("nan")), dict(out=None),
                                dict(kb=None), dict(kb=ODD), dict(sel=ctypes.c_void_p(257)), dict(q=None),
                                dict(bt=None), dict(ct=3, ks=-1.0), dict(nb=0)])
def test_sparse_invalid(pk, kw):
    assert sparse(pk, **kw) == pk.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(D=96), dict(B=1025), dict(nb=2 ** 31), dict(nb=2 ** 28), dict(ct=1),
                                dict(maxlen=2 ** 31 - 1), dict(S=70000), dict(Hq=129, Hkv=1),
                                dict(maxlen=2 ** 19 + 1, B=1)])
def test_sparse_unsupported(pk, kw):
    assert sparse(pk, **kw) == pk.PA_ERR_UNSUPPORTED


def test_sparse_workspace(pk):
    n = pk.sparse_workspace_bytes(64, 32, 8, 128, 16, 32768, 64)
    assert n > 0 and n % 256 == 0
    assert sparse(pk, ws=None) == pk.PA_ERR_WORKSPACE
    assert sparse(pk, ws=ctypes.c_void_p(128)) == pk.PA_ERR_WORKSPACE
    need = pk.sparse_workspace_bytes(2, 32, 8, 128, 16, 100, 4)
    assert sparse(pk, wsb=need - 1) == pk.PA_ERR_WORKSPACE
    for bad in ((64, 30, 8, 128, 16, 100, 4), (64, 32, 8, 128, 16, 100, 0), (64, 32, 8, 128, 0, 100, 4),
                (-1, 32, 8, 128, 16, 100, 4), (64, 32, 8, 128, 16, 2 ** 31 - 1, 4)):
        assert pk.sparse_workspace_bytes(*bad) == 0
    # a workspace for the largest batch, context and selection serves the smaller ones
    for base, step in (((1, 32, 8, 128, 16, 8192, 64), 0), ((3, 32, 8, 128, 16, 1, 64), 5),
                       ((2, 16, 2, 64, 16, 8192, 1), 6)):
        last = 0
        for i in range(1, 400):
            a = list(base)
            a[step] = i * (97 if step == 5 else 1)
            n = pk.sparse_workspace_bytes(*a)
            assert n >= last, a
            last = n


def test_rope_sections(pk):
    assert pk.rope_sections((2, 1, 3)) == b"\0\0\1\2\2\2"


def test_binding_checks_before_the_library(pk):
    """The marshalling module's own refusals: host tensors, wrong objects and types."""
    import torch
    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    kv = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    cs = torch.zeros(8, 64)
    i64 = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA device"):
        pk.rope_and_cache(q, q, kv, kv, cache, cache, cs, i64, i64)
    with pytest.raises(TypeError, match="query must be a tensor"):
        pk.rope_and_cache(q, [1], kv, kv, cache, cache, cs, i64, i64)
    with pytest.raises(TypeError):
        pk.rope_and_cache(q, q)
    bounds = torch.zeros(4, 2, 2, 64, dtype=torch.bfloat16)
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        pk.key_bounds(bounds, cache, torch.zeros(2, 3, dtype=torch.int32), i32, 16)
    with pytest.raises(ValueError, match="CUDA device"):
        pk.sparse_decode(q, q, cache, cache, bounds, torch.zeros(2, 3, dtype=torch.int32), i32, 16, 0.1, 4,
                         torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(TypeError, match="workspace must be a tensor"):
        pk.sparse_decode(q, q, cache, cache, bounds, i32, i32, 16, 0.1, 4, None)


def test_bounds_of_more_warps_than_indices(pk):
    """Touched blocks times KV heads beyond 2^27 (a warp each) are refused: 32-bit thread indices would wrap."""
    assert bounds(pk, new=OK, maxnew=2 ** 24 + 1, maxlen=2 ** 30, B=1, Hkv=8) == pk.PA_ERR_UNSUPPORTED
    assert bounds(pk, new=OK, maxnew=2 ** 30, maxlen=2 ** 30, B=16, Hkv=8) == pk.PA_ERR_UNSUPPORTED
    # at most the context: a larger bound on the new tokens is no reason
    assert bounds(pk, S=0, new=OK, maxnew=2 ** 30, maxlen=2 ** 20) == pk.PA_OK
