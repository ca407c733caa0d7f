"""Argument checks of the block tables on the device, the block-scaled cache and the
draft verification: every refusal comes back before anything is launched (no GPU
here)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_141_gb300 import build
    build.build()
    from paged_kv_cache_141_gb300 import binding
    binding.lib()
    return binding


OK, ODD, HALF = ctypes.c_void_p(256), ctypes.c_void_p(264), ctypes.c_void_p(258)
FOUR = ctypes.c_void_p(260)


def extend(pk, **kw):
    a = dict(bt=OK, mb=8, len=OK, new=OK, S=2, stack=OK, nf=OK, cap=100, B=16, slots=OK, pos=OK, T=10, qs=OK, nl=OK, nn=OK)
    a.update(kw)
    return pk.lib().pa_extend_tables(*a.values(), None, None)


def trim(pk, **kw):
    a = dict(bt=OK, mb=8, len=OK, drop=OK, S=2, stack=OK, nf=OK, cap=100, B=16, shared=None, nl=OK, nn=OK)
    a.update(kw)
    return pk.lib().pa_trim_tables(*a.values(), None, None)


@pytest.mark.parametrize("kw", [dict(S=-1), dict(mb=-1), dict(cap=-1), dict(B=0), dict(len=None), dict(stack=None), dict(nf=None),
                                dict(nl=None), dict(nn=None), dict(bt=None), dict(len=HALF), dict(stack=HALF), dict(nf=HALF)])
def test_tables_invalid(pk, kw):
    assert extend(pk, **kw) == pk.PA_ERR_INVALID_ARG
    assert trim(pk, **kw) == pk.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(new=None), dict(slots=None), dict(qs=None), dict(T=-1), dict(slots=FOUR), dict(pos=FOUR), dict(qs=HALF)])
def test_extend_invalid(pk, kw):
    assert extend(pk, **kw) == pk.PA_ERR_INVALID_ARG


def test_tables_unsupported(pk):
    assert extend(pk, S=16385) == trim(pk, S=16385) == pk.PA_ERR_UNSUPPORTED
    assert extend(pk, B=1025) == trim(pk, B=1025) == pk.PA_ERR_UNSUPPORTED
    assert extend(pk, T=2 ** 31) == extend(pk, cap=2 ** 31) == pk.PA_ERR_UNSUPPORTED
    assert trim(pk, shared=HALF) == pk.PA_ERR_INVALID_ARG


def append(pk, **kw):
    a = dict(k=OK, ks=1024, v=OK, vs=1024, kc=OK, vc=OK, ksc=OK, vsc=OK, bt=OK, mb=8, len=OK, qs=OK, T=4, most=4, S=2, H=8, D=128, B=16,
             nb=10, dt=pk.PA_BF16, ct=pk.PA_INT8)
    a.update(kw)
    return pk.lib().pa_scaled_append(*a.values(), None, None)


@pytest.mark.parametrize("kw", [dict(S=-1), dict(H=0), dict(D=0), dict(B=0), dict(nb=-1), dict(mb=-1), dict(T=-1), dict(most=-1), dict(ks=1020),
                                dict(vs=1016), dict(ks=1028), dict(k=None), dict(v=None), dict(kc=None), dict(vc=None), dict(ksc=None),
                                dict(vsc=None), dict(bt=None), dict(len=None), dict(mb=0), dict(k=ODD), dict(vc=ODD), dict(ksc=HALF),
                                dict(qs=HALF), dict(dt=5), dict(ct=-1), dict(ct=5), dict(qs=None), dict(qs=None, most=1, T=3)])
def test_append_invalid(pk, kw):
    assert append(pk, **kw) == pk.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(D=96), dict(B=1025), dict(S=65536), dict(dt=3), dict(dt=4), dict(ct=0), dict(ct=2)])
def test_append_unsupported(pk, kw):
    assert append(pk, **kw) == pk.PA_ERR_UNSUPPORTED


def attention(pk, **kw):
    a = dict(out=OK, q=OK, kc=OK, vc=OK, ksc=OK, vsc=OK, bt=OK, mb=8, len=OK, qs=OK, T=4, most=2, S=2, Hq=32, H=8, D=128, B=16, nb=10,
             maxlen=100, scale=0.1, dt=pk.PA_BF16, ct=pk.PA_INT8, ws=OK, wsb=1 << 40)
    a.update(kw)
    return pk.lib().pa_scaled_attention(*a.values(), None, None)


@pytest.mark.parametrize("kw", [dict(S=-1), dict(T=-1), dict(most=-1), dict(most=0), dict(Hq=0), dict(H=0), dict(Hq=33), dict(D=0), dict(B=0),
                                dict(nb=-1), dict(mb=0), dict(maxlen=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                                dict(scale=float("inf")), dict(dt=5), dict(ct=-1), dict(out=None), dict(q=None), dict(kc=None),
                                dict(vc=None), dict(ksc=None), dict(vsc=None), dict(bt=None), dict(len=None), dict(out=ODD), dict(q=ODD),
                                dict(kc=ODD), dict(ksc=HALF), dict(len=HALF), dict(qs=HALF), dict(qs=None), dict(qs=None, most=1),
                                dict(S=0)])
def test_attention_invalid(pk, kw):
    assert attention(pk, **kw) == pk.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(dt=0), dict(dt=3), dict(dt=4), dict(ct=1), dict(ct=0), dict(D=96), dict(B=1025), dict(S=65536, T=65536),
                                dict(maxlen=2 ** 30 + 1), dict(nb=2 ** 28)])
def test_attention_unsupported(pk, kw):
    assert attention(pk, **kw) == pk.PA_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [{}, dict(most=200, T=400), dict(D=256, most=64, T=128)])
def test_attention_workspace(pk, kw):
    a = dict(S=2, T=4, most=2, D=128)
    a.update(kw)
    need = pk.scaled_workspace_bytes(a["S"], a["T"], 32, 8, a["D"], a["most"], 100)
    assert need > 0 and need % 256 == 0
    # every block size gets along with it (a byte less is refused for one of them at least)
    got = [attention(pk, **kw, B=B, wsb=need - 1) for B in (1, 16)]
    assert pk.PA_ERR_WORKSPACE in got
    assert pk.PA_ERR_WORKSPACE in [attention(pk, **kw, B=B, ws=None) for B in (1, 16)]
    assert pk.PA_ERR_WORKSPACE in [attention(pk, **kw, B=B, ws=ctypes.c_void_p(384)) for B in (1, 16)]


def test_attention_workspace_sizes(pk):
    ws = pk.scaled_workspace_bytes
    assert ws(0, 1, 32, 8, 128, 1, 100) == ws(1, 1, 33, 8, 128, 1, 100) == ws(1, 1, 32, 8, 96, 1, 100) == 0
    assert ws(1, 1, 32, 8, 128, 1, 2 ** 30 + 1) == 0
    # one wave of warps, whatever the batch and its lengths
    assert ws(256, 256, 32, 8, 128, 1, 131072) - ws(1, 1, 32, 8, 128, 1, 16) <= 4096
    # the bound of the queries counts up to their number
    assert ws(4, 20, 32, 8, 128, 100, 5000) == ws(4, 20, 32, 8, 128, 20, 5000)


def verify(pk, **kw):
    a = dict(out=OK, acc=OK, rej=OK, tp=OK, ts=1000, rows=10, dp=OK, ds=1000, dt=OK, u=OK, qs=OK, S=2, K=4, V=1000)
    a.update(kw)
    return pk.lib().pa_verify_drafts(*a.values(), None, None)


@pytest.mark.parametrize("kw", [dict(S=-1), dict(K=-1), dict(V=0), dict(rows=-1), dict(ts=999), dict(ds=999), dict(out=None), dict(acc=None),
                                dict(tp=None), dict(dt=None), dict(u=None), dict(qs=None), dict(out=FOUR), dict(dt=FOUR), dict(acc=HALF),
                                dict(rej=HALF), dict(tp=HALF), dict(dp=HALF), dict(u=HALF), dict(qs=HALF)])
def test_verify_invalid(pk, kw):
    assert verify(pk, **kw) == pk.PA_ERR_INVALID_ARG


def test_verify_unsupported(pk):
    assert verify(pk, V=2 ** 22 + 1, ts=2 ** 23, ds=2 ** 23) == verify(pk, S=65536) == verify(pk, K=65536) == pk.PA_ERR_UNSUPPORTED


def test_no_work_is_no_launch(pk):
    assert append(pk, S=0, k=None, v=None, kc=None, vc=None, ksc=None, vsc=None, bt=None, len=None) == pk.PA_OK
    assert append(pk, T=0) == append(pk, most=0) == pk.PA_OK
    assert attention(pk, T=0, out=None, q=None) == pk.PA_OK
    assert verify(pk, S=0, out=None, acc=None, u=None, qs=None) == pk.PA_OK


def test_integer_codes_belong_to_the_scaled_calls(pk):
    L, i8 = pk.lib(), pk.PA_INT8
    assert L.pa_reshape_and_cache(OK, OK, OK, OK, OK, 4, 8, 128, 16, 10, pk.PA_BF16, i8, 1.0, 1.0, None, None) == pk.PA_ERR_INVALID_ARG
    assert L.pa_decode(OK, OK, OK, OK, OK, 4, OK, 2, 8, 8, 128, 16, 10, 64, 0.1, pk.PA_BF16, i8, 1.0, 1.0, None, None) == pk.PA_ERR_INVALID_ARG


def test_the_binding_refuses_what_is_not_on_a_device(pk):
    import torch
    t = lambda *s, d=torch.int32: torch.zeros(*s, dtype=d)  # noqa: E731
    with pytest.raises(ValueError):
        pk.extend_tables(t(2, 4), t(2), t(2), t(8), t(1), t(4, d=torch.int64), t(3), 16)
    with pytest.raises(ValueError):
        pk.trim_tables(t(2, 4), t(2), t(2), t(8), t(1), 16)
    x = torch.zeros(2, 2, 64)
    c = t(4, 2, 16, 64, d=torch.int8)
    with pytest.raises(ValueError):
        pk.scaled_append(x, x, c, c, torch.zeros(4, 2), torch.zeros(4, 2), t(2, 4), t(2))
    with pytest.raises(ValueError):
        pk.scaled_attention(x, x, c, c, torch.zeros(4, 2), torch.zeros(4, 2), t(2, 4), t(2), 16, 0.1, None)
    with pytest.raises(ValueError):
        pk.verify_drafts(t(2, 2, d=torch.int64), t(2), torch.zeros(4, 8), t(2, 1, d=torch.int64), torch.zeros(2, 2), t(3))
    with pytest.raises(TypeError):
        pk.verify_drafts(None, t(2), torch.zeros(4, 8), t(2, 1, d=torch.int64), torch.zeros(2, 2), t(3))
