"""CPU checks of the attention-side entry points: bad arguments are refused on
the host with the documented codes, and empty calls launch nothing."""
import ctypes

import pytest

import sharded_gemm_gb300 as tp
from sharded_gemm_gb300 import build as tpbuild

FAKE = 0x10000  # a non-null, aligned address that is never dereferenced


@pytest.fixture(scope="module")
def L():
    tpbuild.build()
    return tp.lib()


def _arr(n, v=FAKE):
    a = (ctypes.c_void_p * n)(*([v] * n))
    return ctypes.cast(a, ctypes.POINTER(ctypes.c_void_p)), a


def _append(L, **kw):
    p, _ = _arr(2)
    d = dict(N=2, qkv=p, T=4, ld=16 * 64, in_dt=tp.TP_BF16, Hq=8, Hk=4, D=64, qn=None, kn=None, eps=1e-6, rope=FAKE,
             rows=10, rot=64, inter=0, pos=FAKE, slots=FAKE, q=p, ldq=512, kc=p, vc=p, pages=4, page=16,
             ldp=4 * 16 * 64, dt=tp.TP_BF16, stream=None)
    assert set(kw) <= set(d)
    d.update(kw)
    return L.tp_qkv_append(*d.values())


def _attn(L, prefill, **kw):
    p, _ = _arr(2)
    d = dict(N=2, q=p, T=3, ldq=512, Hq=8, Hk=4, D=64, kc=p, vc=p, pages=4, page=16, ldp=4 * 16 * 64, table=FAKE)
    if prefill:
        d.update(B=2)
    d.update(width=2, ldt=2)
    if prefill:
        d.update(cu=FAKE)
    d.update(lens=FAKE)
    if prefill:
        d.update(prefix=None)
    d.update(scale=0.125, cap=0.0, window=0, dt=tp.TP_BF16, o=p, ldo=512, stream=None)
    assert set(kw) <= set(d)
    d.update(kw)
    return (L.tp_paged_prefill if prefill else L.tp_paged_decode)(*d.values())


def _sample(L, **kw):
    d = dict(x=FAKE, B=2, V=10, ld=10, dt=tp.TP_F32, u=FAKE, t=None, k=None, p=None, m=None, tok=FAKE, lp=None,
             stream=None)
    assert set(kw) <= set(d)
    d.update(kw)
    return L.tp_sample(*d.values())


CACHE_REFUSALS = [
    (dict(N=0), tp.TP_ERR_INVALID_ARG), (dict(N=65), tp.TP_ERR_INVALID_ARG),
    (dict(dt=tp.TP_F32), tp.TP_ERR_INVALID_ARG), (dict(Hk=0), tp.TP_ERR_INVALID_ARG),
    (dict(Hk=3), tp.TP_ERR_NOT_DIVISIBLE), (dict(D=96), tp.TP_ERR_UNSUPPORTED),
    (dict(page=24), tp.TP_ERR_UNSUPPORTED), (dict(page=8), tp.TP_ERR_UNSUPPORTED),
    (dict(page=512), tp.TP_ERR_UNSUPPORTED), (dict(pages=-1), tp.TP_ERR_INVALID_ARG),
    (dict(ldp=4 * 16 * 64 - 64), tp.TP_ERR_INVALID_ARG), (dict(ldp=4 * 16 * 64 + 8), tp.TP_ERR_INVALID_ARG),
    (dict(kc=None), tp.TP_ERR_INVALID_ARG), (dict(vc=_arr(2, None)[0]), tp.TP_ERR_INVALID_ARG),
    (dict(kc=_arr(2, FAKE + 2)[0]), tp.TP_ERR_ALIGNMENT),
]


@pytest.mark.parametrize("kw,code", CACHE_REFUSALS + [
    (dict(T=-1), tp.TP_ERR_INVALID_ARG), (dict(in_dt=7), tp.TP_ERR_INVALID_ARG), (dict(eps=-1.0), tp.TP_ERR_INVALID_ARG),
    (dict(eps=float("nan")), tp.TP_ERR_INVALID_ARG),
    (dict(rot=24), tp.TP_ERR_UNSUPPORTED), (dict(rot=80), tp.TP_ERR_UNSUPPORTED), (dict(rows=0), tp.TP_ERR_INVALID_ARG),
    (dict(ld=1000), tp.TP_ERR_INVALID_ARG), (dict(ldq=500), tp.TP_ERR_INVALID_ARG),
    (dict(slots=None), tp.TP_ERR_INVALID_ARG), (dict(pos=None), tp.TP_ERR_INVALID_ARG),
    (dict(slots=FAKE + 4), tp.TP_ERR_ALIGNMENT), (dict(qkv=_arr(2, None)[0]), tp.TP_ERR_INVALID_ARG),
    (dict(qkv=_arr(2, FAKE + 1)[0]), tp.TP_ERR_ALIGNMENT), (dict(q=None), tp.TP_ERR_INVALID_ARG)])
def test_append_refusals(L, kw, code):
    assert _append(L, **kw) == code
    assert tp.tp_last_error()


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("kw,code", CACHE_REFUSALS + [
    (dict(T=-1), tp.TP_ERR_INVALID_ARG), (dict(scale=0.0), tp.TP_ERR_INVALID_ARG),
    (dict(scale=float("nan")), tp.TP_ERR_INVALID_ARG), (dict(scale=float("inf")), tp.TP_ERR_INVALID_ARG),
    (dict(cap=-1.0), tp.TP_ERR_INVALID_ARG), (dict(cap=float("nan")), tp.TP_ERR_INVALID_ARG),
    (dict(window=-1), tp.TP_ERR_INVALID_ARG), (dict(ldt=1), tp.TP_ERR_INVALID_ARG),
    (dict(ldq=511), tp.TP_ERR_INVALID_ARG), (dict(ldo=511), tp.TP_ERR_INVALID_ARG),
    (dict(table=None), tp.TP_ERR_INVALID_ARG), (dict(lens=None), tp.TP_ERR_INVALID_ARG),
    (dict(lens=FAKE + 2), tp.TP_ERR_ALIGNMENT), (dict(o=_arr(2, FAKE + 1)[0]), tp.TP_ERR_ALIGNMENT)])
def test_attention_refusals(L, prefill, kw, code):
    assert _attn(L, prefill, **kw) == code
    assert tp.tp_last_error()


def test_prefill_refusals(L):
    assert _attn(L, True, cu=None) == tp.TP_ERR_INVALID_ARG
    assert _attn(L, True, cu=FAKE + 2) == tp.TP_ERR_ALIGNMENT
    assert _attn(L, True, prefix=FAKE + 2) == tp.TP_ERR_ALIGNMENT
    assert _attn(L, True, B=0) == tp.TP_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,code", [
    (dict(dt=9), tp.TP_ERR_INVALID_ARG), (dict(B=-1), tp.TP_ERR_INVALID_ARG), (dict(V=0), tp.TP_ERR_INVALID_ARG),
    (dict(V=(1 << 22) + 1, ld=1 << 23), tp.TP_ERR_UNSUPPORTED), (dict(ld=9), tp.TP_ERR_INVALID_ARG),
    (dict(x=None), tp.TP_ERR_INVALID_ARG), (dict(u=None), tp.TP_ERR_INVALID_ARG), (dict(tok=None), tp.TP_ERR_INVALID_ARG),
    (dict(tok=FAKE + 4), tp.TP_ERR_ALIGNMENT), (dict(x=FAKE + 2), tp.TP_ERR_ALIGNMENT),
    (dict(k=FAKE + 1), tp.TP_ERR_ALIGNMENT)])
def test_sample_refusals(L, kw, code):
    assert _sample(L, **kw) == code
    assert tp.tp_last_error()


def test_empty_calls_launch_nothing(L):
    before = L.tp_launch_count()
    assert _append(L, T=0) == tp.TP_OK
    assert _attn(L, False, T=0) == tp.TP_OK
    assert _attn(L, True, T=0, B=0) == tp.TP_OK
    assert _sample(L, B=0) == tp.TP_OK
    assert L.tp_launch_count() == before


@pytest.mark.parametrize("prefill", [False, True])
def test_attention_of_more_than_2_to_30_rows_is_refused(L, prefill):
    assert _attn(L, prefill, T=(1 << 30) + 1) == tp.TP_ERR_UNSUPPORTED
    assert tp.tp_last_error()


@pytest.mark.parametrize("heads", [dict(Hq=65534, Hk=1), dict(Hq=1 << 30, Hk=1 << 30), dict(Hq=(1 << 31) - 1, Hk=1),
                                   dict(Hq=65536, Hk=4)])
def test_too_many_heads_are_refused(L, heads):
    """Before any product of them is taken in 32 bits."""
    wide = dict(ldp=1 << 45)
    assert _append(L, ld=1 << 40, ldq=1 << 40, **heads, **wide) == tp.TP_ERR_UNSUPPORTED
    for prefill in (False, True):
        assert _attn(L, prefill, ldq=1 << 40, ldo=1 << 40, **heads, **wide) == tp.TP_ERR_UNSUPPORTED
