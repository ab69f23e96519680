"""CPU checks of the operators that serve many requests at once: bad arguments are refused on
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
    return ctypes.cast((ctypes.c_void_p * n)(*([v] * n)), ctypes.POINTER(ctypes.c_void_p))


def _of(fn, d, kw):
    assert set(kw) <= set(d)
    return fn(*{**d, **kw}.values())


def _plan(L, **kw):
    return _of(L.tp_paged_plan, dict(
        B=2, counts=FAKE, rejected=None, lens=FAKE, owned=FAKE, table=FAKE, width=4, ldt=4, pool=FAKE, pages=8, free=FAKE,
        page=16, T=4, nlens=FAKE, nowned=FAKE, nfree=FAKE, missing=FAKE, cu=FAKE, pos=FAKE, slots=FAKE, stream=None), kw)


def _groups(L, **kw):
    return _of(L.tp_lora_plan, dict(B=2, ids=FAKE, cu=FAKE, T=4, n=3, plan=FAKE, stream=None), kw)


def _column(L, **kw):
    size = L.tp_lora_plan_ints(kw.get("T", 4), kw.get("n", 3))
    return _of(L.tp_lora_all_to_sharded, dict(
        N=2, x=FAKE, T=4, K=64, ldx=64, a=FAKE, b=_arr(2), n=3, R=8, O=32, scales=None, plan=FAKE, size=size,
        ws=None, dt=tp.TP_BF16, y=_arr(2), ldy=16, out=_arr(2), ldo=16, odt=tp.TP_BF16, stream=None), kw)


def _row(L, **kw):
    size = L.tp_lora_plan_ints(kw.get("T", 4), kw.get("n", 3))
    return _of(L.tp_lora_sharded_to_all, dict(
        N=2, x=_arr(2), T=4, K=64, ldx=32, a=_arr(2), b=FAKE, n=3, R=8, O=32, scales=None, plan=FAKE, size=size,
        ws=None, dt=tp.TP_F16, y=FAKE, ldy=32, out=FAKE, ldo=32, odt=tp.TP_F32, stream=None), kw)


def _verify(L, **kw):
    return _of(L.tp_verify, dict(
        x=FAKE, T=6, V=10, ld=10, dt=tp.TP_F32, drafts=FAKE, q=FAKE, ldq=10, qdt=tp.TP_BF16, seqs=2, cu=FAKE, u=FAKE,
        t=None, k=None, p=None, m=None, tok=FAKE, lp=None, acc=None, rej=None, stream=None), kw)


BAD, ALIGN, UNSUP, DIV = tp.TP_ERR_INVALID_ARG, tp.TP_ERR_ALIGNMENT, tp.TP_ERR_UNSUPPORTED, tp.TP_ERR_NOT_DIVISIBLE


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), BAD), (dict(B=8193), UNSUP), (dict(T=-1), BAD), (dict(T=1 << 31), BAD), (dict(pages=-1), BAD),
    (dict(width=-1), BAD), (dict(page=24), UNSUP), (dict(page=8), UNSUP), (dict(page=512), UNSUP), (dict(ldt=3), BAD),
    (dict(counts=None), BAD), (dict(lens=None), BAD), (dict(owned=None), BAD), (dict(table=None), BAD),
    (dict(pool=None), BAD), (dict(free=None), BAD), (dict(nlens=None), BAD), (dict(nowned=None), BAD),
    (dict(nfree=None), BAD), (dict(missing=None), BAD), (dict(cu=None), BAD), (dict(pos=None), BAD),
    (dict(slots=None), BAD), (dict(slots=FAKE + 4), ALIGN), (dict(pos=FAKE + 2), ALIGN), (dict(rejected=FAKE + 1), ALIGN)])
def test_plan_refusals(L, kw, code):
    assert _plan(L, **kw) == code
    assert tp.tp_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), BAD), (dict(T=-1), BAD), (dict(n=0), BAD), (dict(n=16385), UNSUP), (dict(B=8193), UNSUP),
    (dict(cu=None), BAD), (dict(ids=None), BAD), (dict(plan=None), BAD), (dict(plan=FAKE + 4), ALIGN),
    (dict(ids=FAKE + 2), ALIGN), (dict(cu=FAKE + 2), ALIGN)])
def test_adapter_plan_refusals(L, kw, code):
    assert _groups(L, **kw) == code
    assert tp.tp_last_error()


BOTH = [(dict(N=0), BAD), (dict(N=65), BAD), (dict(T=-1), BAD), (dict(K=0), BAD), (dict(O=0), BAD), (dict(n=0), BAD),
        (dict(n=16385), UNSUP), (dict(R=0), BAD), (dict(R=129), UNSUP), (dict(dt=tp.TP_F32), BAD), (dict(odt=5), BAD),
        (dict(ldx=31), BAD), (dict(ldy=15), BAD), (dict(ldo=15), BAD), (dict(plan=None), BAD), (dict(plan=FAKE + 8), ALIGN),
        (dict(scales=FAKE + 2), ALIGN), (dict(size=4), BAD), (dict(ws=FAKE + 8), ALIGN), (dict(x=None), BAD), (dict(a=None), BAD), (dict(b=None), BAD),
        (dict(y=None), BAD), (dict(out=None), BAD)]


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(O=33), DIV), (dict(b=_arr(2, None)), BAD), (dict(x=FAKE + 1), ALIGN), (dict(y=_arr(2, FAKE + 1)), ALIGN),
    (dict(ldo=24), BAD)])  # out is y: one row stride
def test_column_adapter_refusals(L, kw, code):
    assert _column(L, **kw) == code
    assert tp.tp_last_error()


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(K=65), DIV), (dict(x=_arr(2, None)), BAD), (dict(a=_arr(2, FAKE + 1)), ALIGN), (dict(out=FAKE + 2), ALIGN)])
def test_row_adapter_refusals(L, kw, code):
    assert _row(L, **kw) == code
    assert tp.tp_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(dt=9), BAD), (dict(qdt=9), BAD), (dict(T=-1), BAD), (dict(V=0), BAD), (dict(seqs=-1), BAD), (dict(ld=9), BAD),
    (dict(ldq=9), BAD), (dict(V=417793, ld=1 << 20, ldq=1 << 20), UNSUP), (dict(T=1 << 30), UNSUP), (dict(x=None), BAD),
    (dict(drafts=None), BAD), (dict(cu=None), BAD), (dict(u=None), BAD), (dict(tok=None), BAD), (dict(tok=FAKE + 4), ALIGN),
    (dict(drafts=FAKE + 4), ALIGN), (dict(q=FAKE + 1), ALIGN), (dict(x=FAKE + 2), ALIGN), (dict(acc=FAKE + 2), ALIGN)])
def test_verify_refusals(L, kw, code):
    assert _verify(L, **kw) == code
    assert tp.tp_last_error()


def test_sizes_of_adapter_plans(L):
    assert L.tp_lora_plan_ints(0, 5) == 4
    assert L.tp_lora_plan_ints(3, 5) == 4 + 12 + 3
    assert L.tp_lora_plan_ints(100, 5) == 4 + 24 + 100


def test_sizes_of_adapter_workspaces(L):
    assert L.tp_lora_workspace_floats(1024, 16) == 0
    assert [L.tp_lora_workspace_floats(1025, r) for r in (1, 16, 17, 64, 65, 128)] == \
        [8 * 1025 * r for r in (16, 16, 32, 64, 128, 128)]
    assert [L.tp_lora_workspace_floats(t, 16) // (16 * t) for t in (4096, 4097, 8192, 8193, 16384, 16385)] == [8, 4, 4, 2, 2, 1]
    assert L.tp_lora_workspace_floats(2000, 129) == 0 and L.tp_lora_workspace_floats(-1, 8) == 0


def test_high_ranks_take_two_passes_earlier(L):
    assert [L.tp_lora_workspace_floats(512, r) for r in (64, 65, 128)] == [0, 0, 0]
    assert [L.tp_lora_workspace_floats(513, r) for r in (64, 65, 128)] == [0] + [8 * 513 * 128] * 2


def test_empty_calls_launch_nothing(L):
    before = L.tp_launch_count()
    assert _column(L, T=0) == tp.TP_OK
    assert _row(L, T=0) == tp.TP_OK
    assert _verify(L, T=0, seqs=0) == tp.TP_OK
    assert L.tp_launch_count() == before
