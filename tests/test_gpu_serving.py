"""GPU parity of the operators that serve many requests at once: the step's plan over a shared pool of
pages, the adapters beside the projections, the verification of drafted tokens, and all of them together.

Whole numbers have one right answer and are compared as such.  Tolerances of the adapters: with u the unit
roundoff of a type (2^-8 for bfloat16, 2^-11 for float16, 2^-24 for float32) an output is rounded once (u |out|).
The sum over x meets B as terms of the operands' type: one where the outputs have no more bits than it, which
loses at most its u of it; two of bfloat16 for float16 outputs, 2^-16 (8 + 8 bits); for float32 ones two of
float16, 2^-21 (11 + 11 bits, less what falls below the smallest), or three of bfloat16, 2^-22 and less.  The two
products are summed in float32, (K + R) adds of at most 2^-23 of the sum of their terms' sizes.
"""
import numpy as np
import pytest
import torch

import sharded_gemm_gb300 as tp
from sharded_gemm_gb300 import build as tpbuild
from sharded_gemm_gb300 import synth
from sharded_gemm_gb300.workloads import PagedServing, SharedServing
from gpu_util import check_close

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def built():
    tpbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    tp.tp_set_policy(tp.TP_POLICY_AUTO)


def status():
    torch.cuda.synchronize()
    return tp.tp_query_status()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def i32(a):
    return dev(np.asarray(a, np.int32))


# ------------------------------------------------------------------ the step's plan
def plan_ref(counts, rejected, lens, owned, table, pool, free, page, T):
    """The definition, one sequence and one page after the other: (lens, owned, free, missing, cu, positions,
    slots, table, pool)."""
    table, pool = [list(r) for r in table], list(pool)
    B, width, pages = len(counts), len(table[0]) if len(table) else 0, len(pool)
    cap = min(width * page, 1 << 30)
    empty = (list(lens), list(owned), free, [0] * (B + 1), [0] * T, [-1] * T, table, pool)

    def given_up(missing):
        return (*empty[:3], missing, *empty[3:])
    bad = free < 0 or free > pages or sum(max(c, 0) for c in counts) > T
    need = back = 0
    for b in range(B):
        own = owned[b]
        if own < 0 or own > width:
            bad = True
        elif counts[b] < 0:
            back += own
        else:
            end = lens[b] - rejected[b] + counts[b]
            if lens[b] < 0 or rejected[b] < 0 or rejected[b] > lens[b] or end > cap or own * page < lens[b] - rejected[b]:
                bad = True
            need += max(0, -(-end // page) - own)
    if bad or free + back > pages:
        return given_up(-1)
    if need > free + back:
        return given_up(need - free - back)
    for b in range(B):
        if counts[b] < 0:
            for j in range(owned[b]):
                pool[free] = table[b][j]
                free += 1
    lens2, owned2, cu, positions, slots = [], [], [0], [], []
    for b in range(B):
        if counts[b] < 0:
            lens2.append(0), owned2.append(0), cu.append(cu[-1])
            continue
        start, own = lens[b] - rejected[b], owned[b]
        end = start + counts[b]
        while own * page < end:
            free -= 1
            table[b][own] = pool[free]
            own += 1
        for i in range(start, end):
            positions.append(i)
            p = table[b][i // page]
            slots.append(p * page + i % page if 0 <= p < pages else -1)
        lens2.append(end), owned2.append(own), cu.append(cu[-1] + counts[b])
    pad = T - len(positions)
    return lens2, owned2, free, 0, cu, positions + [0] * pad, slots + [-1] * pad, table, pool


def run_plan(counts, rejected, lens, owned, table, pool, free, page, T, in_place=False, stream=None):
    t = i32(table)
    args = [i32(counts), i32(lens), i32(owned), t, i32(pool), i32([free])]
    less = None if rejected is None else i32(rejected)
    torch.cuda.synchronize()
    out = None
    if in_place:
        out = [args[1], args[2], args[5], torch.empty(1, dtype=torch.int32, device="cuda"),
               torch.empty(len(counts) + 1, dtype=torch.int32, device="cuda"),
               torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(T, dtype=torch.int64, device="cuda")]
    p = tp.tp_paged_plan(*args, page, T, rejected=less, out=out, stream=stream)
    torch.cuda.synchronize()
    return (p.seq_lens.tolist(), p.owned.tolist(), int(p.free_count), int(p.missing), p.cu_seqlens.tolist(),
            p.positions.tolist(), p.slots.tolist(), t.tolist(), args[4].tolist())


def some_step(B, page, hi, most, ends, seed, short=False, rejects=True):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, hi + 1, B)
    counts = rng.integers(0, most + 1, B)
    back = np.minimum(rng.integers(0, 5, B), lens) if rejects else np.zeros(B, int)
    held = -(-lens // page)
    ended = rng.random(B) < ends
    need = np.where(ended, 0, np.maximum(0, -(-(lens - back + counts) // page) - held))
    width = max(1, -(-(hi + most) // page))
    total = int(need.sum())
    spare = max(0, total - int(held[ended].sum()) - 1) if short else total + 3
    pages = int(held.sum()) + spare
    names = rng.permutation(pages)
    table = np.full((B, width), -1)
    table[np.arange(width)[None] < held[:, None]] = names[:held.sum()]
    pool = np.full(pages, -1)
    pool[:spare] = names[held.sum():]
    counts = np.where(ended, -1 - rng.integers(0, 3, B), counts)
    T = int(np.maximum(counts, 0).sum()) + seed % 4
    return (counts.tolist(), back.tolist(), lens.tolist(), held.tolist(), table.tolist(), pool.tolist(), spare, page, T)


@pytest.mark.parametrize("B,page,hi,most,ends", [
    (1, 16, 0, 1, 0.0), (1, 16, 40, 1, 0.0), (3, 16, 31, 5, 0.0), (33, 32, 100, 8, 0.2), (256, 16, 700, 8, 0.1),
    (1023, 16, 50, 2, 0.3), (1025, 64, 300, 1, 0.1), (40, 128, 1000, 600, 0.1), (70, 16, 300, 300, 0.4),
    (8192, 16, 20, 1, 0.2), (5, 256, 3000, 4000, 0.0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(B, page, hi, most, ends, in_place):
    for seed in range(3):
        step = some_step(B, page, hi, most, ends, seed)
        assert run_plan(*step, in_place=in_place) == plan_ref(*step)
    assert status() == 0


@pytest.mark.parametrize("B,most", [(4, 40), (300, 3), (64, 200)])
def test_plan_without_enough_pages_is_empty(B, most):
    steps = (some_step(B, 16, 100, most, 0.0, seed, short=True) for seed in range(5, 50))
    step = next(s for s in steps if plan_ref(*s)[3] > 0)
    ref = plan_ref(*step)
    assert run_plan(*step) == ref and run_plan(*step, in_place=True) == ref
    assert status() == 0  # the caller is told by `missing`


def test_plan_takes_the_last_page_and_pages_given_back_just_now():
    # 0 ends and gives back 5, 6; 1 needs two pages: 6 and 5; the pool of one page keeps it
    step = ([-1, 20], [0, 0], [32, 0], [2, 0], [[5, 6], [-1, -1]], [3, -1, -1, -1, -1, -1, -1], 1, 16, 20)
    got = run_plan(*step)
    assert got == plan_ref(*step)
    assert got[1] == [0, 2] and got[2] == 1 and got[7][1] == [6, 5]
    # the same with an empty pool and exactly what is needed
    step = ([-1, 20], [0, 0], [32, 0], [2, 0], [[5, 6], [-1, -1]], [-1] * 7, 0, 16, 20)
    assert run_plan(*step)[2:4] == (0, 0)
    assert status() == 0


def test_plan_rejected_tokens_keep_their_pages():
    # 17 positions on two pages, two refused: the next token is position 15, on a page held already
    step = ([3], [2], [17], [2], [[4, 9, -1]], list(range(12)), 2, 16, 3)
    got = run_plan(*step)
    assert got == plan_ref(*step)
    assert got[5] == [15, 16, 17] and got[6] == [4 * 16 + 15, 9 * 16, 9 * 16 + 1] and got[2] == 2


@pytest.mark.parametrize("change", [
    dict(lens=[-1, 3]), dict(rejected=[4, 0]), dict(rejected=[-1, 0]), dict(owned=[-1, 1]), dict(owned=[5, 1]),
    dict(counts=[62, 1]), dict(counts=[2 ** 31 - 1, 2 ** 31 - 1]), dict(owned=[0, 1]), dict(free=-1), dict(free=9),
    dict(T=3), dict(counts=[-1, 1], free=8)])
def test_plan_of_values_out_of_range_is_empty_and_recorded(change):
    step = dict(counts=[2, 3], rejected=[0, 0], lens=[3, 16], owned=[1, 1], table=[[1, -1, -1, -1], [2, -1, -1, -1]],
                pool=[0, 3, 4, 5, 6, 7, -1, -1], free=6, page=16, T=8)
    assert plan_ref(*step.values())[3] == 0
    step.update(change)
    ref = plan_ref(*step.values())
    assert ref[3] == -1
    assert run_plan(*step.values()) == ref
    assert status() == tp.TP_ERR_INVALID_ARG


def test_plan_page_numbers_out_of_range_give_no_slot():
    step = ([2, 1], [0, 0], [15, 0], [1, 0], [[70000, -1], [-1, -1]], [3, 2, -9], 3, 16, 4)
    ref = plan_ref(*step)
    assert ref[6] == [-1, -1, 2 * 16, -1]
    assert run_plan(*step) == ref
    assert status() == tp.TP_ERR_INVALID_ARG


def test_plan_of_no_sequences():
    got = run_plan([], None, [], [], np.zeros((0, 3)), [0, 1], 2, 16, 3)
    assert got == ([], [], 2, 0, [0], [0] * 3, [-1] * 3, [], [0, 1])
    assert status() == 0


# ------------------------------------------------------------------ tokens by adapter
def groups_ref(ids, cu, T, n):
    """The plan's values."""
    kind = [-2] * T
    for b, i in enumerate(ids):
        for t in range(cu[b], cu[b + 1]):
            kind[t] = i if 0 <= i < n else -1
    order, groups = [], []
    for i in [*range(n), -1]:
        mine = [t for t in range(T) if kind[t] == i]
        if mine:
            groups.append((i, len(order), len(mine), 0))
        order += mine
    most = min(T, n + 1)
    head = [len(groups), sum(g[2] for g in groups if g[0] >= 0), 0, 0]
    return head + [v for g in groups for v in g] + [-1] * (4 * (most - len(groups))) + order + [-1] * (T - len(order))


@pytest.mark.parametrize("B,most,n", [(1, 1, 1), (1, 9, 4), (5, 4, 3), (64, 1, 200), (100, 3, 7), (1000, 2, 33),
                                      (1025, 9, 1000), (8192, 1, 16384), (30, 400, 5)])
def test_adapter_plan(B, most, n):
    rng = np.random.default_rng(B + n)
    for pad in (0, 3):
        ids = rng.integers(-1, n, B)
        lens = rng.integers(0, most + 1, B) if most > 1 else np.ones(B, int)
        cu = np.concatenate([[0], np.cumsum(lens)])
        T = int(cu[-1]) + pad
        got = tp.tp_lora_plan(i32(ids), T, n, cu_seqlens=i32(cu))
        assert got.tolist() == groups_ref(ids.tolist(), cu.tolist(), T, n)
        if most == 1:
            assert tp.tp_lora_plan(i32(ids), B, n).tolist() == groups_ref(ids.tolist(), cu.tolist(), B, n)
    assert status() == 0


def test_adapter_plan_of_bad_values():
    got = tp.tp_lora_plan(i32([1, 5, -7]), 3, 2)  # an adapter there is none of: none
    assert got.tolist() == groups_ref([1, -1, -1], [0, 1, 2, 3], 3, 2)
    assert status() == tp.TP_ERR_INVALID_ARG
    for cu in ([0, 3, 2, 4], [0, 1, 2, 9], [1, 2, 3, 4], [-1, 0, 1, 2]):
        got = tp.tp_lora_plan(i32([0, 1, 0]), 4, 2, cu_seqlens=i32(cu))
        assert got.tolist() == [0] * 4 + [-1] * 12 + [-1] * 4
        assert status() == tp.TP_ERR_INVALID_ARG


# ------------------------------------------------------------------ the adapters
def lora_ref(x, a, b, ids, scales, y):
    """(outputs, sizes of what was summed) in float64, per rank; ids per token, -2: no sequence's."""
    x, a, b = ([t.double() for t in v] for v in (x, a, b))
    out, big = [t.double().clone() for t in y], [torch.zeros_like(t, dtype=torch.float64) for t in y]
    for i in set(ids.tolist()) - {-1, -2}:
        rows = (ids == i).nonzero()[:, 0]
        s = 1.0 if scales is None else float(scales[i])
        h = s * sum(xr[rows] @ ar[i].T for xr, ar in zip(x, a))
        hb = abs(s) * sum(xr[rows].abs() @ ar[i].abs().T for xr, ar in zip(x, a))
        for r in range(len(b)):
            out[r][rows] += h @ b[r][i].T
            big[r][rows] += hb @ b[r][i].abs().T
    return out, big


def check_lora(got, x, a, b, ids, scales, y, dt):
    ref, big = lora_ref(x, a, b, ids, scales, y)
    K, R = sum(t.shape[1] for t in x), a[0].shape[1]
    if got[0].dtype == F32:
        lost = 2.0 ** -22 if dt == BF16 else 2.0 ** -20
    else:
        lost = 2.0 ** -16 if dt == BF16 and got[0].dtype == F16 else U[dt]
    lost += (K + R) * 2.0 ** -23
    live = ids > -2
    for g, f, s, start in zip(got, ref, big, y):
        assert torch.equal(g[~live], start[~live])
        d = (g.double() - f).abs()[live]
        tol = (U[g.dtype] * f.abs() + lost * s)[live] + 2.0 ** -24
        assert (d <= tol).all(), float((d / tol).max())
        none = ids == -1
        assert torch.equal(g[none], start[none])


def lora_data(form, T, N, K, O, R, n, dt, out_dt, seed, some_without=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nx, ny = (N, 1) if form == "row" else (1, N)

    def normal(shape, std, d):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(d)
    x = [normal((T, K // nx), 1, dt) for _ in range(nx)]
    a = [normal((n, R, K // nx), K ** -0.5, dt) for _ in range(nx)]
    b = [normal((n, O // ny, R), R ** -0.5, dt) for _ in range(ny)]
    y = [normal((T, O // ny), 1, out_dt) for _ in range(ny)]
    scales = torch.rand(n, generator=g, device="cuda") * 2
    return x, a, b, y, scales


def call_lora(form, x, a, b, plan, y, **kw):
    if form == "column":
        return tp.tp_lora_all_to_sharded(x[0], a[0], b, plan, y, **kw)
    out = kw.pop("out", None)
    return [tp.tp_lora_sharded_to_all(x, a, b[0], plan, y[0], out=None if out is None else out[0], **kw)]


@pytest.fixture(params=[tp.TP_POLICY_AUTO, tp.TP_POLICY_SIMT], ids=["auto", "simt"])
def policy(request):
    tp.tp_set_policy(request.param)
    yield request.param
    tp.tp_set_policy(tp.TP_POLICY_AUTO)


@pytest.mark.parametrize("form", ["column", "row"])
@pytest.mark.parametrize("T,N,K,O,R,n,dt,out_dt", [
    (1, 1, 64, 64, 16, 1, BF16, BF16), (1, 8, 4096, 4096, 16, 3, BF16, F32), (3, 2, 96, 40, 8, 2, F16, F16),
    (17, 4, 512, 256, 4, 20, BF16, BF16), (64, 1, 1000, 333, 16, 64, BF16, F32), (33, 3, 333, 99, 5, 4, F16, BF16),
    (100, 2, 2048, 1024, 64, 7, F16, F32), (50, 8, 640, 128, 128, 5, BF16, F16), (40, 1, 72, 200, 33, 3, BF16, BF16),
    (1025, 2, 256, 320, 32, 9, BF16, BF16), (1500, 4, 128, 96, 16, 3, F16, F32), (1100, 1, 520, 72, 128, 2, BF16, F32),
    (2000, 1, 100, 64, 64, 1, F16, BF16), (1030, 2, 30, 10, 1, 50, BF16, F32)])
def test_adapters(policy, form, T, N, K, O, R, n, dt, out_dt):
    if (K if form == "row" else O) % N:
        K, O = -(-K // N) * N, -(-O // N) * N
    x, a, b, y, scales = lora_data(form, T, N, K, O, R, n, dt, out_dt, T + R)
    rng = np.random.default_rng(T)
    for pad, s, in_place in ((0, None, False), (min(5, T - 1), scales, True)):
        ids = rng.integers(-1, n, T)
        ids[T - pad:] = -2
        plan = tp.tp_lora_plan(i32(ids[:T - pad]), T, n, cu_seqlens=i32(np.arange(T - pad + 1)))
        y0 = [t.clone() for t in y]
        if in_place:
            got = call_lora(form, x, a, b, plan, y, scales=s)
            assert all(p.data_ptr() == t.data_ptr() for p, t in zip(got, y))
        else:
            out = [torch.full_like(t, 7) for t in y]
            got = call_lora(form, x, a, b, plan, y, scales=s, out=out)
            assert all(torch.equal(p, t) for p, t in zip(y, y0))
        check_lora(got, x, a, b, dev(ids), s, y0, dt)
    assert status() == 0


@pytest.mark.parametrize("R,dt,out_dt", [(16, BF16, BF16), (16, F16, F32), (32, BF16, F32), (64, F16, F16),
                                         (64, BF16, F32), (100, BF16, F16), (128, F16, F32)])
@pytest.mark.parametrize("T,n,most", [(70, 60, 60), (150, 140, 140), (300, 200, 200), (512, 2000, 2000),
                                      (1024, 900, 900), (400, 300, 3), (500, 120, 30), (200, 256, 1)])
def test_adapters_of_many_requests(T, n, most, R, dt, out_dt):
    """Tiles from fewer than clusters that run at once to many times as many, of `most` of n adapters."""
    K, O, form, N = (328, 264, "column", 1) if T % 100 else (512, 320, "row", 2)
    x, a, b, y, scales = lora_data(form, T, N, K, O, R, n, dt, out_dt, T + R)
    rng = np.random.default_rng(T)
    for pad, s, in_place in ((0, scales, False), (7, None, True)):
        ids = rng.integers(-1, most, T) * (n // most)
        ids[ids < 0] = -1
        ids[T - pad:] = -2
        plan = tp.tp_lora_plan(i32(ids[:T - pad]), T, n, cu_seqlens=i32(np.arange(T - pad + 1)))
        y0 = [t.clone() for t in y]
        got = call_lora(form, x, a, b, plan, y, scales=s, out=None if in_place else [torch.full_like(t, 7) for t in y])
        # (rows of no sequence are left as they were)
        check_lora(got, x, a, b, dev(ids), s, y0, dt)
        again = [t.clone() for t in y0]
        again = call_lora(form, x, a, b, plan, again, scales=s, out=None if in_place else [torch.full_like(t, 7) for t in y])
        assert all(torch.equal(p, q) for p, q in zip(got, again))
    assert status() == 0


@pytest.mark.parametrize("R,dt,out_dt", [(16, BF16, F32), (16, F16, F16), (32, BF16, BF16), (64, BF16, F16), (64, F16, F32),
                                         (128, BF16, BF16), (128, F16, F32)])
@pytest.mark.parametrize("lens", [[600] + [1, 2] * 200, [31, 32, 33, 15, 16, 17, 63, 64, 65, 47, 48, 49, 127, 128, 129, 500],
                                  [1] * 1100])
def test_adapters_of_prompts_beside_many_requests(lens, R, dt, out_dt):
    """Tiles of one to all blocks of tokens in one step of two passes."""
    n, T, K, O = len(lens), sum(lens), 520, 264
    x, a, b, y, scales = lora_data("column", T, 2, K, O, R, n, dt, out_dt, T + R)
    ids = np.random.default_rng(R).permutation(n)
    plan = tp.tp_lora_plan(i32(ids), T, n, cu_seqlens=i32(np.concatenate([[0], np.cumsum(lens)])))
    got = call_lora("column", x, a, b, plan, y, scales=scales, out=[torch.full_like(t, 7) for t in y])
    check_lora(got, x, a, b, dev(np.repeat(ids, lens)), scales, y, dt)
    assert status() == 0


@pytest.mark.parametrize("T", [40, 1200])
@pytest.mark.parametrize("form", ["column", "row"])
def test_adapters_of_strided_and_unaligned_rows(form, T):
    """Rows with a stride, that begin at any element; outputs that are columns of one buffer."""
    N, K, O, R, n = 2, 256, 128, 16, 4
    x, a, b, y, s = lora_data(form, T, N, K, O, R, n, BF16, F32, 3)
    ids = np.random.default_rng(1).integers(-1, n, T)
    plan = tp.tp_lora_plan(i32(ids), T, n)
    for off in (0, 1):
        xs = []
        for t in x:
            wide = torch.zeros((T, t.shape[1] + 24), dtype=BF16, device="cuda")
            wide[:, off:off + t.shape[1]] = t
            xs.append(wide[:, off:off + t.shape[1]])
        cols = y[0].shape[1]
        one = torch.full((T, cols * len(y) + 8), 9.0, device="cuda")
        out = [one[:, off + r * cols:off + (r + 1) * cols] for r in range(len(y))]
        got = call_lora(form, xs, a, b, plan, y, scales=s, out=out)
        check_lora(got, x, a, b, dev(ids), s, y, BF16)
        assert bool((one[:, :off] == 9).all()) and bool((one[:, off + cols * len(y):] == 9).all())
    assert status() == 0


def test_adapters_give_the_same_bytes_again_and_alone():
    """Twice the same, and a token's outputs do not depend on the tokens beside it."""
    T, N, K, O, R, n = 200, 2, 1024, 512, 16, 5
    x, a, b, y, s = lora_data("column", T, N, K, O, R, n, BF16, BF16, 8)
    ids = np.random.default_rng(2).integers(0, n, T)
    plan = tp.tp_lora_plan(i32(ids), T, n)
    outs = [call_lora("column", x, a, b, plan, y, scales=s, out=[torch.empty_like(t) for t in y]) for _ in range(2)]
    assert all(torch.equal(p, q) for p, q in zip(*outs))
    for t in (0, 77, 199):
        alone = tp.tp_lora_plan(i32(ids[t:t + 1]), 1, n)
        got = call_lora("column", [x[0][t:t + 1]], a, b, alone, [v[t:t + 1] for v in y], scales=s,
                        out=[torch.empty_like(v[t:t + 1]) for v in y])
        assert all(torch.equal(g[0], o[t]) for g, o in zip(got, outs[0]))


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("T", [30, 1100])
def test_adapters_not_finite_and_extreme(dt, T):
    """What is not finite stays in its token and its adapter; sizes from one end of the type to the other."""
    K, O, R, n = 128, 64, 16, 3
    x, a, b, y, _ = lora_data("column", T, 1, K, O, R, n, dt, F32, 4)
    ids = np.arange(T) % n
    ids[9] = 0
    big = 2.0 ** 60 if dt == BF16 else 6e4
    for t, v in ((3, big), (4, 1 / big), (6, 2.0 ** -20)):
        x[0][t] = (x[0][t].float() * v).to(dt).clamp(-6e4 if dt == F16 else -big * 8, 6e4 if dt == F16 else big * 8)
    plan = tp.tp_lora_plan(i32(ids), T, n)
    clean = call_lora("column", x, a, b, plan, y, out=[torch.empty_like(t) for t in y])
    check_lora(clean, x, a, b, dev(ids), None, y, dt)
    x2, a2 = [x[0].clone()], [a[0].clone()]
    x2[0][9, 5] = float("nan")
    x2[0][12, 7] = float("inf")
    a2[0][1, 3, 2] = float("nan")
    got = call_lora("column", x2, a2, b, plan, y, out=[torch.empty_like(t) for t in y])[0]
    assert torch.isnan(got[9]).all() and not torch.isfinite(got[12]).any()
    assert torch.isnan(got[dev(ids == 1)]).all()
    same = dev((ids != 1) & (np.arange(T) != 9) & (np.arange(T) != 12))
    assert torch.equal(got[same], clean[0][same])


def test_adapters_infinite_sums():
    """An infinite sum gives infinite outputs of its sign, as in float32, not NaN."""
    x = torch.ones((2, 32), dtype=BF16, device="cuda")
    x[1, 0] = float("inf")
    a = torch.ones((1, 16, 32), dtype=BF16, device="cuda")
    b = torch.ones((1, 24, 16), dtype=BF16, device="cuda")
    b[0, 1::2] = -1
    y = torch.zeros((2, 24), device="cuda")
    got = tp.tp_lora_all_to_sharded(x, a, [b], tp.tp_lora_plan(i32([0, 0]), 2, 1), [y])[0]
    assert got[0, 0] == 512 and got[0, 1] == -512
    assert (got[1, 0::2] == float("inf")).all() and (got[1, 1::2] == -float("inf")).all()


def test_adapters_of_plans_that_are_none():
    """Values that no plan holds are recorded; nothing outside the tensors is touched."""
    T, n = 8, 2
    x, a, b, y, _ = lora_data("column", T, 1, 64, 64, 16, n, BF16, F32, 4)
    good = tp.tp_lora_plan(i32([0, 1, 0, 1, 0, 1, -1, 0]), T, n)
    for at, v in ((0, 1000), (0, -3), (4, 7), (5, -1), (5, 9), (6, 100), (6, -2), (4 + 4 * 3, 8), (4 + 4 * 3 + 2, -5)):
        bad = good.clone()
        bad[at] = v
        call_lora("column", x, a, b, bad, y, out=[torch.empty_like(t) for t in y])
        assert status() == tp.TP_ERR_INVALID_ARG, (at, v)


def test_adapters_of_many_plans_that_are_none():
    """The same where the plan says how many CTAs take a tile."""
    T, n = 300, 250
    x, a, b, y, _ = lora_data("column", T, 1, 64, 64, 16, n, BF16, F32, 4)
    good = tp.tp_lora_plan(i32(np.arange(T) % n), T, n)
    order = 4 + 4 * (n + 1)
    for at, v in ((0, 1000), (0, -3), (4, 251), (4 + 4 * 200, 250), (5, -1), (5, 500), (6, 1000), (6, -2), (order + 3, 300),
                  (order + 299, -5)):
        bad = good.clone()
        bad[at] = v
        call_lora("column", x, a, b, bad, y, out=[torch.empty_like(t) for t in y])
        assert status() == tp.TP_ERR_INVALID_ARG, (at, v)


# ------------------------------------------------------------------ verification
def part(total, share):
    return (int(total) * int(share)) >> 24


def f32(v):
    return np.float32(v)


def verify_ref(logits, drafts, cu, u, q=None, temperature=None, top_k=None, top_p=None, min_p=None):
    """The definition with whole numbers of any size: tokens, accepted, rejected, logprobs (float64)."""
    T, V = logits.shape
    x = logits.float()
    x = torch.where(torch.isnan(x), -torch.inf, x).clamp(max=float(np.finfo(np.float32).max)) + 0.0
    seq = torch.zeros(T, dtype=torch.long)
    for b in range(len(cu) - 1):
        seq[cu[b]:cu[b + 1]] = b
    t = np.ones(len(cu) - 1, np.float32) if temperature is None else temperature.cpu().numpy()
    greedy = ~(t >= np.float32(2.0 ** -20))
    inv = torch.ones_like(torch.from_numpy(t)).cuda()
    inv = torch.where(dev(greedy), inv, 1.0 / dev(np.minimum(t, np.finfo(np.float32).max)))
    top = x.amax(1, keepdim=True)
    e_all = torch.exp((x - top) * inv[seq.cuda()][:, None]).cpu().numpy()  # the device's exponential
    xs, us = x.cpu().numpy(), u.cpu().numpy()
    qs = None if q is None else np.clip(np.nan_to_num(q.float().cpu().numpy(), nan=0.0, posinf=1.0, neginf=0.0), 0, 1)
    d_all = drafts.cpu().numpy()
    tokens, logprobs = np.full(T, -1), np.zeros(T)
    accepted, rejected = [], []
    for b in range(len(cu) - 1):
        r0, r1 = cu[b], cu[b + 1]
        accepted.append(0), rejected.append(0)
        for i in range(r0, r1):
            row = xs[i]
            if row.max() == -np.inf:
                logprobs[i], rejected[b] = -np.inf, r1 - 1 - i
                break
            e = e_all[i]
            w = [int(v) for v in np.floor(e.astype(np.float64) * 2.0 ** 40)]
            order = np.argsort(-row, kind="stable")
            k = 1 if greedy[b] else int(top_k[b]) if top_k is not None and 0 < int(top_k[b]) < V else V
            kept = list(order[:k])
            p = 1.0 if top_p is None else float(top_p[b])
            if p < 1 and not (greedy[b] or k == 1):
                cut, before, n = part(sum(w[j] for j in kept), int(f32(max(p, 0)) * f32(2 ** 24))), 0, 0
                for j in kept:
                    if n and before >= cut:
                        break
                    before, n = before + w[j], n + 1
                kept = kept[:n]
            m = 0.0 if min_p is None else float(min_p[b])
            m = min(m, 1.0) if m > 0 else 0.0
            kept = [j for j in kept if not e[j] < f32(m)]
            W = sum(w[j] for j in kept)
            s = f32(1) / (f32(W) * f32(2.0 ** -40))
            prob = np.zeros(V, np.float32)
            prob[kept] = e[kept] * s
            wk = np.zeros(V, object)
            wk[kept] = [w[j] for j in kept]
            d = int(d_all[i]) if i < r1 - 1 else -1
            z = np.log(np.sum(np.exp(row.astype(np.float64) - row.max())))
            if d >= 0:
                theirs = qs[i] if qs is not None else (np.arange(V) == d).astype(np.float32)
                ui = min(f32(us[i]), f32(1 - 2.0 ** -24)) if us[i] > 0 else f32(0)
                if ui * theirs[d] < prob[d]:
                    tokens[i], logprobs[i] = d, float(row[d]) - row.max() - z
                    accepted[b] += 1
                    continue
                rest = np.floor(np.maximum(prob - theirs, f32(0)).astype(np.float64) * 2.0 ** 40)
                if rest.sum() > 0:
                    wk = np.array([int(v) for v in rest], object)
            ul = us[r1 - 1]
            share = min(int(min(f32(ul), f32(1)) * f32(2 ** 24)), 2 ** 24 - 1) if ul > 0 else 0
            run, r = np.cumsum(wk), part(sum(wk), share)
            tokens[i] = int(np.argmax(run > r))
            logprobs[i] = float(row[tokens[i]]) - row.max() - z
            rejected[b] = r1 - 1 - i
            break
    return tokens, logprobs, accepted, rejected


def check_verify(got, ref):
    tokens, logprobs, accepted, rejected = got
    torch.cuda.synchronize()
    assert accepted.tolist() == ref[2]
    assert rejected.tolist() == ref[3]
    assert tokens.tolist() == ref[0].tolist()
    lp = logprobs.double().cpu().numpy()
    assert np.array_equal(np.isinf(lp), np.isinf(ref[1]))
    # float32 subtraction of logits, and a logarithm of a sum whose terms are 2^-20 off at most
    live = np.isfinite(lp)
    assert np.all(np.abs(lp[live] - ref[1][live]) <= 2.0 ** -18 * (1 + np.abs(ref[1][live])))


def drafted(B, lo, hi, V, dt, q_dt, seed, std=2.5, noise=0.7):
    """Logits, drafts of a nearby distribution, offsets, random numbers, the distribution."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    n = rng.integers(lo, hi + 1, B)
    cu = np.concatenate([[0], np.cumsum(n + 1)])
    T = int(cu[-1])
    x = torch.randn((T, V), generator=g, device="cuda") * std
    q = torch.softmax(x + noise * torch.randn((T, V), generator=g, device="cuda"), 1)
    pick = torch.rand((T, 1), generator=g, device="cuda", dtype=torch.float64)
    d = (q.double().cumsum(1) < pick).sum(1).clamp(max=V - 1)
    u = torch.rand(T, generator=g, device="cuda")
    return x.to(dt), d, cu.tolist(), u, None if q_dt is None else q.to(q_dt)


def settings_of(B, seed):
    rng = np.random.default_rng(seed)
    return dict(temperature=dev(rng.choice(np.float32([0, 0.3, 0.7, 1, 1, 1.5]), B)),
                top_k=i32(rng.choice([0, 0, 1, 2, 20, 700], B)), top_p=dev(rng.choice(np.float32([1, 0.999, 0.9, 0.5, 0], ), B)),
                min_p=dev(rng.choice(np.float32([0, 0, 0.05, 1]), B)))


@pytest.mark.parametrize("B,lo,hi,V,dt,q_dt", [
    (1, 0, 0, 1, F32, F32), (1, 4, 4, 50, F32, F32), (5, 0, 6, 1000, F32, None), (7, 1, 3, 4097, BF16, F32),
    (3, 2, 2, 50272, F32, BF16), (40, 0, 5, 333, F16, F16), (200, 1, 1, 30, F32, F32), (2, 1, 1, 60001, BF16, None),
    (1, 40, 40, 517, F32, F32)])
@pytest.mark.parametrize("filters", [False, True, "temperature"])
def test_verify(B, lo, hi, V, dt, q_dt, filters):
    x, d, cu, u, q = drafted(B, lo, hi, V, dt, q_dt, B + V)
    s = settings_of(B, V) if filters else {}
    if filters == "temperature":
        s = dict(temperature=s["temperature"])
    got = tp.tp_verify(x, d, i32(cu), u, draft_probs=q, **s)
    check_verify(got, verify_ref(x, d, cu, u, q, **s))
    assert status() == 0


@pytest.mark.parametrize("B,lo,hi", [(90, 0, 4), (200, 0, 1), (5, 60, 80), (1100, 0, 2), (1, 400, 400)])
def test_verify_more_rows_than_the_gpu_holds(B, lo, hi):
    """Rows are taken in another order, and those behind an ended one left out; the results keep their places."""
    V = 2000 if B == 90 else 100
    x, d, cu, u, q = drafted(B, lo, hi, V, F32, F32, B, noise=0.1 if hi > 50 else 0.7)
    for s in ({}, settings_of(B, 3), dict(temperature=settings_of(B, 4)["temperature"])):
        ref = verify_ref(x, d, cu, u, q, **s)
        for _ in range(3):
            check_verify(tp.tp_verify(x, d, i32(cu), u, draft_probs=q, **s), ref)
    assert status() == 0


def test_verify_more_long_rows_than_the_gpu_holds():
    x, d, cu, u, q = drafted(40, 1, 3, 60007, BF16, BF16, 7)
    for s in (settings_of(40, 5), dict(temperature=settings_of(40, 6)["temperature"])):
        check_verify(tp.tp_verify(x, d, i32(cu), u, draft_probs=q, **s), verify_ref(x, d, cu, u, q, **s))


def test_verify_without_filters_reads_rows_of_any_alignment():
    """Logits and probabilities whose rows begin at any element, and a vocabulary that ends inside a vector."""
    for V, dt, q_dt in ((1001, F32, F16), (1003, BF16, F32), (514, F16, BF16)):
        x, d, cu, u, q = drafted(30, 0, 3, V, dt, q_dt, V)
        T = len(d)
        ref = verify_ref(x, d, cu, u, q)
        for off in (0, 1, 2, 3):
            wide, wide_q = torch.zeros((T, V + 6), dtype=dt, device="cuda"), torch.zeros((T, V + 5), dtype=q_dt, device="cuda")
            wide[:, off:off + V], wide_q[:, off:off + V] = x, q
            check_verify(tp.tp_verify(wide[:, off:off + V], d, i32(cu), u, draft_probs=wide_q[:, off:off + V]), ref)
    assert status() == 0


def test_verify_many_rows_between_rows_of_none():
    """Rows in front of the first sequence and behind the last are left alone, in any order of the others."""
    x, d, _, u, q = drafted(100, 3, 3, 50, F32, F32, 2)
    cu = np.arange(5, 391, 4).tolist()
    keep = torch.full((len(d),), 77, dtype=torch.int64, device="cuda")
    got = tp.tp_verify(x, d, i32(cu), u, draft_probs=q, tokens=keep)
    ref = verify_ref(x, d, cu, u, q)
    assert got[0][:5].tolist() == [77] * 5 and got[0][cu[-1]:].tolist() == [77] * (400 - cu[-1])
    assert got[0][5:cu[-1]].tolist() == ref[0][5:cu[-1]].tolist()
    assert got[2].tolist() == ref[2] and got[3].tolist() == ref[3]


@pytest.mark.parametrize("C_rows", [1, 3])
def test_verify_long_rows_of_several_ctas(C_rows):
    x, d, cu, u, q = drafted(C_rows, 1, 2, 130003, F16, F16, 5, std=1.0)
    for s in ({}, settings_of(C_rows, 2)):
        check_verify(tp.tp_verify(x, d, i32(cu), u, draft_probs=q, **s), verify_ref(x, d, cu, u, q, **s))


def test_verify_strides_and_given_outputs():
    x, d, cu, u, q = drafted(6, 0, 3, 77, F32, F16, 9)
    T = len(d)
    wide, wide_q = torch.zeros((T, 100), device="cuda"), torch.zeros((T, 83), dtype=F16, device="cuda")
    wide[:, 3:80], wide_q[:, 1:78] = x, q
    out = [torch.empty(T, dtype=torch.int64, device="cuda"), torch.empty(T, device="cuda"),
           torch.empty(6, dtype=torch.int32, device="cuda"), torch.empty(6, dtype=torch.int32, device="cuda")]
    got = tp.tp_verify(wide[:, 3:80], d, i32(cu), u, draft_probs=wide_q[:, 1:78], tokens=out[0], logprobs=out[1],
                       accepted=out[2], rejected=out[3])
    assert all(a is b for a, b in zip(got, out))
    check_verify(got, verify_ref(x, d, cu, u, q))


def test_verify_borders():
    """Random numbers at both ends, drafts that are certain or impossible, nothing left over, no draft, equal logits."""
    V = 12
    x = torch.zeros((24, V), device="cuda")
    x[8:12, 3:] = -float("inf")
    x[12:14] = -float("inf")
    x[14:16, 5] = float("inf")
    x[16:18, 2] = float("nan")
    d = torch.tensor([0, 5, 11, 0, 3, -1, 4, 0, 1, 7, 2, 0, 3, 0, 5, 0, 2, 0, 9, 9, 9, 9, 9, 0], device="cuda")
    cu = [0, 4, 8, 12, 14, 16, 18, 24]
    u = torch.tensor([0, 0.999, 1.0, 0, 0, 0.5, 0, 0.999999, 0.5, 0, 0, 0.3, 0, 0.5, 0.9, 0.5, 0, 1.0, float("nan"), -1, 0,
                      0.01, 0.02, 2.0], device="cuda")
    q = torch.softmax(x.nan_to_num(0, 1, -50), 1)  # as the target itself: nothing left over
    q[20] = float("nan")
    q[21] = -1
    q[22] = float("inf")
    for probs in (q, None, torch.zeros_like(q), torch.ones_like(q)):
        check_verify(tp.tp_verify(x, d, i32(cu), u, draft_probs=probs), verify_ref(x, d, cu, u, probs))
        s = dict(temperature=dev(np.float32([0, 1, np.inf, 1, 1, 0.5, 1])), top_k=i32([0, 3, 2, 1, 0, 500, 4]),
                 top_p=dev(np.float32([1, 0.5, 1, 0, 0.9, 2, -1])), min_p=dev(np.float32([0, 1, 5, 0, 0.5, -1, 0])))
        check_verify(tp.tp_verify(x, d, i32(cu), u, draft_probs=probs, **s), verify_ref(x, d, cu, u, probs, **s))
        s = dict(temperature=s["temperature"])
        check_verify(tp.tp_verify(x, d, i32(cu), u, draft_probs=probs, **s), verify_ref(x, d, cu, u, probs, **s))
    assert status() == 0


def test_verify_empty_sequences_and_rows_of_none():
    x, d, _, u, q = drafted(4, 1, 1, 40, F32, F32, 2)
    cu = [0, 0, 3, 3, 5, 5]
    keep = torch.full((len(d),), 77, dtype=torch.int64, device="cuda")
    got = tp.tp_verify(x, d, i32(cu), u, draft_probs=q, tokens=keep)
    ref = verify_ref(x, d, cu, u, q)
    assert got[0][5:].tolist() == [77] * 3  # rows of no sequence are left alone
    assert got[0][:5].tolist() == ref[0][:5].tolist()
    assert got[2].tolist() == ref[2] and got[3].tolist() == ref[3]
    none = tp.tp_verify(x[:0], d[:0], i32([0, 0, 0]), u[:0])
    assert none[2].tolist() == [0, 0] and none[3].tolist() == [0, 0]
    assert status() == 0


def test_verify_bad_values_are_recorded():
    x, d, cu, u, q = drafted(3, 2, 2, 40, F32, F32, 2)
    bad = d.clone()
    bad[1] = 40
    got = tp.tp_verify(x, bad, i32(cu), u, draft_probs=q)
    assert status() == tp.TP_ERR_INVALID_ARG
    ended = d.clone()
    ended[1] = -1
    ref = verify_ref(x, ended, cu, u, q)
    assert got[0].tolist() == ref[0].tolist()
    for off in ([0, 3, 2, 9], [0, 3, 6, 10], [-1, 3, 6, 9]):
        got = tp.tp_verify(x, d, i32(off), u, draft_probs=q)
        assert status() == tp.TP_ERR_INVALID_ARG
        assert got[2].min() >= 0
    x, d, cu, u, q = drafted(100, 3, 3, 20, F32, F32, 2)
    for at, v in ((0, -4), (100, 401), (40, 10), (40, 390), (1, -1)):
        off = np.array(cu)
        off[at] = v
        tp.tp_verify(x, d, i32(off), u, draft_probs=q)
        assert status() == tp.TP_ERR_INVALID_ARG, (at, v)


@pytest.mark.parametrize("with_q", [True, False])
def test_verified_tokens_follow_the_target(with_q):
    """Whatever the draft is, the first token is distributed as the target says: 200000 sequences, 5 deviations."""
    V, B = 6, 200000
    logits = torch.tensor([0.5, -1.0, 2.0, 0.0, 1.0, -3.0], device="cuda")
    draft = torch.tensor([0.3, 0.25, 0.05, 0.2, 0.1, 0.1], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    d = torch.zeros((B, 2), dtype=torch.int64, device="cuda")
    d[:, 0] = torch.multinomial(draft, B, replacement=True, generator=g)
    if not with_q:
        d[:, 0] = 4
    u = torch.rand((B, 2), generator=g, device="cuda").flatten()
    x = logits.expand(2 * B, V).contiguous()
    q = draft.expand(2 * B, V).contiguous() if with_q else None
    tokens, _, accepted, _ = tp.tp_verify(x, d.flatten(), i32(np.arange(B + 1) * 2), u, draft_probs=q)
    p = torch.softmax(logits.double(), 0).cpu().numpy()
    seen = np.bincount(tokens.view(B, 2)[:, 0].cpu().numpy(), minlength=V) / B
    assert np.all(np.abs(seen - p) <= 5 * np.sqrt(p * (1 - p) / B))
    rate = np.minimum(p, draft.double().cpu().numpy()).sum() if with_q else p[4]
    assert abs(float(accepted.double().mean()) - rate) <= 5 * np.sqrt(rate * (1 - rate) / B)


# ------------------------------------------------------------------ all of them together
def embeddings(V, D, seed=11):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((V, D), generator=g, device="cuda").to(BF16)


def make_adapters(n, R, D, seed=5, size=0.05):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return (torch.randn(shape, generator=g, device="cuda") * size).to(BF16)
    return dict(qkv_a=normal(n, R, D), qkv_b=normal(n, 3 * D, R), o_a=normal(n, R, D), o_b=normal(n, D, R),
                scales=torch.rand(n, generator=g, device="cuda") + 0.5)


def padded(rows, x):
    out = torch.full((rows, x.shape[1]), float("nan"), dtype=BF16, device="cuda")
    out[:len(x)] = x
    return out


@pytest.mark.parametrize("N", [1, 2])
def test_shared_serving_is_paged_serving(N):
    """Without adapters and drafts the pool changes where rows lie and nothing else: the same bytes of steps whose
    rows are all used (the linears choose their kernels by the rows), and nearly the same of padded ones."""
    cfg = synth.qkv(seed=6, T=1, D=256, V=512, N=N)
    table = embeddings(512, 256)
    a, a2 = (PagedServing(cfg, heads=4, batch=3, capacity=96, page=16) for _ in range(2))
    b = SharedServing(cfg, heads=4, batch=3, pages=18, capacity=96, rows=40, page=16)
    c = SharedServing(cfg, heads=4, batch=3, pages=18, capacity=96, rows=40, page=16)
    ids = torch.randint(0, 512, (40,), generator=torch.Generator().manual_seed(1)).cuda()
    u = torch.tensor([0.2, 0.5, 0.9], device="cuda")
    for counts in ([30, 3, 7], [1, 38, 1], [5, 5, 30]):
        t0, y0 = a.step(table[ids], counts, u)
        t1, y1 = b.step(table[ids], i32(counts), u)
        assert torch.equal(y0, y1) and torch.equal(t0, t1)
    assert b.plan[0].tolist() == a.lens and int(b.plan[3]) == 0
    for counts in ([21, 5, 1], [2, 1, 9], [1, 1, 1]):
        T = sum(counts)
        _, y0 = a2.step(table[ids[:T]], counts, u)
        _, y1 = c.step(padded(40, table[ids[:T]]), i32(counts), u)
        check_close(y1[:T].cpu().numpy(), y0.cpu().numpy())
    # a sequence ends, another takes its place and its pages
    free, held = int(b.plan[2]), int(b.plan[1][0])
    b.step(padded(40, table[ids[:2]]), i32([-1, 1, 1]), u)
    assert int(b.plan[2]) == free + held
    _, y = b.step(table[ids], i32([38, 1, 1]), u)
    _, alone = PagedServing(cfg, heads=4, batch=1, capacity=96, page=16).step(table[ids[:38]], [38], u[:1])
    check_close(y[:38].cpu().numpy(), alone.cpu().numpy())
    assert status() == 0


def test_shared_serving_with_adapters_against_merged_weights():
    """An adapter beside a projection is the projection with the adapter's product added to its weight."""
    D, V, N, R, n = 256, 512, 2, 16, 3
    cfg = synth.qkv(seed=6, T=1, D=D, V=V, N=N)
    table, lora = embeddings(V, D), make_adapters(n, R, D)
    ids = torch.randint(0, V, (60,), generator=torch.Generator().manual_seed(1)).cuda()
    serve = SharedServing(cfg, heads=4, batch=3, pages=20, capacity=96, rows=64, page=16, adapters=lora)
    u = torch.full((3,), 0.5, device="cuda")
    adapter_ids = i32([2, -1, 0])
    _, y = serve.step(padded(64, table[ids[:50]]), i32([20, 13, 17]), u, adapter_ids=adapter_ids)
    start = 0
    for which, count in ((2, 20), (-1, 13), (0, 17)):
        merged = dict(cfg)
        if which >= 0:
            for w, a, b in (("w_qkv", "qkv_a", "qkv_b"), ("w_o", "o_a", "o_b")):
                full = torch.from_numpy(np.ascontiguousarray(cfg[w]).view(np.int16)).view(BF16).cuda().double()
                full = full + float(lora["scales"][which]) * lora[b][which].double() @ lora[a][which].double()
                merged[w] = full.to(BF16).cpu().view(torch.int16).numpy().view(np.uint16)
        alone = PagedServing(merged, heads=4, batch=1, capacity=96, page=16)
        _, ref = alone.step(table[ids[start:start + count]], [count], u[:1])
        got = y[start:start + count]
        # the merged weight and both sides' intermediates are rounded to bfloat16: a few of its steps
        torch.testing.assert_close(got, ref, rtol=0, atol=2 ** -5 * float(ref.abs().max()))
        err = float((got - ref).norm() / ref.norm())
        assert err <= 2 ** -6, err
        start += count
    assert status() == 0


def greedy_loop(serve, table, prompts, steps, guess, adapter_ids):
    """Greedy decoding with drafts guess(b, position): the tokens of each sequence and the steps that it took."""
    B, rows = serve.batch, serve.rows
    done = [list(p) for p in prompts]
    settings = dict(temperature=torch.zeros(B, device="cuda"))
    ids = torch.tensor([t for p in prompts for t in p], device="cuda")
    tokens, _ = serve.step(padded(rows, table[ids]), i32([len(p) for p in prompts]), torch.zeros(B, device="cuda"),
                           adapter_ids=adapter_ids, **settings)
    for b, t in enumerate(tokens.tolist()):
        done[b].append(t)
    for _ in range(steps):
        counts, fed, drafts = [], [], []
        for b in range(B):
            g = guess(b, len(done[b]))
            counts.append(1 + len(g))
            fed += [done[b][-1], *g]
            drafts += [*g, -1]
        d = torch.full((rows,), -1, dtype=torch.int64, device="cuda")
        d[:len(drafts)] = torch.tensor(drafts, device="cuda")
        got, accepted, _ = serve.verify(padded(rows, table[torch.tensor(fed, device="cuda")]), i32(counts), d,
                                        torch.zeros(rows, device="cuda"), adapter_ids=adapter_ids, **settings)
        best, at = serve.logits.argmax(1).tolist(), 0
        for b in range(B):
            n = int(accepted[b]) + 1
            emitted = got[at:at + n].tolist()
            assert emitted == best[at:at + n]  # greedy: each row's largest logit
            assert got[at + n:at + counts[b]].tolist() == [-1] * (counts[b] - n)
            assert int(serve.rejected[b]) == counts[b] - n
            assert drafts[at:at + n - 1] == emitted[:-1]
            done[b] += emitted
            at += counts[b]
    return done


def test_drafts_change_how_fast_tokens_come_and_not_which():
    D, V, N = 256, 512, 2
    cfg = synth.qkv(seed=9, T=1, D=D, V=V, N=N)
    table, lora = embeddings(V, D), make_adapters(2, 8, D)
    prompts = [[3, 77, 12], [500], [9, 9, 8, 7, 6]]
    ids = i32([1, -1, 0])

    def fresh():
        return SharedServing(cfg, heads=4, batch=3, pages=30, capacity=128, rows=32, page=16, adapters=lora)
    plain = greedy_loop(fresh(), table, prompts, 24, lambda b, n: [], ids)
    rng = np.random.default_rng(2)

    def guess(b, n):  # right for a while, then wrong
        known = plain[b][n:n + int(rng.integers(0, 5))]
        return [t if rng.random() < 0.7 else int(rng.integers(0, V)) for t in known]
    serve = fresh()
    drafted_ = greedy_loop(serve, table, prompts, 10, guess, ids)
    for a, b, p in zip(plain, drafted_, prompts):
        n = min(len(a), len(b))
        assert a[:n] == b[:n]
    assert sum(map(len, drafted_)) > sum(map(len, prompts)) + 3 + 3 * 10  # some drafts were right
    assert status() == 0


def test_shared_serving_step_captured_and_replayed():
    """A step with adapters and drafts as a graph: replays on new inputs are the eager steps, byte for byte."""
    D, V, N, B, rows = 256, 512, 2, 3, 24
    cfg = synth.qkv(seed=9, T=1, D=D, V=V, N=N)
    table, lora = embeddings(V, D), make_adapters(2, 8, D)
    g = torch.Generator().manual_seed(4)

    def inputs():
        counts = torch.randint(1, 7, (B,), generator=g).to(torch.int32)
        toks = torch.randint(0, V, (rows,), generator=g)
        return (table[toks.cuda()], counts.cuda(), torch.randint(0, V, (rows,), generator=g).cuda(),
                torch.rand(rows, generator=g).cuda(), i32(torch.randint(-1, 2, (B,), generator=g).numpy()))
    steps = [inputs() for _ in range(6)]

    def fresh():
        return SharedServing(cfg, heads=4, batch=B, pages=20, capacity=96, rows=rows, page=16, adapters=lora)
    eager = fresh()
    want = []
    for x, counts, d, u, ids in steps:
        out = eager.verify(x, counts, d, u, adapter_ids=ids)
        want.append([t.clone() for t in out] + [t.clone() for t in eager.plan] + [eager.rejected.clone()])
    serve = fresh()
    static = [t.clone() for t in steps[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        serve.verify(*static[:4], adapter_ids=static[4])  # what the library allocates, it allocates now
    torch.cuda.current_stream().wait_stream(side)
    for to, t in zip([*serve.plan, serve.rejected, serve.block_table, serve.free_pages],
                     [*fresh().plan, fresh().rejected, fresh().block_table, fresh().free_pages]):
        to.copy_(t)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = serve.verify(*static[:4], adapter_ids=static[4])
    for step, ref in zip(steps, want):
        for to, t in zip(static, step):
            to.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for got, r in zip([*out, *serve.plan, serve.rejected], ref):
            assert torch.equal(got, r)
    assert status() == 0


def test_adapters_two_graphs_at_once():
    """Steps of many tokens captured on one stream and replayed on two: each graph has its own memory."""
    T, K, O, R, n = 2048, 512, 512, 16, 4
    ids = np.random.default_rng(1).integers(0, n, T)
    plan = tp.tp_lora_plan(i32(ids), T, n)
    side = torch.cuda.Stream()
    work = []
    for seed in (1, 2):
        x, a, b, y, s = lora_data("column", T, 1, K, O, R, n, BF16, F32, seed)
        out = [torch.empty_like(t) for t in y]
        want = call_lora("column", x, a, b, plan, y, scales=s, out=[torch.empty_like(t) for t in y])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            call_lora("column", x, a, b, plan, y, scales=s, out=out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for _ in range(20):
                call_lora("column", x, a, b, plan, y, scales=s, out=out)
        work.append((graph, out, want, (x, a, b, y, s)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for (graph, _, _, _), st in zip(work, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for _, out, want, _ in work:
        assert all(torch.equal(o, w) for o, w in zip(out, want))


def test_calls_on_a_named_stream():
    """The operators on a stream that is not the current one, behind work that is still running there."""
    T, K, O, R, n = 1500, 256, 256, 16, 4
    x, a, b, y, s = lora_data("column", T, 1, K, O, R, n, BF16, F32, 1)
    ids = i32(np.random.default_rng(1).integers(0, n, T))
    want = call_lora("column", x, a, b, tp.tp_lora_plan(ids, T, n), y, scales=s, out=[torch.empty_like(t) for t in y])[0]
    step = some_step(20, 16, 100, 8, 0.1, 1)
    ref = plan_ref(*step)
    v = drafted(5, 0, 3, 300, F32, F32, 1)
    cu = i32(v[2])  # kept, as all inputs, until the other stream is done with it
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for st in (side, side.cuda_stream):
        out = torch.empty_like(y[0])
        late = torch.empty_like(x[0])
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
            late.copy_(x[0])
        plan = tp.tp_lora_plan(ids, T, n, stream=st)
        tp.tp_lora_all_to_sharded(late, a[0], b, plan, y, scales=s, out=[out], stream=st)
        got = tp.tp_verify(v[0], v[1], cu, v[3], draft_probs=v[4], stream=st)
        assert run_plan(*step, stream=st) == ref
        side.synchronize()
        assert torch.equal(out, want)
        check_verify(got, verify_ref(v[0], v[1], v[2], v[3], v[4]))


def test_prepared_calls_are_replayed():
    T, K, O, R, n = 1300, 256, 256, 16, 4
    x, a, b, y, s = lora_data("column", T, 1, K, O, R, n, BF16, F32, 1)
    plan = tp.tp_lora_plan(i32(np.random.default_rng(1).integers(0, n, T)), T, n)
    want = call_lora("column", x, a, b, plan, y, scales=s, out=[torch.empty_like(t) for t in y])[0].clone()
    out = [torch.zeros_like(t) for t in y]
    call = tp.prepare(tp.tp_lora_all_to_sharded, x[0], a[0], b, plan, y, scales=s, out=out)
    torch.cuda.synchronize()
    assert not out[0].any()
    other = [torch.full((8 * T * 16,), 7.0, device="cuda") for _ in range(3)]  # in memory that the call has given back
    call()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want) and all(bool((t == 7).all()) for t in other)
    xl, d, cu, u, q = drafted(4, 1, 3, 100, F32, F32, 1)
    call = tp.prepare(tp.tp_verify, xl, d, i32(cu), u, draft_probs=q)
    check_verify(call(), verify_ref(xl, d, cu, u, q))
    xr, ar, br, yr, s = lora_data("row", 9, 2, 64, 64, 8, 3, F16, BF16, 2)
    plan = tp.tp_lora_plan(i32([0, 1, 2, 0, 1, 2, -1, -1, 0]), 9, 3)
    out = torch.zeros_like(yr[0])
    tp.prepare(tp.tp_lora_sharded_to_all, xr, ar, br[0], plan, yr[0], out=out)()
    assert torch.equal(out, tp.tp_lora_sharded_to_all(xr, ar, br[0], plan, yr[0], out=torch.empty_like(out)))
    step = some_step(6, 16, 50, 3, 0.1, 2)
    t, pool = i32(step[4]), i32(step[5])
    call = tp.prepare(tp.tp_paged_plan, i32(step[0]), i32(step[2]), i32(step[3]), t, pool, i32([step[6]]), step[7], step[8],
                      rejected=i32(step[1]))
    p = call()
    torch.cuda.synchronize()
    ref = plan_ref(*step)
    assert (p[0].tolist(), p[5].tolist(), p[6].tolist(), t.tolist(), pool.tolist()) == (ref[0], ref[5], ref[6], ref[7], ref[8])
    ids = i32([1, 0, 2])
    call = tp.prepare(tp.tp_lora_plan, ids, 3, 3)
    assert call().tolist() == groups_ref([1, 0, 2], [0, 1, 2, 3], 3, 3)


def test_binding_refusals():
    x, a, b, y, s = lora_data("column", 8, 2, 64, 64, 16, 3, BF16, BF16, 1)
    plan = tp.tp_lora_plan(i32([0] * 8), 8, 3)
    ok = dict(x=x[0], a=a[0], b=b, plan=plan, y=y)
    for kw in (dict(x=x[0].float()), dict(a=a[0].half()), dict(b=b[:1]), dict(y=y[:1]), dict(y=[y[0], y[1].float()]),
               dict(plan=plan.long()), dict(plan=plan.cpu()), dict(x=x), dict(a=a[0].transpose(1, 2)), dict(out=[y[0]]),
               dict(out=[t.float() for t in y]), dict(scales=s.double()), dict(scales=s[:2]), dict(x=x[0][:, ::2])):
        with pytest.raises((ValueError, TypeError)):
            tp.tp_lora_all_to_sharded(**{**ok, **kw})
    with pytest.raises(tp.TPError):  # a plan of another step
        tp.tp_lora_all_to_sharded(**{**ok, "plan": tp.tp_lora_plan(i32([0] * 9), 9, 3)})
    with pytest.raises(tp.TPError):
        tp.tp_lora_all_to_sharded(**ok, out=[y[0], torch.empty_like(y[1])])
    with pytest.raises(ValueError):
        tp.tp_lora_sharded_to_all(x, a, b, plan, y[0])
    ints = i32([1, 2])
    good = [ints, ints, ints, i32([[0, 1], [2, 3]]), i32([0] * 8), i32([4]), 16, 4]
    for at, v in ((0, ints.long()), (1, i32([1])), (3, i32([[0, 1]])), (3, ints), (4, ints.float()), (5, ints), (7, -1)):
        args = list(good)
        args[at] = v
        with pytest.raises((ValueError, TypeError)):
            tp.tp_paged_plan(*args)
    with pytest.raises(ValueError):
        tp.tp_paged_plan(*good, out=[ints])
    xl, d, cu, u, q = drafted(4, 1, 3, 100, F32, F32, 1)
    for kw in (dict(drafts=d.int()), dict(drafts=d[:3]), dict(u=u[:3]), dict(draft_probs=q[:, :50]), dict(cu_rows=i32(cu).long()),
               dict(temperature=u), dict(tokens=d[:2]), dict(draft_probs=q.t()), dict(logits=xl.double())):
        with pytest.raises((ValueError, TypeError)):
            tp.tp_verify(**{**dict(logits=xl, drafts=d, cu_rows=i32(cu), u=u, draft_probs=q), **kw})
    with pytest.raises(tp.TPError):
        tp.tp_lora_plan(i32([0, 1]), 3, 2)


# ------------------------------------------------------------------ far addresses
@pytest.mark.parametrize("T", [40, 1500])
def test_adapters_beyond_32_bits(T):
    """Rows, adapters and outputs more than 2^31 elements apart."""
    n, R, K, O = 16384, 128, 1032, 1032  # 2.2 G elements a pool
    g = torch.Generator(device="cuda").manual_seed(1)
    a, b = (torch.empty((n, *shape), dtype=BF16, device="cuda") for shape in ((R, K), (O, R)))
    used = [0, 5, n - 1]
    for i in used:
        a[i] = torch.randn((R, K), generator=g, device="cuda") * K ** -0.5
        b[i] = torch.randn((O, R), generator=g, device="cuda") * R ** -0.5
    ld = (1 << 31) // T // 8 * 8 + 2048
    x = torch.empty((T, ld), dtype=BF16, device="cuda")[:, :K]
    y = torch.empty((T, ld), dtype=F32, device="cuda")[:, :O]
    x.copy_(torch.randn((T, K), generator=g, device="cuda"))
    y.copy_(torch.randn((T, O), generator=g, device="cuda"))
    ids = np.array(used)[np.arange(T) % 3]
    plan = tp.tp_lora_plan(i32(ids), T, n)
    y0 = y.clone()
    got = tp.tp_lora_all_to_sharded(x, a, [b], plan, [y])
    d, names = dev(np.arange(T) % 3), torch.tensor(used, device="cuda")
    check_lora(got, [x.clone()], [a[names]], [b[names]], d, None, [y0], BF16)
    assert status() == 0


def test_verify_beyond_32_bits():
    V, T = 50000, 44000  # 2.2 G logits, of which the last sequences' are used
    x = torch.empty((T, V), dtype=F32, device="cuda")
    q = torch.empty((T, V), dtype=F16, device="cuda")
    xs, ds, cu, us, qs = drafted(3, 2, 2, V, F32, F16, 4)
    x[-9:], q[-9:] = xs, qs
    d = torch.zeros(T, dtype=torch.int64, device="cuda")
    u = torch.zeros(T, device="cuda")
    d[-9:], u[-9:] = ds, us
    keep = torch.full((T,), 77, dtype=torch.int64, device="cuda")
    got = tp.tp_verify(x, d, i32([T - 9 + c for c in cu]), u, draft_probs=q, tokens=keep)
    check_verify((keep[-9:], got[1][-9:], got[2], got[3]), verify_ref(xs, ds, cu, us, qs))
    assert bool((keep[:-9] == 77).all())
    assert status() == 0


def test_plan_beyond_32_bits():
    B, width = 8192, 270000  # entries of the block table
    table = torch.empty((B, width), dtype=torch.int32, device="cuda")
    pages = 1000
    table[B - 1, :3] = torch.tensor([4, 7, 9], dtype=torch.int32)
    table[B - 2, :2] = torch.tensor([11, 12], dtype=torch.int32)
    lens, owned, counts = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
    lens[B - 1], owned[B - 1], counts[B - 1] = 40, 3, 20
    lens[B - 2], owned[B - 2], counts[B - 2] = 32, 2, -1
    pool = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    pool[:2] = torch.tensor([1, 2], dtype=torch.int32)
    p = tp.tp_paged_plan(counts, lens, owned, table, pool, i32([2]), 16, 20)
    assert p.positions.tolist() == list(range(40, 60)) and int(p.free_count) == 3
    assert table[B - 1, :4].tolist() == [4, 7, 9, 12]
    assert p.slots.tolist() == [9 * 16 + i % 16 for i in range(40, 48)] + [12 * 16 + i % 16 for i in range(48, 60)]
    assert status() == 0
