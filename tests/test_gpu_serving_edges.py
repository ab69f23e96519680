"""Edges of the operators that serve many requests at once, and of the serving step that runs them.

Tolerances of the adapters, with u the unit roundoff of the outputs' type: an output is rounded once (u |out|); the
sum over x meets B as two or more terms of the operands' type, which lose at most 2^-16 of it for bfloat16 (8 + 8 bits)
and 2^-20 for float16 (11 + 11 bits, less what falls below the smallest); the two products are summed in float32,
(K + R) adds of at most 2^-23 of the sum of their terms' sizes; where the second product is summed onto the old value,
16 of them at most are of its size.
"""
import numpy as np
import pytest
import torch

import sharded_gemm_gb300 as tp
from sharded_gemm_gb300 import build as tpbuild
from sharded_gemm_gb300 import synth
from sharded_gemm_gb300.workloads import PagedServing, SharedServing
from test_gpu_serving import (BF16, F16, F32, U, call_lora, check_verify, dev, drafted, embeddings, i32, lora_data,
                              lora_ref, make_adapters, padded, settings_of, status, verify_ref)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    tpbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    tp.tp_set_policy(tp.TP_POLICY_AUTO)


# ------------------------------------------------------------------ the bits of h
@pytest.mark.parametrize("dt,out_dt", [(BF16, BF16), (F16, F16), (BF16, F16), (F16, BF16)])
@pytest.mark.parametrize("T,R", [(1, 16), (40, 16), (300, 64), (600, 128), (1100, 16), (1500, 64), (1030, 32)])
def test_adapters_keep_16_bits_of_the_sum_over_x(T, R, dt, out_dt):
    """Where an adapter's outputs cancel, what is left is as exact as the outputs' type holds it."""
    n, K, O = 3, 512, 256
    x, a, b, y, s = lora_data("column", T, 2, K, O, R, n, dt, out_dt, T + R)
    ids = np.random.default_rng(T).integers(0, n, T)
    plan = tp.tp_lora_plan(i32(ids), T, n)
    lost = (2.0 ** -16 if dt == BF16 else 2.0 ** -20) + (K + R) * 2.0 ** -23
    for start in ([torch.zeros_like(t) for t in y], y):
        got = call_lora("column", x, a, b, plan, start, scales=s, out=[torch.empty_like(t) for t in y])
        ref, big = lora_ref(x, a, b, dev(ids), s, start)
        for g, f, size, old in zip(got, ref, big, start):
            tol = U[out_dt] * f.abs() + lost * size + 2.0 ** -19 * old.double().abs() + 2.0 ** -24
            worst = ((g.double() - f).abs() / tol).max()
            assert worst <= 1, float(worst)
    assert status() == 0


# ------------------------------------------------------------------ steps that cannot be made
def a_step(kind, counts, V, rows, seed):
    """Tokens, drafts and random numbers of a step; `kind` is "verify" or "step"."""
    g = torch.Generator().manual_seed(seed)
    return (kind, counts, torch.randint(0, V, (rows,), generator=g).cuda(), torch.randint(0, V, (rows,), generator=g).cuda(),
            torch.rand(rows, generator=g).cuda())


def make_step(serve, table, step, ids):
    kind, counts, toks, drafts, u = step
    x = table[toks]
    if kind == "step":
        return serve.step(x, i32(counts), u[:serve.batch], adapter_ids=ids)
    return serve.verify(x, i32(counts), drafts, u, adapter_ids=ids)


def state_of(serve):
    return [serve.plan[0].tolist(), serve.rejected.tolist()]


@pytest.mark.parametrize("fails", ["step", "verify", "rows", "rows twice"])
def test_a_step_that_cannot_be_made_changes_nothing(fails):
    """What the last step refused stays refused over an empty step: the steps behind it are those of a server that was
    never asked for it."""
    D, V, N, B, rows = 256, 512, 2, 3, 48
    cfg = synth.qkv(seed=9, T=1, D=D, V=V, N=N)
    table, lora, ids = embeddings(V, D), make_adapters(2, 8, D), i32([1, -1, 0])
    small, large = (SharedServing(cfg, heads=4, batch=B, pages=p, capacity=128, rows=rows, page=16, adapters=lora)
                    for p in (6, 30))
    script = [a_step("step", [20, 14, 9], V, rows, 1), a_step("verify", [9, 5, 7], V, rows, 2)]
    for step in script:
        for serve in (small, large):
            make_step(serve, table, step, ids)
    assert state_of(small) == state_of(large) and int(small.plan[3]) == 0
    assert sum(small.rejected.tolist()) > 6  # random drafts are mostly refused
    assert status() == 0
    for _ in range(2 if fails == "rows twice" else 1):
        before = state_of(small)
        counts = [20, 20, 20] if "rows" in fails else [16, 16, 16]
        make_step(small, table, a_step("verify" if "rows" in fails else fails, counts, V, rows, 3), ids)
        assert int(small.plan[3]) == -1 if "rows" in fails else int(small.plan[3]) > 0
        assert state_of(small) == before
        assert status() == (tp.TP_ERR_INVALID_ARG if "rows" in fails else 0)
    for i, (kind, counts) in enumerate([("verify", [4, -1, 5]), ("step", [1, 6, 1]), ("verify", [3, 3, 3])]):
        step = a_step(kind, counts, V, rows, 10 + i)
        got, want = (make_step(serve, table, step, ids) for serve in (small, large))
        assert int(small.plan[3]) == 0
        assert state_of(small) == state_of(large)
        used = sum(max(c, 0) for c in counts)
        assert torch.equal(got[-1][:used], want[-1][:used])
        for p, q in zip(got[:-1], want[:-1]):
            live = torch.tensor([c > 0 for c in counts], device="cuda") if kind == "step" else slice(None)
            assert torch.equal(p[live], q[live])
    assert status() == 0


def test_a_captured_step_that_cannot_be_made_changes_nothing():
    """The same as a graph that is replayed."""
    D, V, N, B, rows = 256, 512, 2, 3, 48
    cfg = synth.qkv(seed=9, T=1, D=D, V=V, N=N)
    table, lora, ids = embeddings(V, D), make_adapters(2, 8, D), i32([1, -1, 0])

    def fresh(pages):
        return SharedServing(cfg, heads=4, batch=B, pages=pages, capacity=128, rows=rows, page=16, adapters=lora)
    small, large = fresh(4), fresh(30)
    counts, toks, drafts, u = i32([1, 1, 1]), *(t.clone() for t in a_step("verify", [], V, rows, 0)[2:])

    def call():
        return small.verify(table[toks], counts, drafts, u, adapter_ids=ids)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    new = fresh(4)
    for to, t in zip([*small.plan, small.rejected, small.block_table, small.free_pages],
                     [*new.plan, new.rejected, new.block_table, new.free_pages]):
        to.copy_(t)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = call()
    for i, c in enumerate([[20, 14, 9], [9, 5, 7], [16, 16, 16], [16, 16, 16], [4, -1, 5], [1, 6, 1], [3, 3, 3]]):
        step = a_step("verify", c, V, rows, 20 + i)
        for to, t in zip((counts, toks, drafts, u), (i32(c), *step[2:])):
            to.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        if sum(c) == 48:
            assert int(small.plan[3]) > 0
        else:
            want = make_step(large, table, step, ids)
            used = sum(max(n, 0) for n in c)
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
            assert torch.equal(out[2][:used], want[2][:used])
        assert state_of(small) == state_of(large)
    assert status() == 0


@pytest.mark.parametrize("kind", ["step", "verify"])
def test_refused_steps_change_nothing(kind):
    """A call that is refused for its arguments leaves lengths, pages and refusals as they were."""
    D, V, N, B, rows = 256, 512, 2, 3, 48
    cfg = synth.qkv(seed=9, T=1, D=D, V=V, N=N)
    table, ids = embeddings(V, D), i32([1, -1, 0])
    plain, full = (SharedServing(cfg, heads=4, batch=B, pages=30, capacity=128, rows=rows, page=16, adapters=a)
                   for a in (None, make_adapters(2, 8, D)))
    _, _, toks, drafts, u = a_step(kind, [], V, rows, 5)
    ok = dict(x=table[toks], counts=i32([5, 4, 3]), u=u[:B] if kind == "step" else u, adapter_ids=ids)
    if kind == "verify":
        ok["drafts"] = drafts
    for serve, bad in [(plain, {})] + [(full, b) for b in (
            dict(adapter_ids=i32([1, 0])), dict(adapter_ids=ids.long()), dict(x=table[toks][:40]), dict(x=table[toks].float()),
            dict(x=table[toks][:, :128]), dict(counts=i32([1, 2])), dict(counts=ids.long()), dict(u=u[:2]), dict(u=u.double()),
            dict(temperature=u[:2]), dict(top_k=u[:3]), dict(top_q=u[:3]), dict(x=table[toks].cpu()), dict(x=table[:1].expand(rows, D)))] + [(full, b) for b in (
                dict(drafts=drafts[:4]), dict(drafts=drafts.int()), dict(draft_probs=torch.zeros((rows, V - 1), device="cuda")),
                dict(draft_probs=torch.zeros((rows, V), dtype=torch.float64, device="cuda"))) if kind == "verify"]:
        make_step(serve, table, a_step("verify", [9, 5, 7], V, rows, 2), None)
        state = [t.clone() for t in (*serve.plan[:3], serve.rejected, serve.block_table, serve.free_pages)]
        assert sum(serve.rejected.tolist()) > 0
        with pytest.raises((ValueError, TypeError)):
            getattr(serve, kind)(**{**ok, **bad})
        now = (*serve.plan[:3], serve.rejected, serve.block_table, serve.free_pages)
        assert all(torch.equal(p, q) for p, q in zip(now, state)), bad
        serve.step(table[toks], i32([-1, -1, -1]), u[:B])  # all end: room for the next
    getattr(full, kind)(**ok)
    assert full.plan[0].tolist() == [5, 4, 3]
    assert status() == 0


def test_adapters_that_no_step_takes_are_refused_at_once():
    cfg, good = synth.qkv(seed=9, T=1, D=256, V=512, N=2), make_adapters(2, 8, 256)
    wide = make_adapters(2, 129, 256)
    for bad in (dict(qkv_a=wide["qkv_a"], qkv_b=wide["qkv_b"]), dict(o_b=good["o_b"].float()), dict(o_a=good["o_a"][:1]),
                dict(scales=good["scales"].double()), dict(qkv_b=good["qkv_b"][:, :256]),
                dict(qkv_a=good["qkv_a"].transpose(1, 2).contiguous().transpose(1, 2)), dict(o_b=good["o_b"].cpu())):
        with pytest.raises(ValueError):
            SharedServing(cfg, heads=4, batch=1, pages=8, capacity=64, rows=8, page=16, adapters={**good, **bad})
    kept = SharedServing(cfg, heads=4, batch=1, pages=8, capacity=64, rows=8, page=16, adapters={**good, "scales": None})
    out = torch.zeros(8, device="cuda")
    x, u = embeddings(512, 256)[:8], torch.full((8,), 0.5, device="cuda")
    kept.verify(x, i32([8]), torch.zeros(8, dtype=torch.int64, device="cuda"), u, adapter_ids=i32([1]), logprobs=out)
    assert kept.logprobs is out and bool(out[0] < 0)


@pytest.mark.parametrize("capacity,page", [(40, 16), (1, 16), (33, 32)])
def test_capacities_end_with_a_page(capacity, page):
    """Positions up to the end of a sequence's last page are rotated by their own angles."""
    cfg = synth.qkv(seed=6, T=1, D=256, V=512, N=2)
    table = embeddings(512, 256)
    whole = -(-capacity // page) * page
    a, b = (SharedServing(cfg, heads=4, batch=1, pages=8, capacity=c, rows=64, page=page) for c in (capacity, whole))
    ids = torch.randint(0, 512, (64,), generator=torch.Generator().manual_seed(1)).cuda()
    u = torch.tensor([0.5], device="cuda")
    for count in (whole - 1, 1):
        (t0, y0), (t1, y1) = (serve.step(table[ids], i32([count]), u) for serve in (a, b))
        assert torch.equal(y0[:count], y1[:count]) and torch.equal(t0, t1)
    assert a.plan[0].tolist() == [whole] and int(a.plan[3]) == 0
    assert status() == 0


# ------------------------------------------------------------------ streams
def test_the_default_stream_by_its_handle(monkeypatch):
    """0 names the default stream: the call's memory is of that stream, and a serving step runs there."""
    seen = []

    def empty(*args, real=torch.empty, **kwargs):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return real(*args, **kwargs)
    with torch.cuda.stream(torch.cuda.Stream()):
        monkeypatch.setattr(torch, "empty", empty)
        ws = tp._lora_workspace(2048, 16, torch.cuda.current_device(), 0)
        monkeypatch.undo()
    assert ws.numel() >= 2048 * 16 and seen == [0]
    cfg = synth.qkv(seed=6, T=1, D=256, V=512, N=2)
    table, u = embeddings(512, 256), torch.tensor([0.5], device="cuda")
    a, b = (PagedServing(cfg, heads=4, batch=1, capacity=64, page=16) for _ in range(2))
    real, where = b._step, []
    b._step = lambda *args: (where.append(torch.cuda.current_stream().cuda_stream), real(*args))[1]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        want, got = a.step(table[:9], [9], u), b.step(table[:9], [9], u, stream=0)
    torch.cuda.synchronize()
    assert where == [0] and all(torch.equal(p, q) for p, q in zip(got, want))


def test_adapters_on_the_default_stream_by_its_handle():
    """Many tokens on stream 0 behind work that is still running there, called from another stream."""
    T, K, O, R, n = 1500, 256, 256, 16, 4
    x, a, b, y, s = lora_data("column", T, 1, K, O, R, n, BF16, F32, 1)
    ids = i32(np.random.default_rng(1).integers(0, n, T))
    plan = tp.tp_lora_plan(ids, T, n)
    want = call_lora("column", x, a, b, plan, y, scales=s, out=[torch.empty_like(t) for t in y])[0]
    out = torch.empty_like(y[0])
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    with torch.cuda.stream(torch.cuda.Stream()):
        tp.tp_lora_all_to_sharded(x[0], a[0], b, plan, y, scales=s, out=[out], stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# ------------------------------------------------------------------ what is not finite, and sizes from end to end
@pytest.mark.parametrize("policy", [tp.TP_POLICY_AUTO, tp.TP_POLICY_SIMT], ids=["auto", "simt"])
@pytest.mark.parametrize("dt,out_dt", [(BF16, F32), (BF16, BF16), (F16, F32), (F16, F16)])
@pytest.mark.parametrize("R,O", [(1, 24), (4, 24), (5, 24), (8, 24), (16, 24), (24, 24), (24, 23), (40, 24), (100, 24), (128, 24)])
@pytest.mark.parametrize("T", [2, 1100])
def test_adapters_infinite_sums_of_any_rank(policy, T, R, O, dt, out_dt):
    """An infinite sum gives infinite outputs of its sign whatever the rank is rounded up to inside."""
    x = torch.ones((T, 32), dtype=dt, device="cuda")
    x[1, 0] = float("inf")
    x[T - 1, 31] = -float("inf") if T > 2 else x[T - 1, 31]
    a = torch.ones((1, R, 32), dtype=dt, device="cuda")
    b = torch.ones((1, O, R), dtype=dt, device="cuda")
    b[0, 1::2] = -1
    y = torch.zeros((T, O), dtype=out_dt, device="cuda")
    tp.tp_set_policy(policy)
    try:
        got = tp.tp_lora_all_to_sharded(x, a, [b], tp.tp_lora_plan(i32([0] * T), T, 1), [y])[0].float()
    finally:
        tp.tp_set_policy(tp.TP_POLICY_AUTO)
    sign = torch.ones(O, device="cuda")
    sign[1::2] = -1
    assert torch.equal(got[1], sign * float("inf"))
    if T > 2:
        assert torch.equal(got[T - 1], sign * -float("inf"))
    rest = torch.cat([got[:1], got[2:T - 1]]) if T > 2 else got[:1]
    assert torch.equal(rest, (sign * 32 * R).expand_as(rest))  # whole numbers that all types hold
    assert status() == 0


@pytest.mark.parametrize("form,R,out_dt", [("column", 16, BF16), ("column", 64, F32), ("row", 128, F32)])
def test_adapters_of_many_tokens_behind_a_plan_that_is_written_anew(form, R, out_dt):
    """A step's plan and its adapters as a graph, replayed on other adapters, other offsets and other tokens."""
    T, N, K, O, n, B = 1500, 2, 256, 320, 40, 60
    x, a, b, y, s = lora_data(form, T, N, K, O, R, n, BF16, out_dt, 3)
    ids, cu = i32([0] * B), i32([0] * (B + 1))
    rng = np.random.default_rng(5)
    steps = []
    for i in range(8):
        cuts = np.sort(rng.integers(0, T + 1 - 100 * (i % 2), B - 1))
        steps.append((rng.integers(-1, n, B) if i % 3 else np.full(B, i), np.concatenate([[0], cuts, [T - 100 * (i % 2)]])))
    out = [torch.empty_like(t) for t in y]
    plan = tp.tp_lora_plan(ids, T, n, cu_seqlens=cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        tp.tp_lora_plan(ids, T, n, cu_seqlens=cu, out=plan)
        call_lora(form, x, a, b, plan, y, scales=s, out=out)
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for names, offsets in steps * 3:
        ids.copy_(i32(names))
        cu.copy_(i32(offsets))
        for t in out:
            t.fill_(7)
        graph.replay()
        fresh = tp.tp_lora_plan(i32(names), T, n, cu_seqlens=i32(offsets))
        want = call_lora(form, x, a, b, fresh, y, scales=s, out=[torch.full_like(t, 7) for t in y])
        assert torch.equal(plan, fresh)
        assert all(torch.equal(p, q) for p, q in zip(out, want))
    assert status() == 0


# ------------------------------------------------------------------ offsets that do not ascend
def rows_of(off, T, s):
    """The rows of sequence s: none where its offsets or others leave them unclear."""
    r0, r1 = off[s], off[s + 1]
    clear = 0 <= r0 <= r1 <= T and all(
        (o <= r0 if j < s else o >= r1) for j, o in enumerate(off) if j not in (s, s + 1) and 0 <= o <= T)
    return (r0, r1) if clear else (0, 0)


def check_offsets(x, d, off, u, q, settings):
    """Sequences whose rows are clear are served, the others' rows stay as they were."""
    T, B = len(d), len(off) - 1
    tokens = torch.full((T,), 77, dtype=torch.int64, device="cuda")
    logprobs = torch.full((T,), 7.0, device="cuda")
    got = tp.tp_verify(x, d, i32(off), u, draft_probs=q, tokens=tokens, logprobs=logprobs, **settings)
    bad = any(not 0 <= off[s] <= off[s + 1] <= T for s in range(B))
    assert status() == (tp.TP_ERR_INVALID_ARG if bad else 0)
    used = torch.zeros(T, dtype=torch.bool, device="cuda")
    for s in range(B):
        r0, r1 = rows_of(off, T, s)
        if r0 == r1:
            assert (int(got[2][s]), int(got[3][s])) == (0, 0)
            continue
        used[r0:r1] = True
        mine = {k: v[s:s + 1] for k, v in settings.items()}
        ref = verify_ref(x[r0:r1], d[r0:r1], [0, r1 - r0], u[r0:r1], None if q is None else q[r0:r1], **mine)
        check_verify((tokens[r0:r1], logprobs[r0:r1], got[2][s:s + 1], got[3][s:s + 1]), ref)
    assert bool((tokens[~used] == 77).all()) and bool((logprobs[~used] == 7).all())


@pytest.mark.parametrize("V", [40, 60001, 130003])
@pytest.mark.parametrize("off", [[0, 5, 2, 6], [0, 3, 2, 9], [0, 3, 6, 10], [-1, 3, 6, 9], [4, 1, 6, 9], [9, 6, 3, 0],
                                 [0, 9, 0, 9], [0, 3, 99, 4, 9], [0, 2, 5, 4, 4, 9], [3, 3, 0, 3], [0, 4, 4, 2, 8, 9], [1, 1, 4, 8]])
def test_verify_of_offsets_that_do_not_ascend(off, V):
    x, d, _, u, q = drafted(3, 2, 2, V, F32, F32, 2)
    for settings in ({}, settings_of(len(off) - 1, 7)):
        check_offsets(x, d, off, u, q, settings)


@pytest.mark.parametrize("changes", [{0: -4}, {100: 401}, {40: 10}, {40: 390}, {1: -1}, {99: 0}, {100: 0}, {50: 203, 60: 2 ** 30},
                                     {3: 11, 4: 11, 97: 3}, {}])
def test_verify_of_many_rows_of_offsets_that_do_not_ascend(changes):
    """The same where the rows are more than the GPU holds at once."""
    x, d, cu, u, q = drafted(100, 3, 3, 20, F32, F32, 2)
    off = list(cu)
    for at, v in changes.items():
        off[at] = v
    for settings in ({}, settings_of(100, 7)):
        check_offsets(x, d, off, u, q, settings)


def test_verify_of_many_long_rows_of_offsets_that_do_not_ascend():
    x, d, cu, u, q = drafted(60, 1, 3, 60007, BF16, BF16, 7)
    for at, v in ((30, 5), (60, len(d) + 1), (0, -1)):
        off = list(cu)
        off[at] = v
        check_offsets(x, d, off, u, q, settings_of(60, 5))


def test_verify_of_no_rows_and_offsets_that_claim_some():
    none = torch.empty((0, 40), device="cuda")
    got = tp.tp_verify(none, torch.empty(0, dtype=torch.int64, device="cuda"), i32([0, 0, 3]), torch.empty(0, device="cuda"))
    assert got[2].tolist() == [0, 0] and got[3].tolist() == [0, 0]
    assert status() == tp.TP_ERR_INVALID_ARG


@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** 122, 2.0 ** -100, 2.0 ** -120])
@pytest.mark.parametrize("T", [3, 1100])
def test_adapters_of_float16_with_scales_from_end_to_end(T, size):
    """Sums over x near float32's largest and smallest numbers meet B with the bits that others do."""
    n, K, O, R = 2, 64, 40, 16
    x, a, b, y, _ = lora_data("column", T, 1, K, O, R, n, F16, F32, 4)
    y = [torch.zeros_like(t) for t in y]
    b = [t * 2.0 ** (-4 if size > 1 else 4) for t in b]
    scales = torch.tensor([size, -size / 2], device="cuda")
    ids = np.arange(T) % n
    got = call_lora("column", x, a, b, tp.tp_lora_plan(i32(ids), T, n), y, scales=scales)[0]
    ref, big = lora_ref(x, a, b, dev(ids), scales, [torch.zeros_like(t) for t in y])
    tol = U[F32] * ref[0].abs() + (2.0 ** -20 + (K + R) * 2.0 ** -23) * big[0]
    assert ((got.double() - ref[0]).abs() <= tol).all()
    assert status() == 0


def test_plan_of_a_page_size_beyond_32_bits_is_refused():
    ints = i32([1, 2])
    with pytest.raises((ValueError, tp.TPError)):
        tp.tp_paged_plan(ints, i32([0, 0]), i32([0, 0]), i32([[0, 1], [2, 3]]), i32([0] * 8), i32([4]), 2 ** 32 + 16, 4)
