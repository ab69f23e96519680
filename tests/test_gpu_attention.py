"""GPU parity of the attention-side operators against plain float64 forms.

Tolerances.  With u the unit roundoff of the 16-bit type (2^-8 for bfloat16,
2^-11 for float16), an attention output is rounded once (u |o|) and each
softmax term is rounded once before it meets its value (u sum_j p_j |v_j|);
float32 scores and exponentials add less than 2^-13 of that sum.  A float16
term below 2^-14 of the largest has an absolute error of 2^-25 instead.
An appended value is rounded once, after at most 2^-20 of relative error of its
norm and rotation.
"""
import numpy as np
import pytest
import torch

import oracle
import sharded_gemm_gb300 as tp
from sharded_gemm_gb300 import build as tpbuild
from sharded_gemm_gb300 import synth
from sharded_gemm_gb300.workloads import PagedServing, to_device, to_host
from gpu_util import check_close

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    tpbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    tp.tp_set_policy(tp.TP_POLICY_AUTO)


@pytest.fixture(params=[tp.TP_POLICY_AUTO, tp.TP_POLICY_SIMT], ids=["auto", "simt"])
def policy(request):
    tp.tp_set_policy(request.param)
    yield request.param
    tp.tp_set_policy(tp.TP_POLICY_AUTO)


def status_ok():
    torch.cuda.synchronize()
    assert tp.tp_query_status() == 0


# ------------------------------------------------------------------ append
def append_ref(x, Hq, Hk, D, qn, kn, eps, rope, pos, interleaved):
    """(q, k, v) of x (T, (Hq + 2 Hk) D) in float64."""
    x = x.double().cpu().reshape(len(x), Hq + 2 * Hk, D)
    y = x[:, :Hq + Hk].clone()
    for lo, hi, g in ((0, Hq, qn), (Hq, Hq + Hk, kn)):
        if g is not None:
            z = y[:, lo:hi]
            y[:, lo:hi] = z / torch.sqrt(z.pow(2).mean(-1, keepdim=True) + eps) * g.double().cpu()
    if rope is not None:
        rot = rope.shape[1]
        row = rope.double().cpu()[pos.long().cpu()]
        c, s = row[:, None, :rot // 2], row[:, None, rot // 2:]
        ia = torch.arange(rot // 2) * 2 if interleaved else torch.arange(rot // 2)
        ib = ia + 1 if interleaved else ia + rot // 2
        a, b = y[..., ia].clone(), y[..., ib].clone()
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y[:, :Hq], y[:, Hq:], x[:, Hq + Hk:]


def rope_table(rows, rot):
    ang = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(rot // 2) * 2.0 / rot)
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()


@pytest.mark.parametrize("T,N,Hq,Hk,D,page,rot,inter,norm,in_dt,dt", [
    (1, 1, 1, 1, 64, 16, 64, False, True, torch.bfloat16, torch.bfloat16),
    (1, 2, 32, 8, 128, 16, 128, False, True, torch.bfloat16, torch.bfloat16),
    (37, 3, 6, 2, 64, 32, 32, True, False, torch.float32, torch.float16),
    (37, 1, 5, 5, 128, 64, 16, False, True, torch.float16, torch.float16),
    (333, 2, 7, 1, 128, 256, 48, True, True, torch.float32, torch.bfloat16),
    (1025, 4, 12, 3, 64, 16, 0, False, True, torch.bfloat16, torch.bfloat16),
    (700, 1, 4, 4, 128, 128, 128, False, False, torch.float16, torch.bfloat16)])
def test_append(T, N, Hq, Hk, D, page, rot, inter, norm, in_dt, dt):
    g = torch.Generator(device="cuda").manual_seed(T + N)
    rng = np.random.default_rng(T * N)
    pages = -(-T // page) + 3
    wide = (Hq + 2 * Hk) * D
    qkv = [torch.randn((T, wide), generator=g, device="cuda").to(in_dt) for _ in range(N)]
    kc = torch.randn((N, pages, Hk, page, D), generator=g, device="cuda").to(dt)
    vc = torch.randn((N, pages, Hk, page, D), generator=g, device="cuda").to(dt)
    slots = torch.from_numpy(rng.permutation(pages * page)[:T].astype(np.int64)).cuda()
    if T > 4:
        slots[3] = -1  # padding
    pos = torch.from_numpy(rng.integers(0, 500, T).astype(np.int32)).cuda()
    rope = rope_table(500, rot) if rot else None
    qn = torch.rand(D, generator=g, device="cuda") + 0.5 if norm else None
    kn = torch.rand(D, generator=g, device="cuda") + 0.5 if norm else None
    k0, v0 = kc.clone(), vc.clone()
    q = tp.tp_qkv_append(qkv, kc, vc, slots, positions=pos, rope=rope, q_norm=qn, k_norm=kn, eps=1e-5, interleaved=inter)
    status_ok()
    live = slots >= 0
    at, off = slots[live] // page, slots[live] % page
    for r in range(N):
        rq, rk, rv = append_ref(qkv[r], Hq, Hk, D, qn, kn, 1e-5, rope, pos, inter)
        tol = U[dt] + 2.0 ** -20
        got = q[r].double().cpu().reshape(T, Hq, D)
        # the rotated value's own size bounds the float32 error, its pair's size that of the sum
        big = rq.abs().amax(-1, keepdim=True)
        assert ((got - rq).abs() <= U[dt] * rq.abs() + 2.0 ** -20 * big + 2.0 ** -24).all()
        gk = kc[r][at, :, off].double().cpu()
        rk, rv = rk[live.cpu()], rv[live.cpu()]
        assert ((gk - rk).abs() <= U[dt] * rk.abs() + 2.0 ** -20 * rk.abs().amax(-1, keepdim=True) + 2.0 ** -24).all()
        assert torch.equal(vc[r][at, :, off].cpu(), rv.to(dt)), tol
        k0[r][at, :, off], v0[r][at, :, off] = kc[r][at, :, off], vc[r][at, :, off]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)  # nothing else was written


F32 = torch.float32


def takes_ring(T, N, Hq, Hk, D):
    """Whether an append of aligned rows is a prompt batch: its blocks of tokens fill the GPU twice."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tokens, stretches = 256 // (D // 8), -(-(Hq + 2 * Hk) // 4)
    return -(-T // tokens) >= 2 * -(-3 * sms // (stretches * N))


@pytest.mark.parametrize("T,N,Hq,Hk,D,page,rot,inter,norms,in_dt,dt", [
    (16391, 1, 6, 2, 64, 16, 64, False, "qk", F32, torch.bfloat16),
    (8209, 1, 2, 2, 128, 64, 128, True, "qk", torch.bfloat16, torch.bfloat16),
    (3001, 8, 7, 1, 128, 256, 16, True, "qk", torch.float16, torch.bfloat16),
    (3001, 8, 5, 1, 64, 32, 48, False, "q", F32, torch.float16),
    (3000, 8, 2, 1, 128, 16, 128, False, "k", F32, torch.bfloat16),
    (8199, 4, 1, 1, 64, 16, 0, False, "", torch.bfloat16, torch.float16),
    (4099, 4, 4, 4, 64, 128, 32, True, "qk", F32, torch.bfloat16),
    (1500, 64, 1, 1, 128, 64, 128, False, "qk", torch.float16, torch.float16),
    (5003, 2, 9, 3, 128, 64, 0, False, "k", F32, torch.float16)])
@pytest.mark.parametrize("odd_out", [False, True])
def test_append_prompt_batches(T, N, Hq, Hk, D, page, rot, inter, norms, in_dt, dt, odd_out):
    """Prompt batches, which the ring kernel takes: stretches of four heads that mix queries, keys and values and
    do not end with them, tokens that do not end with a block, padding, and query rows without alignment."""
    assert takes_ring(T, N, Hq, Hk, D)
    g = torch.Generator(device="cuda").manual_seed(T + N)
    rng = np.random.default_rng(T * N)
    pages = -(-T // page) + 3
    wide = (Hq + 2 * Hk) * D
    qkv = [torch.randn((T, wide + 8), generator=g, device="cuda").to(in_dt)[:, :wide] for _ in range(N)]
    kc = torch.randn((N, pages, Hk, page, D), generator=g, device="cuda").to(dt)
    vc = torch.randn((N, pages, Hk, page, D), generator=g, device="cuda").to(dt)
    slots = torch.from_numpy(rng.permutation(pages * page)[:T].astype(np.int64)).cuda()
    slots[torch.from_numpy(rng.integers(0, T, 20)).cuda()] = -1
    slots[T - 1] = -(1 << 40)
    pos = torch.from_numpy(rng.integers(0, 500, T).astype(np.int32)).cuda()
    rope = rope_table(500, rot) if rot else None
    qn = torch.rand(D, generator=g, device="cuda") + 0.5 if "q" in norms else None
    kn = torch.rand(D, generator=g, device="cuda") + 0.5 if "k" in norms else None
    k0, v0 = kc.clone(), vc.clone()
    obuf = torch.full((N, T, Hq * D + 6), 7.0, device="cuda").to(dt)
    lo = 3 if odd_out else 0
    tp.tp_qkv_append(qkv, kc, vc, slots, positions=pos, rope=rope, q_norm=qn, k_norm=kn, eps=1e-5, interleaved=inter,
                     out=obuf[:, :, lo:lo + Hq * D])
    status_ok()
    live = slots >= 0
    at, off = slots[live] // page, slots[live] % page
    for r in range(N):
        rq, rk, rv = append_ref(qkv[r], Hq, Hk, D, qn, kn, 1e-5, rope, pos, inter)
        got = obuf[r, :, lo:lo + Hq * D].double().cpu().reshape(T, Hq, D)
        big = rq.abs().amax(-1, keepdim=True)
        assert ((got - rq).abs() <= U[dt] * rq.abs() + 2.0 ** -20 * big + 2.0 ** -24).all()
        gk = kc[r][at, :, off].double().cpu()
        rk, rv = rk[live.cpu()], rv[live.cpu()]
        assert ((gk - rk).abs() <= U[dt] * rk.abs() + 2.0 ** -20 * rk.abs().amax(-1, keepdim=True) + 2.0 ** -24).all()
        assert torch.equal(vc[r][at, :, off].cpu(), rv.to(dt))
        k0[r][at, :, off], v0[r][at, :, off] = kc[r][at, :, off], vc[r][at, :, off]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)  # nothing else was written
    assert (obuf[:, :, :lo] == 7).all() and (obuf[:, :, lo + Hq * D:] == 7).all()


@pytest.mark.parametrize("in_dt", [F32, torch.bfloat16])
def test_append_prompt_batch_with_bad_slots_and_positions(in_dt):
    """They are recorded; every other token is as without them."""
    T, N, Hq, Hk, D, page = 4099, 2, 6, 1, 128, 16
    assert takes_ring(T, N, Hq, Hk, D)
    pages = -(-T // page) + 1
    qkv = torch.randn((N, T, (Hq + 2 * Hk) * D), device="cuda").to(in_dt)
    kc = torch.zeros((N, pages, Hk, page, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    slots, pos = torch.arange(T, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda") % 90
    rope = rope_table(90, D)
    q = tp.tp_qkv_append(qkv, kc, vc, slots, positions=pos, rope=rope)
    status_ok()
    for bad_slot, bad_pos in ((pages * page, None), (1 << 60, None), (None, 90), (None, -1), (None, 2 ** 31 - 1)):
        k2, v2, s2, p2 = torch.zeros_like(kc), torch.zeros_like(vc), slots.clone(), pos.clone()
        if bad_slot is not None:
            s2[[5, T - 1]] = bad_slot
        else:
            p2[[5, T - 1]] = bad_pos
        q2 = tp.tp_qkv_append(qkv, k2, v2, s2, positions=p2, rope=rope)
        assert tp.tp_query_status() == tp.TP_ERR_INVALID_ARG
        rest = torch.ones(T, dtype=torch.bool, device="cuda")
        rest[[5, T - 1]] = False
        at, off = slots[rest] // page, slots[rest] % page
        assert torch.equal(q2[:, rest], q[:, rest])
        assert torch.equal(k2[:, at, :, off], kc[:, at, :, off]) and torch.equal(v2[:, at, :, off], vc[:, at, :, off])
        if bad_slot is not None:  # and nothing is written for them
            lost = slots[~rest]
            assert (k2[:, lost // page, :, lost % page] == 0).all() and (v2[:, lost // page, :, lost % page] == 0).all()
    status_ok()


def test_append_strides_and_unaligned_rows():
    T, Hq, Hk, D, page = 19, 3, 1, 64, 16
    g = torch.Generator(device="cuda").manual_seed(5)
    wide = (Hq + 2 * Hk) * D
    buf = torch.randn((T, wide + 3), generator=g, device="cuda").to(torch.bfloat16)
    qkv = buf[:, 1:wide + 1]  # odd row stride, base not 16-byte aligned
    kv = torch.zeros((4, 2, Hk, page, D), dtype=torch.bfloat16, device="cuda")  # keys and values of a page together
    obuf = torch.zeros((T, Hq * D + 5), dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(T, device="cuda") + 20
    got = tp.tp_qkv_append([qkv], [kv[:, 0]], [kv[:, 1]], slots, out=[obuf[:, 3:3 + Hq * D]])[0]
    status_ok()
    assert torch.equal(got, qkv[:, :Hq * D])
    assert torch.equal(kv[slots // page, 0, 0, slots % page], qkv[:, Hq * D:(Hq + 1) * D])
    assert torch.equal(kv[slots // page, 1, 0, slots % page], qkv[:, (Hq + 1) * D:])
    assert (obuf[:, :3] == 0).all() and (obuf[:, 3 + Hq * D:] == 0).all()


def test_append_bad_slot_and_position_are_recorded():
    qkv = torch.ones((2, 3 * 64), dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    tp.tp_qkv_append([qkv], [kc], [vc], torch.tensor([0, 32], device="cuda"), positions=pos)
    assert tp.tp_query_status() == tp.TP_ERR_INVALID_ARG
    assert (vc[1] == 0).all() and (vc[0, :, 1:] == 0).all() and (vc[0, :, 0] == 1).all()
    tp.tp_qkv_append([qkv], [kc], [vc], torch.tensor([0, 1], device="cuda"), positions=pos + 9, rope=rope_table(9, 64))
    assert tp.tp_query_status() == tp.TP_ERR_INVALID_ARG
    assert tp.tp_query_status() == 0


# ------------------------------------------------------------------ attention
def paged(lens, N, Hk, D, page, dt, seed, fill=NAN, spare=2, std=1.0):
    """Caches whose rows outside every sequence hold `fill`, the block table (unused entries -1) and each
    sequence's keys and values (N, Hk, len, D)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    ids = rng.permutation(pages)[:sum(need)]
    width = max(need + [0]) + 1
    table = np.full((len(lens), width), -1, np.int32)
    kc = torch.full((N, pages, Hk, page, D), fill, device="cuda").to(dt)
    vc = torch.full((N, pages, Hk, page, D), fill, device="cuda").to(dt)
    kv, at = [], 0
    for b, n in enumerate(lens):
        mine = ids[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = mine
        k = (torch.randn((N, Hk, n, D), generator=g, device="cuda") * std).to(dt)
        v = torch.randn((N, Hk, n, D), generator=g, device="cuda").to(dt)
        for i, p in enumerate(mine):
            m = min(page, n - i * page)
            kc[:, p, :, :m], vc[:, p, :, :m] = k[:, :, i * page:i * page + m], v[:, :, i * page:i * page + m]
        kv.append((k, v))
    return kc, vc, torch.from_numpy(table).cuda(), kv


def attn_ref(q, k, v, seen, scale, cap):
    """q (R, G, D), k / v (n, D), seen (R, n): (o, sum_j p_j |v_j|) in float64, zero where a row sees nothing."""
    s = torch.einsum("rgd,nd->rgn", q.double(), k.double()) * scale
    if cap:
        s = cap * torch.tanh(s / cap)
    s = s.masked_fill(~seen[:, None], -float("inf"))
    p = torch.nan_to_num(torch.softmax(s, -1), nan=0.0) if s.shape[-1] else s
    return torch.einsum("rgn,nd->rgd", p, v.double()), torch.einsum("rgn,nd->rgd", p, v.double().abs())


def check_attention(got, q, kv, rows, lens, Hq, Hk, D, dt, scale, cap, window, prefix=None):
    """got, q (N, T, Hq D); rows[b] = (first row, rows)."""
    N, G = q.shape[0], Hq // Hk
    assert torch.isfinite(got.float()).all()
    for b, n in enumerate(lens):
        t0, m = rows[b]
        pos = n - m + torch.arange(m, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")[None]
        seen = j <= pos
        if window:
            seen = seen & (j > pos - window)
        if prefix is not None:
            seen = seen | (j < prefix[b])
        for r in range(N):
            for h in range(Hk):
                qq = q[r, t0:t0 + m].reshape(m, Hq, D)[:, h * G:(h + 1) * G]
                ref, mass = attn_ref(qq, kv[b][0][r, h], kv[b][1][r, h], seen, scale, cap)
                o = got[r, t0:t0 + m].reshape(m, Hq, D)[:, h * G:(h + 1) * G].double()
                tol = U[dt] * ref.abs() + (U[dt] + 2.0 ** -13) * mass + 2.0 ** -24
                if dt == torch.float16:
                    tol = tol + n * 2.0 ** -25 * 6
                bad = (o - ref).abs() > tol
                assert not bad.any(), (b, r, h, float(((o - ref).abs() / tol).max()))
                assert (o[~seen.any(1)] == 0).all()


def run_decode(lens, N, Hq, Hk, D, page, dt, cap=0.0, window=0, seed=0, std=1.0):
    kc, vc, table, kv = paged(lens, N, Hk, D, page, dt, seed, std=std)
    B = len(lens)
    q = torch.randn((N, B, Hq * D), device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed + 1)).to(dt)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o = tp.tp_paged_decode(q, kc, vc, table, seq, softcap=cap, window=window)
    status_ok()
    check_attention(o, q, kv, [(b, 1) for b in range(B)], lens, Hq, Hk, D, dt, D ** -0.5, cap, window)
    return o, (q, kc, vc, table, seq)


BF, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("lens,N,Hq,Hk,D,page,dt,cap,window", [
    ([1], 1, 1, 1, 128, 16, BF, 0.0, 0),
    ([0], 1, 4, 2, 64, 16, BF, 0.0, 0),
    ([0, 0, 17, 0], 2, 4, 2, 128, 16, F16, 0.0, 0),
    ([1, 15, 16, 17, 31, 127, 128, 129, 255, 257], 1, 8, 2, 128, 16, BF, 0.0, 0),
    ([1, 2, 63, 64, 65, 300], 3, 6, 2, 64, 32, F16, 0.0, 0),
    ([517], 1, 32, 8, 128, 16, BF, 0.0, 0),
    ([1000, 3, 0, 777], 2, 16, 1, 128, 256, BF, 0.0, 0),
    ([1000, 3, 0, 777], 2, 9, 1, 64, 64, BF, 0.0, 0),
    ([400, 90], 1, 40, 2, 128, 128, F16, 0.0, 0),
    ([300, 41], 1, 71, 1, 64, 16, BF, 0.0, 0),
    ([2000, 1999, 100, 5], 2, 5, 5, 128, 64, F16, 20.0, 0),
    ([2000, 1999, 100, 5, 0], 1, 14, 2, 64, 16, BF, 0.0, 100),
    ([513, 1, 16, 17], 1, 8, 8, 128, 32, BF, 5.0, 1),
    ([513, 129, 16, 17], 4, 3, 3, 64, 128, F16, 50.0, 16),
    ([9001], 1, 2, 1, 128, 64, BF, 0.0, 0),
    ([20000, 1], 1, 8, 1, 64, 16, F16, 0.0, 0)])
def test_decode(policy, lens, N, Hq, Hk, D, page, dt, cap, window):
    run_decode(lens, N, Hq, Hk, D, page, dt, cap, window)


@pytest.mark.parametrize("cap", [0.25, 1e3, 1e4, 1e6, 1e30])
def test_caps_far_from_the_scores(policy, cap):
    """Scores far below the cap are themselves; far above it they are the cap."""
    run_decode([700, 33], 1, 8, 2, 64, 16, F16, cap)
    run_prefill([(40, 300), (150, 150)], 1, 8, 2, 64, 16, F16, cap)


def test_decode_many_sequences(policy):
    rng = np.random.default_rng(3)
    run_decode([int(n) for n in rng.integers(0, 90, 700)], 1, 4, 2, 64, 16, BF)


def test_decode_large_scores(policy):
    run_decode([300, 33, 700], 1, 8, 2, 128, 16, BF, std=30.0)


def test_decode_peak_at_the_end_and_the_front(policy):
    """The running maximum rises late, and falls: the sums have to be rescaled, and not by a stale maximum."""
    D, n = 64, 640
    for peak in (0, 5, 127, 128, 639):
        kc, vc, table, kv = paged([n], 1, 1, D, 16, F16, seed=peak)
        k = kv[0][0]
        k.mul_(0.01)
        k[0, 0, peak] = 4.0
        for i in range(n // 16):
            kc[0, table[0, i], 0] = k[0, 0, 16 * i:16 * i + 16]
        q = torch.full((1, 1, D), 2.0, dtype=F16, device="cuda")
        o = tp.tp_paged_decode(q, kc, vc, table, torch.tensor([n], dtype=torch.int32, device="cuda"))
        status_ok()
        check_attention(o, q, kv, [(0, 1)], [n], 1, 1, D, F16, D ** -0.5, 0.0, 0)


def test_decode_repeats_bit_for_bit():
    o, args = run_decode([3000, 1, 700, 0, 64], 2, 8, 2, 128, 64, BF)
    for _ in range(4):
        assert torch.equal(tp.tp_paged_decode(*args), o)


def test_decode_lists_strides_other_stream_and_prepare():
    lens, N, Hq, Hk, D, page = [77, 300, 16], 2, 8, 2, 64, 16
    o, (q, kc, vc, table, seq) = run_decode(lens, N, Hq, Hk, D, page, BF)
    B, P = len(lens), kc.shape[1]
    kv = [torch.zeros((P, 2, Hk, page, D), dtype=BF, device="cuda") for _ in range(N)]
    qw = [torch.zeros((B, Hq * D + 7), dtype=BF, device="cuda") for _ in range(N)]
    ow = [torch.zeros((B, Hq * D + 9), dtype=BF, device="cuda") for _ in range(N)]
    wide = torch.full((B, table.shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    for r in range(N):
        kv[r][:, 0], kv[r][:, 1], qw[r][:, 5:5 + Hq * D] = kc[r], vc[r], q[r]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = ([x[:, 5:5 + Hq * D] for x in qw], [x[:, 0] for x in kv], [x[:, 1] for x in kv], wide[:, :table.shape[1]], seq)
    out = [x[:, 1:1 + Hq * D] for x in ow]
    call = tp.prepare(tp.tp_paged_decode, *args, out=out)
    call(s)
    s.synchronize()
    for r in range(N):
        assert torch.equal(out[r], o[r])
        assert (ow[r][:, 0] == 0).all() and (ow[r][:, 1 + Hq * D:] == 0).all()


def test_decode_in_a_graph():
    o, args = run_decode([3000, 1, 700, 0, 64], 2, 8, 2, 128, 64, BF)
    out = torch.zeros_like(o)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    tp.tp_paged_decode(*args, out=out, stream=s)  # the stream's workspace
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        tp.tp_paged_decode(*args, out=out, stream=s)
    out.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o)


def test_decode_bad_page_and_length_are_recorded(policy):
    _, (q, kc, vc, table, seq) = run_decode([40, 20], 1, 2, 1, 64, 16, BF)
    for bad in (-1, kc.shape[1], 1 << 30):
        t2 = table.clone()
        t2[0, 1] = bad
        tp.tp_paged_decode(q, kc, vc, t2, seq)
        assert tp.tp_query_status() == tp.TP_ERR_INVALID_ARG
    tp.tp_paged_decode(q, kc, vc, table, seq + 100000)
    assert tp.tp_query_status() == tp.TP_ERR_INVALID_ARG
    tp.tp_paged_decode(q, kc, vc, table, seq - 100000)  # a negative length is an empty sequence
    torch.cuda.synchronize()
    assert tp.tp_query_status() in (0, tp.TP_ERR_INVALID_ARG)
    tp.tp_paged_decode(q, kc, vc, table, seq)
    assert tp.tp_query_status() == 0


def test_negative_lengths_and_disordered_offsets_are_recorded(policy):
    """A negative length is out of range, and counts as an empty sequence; so are offsets that do not ascend."""
    _, (q, kc, vc, table, seq) = run_decode([40, 20, 33], 1, 2, 1, 64, 16, BF)
    for n in (-1, -100000, -2 ** 31):
        bad = seq.clone()
        bad[1] = n
        o = tp.tp_paged_decode(q, kc, vc, table, bad)
        assert tp.tp_query_status() == tp.TP_ERR_INVALID_ARG
        assert (o[0, 1] == 0).all()
    o, (q, kc, vc, table, cu, seq, _) = run_prefill([(40, 0), (20, 4), (33, 50)], 1, 2, 1, 64, 16, BF)
    for n in (-1, -100000, -2 ** 31):
        bad = seq.clone()
        bad[1] = n
        got = tp.tp_paged_prefill(q, kc, vc, table, cu, bad)
        assert tp.tp_query_status() == tp.TP_ERR_INVALID_ARG
        assert (got[0, 40:60] == 0).all()
    for at, n in ((0, -1), (1, 61), (3, 94), (2, 1000)):
        bad = cu.clone()
        bad[at] = n
        tp.tp_paged_prefill(q, kc, vc, table, bad, seq)
        assert tp.tp_query_status() == tp.TP_ERR_INVALID_ARG, (at, n)
    assert torch.equal(tp.tp_paged_prefill(q, kc, vc, table, cu, seq), o)
    status_ok()


def test_prefix_lengths_beyond_the_sequence(policy):
    """A prefix longer than its sequence is the whole of it, one below zero is none: no error."""
    chunks = [(40, 30), (20, 4), (33, 50)]
    same, args = run_prefill(chunks, 1, 4, 2, 64, 16, F16, prefix=[70, 0, 83])
    over = torch.tensor([2 ** 31 - 1, -2 ** 31, 1000], dtype=torch.int32, device="cuda")
    assert torch.equal(tp.tp_paged_prefill(*args[:6], over), same)
    status_ok()


def test_the_longest_sequences(policy):
    """Positions up to 2^30 (a table of one page repeated, the window at the end); one more is out of range."""
    page, D, W = 256, 64, 40
    kc = torch.randn((1, 1, 1, page, D), device="cuda").to(BF)
    vc = torch.randn((1, 1, 1, page, D), device="cuda").to(BF)
    table = torch.zeros((1, 1 << 23), dtype=torch.int32, device="cuda")
    q = torch.randn((1, 5, 2 * D), device="cuda").to(BF)
    cu = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    for n in (1 << 30, (1 << 30) - 77):
        seq = torch.tensor([n], dtype=torch.int32, device="cuda")
        o = tp.tp_paged_prefill(q, kc, vc, table, cu, seq, window=W)
        d = tp.tp_paged_decode(q[:, 4:], kc, vc, table, seq, window=W)
        status_ok()
        at = torch.arange(n - 4 - W, n, device="cuda") % page  # what the five rows can see
        kv = [(kc[:, 0][:, :, at], vc[:, 0][:, :, at])]
        check_attention(o, q, kv, [(0, 5)], [W + 4], 2, 1, D, BF, D ** -0.5, 0.0, W)
        check_attention(d, q[:, 4:], kv, [(0, 1)], [W + 4], 2, 1, D, BF, D ** -0.5, 0.0, W)
    for n in ((1 << 30) + 1, (1 << 31) - 1):
        seq = torch.tensor([n], dtype=torch.int32, device="cuda")
        tp.tp_paged_prefill(q, kc, vc, table, cu, seq, window=W)
        assert tp.tp_query_status() == tp.TP_ERR_INVALID_ARG
        tp.tp_paged_decode(q[:, 4:], kc, vc, table, seq, window=W)
        assert tp.tp_query_status() == tp.TP_ERR_INVALID_ARG


def test_the_widest_window_hides_nothing(policy):
    """A window of 2^31 - 1, with rows before the first position too, is no window."""
    kc, vc, table, kv = paged([10, 300], 1, 1, 64, 16, BF, seed=8)
    q = torch.randn((1, 320, 128), device="cuda").to(BF)
    cu = torch.tensor([0, 17, 320], dtype=torch.int32, device="cuda")
    seq = torch.tensor([10, 300], dtype=torch.int32, device="cuda")
    for window in (2 ** 31 - 1, 2 ** 31 - 20, 2 ** 30):
        o = tp.tp_paged_prefill(q, kc, vc, table, cu, seq, window=window)
        status_ok()
        assert torch.equal(o, tp.tp_paged_prefill(q, kc, vc, table, cu, seq))
        check_attention(o, q, kv, [(0, 17), (17, 303)], [10, 300], 2, 1, 64, BF, 0.125, 0.0, 0)
        d = tp.tp_paged_decode(q[:, :2], kc, vc, table, seq, window=window)
        assert torch.equal(d, tp.tp_paged_decode(q[:, :2], kc, vc, table, seq))


def test_a_bad_value_on_one_stream_leaves_others_alone():
    """Asking for the status while other streams' kernels join their parts: they count on, and leave no count behind."""
    d, dargs = run_decode([9000, 1, 700, 64], 1, 8, 2, 128, 64, BF)
    p, pargs = run_prefill([(4, 9000), (20, 300)], 1, 8, 2, 128, 64, BF)
    qkv = torch.ones((2, 3 * 64), dtype=BF, device="cuda")
    kc = torch.zeros((2, 1, 16, 64), dtype=BF, device="cuda")
    bad = torch.tensor([0, 32], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs, seen = [], 0
    for _ in range(60):
        with torch.cuda.stream(side):
            for _ in range(8):
                outs.append((tp.tp_paged_decode(*dargs), tp.tp_paged_prefill(*pargs)))
        tp.tp_qkv_append([qkv], [kc], [kc.clone()], bad)
        seen += tp.tp_query_status() == tp.TP_ERR_INVALID_ARG
    assert seen == 60
    side.synchronize()
    for a, b in outs:
        assert torch.equal(a, d) and torch.equal(b, p)
    status_ok()


def test_errors_behind_a_cleared_status_are_kept():
    """The word is clear when the query returns: a call on another stream right behind it may set it again."""
    qkv = torch.ones((2, 3 * 64), dtype=BF, device="cuda")
    kc, vc = (torch.zeros((2, 1, 16, 64), dtype=BF, device="cuda") for _ in range(2))
    bad = torch.tensor([0, 32], device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    tp.tp_qkv_append([qkv], [kc], [vc], bad)
    for _ in range(200):
        assert tp.tp_query_status() == tp.TP_ERR_INVALID_ARG
        with torch.cuda.stream(side):
            tp.tp_qkv_append([qkv], [kc], [vc], bad)
        side.synchronize()
    assert tp.tp_query_status() == tp.TP_ERR_INVALID_ARG
    status_ok()


def test_timeouts_stay_over_bad_values():
    """Both in the status word: the timeout is reported, as the counters have to be cleared after it."""
    qkv = torch.ones((2, 3 * 64), dtype=BF, device="cuda")
    kc = torch.zeros((2, 1, 16, 64), dtype=BF, device="cuda")
    bad = torch.tensor([0, 32], device="cuda")
    for first in (True, False):
        if first:
            tp.tp_qkv_append([qkv], [kc], [kc.clone()], bad)
        tp.tp_debug_wait_timeout(2000000)
        if not first:
            tp.tp_qkv_append([qkv], [kc], [kc.clone()], bad)
        assert tp.tp_query_status() == tp.TP_ERR_TIMEOUT
        assert tp.tp_query_status() == 0


def test_a_cache_beyond_32_bit_offsets():
    """Pages whose byte and element offsets pass 2^32 (a 17 GB key cache)."""
    Hk, page, D = 8, 256, 128
    pages = (1 << 33) // (Hk * page * D) + 2
    kc = torch.zeros((pages, Hk, page, D), dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    q = torch.randn((1, 1, Hk * D), device="cuda").to(BF)
    x = torch.randn((1, 300, 3 * Hk * D), device="cuda").to(BF)
    slots = torch.cat([torch.arange(256, device="cuda") + (pages - 1) * page, torch.arange(44, device="cuda") + page])
    tp.tp_qkv_append(x, [kc], [vc], slots)
    status_ok()
    k, v = (x[0, :, i * Hk * D:(i + 1) * Hk * D].view(300, Hk, D).transpose(0, 1) for i in (1, 2))
    assert torch.equal(kc[pages - 1], k[:, :256]) and torch.equal(vc[pages - 1], v[:, :256])
    assert torch.equal(kc[1, :, :44], k[:, 256:]) and (kc[1, :, 44:] == 0).all()
    table = torch.tensor([[pages - 1, 1]], dtype=torch.int32, device="cuda")
    for chunk in (False, True):
        n = torch.tensor([300], dtype=torch.int32, device="cuda")
        if chunk:
            o = tp.tp_paged_prefill(q, [kc], [vc], table, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), n)
        else:
            o = tp.tp_paged_decode(q, [kc], [vc], table, n)
        status_ok()
        check_attention(o, q, [(k[None], v[None])], [(0, 1)], [300], Hk, Hk, D, BF, D ** -0.5, 0.0, 0)


def run_prefill(chunks, N, Hq, Hk, D, page, dt, cap=0.0, window=0, prefix=None, seed=0, std=1.0):
    """chunks: (new tokens, cached before them) of each sequence."""
    lens = [m + c for m, c in chunks]
    kc, vc, table, kv = paged(lens, N, Hk, D, page, dt, seed, std=std)
    cu = np.concatenate([[0], np.cumsum([m for m, _ in chunks])]).astype(np.int32)
    T = int(cu[-1])
    q = torch.randn((N, T, Hq * D), device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed + 1)).to(dt)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pre = torch.tensor(prefix, dtype=torch.int32, device="cuda") if prefix is not None else None
    args = (q, kc, vc, table, torch.from_numpy(cu).cuda(), seq, pre)
    o = tp.tp_paged_prefill(*args, softcap=cap, window=window)
    status_ok()
    check_attention(o, q, kv, [(int(cu[b]), chunks[b][0]) for b in range(len(chunks))], lens, Hq, Hk, D, dt, D ** -0.5,
                    cap, window, prefix)
    return o, args


@pytest.mark.parametrize("chunks,N,Hq,Hk,D,page,dt,cap,window,prefix", [
    ([(1, 0)], 1, 1, 1, 128, 16, BF, 0.0, 0, None),
    ([(1, 40)], 1, 8, 2, 64, 16, F16, 0.0, 0, None),
    ([(0, 5), (3, 0), (0, 0), (20, 0)], 2, 4, 2, 128, 16, BF, 0.0, 0, None),
    ([(127, 0), (128, 0), (129, 0)], 1, 2, 2, 128, 64, BF, 0.0, 0, None),
    ([(150, 60), (7, 90), (33, 1), (64, 64)], 2, 8, 2, 64, 16, F16, 20.0, 0, None),
    ([(300, 0)], 1, 7, 1, 128, 128, BF, 0.0, 0, None),
    ([(300, 200)], 1, 5, 1, 64, 256, BF, 0.0, 0, None),
    ([(77, 300)], 2, 48, 3, 128, 32, F16, 0.0, 0, None),
    ([(40, 3)], 1, 130, 1, 64, 16, BF, 0.0, 0, None),
    ([(600, 100), (1, 500)], 1, 8, 2, 128, 16, BF, 0.0, 100, None),
    ([(600, 0)], 1, 4, 4, 64, 64, F16, 30.0, 1, None),
    ([(300, 100), (90, 0), (5, 200)], 1, 8, 2, 128, 16, BF, 0.0, 0, [350, 0, 1]),
    ([(700, 100), (90, 0)], 1, 4, 1, 64, 32, BF, 0.0, 33, [90, 90]),
    ([(1030, 2000)], 1, 4, 1, 128, 64, BF, 0.0, 0, None)])
def test_prefill(policy, chunks, N, Hq, Hk, D, page, dt, cap, window, prefix):
    run_prefill(chunks, N, Hq, Hk, D, page, dt, cap, window, prefix)


@pytest.mark.parametrize("N,Hq,Hk,D,chunks", [(9, 2, 1, 64, [(40, 3), (1, 100)]), (64, 1, 1, 128, [(130, 0)]),
                                              (64, 3, 1, 64, [(3, 4000), (2, 17)]), (33, 2, 2, 128, [(300, 200)])])
@pytest.mark.parametrize("dt", [BF, F16])
def test_attention_of_many_ranks(policy, N, Hq, Hk, D, chunks, dt):
    """More than eight ranks in one call, up to 64: prefill has a form of its own for them."""
    run_prefill(chunks, N, Hq, Hk, D, 16, dt, prefix=[20] * len(chunks))
    run_decode([m + c for m, c in chunks], N, Hq, Hk, D, 16, dt)


def test_prefill_large_scores(policy):
    run_prefill([(260, 100), (33, 0)], 1, 8, 2, 128, 16, BF, std=30.0)


def test_prefill_many_sequences(policy):
    rng = np.random.default_rng(4)
    run_prefill([(int(a), int(b)) for a, b in zip(rng.integers(0, 9, 300), rng.integers(0, 60, 300))], 1, 4, 2, 64, 16, BF)


def test_prefill_rows_before_the_first_position_and_of_no_sequence(policy):
    """More new tokens than positions: the first rows see nothing.  Rows outside cu_seqlens are zero."""
    kc, vc, table, kv = paged([10, 30], 1, 1, 64, 16, BF, seed=8)
    q = torch.randn((1, 60, 128), device="cuda").to(BF)
    cu = torch.tensor([3, 20, 50], dtype=torch.int32, device="cuda")
    seq = torch.tensor([10, 30], dtype=torch.int32, device="cuda")
    o = tp.tp_paged_prefill(q, kc, vc, table, cu, seq, out=torch.full_like(q, NAN))
    status_ok()
    assert (o[0, :3] == 0).all() and (o[0, 50:] == 0).all()
    check_attention(o, q, kv, [(3, 17), (20, 30)], [10, 30], 2, 1, 64, BF, 0.125, 0.0, 0)


def test_prefill_of_one_token_is_decode():
    lens = [77, 300, 16]
    o, (q, kc, vc, table, seq) = run_decode(lens, 2, 8, 2, 64, 16, BF)
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    o2 = tp.tp_paged_prefill(q, kc, vc, table, cu, seq)
    status_ok()
    assert ((o - o2).float().abs() <= 2 * U[BF] * (o.float().abs() + 1)).all()


@pytest.mark.parametrize("chunks,N,Hq,Hk,D,page,dt,cap,window", [
    ([(1, 9000)], 1, 8, 2, 128, 16, BF, 0.0, 0),
    ([(4, 16000)], 1, 32, 8, 128, 64, F16, 0.0, 0),
    ([(5, 5000), (0, 700), (3, 12), (17, 4097), (2, 1)], 2, 6, 2, 64, 32, BF, 20.0, 0),
    ([(64, 8192)], 1, 4, 4, 128, 128, BF, 0.0, 0),
    ([(300, 6000), (700, 700)], 1, 8, 1, 128, 16, F16, 0.0, 3000),
    ([(1100, 1100)], 1, 2, 2, 128, 16, BF, 0.0, 0),
    ([(129, 3000), (40, 2999), (1, 3001)], 4, 3, 3, 64, 256, F16, 0.0, 0),
    ([(16, 4000)], 1, 150, 1, 64, 16, BF, 0.0, 0),
    ([(2, 300)] * 40 + [(3, 9000)], 1, 4, 2, 64, 16, BF, 0.0, 0)])
def test_prefill_tiles_shared_between_ctas(policy, chunks, N, Hq, Hk, D, page, dt, cap, window):
    """Few rows over long caches: the key tiles of a block are divided, and joined."""
    chunks = [(min(a, b), b) for a, b in chunks]
    run_prefill(chunks, N, Hq, Hk, D, page, dt, cap, window)
    run_prefill(chunks, N, Hq, Hk, D, page, dt, cap, window, seed=5)  # the counters are clear again


@pytest.mark.parametrize("tokens,Hq,Hk,D", [(1, 8, 2, 128), (1, 8, 1, 64), (3, 8, 2, 64), (2, 8, 1, 128), (9, 8, 2, 64),
                                            (40, 8, 1, 128)])
def test_prefill_joins_of_few_and_many_rows_repeat(tokens, Hq, Hk, D):
    """Joins where 8, 16 or all 32 lanes of a warp have rows of their own, again and again with other work between:
    each reads every part that other CTAs have left."""
    o, args = run_prefill([(tokens, 6000), (1, 40)], 2, Hq, Hk, D, 16, BF)
    other = torch.randn((1 << 24,), device="cuda")
    outs = []
    for i in range(40):
        outs.append(tp.tp_paged_prefill(*args))
        if i % 4 == 0:
            other.mul_(1.0)
    status_ok()
    for x in outs:
        assert torch.equal(x, o)


@pytest.mark.parametrize("chunks,N,Hq,Hk,D,page,dt,cap,window,prefix", [
    ([(1, 0), (130, 0), (37, 200)], 1, 4, 2, 64, 16, BF, 0.0, 0, None),
    ([(600, 100), (3, 500)], 2, 6, 2, 128, 32, F16, 0.0, 90, None),
    ([(300, 100), (90, 0)], 1, 7, 1, 128, 128, BF, 20.0, 0, [150, 20]),
    ([(260, 40)], 1, 130, 1, 64, 16, BF, 0.0, 33, [60]),
    ([(5, 6000)], 2, 8, 2, 128, 64, BF, 0.0, 0, None),  # from here on key tiles shared between CTAs
    ([(40, 5000), (9, 700)], 1, 4, 1, 64, 16, F16, 0.0, 0, None),
    ([(64, 8192)], 1, 4, 4, 128, 128, BF, 30.0, 3000, None)])
def test_prefill_values_that_are_not_finite(policy, chunks, N, Hq, Hk, D, page, dt, cap, window, prefix):
    """Infinities and NaN in the values (whole rows, and single columns) and keys of single positions: a row that
    does not see the position is as without it."""
    chunks = [(min(a, b) if b > 1000 else a, b) for a, b in chunks]
    lens = [m + c for m, c in chunks]
    kc, vc, table, kv = paged(lens, N, Hk, D, page, dt, seed=3)
    g = torch.Generator().manual_seed(len(chunks) + Hq)
    poison = []  # of each sequence: (n, D), which values are not finite
    for b, n in enumerate(lens):
        mark = torch.zeros((n, D), dtype=torch.bool, device="cuda")
        # the last positions, which most of the chunk's rows do not see, and some others
        for i, j in enumerate({n - 1, max(0, n - 3), min(n - 1, n - chunks[b][0] // 2), int(torch.randint(n, (1,), generator=g))}):
            cols = slice(None) if i % 2 else slice(5, 6)
            at = int(table[b, j // page])
            row = vc[:, at, :, j % page]  # a view: (N, Hk, D)
            row[..., cols] = [NAN, float("inf"), -float("inf")][i % 3]
            kv[b][1][:, :, j, cols] = 0.0
            mark[j, cols] = True
            if i % 2 and j == n - 1 and chunks[b][0] > 1:  # its key too: rows that see it are NaN all over
                kc[:, at, :, j % page] = NAN
                mark[j] = True
                kv[b][0][:, :, j] = 0.0
        poison.append(mark)
    cu = np.concatenate([[0], np.cumsum([m for m, _ in chunks])]).astype(np.int32)
    q = torch.randn((N, int(cu[-1]), Hq * D), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(dt)
    wide = torch.empty((N, int(cu[-1]), Hq * D + 1), dtype=dt, device="cuda")
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pre = torch.tensor(prefix, dtype=torch.int32, device="cuda") if prefix else None
    for out in (torch.empty_like(q), wide[..., 1:]):
        o = tp.tp_paged_prefill(q, kc, vc, table, torch.from_numpy(cu).cuda(), seq, pre, softcap=cap, window=window, out=out)
        status_ok()
        clean, hit = o.clone(), torch.zeros(q.shape, dtype=torch.bool, device="cuda")
        for b, n in enumerate(lens):
            m, t0 = chunks[b][0], int(cu[b])
            pos, j = n - m + torch.arange(m, device="cuda")[:, None], torch.arange(n, device="cuda")[None]
            seen = (j <= pos) & (j > pos - window if window else j >= 0) | (j < (prefix[b] if prefix else 0))
            bad = (seen.double() @ poison[b].double()) > 0  # (m, D)
            hit[:, t0:t0 + m] = bad.repeat(1, Hq)
            # what sees a poisoned position is not compared with the reference, which lacks it
            for r in range(N):
                for h in range(Hk):
                    G = Hq // Hk
                    ref, mass = attn_ref(q[r, t0:t0 + m].reshape(m, Hq, D)[:, h * G:(h + 1) * G], kv[b][0][r, h],
                                         kv[b][1][r, h], seen, D ** -0.5, cap)
                    got = clean[r, t0:t0 + m].reshape(m, Hq, D)[:, h * G:(h + 1) * G].double()
                    tol = U[dt] * ref.abs() + (U[dt] + 2.0 ** -13) * mass + 2.0 ** -24
                    if dt == torch.float16:
                        tol = tol + n * 2.0 ** -25 * 6
                    assert (((got - ref).abs() <= tol) | bad[:, None]).all(), (b, r, h)
        assert torch.isfinite(o[~hit]).all() and not torch.isfinite(o[hit]).any()


def test_prefill_shared_tiles_repeat_bitwise():
    o, args = run_prefill([(33, 7000), (90, 2500)], 1, 8, 2, 128, 32, BF)
    for _ in range(5):
        assert torch.equal(tp.tp_paged_prefill(*args), o)


def test_prefill_shared_tiles_in_a_graph():
    """Replayed on new queries: the arrival counts are clear after every run."""
    o, args = run_prefill([(4, 9000), (20, 300)], 1, 8, 2, 128, 64, F16)
    q, out = args[0].clone(), torch.empty_like(o)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    tp.tp_paged_prefill(q, *args[1:], out=out, stream=s)  # the stream's workspace
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        tp.tp_paged_prefill(q, *args[1:], out=out, stream=s)
    for seed in range(3):
        q.copy_(torch.randn(q.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, tp.tp_paged_prefill(q, *args[1:]))
    status_ok()


def test_prefill_strides_other_stream():
    o, (q, kc, vc, table, cu, seq, _) = run_prefill([(50, 20), (200, 0)], 2, 4, 2, 128, 16, F16)
    N, T, C = q.shape
    qw = torch.zeros((N, T, C + 8), dtype=F16, device="cuda")
    qw[:, :, :C] = q
    qo = torch.zeros((N, T, C + 1), dtype=F16, device="cuda")
    qo[:, :, 1:] = q
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for view in (qw[:, :, :C], qo[:, :, 1:]):
        ow = torch.zeros((N, T, C + 3), dtype=F16, device="cuda")
        torch.cuda.synchronize()
        tp.tp_paged_prefill(view, kc, vc, table, cu, seq, out=ow[:, :, 2:2 + C], stream=s)
        s.synchronize()
        assert torch.equal(ow[:, :, 2:2 + C], o)
        assert (ow[:, :, :2] == 0).all() and (ow[:, :, 2 + C:] == 0).all()


def test_prefill_bad_page_and_length_are_recorded(policy):
    _, (q, kc, vc, table, cu, seq, _) = run_prefill([(40, 0), (20, 4)], 1, 2, 1, 64, 16, BF)
    t2 = table.clone()
    t2[0, 1] = kc.shape[1]
    tp.tp_paged_prefill(q, kc, vc, t2, cu, seq)
    assert tp.tp_query_status() == tp.TP_ERR_INVALID_ARG
    tp.tp_paged_prefill(q, kc, vc, table, cu, seq + 100000)
    assert tp.tp_query_status() == tp.TP_ERR_INVALID_ARG
    tp.tp_paged_prefill(q, kc, vc, table, cu, seq)
    assert tp.tp_query_status() == 0


# ------------------------------------------------------------------ float16 over long rows
def float16_reference(q, k, v, seen, scale):
    """q (R, G, D), k / v (n, D), seen (R, n) in float64: the output, its tolerance, and the smallest of any 128
    consecutive positions' largest share of the tolerance, were they left out.

    A term e = 2^(s - m) is rounded by 2^-11 of itself, or by 2^-25 where it is below 2^-14.  Every m is a score of
    the row (that of a part of it), so relative to the row's largest score the latter is 2^-25 at most, and 2^-25
    sum |v_j| / L of the output, L being the softmax's sum relative to that score."""
    u = U[torch.float16]
    s = torch.einsum("rgd,nd->rgn", q.double(), k.double()) * scale
    s = s.masked_fill(~seen[:, None], -float("inf"))
    e = torch.exp(s - s.amax(-1, keepdim=True))
    L = e.sum(-1, keepdim=True)
    v = v.double()
    sums = torch.einsum("rgn,nd->rgd", e, v)
    ref, mass = sums / L, torch.einsum("rgn,nd->rgd", e, v.abs()) / L
    small = torch.einsum("rn,nd->rd", seen.double(), v.abs())[:, None] * 2.0 ** -25 / L
    tol = u * ref.abs() + (u + 2.0 ** -13) * mass + small + 2.0 ** -25
    least = float("inf")
    for j in range(0, k.shape[0], 128):
        part = torch.einsum("rgn,nd->rgd", e[..., j:j + 128], v[j:j + 128])
        rest = L - e[..., j:j + 128].sum(-1, keepdim=True)
        without = torch.where(rest > 0, (sums - part) / rest, 0.0)
        least = min(least, float(((without - ref).abs() / tol).max()))
    return ref, tol, least


@pytest.mark.parametrize("tokens,n,Hq,Hk,D,page", [(1, 20060, 8, 1, 64, 16), (1, 9061, 4, 2, 128, 64),
                                                   (1, 4190, 32, 8, 128, 16), (4, 16100, 8, 2, 128, 64),
                                                   (40, 5080, 4, 1, 64, 16), (3, 20063, 4, 2, 64, 256)])
def test_float16_long_rows(policy, tokens, n, Hq, Hk, D, page):
    """Close enough to see any 128 positions left out."""
    kc, vc, table, kv = paged([n], 1, Hk, D, page, F16, seed=n)
    g = torch.Generator(device="cuda").manual_seed(n + 1)  # not the keys' own
    q = torch.randn((1, tokens, Hq * D), generator=g, device="cuda").to(F16)
    seq = torch.tensor([n], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    outs = [tp.tp_paged_prefill(q, kc, vc, table, cu, seq)]
    if tokens == 1:
        outs.append(tp.tp_paged_decode(q, kc, vc, table, seq))
    status_ok()
    G = Hq // Hk
    seen = torch.arange(n, device="cuda")[None] <= n - tokens + torch.arange(tokens, device="cuda")[:, None]
    for h in range(Hk):
        part = slice(h * G, (h + 1) * G)
        ref, tol, least = float16_reference(q[0].reshape(tokens, Hq, D)[:, part], kv[0][0][0, h], kv[0][1][0, h], seen,
                                            D ** -0.5)
        assert least > 1
        for o in outs:
            assert ((o[0].reshape(tokens, Hq, D)[:, part].double() - ref).abs() <= tol).all()


# ------------------------------------------------------------------ sampling
def kept_set(x, t, k, p, m, slack):
    """Indices that may be kept and those that must be, in float64, `slack` the allowed relative error of a share."""
    order = np.argsort(-x, kind="stable")
    e = np.exp((x[order] - x[order[0]]) / t)
    n = len(x) if k <= 0 else min(k, len(x))
    before = np.cumsum(e[:n]) - e[:n]
    total = e[:n].sum()

    def cut(sign):
        keep = np.ones(n, bool) if p >= 1 else before < (p + sign * slack) * total
        keep &= e[:n] >= min(m, 1.0) * (1 - sign * slack)
        keep[0] = True  # the largest is always kept
        return set(order[:n][keep].tolist())
    return cut(+1), cut(-1)


def check_draw(x, token, t, k, p, m, u, slack=2e-5):
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max)).astype(np.float64)
    if t < 2.0 ** -20:
        t, k = 1.0, 1
    may, must = kept_set(x, t, k, p, m, slack)
    assert token in may
    w = np.exp((x - x.max()) / t)
    hi = sum(w[i] for i in may if i <= token) / sum(w[i] for i in must)
    lo = sum(w[i] for i in must if i < token) / sum(w[i] for i in may)
    assert lo - slack <= u <= hi + slack, (lo, u, hi)


@pytest.mark.parametrize("B,V,dt", [(1, 1, torch.float32), (3, 2, torch.float16), (5, 31, torch.bfloat16),
                                    (64, 1000, torch.float32), (40, 5001, torch.bfloat16), (9, 50272, torch.float32),
                                    (7, 50272, torch.float16), (3, 200003, torch.float32), (2, 1 << 20, torch.bfloat16)])
def test_sample(B, V, dt):
    rng = np.random.default_rng(B + V)
    x = torch.from_numpy(rng.standard_normal((B, V + 3)).astype(np.float32) * 2.5).cuda().to(dt)[:, 1:V + 1]
    u = rng.random(B, dtype=np.float32)
    t = rng.choice(np.float32([0, 0.3, 0.7, 1, 1.5, 5]), B).astype(np.float32)
    k = rng.choice([0, -1, 1, 2, 50, 1000, 1 << 30], B).astype(np.int32)
    p = rng.choice(np.float32([1, 0, 1e-4, 0.3, 0.9, 0.999, 2]), B).astype(np.float32)
    m = rng.choice(np.float32([0, 0, 0.01, 0.3, 1, 7]), B).astype(np.float32)
    dev = [torch.from_numpy(a).cuda() for a in (u, t, k, p, m)]
    tok, lp = tp.tp_sample(x, *dev)
    status_ok()
    xh = x.double().cpu().numpy()
    tok, lp = tok.cpu().numpy(), lp.cpu().numpy()
    for b in range(B):
        check_draw(xh[b], int(tok[b]), float(t[b]), int(k[b]), float(p[b]), float(m[b]), float(u[b]))
        z = xh[b] - xh[b].max()
        ref = z[tok[b]] - np.log(np.exp(z).sum())
        assert abs(lp[b] - ref) <= 1e-5 * (1 + abs(ref))


@pytest.mark.parametrize("B,V", [(200, 300), (1500, 77), (170, 60000)])
def test_sample_more_rows_than_the_gpu_holds(B, V):
    """Rows are then taken in another order: each must still get its own parameters and place."""
    rng = np.random.default_rng(B)
    x = torch.from_numpy(rng.standard_normal((B, V)).astype(np.float32) * 2).cuda()
    u = rng.random(B, dtype=np.float32)
    t = rng.choice(np.float32([0, 0.7, 1, 1.5]), B).astype(np.float32)
    k = rng.choice([0, 1, 20, 300, 5000], B).astype(np.int32)
    p = rng.choice(np.float32([1, 0.3, 0.9, 0.999]), B).astype(np.float32)
    m = rng.choice(np.float32([0, 0.01]), B).astype(np.float32)
    tok, _ = tp.tp_sample(x, *[torch.from_numpy(a).cuda() for a in (u, t, k, p, m)])
    status_ok()
    xh, tok = x.double().cpu().numpy(), tok.cpu().numpy()
    for b in range(B):
        check_draw(xh[b], int(tok[b]), float(t[b]), int(k[b]), float(p[b]), float(m[b]), float(u[b]))


@pytest.mark.parametrize("t", [1e-5, 1e-2, 100.0, 1e30, float("inf")])
def test_sample_extreme_temperatures(t):
    """Narrow and flat distributions: top-p ends among few values, or among all of a flat row."""
    B, V = 4, 40000
    x = torch.randn((B, V), device="cuda") * 3
    u = torch.tensor([0.0, 0.3, 0.6, 0.95], device="cuda")
    p = torch.tensor([0.9, 0.5, 1.0, 0.99], device="cuda")
    k = torch.tensor([0, 0, 3000, 1500], dtype=torch.int32, device="cuda")
    tok, _ = tp.tp_sample(x, u, temperature=torch.full((B,), t, device="cuda"), top_k=k, top_p=p)
    status_ok()
    for b in range(B):
        # near a flat row's cut, weights of 2^-24 steps decide: allow what float32 exponentials can differ by
        check_draw(x[b].double().cpu().numpy(), int(tok[b]), t, int(k[b]), float(p[b]), 0.0, float(u[b]), slack=2e-4)


def test_sample_defaults_and_repeat():
    x = torch.randn((33, 777), device="cuda")
    u = torch.rand(33, device="cuda")
    tok, lp = tp.tp_sample(x, u)
    for b in range(33):
        check_draw(x[b].double().cpu().numpy(), int(tok[b]), 1.0, 0, 1.0, 0.0, float(u[b]))
    again, lp2 = tp.tp_sample(x, u)
    assert torch.equal(tok, again) and torch.equal(lp, lp2)


@pytest.mark.parametrize("V", [4, 1000, 50000, 200000])
def test_sample_ties_go_to_the_lowest_index(V):
    """All logits equal: every weight is 2^40, so every filter and draw has one exact answer."""
    B = 6
    x = torch.full((B, V), -3.25, device="cuda")
    x[1] = 0.0
    x[1, ::2] = -0.0  # one zero
    n = V // 2
    k = torch.tensor([1, n, n, 0, 0, n], dtype=torch.int32, device="cuda")
    p = torch.tensor([1, 1, 0.5, 0.25, 1, 0.5], dtype=torch.float32, device="cuda")
    u = torch.tensor([0.9, 0.5, 0.999999, 0.999999, 0.5, 0.0], dtype=torch.float32, device="cuda")
    tok, lp = tp.tp_sample(x, u, top_k=k, top_p=p)
    part = lambda w, f: int(w) * int(np.float32(f) * np.float32(1 << 24)) >> 24  # noqa: E731
    want = []
    for b in range(B):
        kept = int(k[b]) or V
        if float(p[b]) < 1:
            kept = max(1, -(-part(kept << 40, float(p[b])) // (1 << 40)))
        want.append(part(kept << 40, float(u[b])) >> 40)
    assert tok.tolist() == want
    assert np.allclose(lp.cpu().numpy(), -np.log(V), atol=1e-5)


def test_sample_masked_and_special_logits():
    V, inf = 5000, float("inf")
    x = torch.randn((7, V), device="cuda")
    x[0] = -inf                      # nothing to draw
    x[1] = -inf
    x[1, 4321] = -50.0               # one token left
    x[2, 100] = inf                  # the largest float: the only one with weight
    x[3, :] = NAN
    x[3, 17] = 1.0                   # NaN is never drawn
    x[4, :] = -inf
    x[4, [5, 10]] = 0.0
    x[5] = torch.finfo(torch.float32).min
    x[5, 4000:] = 0.0
    x[6, :] = NAN
    u = torch.tensor([0.5, 0.9, 0.99, 0.3, 0.75, 0.0, 0.1], device="cuda")
    k = torch.tensor([0, 10, 0, 3, 2, 0, 1], dtype=torch.int32, device="cuda")
    p = torch.tensor([1, 0.9, 1, 0.5, 0.99, 1, 1], device="cuda")
    tok, lp = tp.tp_sample(x, u, top_k=k, top_p=p)
    assert tok.tolist() == [-1, 4321, 100, 17, 10, 4000, -1]
    lp = lp.tolist()
    assert lp[0] == -inf and lp[6] == -inf and lp[1] == 0.0 and lp[2] == 0.0 and lp[3] == 0.0
    assert abs(lp[4] + np.log(2)) < 1e-6
    # odd parameters: outside [0, 1], NaN
    x = torch.randn((4, V), device="cuda")
    u = torch.tensor([-1.0, 1.0, 2.0, NAN], device="cuda")
    tok, _ = tp.tp_sample(x, u, temperature=torch.tensor([1, 1, 1, NAN], device="cuda"),
                          top_p=torch.tensor([NAN, 1, 1, 1], device="cuda"),
                          min_p=torch.tensor([NAN, 0, 0, 0], device="cuda"))
    assert tok[0] == 0 and tok[3] == int(x[3].argmax())
    assert tok[1] == tok[2] == V - 1 or tok[1] > V - 50


def draw_by_definition(x, u, t, k, p, m):
    """The tokens in whole numbers, from float32 exponentials: every sum exact, the row sorted."""
    x = x.float()
    V = x.shape[1]
    x = torch.where(torch.isnan(x), -float("inf"), x).clamp(max=torch.finfo(torch.float32).max) + 0.0
    part = lambda total, share: (total >> 24) * share + (((total & 0xFFFFFF) * share) >> 24)  # noqa: E731
    greedy = t[:, None] < 2.0 ** -20
    e = torch.exp((x - x.amax(1, keepdim=True)) * torch.where(greedy, 1.0, 1.0 / t[:, None]))
    w = (e * 2.0 ** 40).long()
    order = torch.sort(x, dim=1, descending=True, stable=True)[1]
    rank = torch.arange(V, device=x.device)
    kk = torch.where(greedy, 1, torch.where((k[:, None] <= 0) | (k[:, None] > V), V, k[:, None]))
    ws = torch.where(rank < kk, w.gather(1, order), 0)
    cut = part(ws.sum(1, keepdim=True), (p[:, None] * 2.0 ** 24).long())
    keep = (rank < kk) & ((p[:, None] >= 1) | (ws.cumsum(1) - ws < cut) | (rank == 0))
    keep = torch.zeros_like(keep).scatter(1, order, keep) & (e >= m[:, None].clamp(max=1))
    run = torch.where(keep, w, 0).cumsum(1)
    return (run <= part(run[:, -1:], (u[:, None] * 2.0 ** 24).long())).sum(1)


@pytest.mark.parametrize("seed", range(24))
def test_sample_equals_its_definition(seed):
    rng = np.random.default_rng(seed)
    V = int(rng.choice([3, 100, 1024, 5000, 50272, 60000, 130000]))
    B = int(rng.choice([1, 7, 40, 200]))
    dt = [torch.float32, torch.bfloat16, torch.float16][seed % 3]
    x = torch.from_numpy(rng.standard_normal((B, V)).astype(np.float32) * rng.choice([0.01, 0.5, 3, 20])).cuda().to(dt)
    if seed % 4 == 1:
        x = (x.float() * 2).round().div(2).to(dt)  # many equal logits
    if seed % 5 == 2:
        x[:, ::3] = -float("inf")
    par = [rng.random(B, dtype=np.float32), rng.choice(np.float32([0, 1e-5, 0.5, 1, 1.3, 100]), B),
           rng.choice([0, 0, 1, 3, 50, 600, 1500, 3000, 20000], B).astype(np.int32),
           rng.choice(np.float32([1, 1, 0.5, 0.9, 0.999, 0.9999999]), B), rng.choice(np.float32([0, 0, 0.01, 0.5]), B)]
    par = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in par]
    tok, _ = tp.tp_sample(x, *par)
    status_ok()
    assert torch.equal(tok, draw_by_definition(x, *par))


@pytest.mark.parametrize("B,V", [(1, 25600), (1, 25601), (3, 52224), (3, 52225), (15, 60000), (16, 30000), (36, 60000),
                                 (37, 60000), (2, 104449), (20, 150000), (40, 110000), (1, 208897)])
@pytest.mark.parametrize("with_k", [False, True])
def test_sample_rows_of_every_split(B, V, with_k):
    """Rows on 1, 2, 4 and 8 CTAs, at the sizes where the number changes."""
    rng = np.random.default_rng(B + V)
    x = torch.from_numpy(rng.standard_normal((B, V)).astype(np.float32) * 2.5).cuda()
    par = [rng.random(B, dtype=np.float32), rng.choice(np.float32([0.5, 0.7, 1, 1.3, 20]), B),
           rng.choice([0, 40, 2500] if with_k else [0], B).astype(np.int32),
           rng.choice(np.float32([1, 0.02, 0.5, 0.9, 0.95, 0.999]), B), rng.choice(np.float32([0, 0.02]), B)]
    par = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in par]
    tok, _ = tp.tp_sample(x, par[0], par[1], par[2] if with_k else None, par[3], par[4])
    status_ok()
    assert torch.equal(tok, draw_by_definition(x, *par))


@pytest.mark.parametrize("V", [30000, 50272, 120000])
def test_sample_top_p_where_a_guess_misleads(V):
    """Every fourth part of the row unlike the rest, a ramp, a spike and two levels: the elements that the end
    of top-p is guessed from do not stand for the row."""
    B = 8
    rng = np.random.default_rng(V)
    i = np.arange(V)
    x = rng.standard_normal((B, V)).astype(np.float32)
    x[0] = 10 - 20 * i / V
    x[1] = np.where(i % 49 == 0, 8, x[1])
    x[2] = np.where(i % 49 == 1, 8, x[2])
    x[3] = -30
    x[3, V // 3] = 5
    x[4] = np.where(i < V // 2, 1, 2)
    x[5] = np.where(i < 700, 6, -6) + x[5] * 1e-3
    x[6] = x[6] * 1e-6
    x[7] = np.where(i % 2, -np.inf, x[7] * 4)
    x = torch.from_numpy(x).cuda()
    for p in (0.3, 0.9, 0.99999):
        par = [torch.from_numpy(rng.random(B, dtype=np.float32)).cuda(), torch.full((B,), 0.8, device="cuda"),
               torch.zeros(B, dtype=torch.int32, device="cuda"), torch.full((B,), p, device="cuda"),
               torch.zeros(B, device="cuda")]
        tok, _ = tp.tp_sample(x, par[0], par[1], None, par[3])
        status_ok()
        assert torch.equal(tok, draw_by_definition(x, *par))


def test_sample_distribution():
    """20000 draws of one row: each share within five standard deviations of its probability."""
    V, n = 12, 20000
    row = torch.linspace(-2, 2, V, device="cuda")
    u = torch.from_numpy(np.random.default_rng(1).random(n, dtype=np.float32)).cuda()
    tok, _ = tp.tp_sample(row.expand(n, V).contiguous(), u)
    prob = torch.softmax(row.double(), 0).cpu().numpy()
    share = np.bincount(tok.cpu().numpy(), minlength=V) / n
    assert (np.abs(share - prob) <= 5 * np.sqrt(prob * (1 - prob) / n)).all()


# ------------------------------------------------------------------ the binding
def test_binding_refusals():
    B, N, Hq, Hk, D, page = 2, 2, 4, 2, 64, 16
    cuda = dict(device="cuda")
    q = torch.zeros((N, B, Hq * D), dtype=BF, **cuda)
    kc = torch.zeros((N, 3, Hk, page, D), dtype=BF, **cuda)
    table = torch.zeros((B, 1), dtype=torch.int32, **cuda)
    lens = torch.ones(B, dtype=torch.int32, **cuda)
    ok = dict(q=q, k_cache=kc, v_cache=kc.clone(), block_table=table, seq_lens=lens)
    tp.tp_paged_decode(**ok)
    for change, error in [
            (dict(q=q.cpu()), ValueError), (dict(q=q.half()), TypeError), (dict(q=q[:1]), ValueError),
            (dict(q=[q[0], q[1].float()]), ValueError), (dict(q=q[..., :70]), ValueError), (dict(q=q[0]), ValueError),
            (dict(q=q.double()), TypeError), (dict(q=q.transpose(1, 2)), ValueError), (dict(q=[]), (ValueError, IndexError)),
            (dict(k_cache=kc[:, :2]), ValueError), (dict(k_cache=kc.transpose(2, 3)), ValueError),
            (dict(k_cache=kc[..., ::2], v_cache=kc[..., ::2]), ValueError), (dict(v_cache=kc.half()), ValueError),
            (dict(block_table=table.long()), ValueError), (dict(block_table=table[:1]), ValueError),
            (dict(block_table=table.cpu()), ValueError), (dict(seq_lens=lens.long()), TypeError),
            (dict(seq_lens=lens[:1]), ValueError), (dict(seq_lens=torch.ones(4, dtype=torch.int32, **cuda)[::2]), ValueError),
            (dict(out=q[:1]), ValueError), (dict(out=q.half()), ValueError), (dict(scale="x"), TypeError),
            (dict(scale=-1.0), tp.TPError), (dict(window=-3), tp.TPError), (dict(softcap=-1.0), tp.TPError)]:
        with pytest.raises(error):
            tp.tp_paged_decode(**{**ok, **change})
    slots = torch.zeros(B, dtype=torch.int64, **cuda)
    x = torch.zeros((N, B, (Hq + 2 * Hk) * D), dtype=BF, **cuda)
    rope = torch.zeros((4, D), **cuda)
    for args, error in [
            (dict(rope=rope), ValueError), (dict(rope=rope.half(), positions=lens), ValueError),
            (dict(q_norm=torch.ones(D + 1, **cuda)), ValueError), (dict(k_norm=torch.ones(D, dtype=BF, **cuda)), TypeError),
            (dict(out=q.half()), ValueError), (dict(eps=-1.0), tp.TPError)]:
        with pytest.raises(error):
            tp.tp_qkv_append(x, kc, kc.clone(), slots, **args)
    with pytest.raises(ValueError):
        tp.tp_qkv_append(x[..., :2 * Hk * D], kc, kc.clone(), slots)
    logits, u = torch.zeros((2, 8), **cuda), torch.zeros(2, **cuda)
    for args, error in [
            (dict(logits=logits.double()), TypeError), (dict(logits=logits[0]), ValueError), (dict(u=u.double()), TypeError),
            (dict(top_k=u), TypeError), (dict(top_p=u[:1]), ValueError), (dict(logits=logits.T), ValueError)]:
        with pytest.raises(error):
            tp.tp_sample(**{**dict(logits=logits, u=u), **args})
    status_ok()


def test_prepared_calls_of_every_entry_point():
    """prepare() records the same calls that run directly."""
    x = torch.randn((2, 3, 8 * 64), device="cuda").to(BF)
    kc = torch.zeros((2, 2, 2, 16, 64), dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    slots, pos = torch.arange(3, device="cuda"), torch.arange(3, dtype=torch.int32, device="cuda")
    gain = torch.rand(64, device="cuda")
    call = tp.prepare(tp.tp_qkv_append, x, kc, vc, slots, positions=pos, rope=rope_table(4, 64), q_norm=gain, k_norm=gain,
                      eps=1e-5, interleaved=True)
    q = call().clone()
    k1, v1 = kc.clone(), vc.clone()
    again = tp.tp_qkv_append(x, kc.zero_(), vc.zero_(), slots, positions=pos, rope=rope_table(4, 64), q_norm=gain,
                             k_norm=gain, eps=1e-5, interleaved=True)
    assert torch.equal(q, again) and torch.equal(k1, kc) and torch.equal(v1, vc)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    cu, n = torch.tensor([0, 3], dtype=torch.int32, device="cuda"), torch.tensor([3], dtype=torch.int32, device="cuda")
    args = (q, kc, vc, table, cu, n)
    call = tp.prepare(tp.tp_paged_prefill, *args, prefix_lens=n, softcap=3.0, window=2)
    assert torch.equal(call(), tp.tp_paged_prefill(*args, prefix_lens=n, softcap=3.0, window=2))
    logits, u = torch.randn((4, 100), device="cuda"), torch.rand(4, device="cuda")
    call = tp.prepare(tp.tp_sample, logits, u, temperature=u + 0.5, min_p=u * 0.1)
    for got, want in zip(call(), tp.tp_sample(logits, u, temperature=u + 0.5, min_p=u * 0.1)):
        assert torch.equal(got, want)
    status_ok()


def test_calls_from_two_threads():
    """Draws of different lengths, appends and both attentions from two threads at once, a stream each: no call is
    refused, and every one gives what it gives alone."""
    import threading
    jobs, want, errors = [], [], []
    for i, V in enumerate((1000, 50272)):
        g = torch.Generator(device="cuda").manual_seed(V)
        logits = torch.randn((3, V), generator=g, device="cuda")
        u = torch.rand(3, generator=g, device="cuda")
        kc, vc, table, _ = paged([70 + 300 * i, 33], 1, 2, 64 << i, 16, BF, seed=i, fill=0.0)
        q = torch.randn((1, 2, 8 * (64 << i)), generator=g, device="cuda").to(BF)
        lens = torch.tensor([70 + 300 * i, 33], dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
        x = torch.randn((1, 2, 12 * (64 << i)), generator=g, device="cuda").to(BF)
        ka, va, slots = torch.zeros_like(kc), torch.zeros_like(vc), torch.arange(2, device="cuda")

        def work(logits=logits, u=u, kc=kc, vc=vc, table=table, q=q, lens=lens, cu=cu, x=x, ka=ka, va=va, slots=slots):
            return (*tp.tp_sample(logits, u, top_p=u), tp.tp_paged_decode(q, kc, vc, table, lens),
                    tp.tp_paged_prefill(q, kc, vc, table, cu, lens), tp.tp_qkv_append(x, ka, va, slots))
        jobs.append(work)
        want.append(work())
    torch.cuda.synchronize()

    def loop(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(300):
                    got = jobs[i]()
                torch.cuda.current_stream().synchronize()
            for a, b in zip(got, want[i]):
                assert torch.equal(a, b)
        except BaseException as e:  # noqa: BLE001 - reported by the test's thread
            errors.append(e)
    threads = [threading.Thread(target=loop, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    status_ok()


# ------------------------------------------------------------------ together
def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(BF).double().numpy()


def test_serving_steps_against_float64():
    """Prompts, then decode steps, through the linears, the cache and the draw."""
    N, D, heads, V = 4, 512, 8, 1000
    cfg = synth.qkv(seed=9, T=1, D=D, V=V, N=N, bias_std=0.1)
    gains = [torch.rand(D // heads, device="cuda") + 0.5 for _ in range(2)]
    serve = PagedServing(cfg, heads, batch=3, capacity=90, page=16, q_norm=gains[0], k_norm=gains[1])
    w = {n: oracle.bf16_to_f64(cfg[n]) for n in ("w_qkv", "w_o", "w_lm")}
    rng = np.random.default_rng(2)
    hd = D // heads
    past = [[np.zeros((0, heads, hd))] * 2 for _ in range(3)]
    ang = np.arange(90)[:, None] * 10000.0 ** (-np.arange(hd // 2) * 2.0 / hd)
    for counts in ([40, 1, 23], [1, 1, 1], [1, 1, 1], [5, 30, 1], [1, 1, 1]):
        x = to_device(synth.f32_to_bf16_bits(rng.standard_normal((sum(counts), D)).astype(np.float32)), "bf16")
        u = torch.from_numpy(rng.random(3, dtype=np.float32)).cuda()
        tokens, y = serve.step(x, counts, u, temperature=torch.full((3,), 0.8, device="cuda"),
                               top_k=torch.tensor([50, 0, 1], dtype=torch.int32, device="cuda"))
        status_ok()
        qkv = bf16(oracle.linear(to_host(x), w["w_qkv"], cfg["b_qkv"])).reshape(-1, 3, heads, hd)
        out, t0 = [], 0
        for b, c in enumerate(counts):
            n = len(past[b][0])
            cs, sn = np.cos(ang[n:n + c, None]), np.sin(ang[n:n + c, None])
            qk = []
            for i in range(2):
                z = qkv[t0:t0 + c, i]
                z = z / np.sqrt((z * z).mean(-1, keepdims=True) + 1e-6) * to_host(gains[i])
                a, d = z[..., :hd // 2], z[..., hd // 2:]
                qk.append(bf16(np.concatenate([a * cs - d * sn, d * cs + a * sn], -1)))
            past[b] = [np.concatenate([past[b][0], qk[1]]), np.concatenate([past[b][1], qkv[t0:t0 + c, 2]])]
            s = np.einsum("ihd,jhd->hij", qk[0], past[b][0]) / np.sqrt(hd)
            s[:, np.arange(n + c)[None] > n + np.arange(c)[:, None]] = -np.inf
            p = np.exp(s - s.max(-1, keepdims=True))
            o = np.einsum("hij,jhd->ihd", p / p.sum(-1, keepdims=True), past[b][1])
            out.append(bf16(o).reshape(c, D))
            t0 += c
        ref = oracle.linear(np.concatenate(out), w["w_o"], cfg["b_o"])
        check_close(to_host(y), ref, "attention block")
        last = to_host(y[torch.from_numpy(np.cumsum(counts) - 1).cuda()].to(BF))
        logits = oracle.linear(last, w["w_lm"], None)
        check_close(to_host(serve.logits), logits, "logits")
        for b in range(3):
            check_draw(to_host(serve.logits)[b], int(tokens[b]), float(np.float32(0.8)), [50, 0, 1][b], 1.0, 0.0, float(u[b]))


def test_serving_step_refusals():
    cfg = synth.qkv(seed=9, T=1, D=128, V=64, N=2)
    serve = PagedServing(cfg, 2, batch=2, capacity=20, page=16)
    x = torch.zeros((4, 128), dtype=BF, device="cuda")
    u = torch.zeros(2, device="cuda")
    for counts in ([4], [4, 0], [1, 21]):
        with pytest.raises(ValueError):
            serve.step(x, counts, u)


@pytest.mark.parametrize("raw", [False, True])
def test_serving_steps_on_a_busy_side_stream(raw):
    """Both streams have work queued when a step on another stream is asked for: its inputs are written
    late on the caller's, and its results are read there at once."""
    cfg = synth.qkv(seed=9, T=1, D=512, V=1000, N=4, bias_std=0.1)
    plain, moved = (PagedServing(cfg, 8, batch=3, capacity=90, page=16) for _ in range(2))
    side = torch.cuda.Stream()
    rng = np.random.default_rng(7)
    for counts in ([40, 1, 23], [1, 1, 1], [5, 30, 1], [1, 1, 1]):
        xs = to_device(synth.f32_to_bf16_bits(rng.standard_normal((sum(counts), 512)).astype(np.float32)), "bf16")
        us = torch.from_numpy(rng.random(3, dtype=np.float32)).cuda()
        want = [t.clone() for t in (*plain.step(xs, counts, us), plain.logits, plain.logprobs)]
        torch.cuda.synchronize()
        x, u = torch.zeros_like(xs), torch.zeros_like(us)
        with torch.cuda.stream(side):
            torch.cuda._sleep(3000000)
        torch.cuda._sleep(3000000)
        x.copy_(xs)
        u.copy_(us)
        tokens, y = moved.step(x, counts, u, stream=side.cuda_stream if raw else side)
        got = [t.clone() for t in (tokens, y, moved.logits, moved.logprobs)]
        # what the step freed may be handed out again on either stream
        for s in (torch.cuda.current_stream(), side):
            with torch.cuda.stream(s):
                junk = [torch.full_like(y, NAN) for _ in range(8)]
        del tokens, y, junk
        status_ok()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
