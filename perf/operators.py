"""Cases of the attention-side operators that sit between the sharded linears.

The sharded QKV linear writes one fused buffer per rank; from there a serving
step needs
  append   the per-head norms and the rotation of the queries and keys, and the
           write of the keys and values into a paged cache (tp_qkv_append);
  decode   attention of one new token per sequence over that cache
           (tp_paged_decode);
  prefill  attention of a ragged batch of prompt chunks over that cache
           (tp_paged_prefill);
  sample   the draw of a token from the gathered logits of the vocab-parallel
           head, with given random numbers (tp_sample).

The N ranks' buffers are the slices [r] of one tensor with N as its first
dimension.  ``run`` computes the operators in plain 32-bit torch operations, or
with the library's entry points where ``own`` is true.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
FMAX = float(np.finfo(np.float32).max)


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one sequence decoding: one token enters the cache (launch latency)
        dict(name="append_one", op="append", T=1, N=1, Hq=32, Hk=8, D=128, page=16, in_dt="bf16", dt="bf16",
             norm=True, rot=128, interleaved=False),
        # a decode batch with float32 activations, half of each head rotated in neighbouring pairs
        dict(name="append_batch", op="append", T=97, N=4, Hq=8, Hk=2, D=64, page=32, in_dt="f32", dt="f16",
             norm=False, rot=32, interleaved=True),
        # a 4096-wide fused QKV layer on 8 ranks (4 heads of 128 each), a full prompt batch
        dict(name="append_prompt", op="append", T=16384, N=8, Hq=4, Hk=4, D=128, page=64, in_dt="bf16", dt="bf16",
             norm=True, rot=128, interleaved=False),
        # one chat turn, short context, grouped heads on one rank (latency)
        dict(name="decode_one", op="decode", B=1, N=1, Hq=32, Hk=8, D=128, page=16, dt="bf16", lo=517, hi=517,
             softcap=0.0, window=0),
        # a mixed serving batch with capped scores and a sliding window
        dict(name="decode_window", op="decode", B=48, N=4, Hq=8, Hk=2, D=64, page=32, dt="f16", lo=1, hi=4001,
             softcap=30.0, window=1024),
        # the 16-token decode batch of the 4096-wide fused QKV layer on 8 ranks (as many key as query heads)
        dict(name="decode_mha", op="decode", B=16, N=8, Hq=4, Hk=4, D=128, page=64, dt="bf16", lo=100, hi=4096,
             softcap=0.0, window=0),
        # a large batch of long contexts, one key-value head per rank
        dict(name="decode_long", op="decode", B=64, N=8, Hq=8, Hk=1, D=128, page=64, dt="bf16", lo=1000, hi=16384,
             softcap=0.0, window=0),
        # a few short prompts of odd lengths arriving together, capped scores
        dict(name="prefill_short", op="prefill", B=5, N=2, Hq=8, Hk=2, D=64, page=16, dt="f16", qlo=7, qhi=150,
             clo=0, chi=90, prefix=0.0, softcap=20.0, window=0),
        # chunked prefill: chunks of two prompts against a long cached context, a bidirectional prefix
        dict(name="prefill_chunk", op="prefill", B=2, N=1, Hq=32, Hk=8, D=128, page=64, dt="bf16", qlo=1000,
             qhi=1024, clo=4000, chi=8192, prefix=0.1, softcap=0.0, window=0),
        # one long prompt through the 4096-wide layer's 8 ranks
        dict(name="prefill_long", op="prefill", B=1, N=8, Hq=4, Hk=4, D=128, page=64, dt="bf16", qlo=8192, qhi=8192,
             clo=0, chi=0, prefix=0.0, softcap=0.0, window=0),
        # one token drawn from the 50272-wide head
        dict(name="sample_one", op="sample", B=1, V=50272, dt="f32"),
        # a large decode batch, each row with its own settings
        dict(name="sample_batch", op="sample", B=384, V=50272, dt="f32"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _drawn(rng):
    op = rng.choice(["append", "decode", "prefill", "sample"])
    if op == "sample":
        return dict(op=op, B=_spread(rng, 1, 512), V=_spread(rng, 1000, 200000), dt=rng.choice(["f32", "bf16", "f16"]))
    N = rng.choice([1, 2, 4, 8])
    Hk = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    c = dict(op=op, N=N, Hq=Hk * G, Hk=Hk, D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
             dt=rng.choice(["bf16", "f16"]))
    if op == "append":
        rot = rng.choice([0, 32, 64, c["D"]])
        return c | dict(T=_spread(rng, 1, 16384), in_dt=rng.choice(["bf16", "f16", "f32"]),
                        norm=rng.choice([True, False]), rot=rot, interleaved=rng.choice([True, False]))
    c |= dict(softcap=rng.choice([0.0, 0.0, 15.0, 50.0]), window=rng.choice([0, 0, 0, _spread(rng, 16, 4096)]))
    if op == "decode":
        hi = _spread(rng, 16, 16384)
        return c | dict(B=_spread(rng, 1, 256), lo=rng.choice([0, 1, hi // 2, hi]), hi=hi)
    qhi, chi = _spread(rng, 1, 4096), rng.choice([0, _spread(rng, 1, 8192)])
    return c | dict(B=_spread(rng, 1, 16), qlo=rng.choice([1, qhi, (qhi + 1) // 2]), qhi=qhi, clo=chi // 3, chi=chi,
                    prefix=rng.choice([0.0, 0.0, 0.3]))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = {k: max(w[k], most.get(c["op"], w)[k]) for k in w}
    while True:
        c = _drawn(rng)
        w = work(c)
        if c["op"] in ("decode", "prefill"):  # the plain forms work on the padded batch
            L = (c["hi"] if c["op"] == "decode" else c["qhi"] + c["chi"])
            rows = c["B"] * c["N"] * c["Hq"] * L * (1 if c["op"] == "decode" else c["qhi"])
            kv = c["B"] * c["N"] * c["Hk"] * L * c["D"]
            if rows > (1 << 31) or kv > (1 << 30):
                continue
        if all(w[k] <= most[c["op"]][k] for k in w):
            return c


def _lens(lo, hi, n):
    """n lengths spread over lo..hi, hi among them."""
    return [hi - int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _pairs(case):
    """(keys that have to be read, query-key pairs) of one key-value head's sequences."""
    keys = pairs = 0
    if case["op"] == "decode":
        for s in _lens(case["lo"], case["hi"], case["B"]):
            n = min(s, case["window"]) if case["window"] else s
            keys, pairs = keys + n, pairs + n
        return keys, pairs
    for ql, cl in zip(_lens(case["qlo"], case["qhi"], case["B"]), _lens(case["clo"], case["chi"], case["B"])):
        s = ql + cl
        pre = int(s * case["prefix"])
        pos = np.arange(cl, s, dtype=np.int64)
        first = np.maximum(0, pos + 1 - case["window"]) if case["window"] else np.zeros_like(pos)
        pairs += int(np.sum(pos + 1 - first + np.minimum(pre, first) + np.maximum(0, pre - pos - 1)))
        keys += s - int(max(0, first[0] - pre))
    return keys, pairs


def work(case):
    if case["op"] == "sample":
        B, V = case["B"], case["V"]
        return {"bytes": float(B * V * BYTES[case["dt"]] + B * 32), "flops": float(4 * B * V)}
    N, Hq, Hk, D = case["N"], case["Hq"], case["Hk"], case["D"]
    if case["op"] == "append":
        el = case["T"] * N * (Hq + 2 * Hk) * D
        return {"bytes": float(el * (BYTES[case["in_dt"]] + BYTES[case["dt"]]) + case["T"] * (12 + 4 * case["rot"])),
                "flops": float(el * 5)}
    keys, pairs = _pairs(case)
    toks = case["B"] if case["op"] == "decode" else sum(_lens(case["qlo"], case["qhi"], case["B"]))
    return {"bytes": float(N * D * 2 * (2 * Hk * keys + 2 * Hq * toks)), "flops": float(4 * N * Hq * D * pairs)}


# ---------------------------------------------------------------- inputs
def _normal(g, shape, dt, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32 if dt == "f32" else DT[dt]) * std)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    st = {"case": case}

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()

    if case["op"] == "sample":
        B, V = case["B"], case["V"]
        st["logits"] = torch.randn((B, V), generator=g, device="cuda").mul_(2.5).to(DT[case["dt"]])
        st["u"] = dev(rng.random(B, dtype=np.float32))
        # rows of every kind: greedy, free, narrow and wide filters, alone and together
        st["temperature"] = dev(rng.choice(np.float32([0, 0.5, 0.7, 1, 1, 1.3]), B).astype(np.float32))
        st["top_k"] = dev(rng.choice([0, 0, 1, 20, 50, 1000], B).astype(np.int32))
        st["top_p"] = dev(rng.choice(np.float32([1, 1, 0.5, 0.9, 0.95, 0.999]), B).astype(np.float32))
        st["min_p"] = dev(rng.choice(np.float32([0, 0, 0, 0.02, 0.1]), B).astype(np.float32))
        return st

    N, Hq, Hk, D, page = (case[k] for k in ("N", "Hq", "Hk", "D", "page"))
    if case["op"] == "append":
        T, rot = case["T"], case["rot"]
        pages = -(-T // page) + T // (4 * page) + 2
        st["qkv"] = _normal(g, (N, T, (Hq + 2 * Hk) * D), case["in_dt"])
        st["slots"] = dev(rng.permutation(pages * page)[:T].astype(np.int64) if T < 4096 else
                          (rng.permutation(pages)[:-(-T // page), None] * page + np.arange(page)).reshape(-1)[:T])
        rows = 16384
        st["positions"] = dev(rng.integers(0, rows, T).astype(np.int32))
        st["rope"] = None
        if rot:
            ang = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(rot // 2) * 2.0 / rot)
            st["rope"] = dev(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32))
        st["q_norm"] = dev((1 + 0.1 * rng.standard_normal(D)).astype(np.float32)) if case["norm"] else None
        st["k_norm"] = dev((1 + 0.1 * rng.standard_normal(D)).astype(np.float32)) if case["norm"] else None
    else:
        B = case["B"]
        order = rng.permutation(B)
        if case["op"] == "decode":
            lens = np.array(_lens(case["lo"], case["hi"], B))[order]
            T, top = B, case["hi"]
        else:
            ql = np.array(_lens(case["qlo"], case["qhi"], B))[order]
            lens = ql + np.array(_lens(case["clo"], case["chi"], B))[order]
            T, top = int(ql.sum()), case["qhi"] + case["chi"]
            st["cu_seqlens"] = dev(np.concatenate([[0], np.cumsum(ql)]).astype(np.int32))
            st["prefix_lens"] = dev(np.array([int(s * case["prefix"]) for s in lens]).astype(np.int32)) \
                if case["prefix"] else None
        width = max(1, -(-top // page))
        need = -(-lens // page)
        pages = int(need.sum()) + 1
        table = np.full((B, width), -1, np.int32)  # entries behind a sequence's end name no page
        table[np.arange(width)[None, :] < need[:, None]] = rng.permutation(pages)[:int(need.sum())]
        st["block_table"], st["seq_lens"] = dev(table), dev(lens.astype(np.int32))
        st["q"] = _normal(g, (N, T, Hq * D), case["dt"], 1.5)
    st["k_cache"] = _normal(g, (N, pages, Hk, page, D), case["dt"])
    st["v_cache"] = _normal(g, (N, pages, Hk, page, D), case["dt"])
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    c = st["case"]
    if own:
        import sharded_gemm_gb300 as tp
        if c["op"] == "append":
            q = tp.tp_qkv_append(st["qkv"], st["k_cache"], st["v_cache"], st["slots"], positions=st["positions"],
                                 rope=st["rope"], q_norm=st["q_norm"], k_norm=st["k_norm"], eps=1e-6,
                                 interleaved=c["interleaved"])
            return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
        if c["op"] == "decode":
            return {"o": tp.tp_paged_decode(st["q"], st["k_cache"], st["v_cache"], st["block_table"], st["seq_lens"],
                                            scale=c["D"] ** -0.5, softcap=c["softcap"], window=c["window"])}
        if c["op"] == "prefill":
            return {"o": tp.tp_paged_prefill(st["q"], st["k_cache"], st["v_cache"], st["block_table"],
                                             st["cu_seqlens"], st["seq_lens"], prefix_lens=st["prefix_lens"],
                                             scale=c["D"] ** -0.5, softcap=c["softcap"], window=c["window"])}
        tokens, logprobs = tp.tp_sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"],
                                        top_p=st["top_p"], min_p=st["min_p"])
        return {"tokens": tokens, "logprobs": logprobs}
    return {"append": _append, "decode": _decode, "prefill": _prefill, "sample": _sample}[c["op"]](st)


def _append(st):
    c = st["case"]
    N, T, Hq, Hk, D, page, rot = (c[k] for k in ("N", "T", "Hq", "Hk", "D", "page", "rot"))
    x = st["qkv"].view(N, T, Hq + 2 * Hk, D).float()
    qk, v = x[:, :, :Hq + Hk], x[:, :, Hq + Hk:]
    if c["norm"]:
        qk = qk * torch.rsqrt(qk.square().mean(-1, keepdim=True) + 1e-6)
        qk = torch.cat([qk[:, :, :Hq] * st["q_norm"], qk[:, :, Hq:] * st["k_norm"]], 2)
    if rot:
        table = st["rope"][st["positions"].long()][None, :, None, :]
        cos, sin = table[..., :rot // 2], table[..., rot // 2:]
        if c["interleaved"]:
            a, b = qk[..., 0:rot:2], qk[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = qk[..., :rot // 2], qk[..., rot // 2:rot]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        qk = torch.cat([turned, qk[..., rot:]], -1)
    q = qk[:, :, :Hq].reshape(N, T, Hq * D).to(DT[c["dt"]])
    at, off = st["slots"] // page, st["slots"] % page
    st["k_cache"][:, at, :, off] = qk[:, :, Hq:].transpose(0, 1).to(DT[c["dt"]])
    st["v_cache"][:, at, :, off] = v.transpose(0, 1).to(DT[c["dt"]])
    return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _paged(cache, table, c):
    """(N, B, Hk, L, D) in 32 bits: each sequence's pages one after the other."""
    x = cache[:, table.clamp(min=0).long()]
    return x.permute(0, 1, 3, 2, 4, 5).reshape(c["N"], table.shape[0], c["Hk"], -1, c["D"]).float()


def _attend(q, k, v, seen, c):
    """softmax over the seen keys, zero where a row sees none; q (N, B, Hk, R, D), seen (B, 1, R or 1, L)."""
    s = torch.matmul(q, k.transpose(-1, -2)) * c["D"] ** -0.5
    if c["softcap"]:
        s = c["softcap"] * torch.tanh(s / c["softcap"])
    s = torch.where(seen, s, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-FMAX))
    del s
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total > 0, total, 1.0)


def _decode(st):
    c = st["case"]
    N, B, Hq, Hk, D = (c[k] for k in ("N", "B", "Hq", "Hk", "D"))
    k, v = _paged(st["k_cache"], st["block_table"], c), _paged(st["v_cache"], st["block_table"], c)
    at, n = torch.arange(k.shape[3], device="cuda"), st["seq_lens"][:, None]
    seen = (at < n) & (at >= (n - c["window"] if c["window"] else 0))
    o = _attend(st["q"].view(N, B, Hk, Hq // Hk, D).float(), k, v, seen[:, None, None], c)
    return {"o": o.reshape(N, B, Hq * D).to(DT[c["dt"]])}


def _prefill(st):
    c = st["case"]
    N, B, Hq, Hk, D, qhi = (c[k] for k in ("N", "B", "Hq", "Hk", "D", "qhi"))
    G, T, cu = Hq // Hk, st["q"].shape[1], st["cu_seqlens"].long()
    k, v = _paged(st["k_cache"], st["block_table"], c), _paged(st["v_cache"], st["block_table"], c)
    i = torch.arange(qhi, device="cuda")
    q = st["q"][:, (cu[:-1, None] + i).clamp(max=T - 1)]  # the batch padded to its longest chunk
    q = q.view(N, B, qhi, Hk, G, D).permute(0, 1, 3, 4, 2, 5).reshape(N, B, Hk, G * qhi, D).float()
    n, at = st["seq_lens"][:, None, None], torch.arange(k.shape[3], device="cuda")
    pos = n - (cu[1:] - cu[:-1])[:, None, None] + i[:, None]
    seen = (at <= pos) & (at > pos - c["window"]) if c["window"] else at <= pos
    if st["prefix_lens"] is not None:
        seen = seen | (at < st["prefix_lens"][:, None, None])
    seen = (seen & (at < n)).repeat(1, G, 1)[:, None]
    o = _attend(q, k, v, seen, c)
    o = o.view(N, B, Hk, G, qhi, D).permute(0, 1, 4, 2, 3, 5).reshape(N, B, qhi, Hq * D)
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    return {"o": o[:, b, t - cu[b]].to(DT[c["dt"]])}


def _part(total, share):
    """floor(total * share / 2^24) for whole totals up to 2^62 and shares of 2^24, without leaving 64 bits."""
    return (total >> 24) * share + (((total & 0xFFFFFF) * share) >> 24)


def _sample(st):
    x = st["logits"].float()
    B, V = x.shape
    x = torch.where(torch.isnan(x), -math.inf, x).clamp(max=FMAX) + 0.0
    t, k, p = st["temperature"][:, None], st["top_k"][:, None], st["top_p"][:, None]
    greedy = t < 2.0 ** -20
    top = x.amax(1, keepdim=True)
    e = torch.exp((x - top) * torch.where(greedy, 1.0, 1.0 / t))
    w = (e * 2.0 ** 40).long()  # the tokens' weights as whole numbers: their sums have no order
    xs, order = torch.sort(x, dim=1, descending=True, stable=True)
    ws = w.gather(1, order)
    rank = torch.arange(V, device="cuda")
    k = torch.where(greedy, 1, torch.where(k <= 0, V, k))
    ws = torch.where(rank < k, ws, 0)
    before = ws.cumsum(1) - ws
    cut = _part(ws.sum(1, keepdim=True), (p.clamp(min=0) * 2.0 ** 24).long())
    keep = (rank < k) & ((p >= 1) | (before < cut) | (rank == 0))
    keep = torch.zeros_like(keep).scatter(1, order, keep) & (e >= st["min_p"][:, None].clamp(max=1))
    total = torch.where(keep, w, 0).cumsum(1)
    r = _part(total[:, -1:], (st["u"][:, None] * 2.0 ** 24).long())
    tokens = (total <= r).sum(1)
    logz = torch.log(torch.exp(x - top).sum(1))
    return {"tokens": tokens, "logprobs": x.gather(1, tokens[:, None])[:, 0] - top[:, 0] - logz}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    if case["op"] in ("decode", "prefill") and work(case)["flops"] > 3e12:
        return None
    st = prepare(case, seed)
    with torch.no_grad():
        return {"append": _exact_append, "decode": _exact_attention, "prefill": _exact_attention,
                "sample": _exact_sample}[case["op"]](case, st)


def _exact_append(c, st):
    N, T, Hq, Hk, D = (c[k] for k in ("N", "T", "Hq", "Hk", "D"))
    x = st["qkv"].double().reshape(N, T, Hq + 2 * Hk, D)
    kc, vc = st["k_cache"].double(), st["v_cache"].double()
    q = torch.empty((N, T, Hq, D), dtype=torch.float64, device="cuda")
    at, off = torch.div(st["slots"], c["page"], rounding_mode="floor"), torch.remainder(st["slots"], c["page"])
    half = c["rot"] // 2
    for h in range(Hq + 2 * Hk):
        y = x[:, :, h].clone()
        if h < Hq + Hk:
            if c["norm"]:
                weight = (st["q_norm"] if h < Hq else st["k_norm"]).double()
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + 1e-6) * weight
            if half:
                pairs = torch.complex(y[..., 0:c["rot"]:2], y[..., 1:c["rot"]:2]) if c["interleaved"] else \
                    torch.complex(y[..., :half], y[..., half:c["rot"]])
                rows = st["rope"].double()[st["positions"].long()]
                turned = pairs * torch.complex(rows[:, :half], rows[:, half:])
                if c["interleaved"]:
                    y[..., 0:c["rot"]:2], y[..., 1:c["rot"]:2] = turned.real, turned.imag
                else:
                    y[..., :half], y[..., half:c["rot"]] = turned.real, turned.imag
        if h < Hq:
            q[:, :, h] = y
        elif h < Hq + Hk:
            kc[:, at, h - Hq, off] = y
        else:
            vc[:, at, h - Hq - Hk, off] = y
    return {"q": q.reshape(N, T, Hq * D), "k_cache": kc, "v_cache": vc}


def _exact_attention(c, st):
    N, Hq, Hk, D, page = (c[k] for k in ("N", "Hq", "Hk", "D", "page"))
    G = Hq // Hk
    lens = st["seq_lens"].tolist()
    cu = st["cu_seqlens"].tolist() if c["op"] == "prefill" else list(range(len(lens) + 1))
    pre = st["prefix_lens"].tolist() if st.get("prefix_lens") is not None else [0] * len(lens)
    out = torch.zeros((N, cu[-1], Hq * D), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n == 0:
            continue
        ids = st["block_table"][b, :-(-n // page)].long()
        for r in range(N):
            for h in range(Hk):
                K = st["k_cache"][r, ids, h].reshape(-1, D)[:n].double()
                V = st["v_cache"][r, ids, h].reshape(-1, D)[:n].double()
                for i0 in range(cu[b], cu[b + 1], 1024):
                    i1 = min(i0 + 1024, cu[b + 1])
                    q = st["q"][r, i0:i1].double().reshape(i1 - i0, Hq, D)[:, h * G:(h + 1) * G]
                    s = torch.einsum("igd,jd->igj", q, K) / math.sqrt(D)
                    if c["softcap"]:
                        s = torch.tanh(s / c["softcap"]) * c["softcap"]
                    pos = (torch.arange(i0, i1, device="cuda") - cu[b + 1] + n)[:, None, None]
                    j = torch.arange(n, device="cuda")
                    hidden = j > pos
                    if c["window"]:
                        hidden = hidden | (pos - j >= c["window"])
                    s = s.masked_fill(hidden & (j >= pre[b]), -math.inf)
                    out[r, i0:i1, h * G * D:(h + 1) * G * D] = \
                        torch.einsum("igj,jd->igd", torch.softmax(s, -1), V).reshape(i1 - i0, G * D)
    return {"o": out}


def _exact_sample(c, st):
    x = st["logits"].double().cpu().numpy()
    t, k, p, m, u = (st[n].double().cpu().numpy() for n in ("temperature", "top_k", "top_p", "min_p", "u"))
    logprobs = np.empty(len(x))
    for b, row in enumerate(x):
        order = np.argsort(-row, kind="stable")
        if t[b] == 0:
            order = order[:1]
            tokens = order
        else:
            if k[b] > 0:
                order = order[:int(k[b])]
            w = np.exp((row[order] - row[order[0]]) / t[b])
            if p[b] < 1:
                order = order[:max(1, int(np.sum(np.cumsum(w) - w < p[b] * w.sum())))]
            order = order[w[:len(order)] >= m[b]]
            tokens = np.sort(order)
        w = np.cumsum(np.exp((row[tokens] - row.max()) / (t[b] or 1.0)))
        token = tokens[min(len(tokens) - 1, int(np.searchsorted(w, u[b] * w[-1], side="right")))]
        logprobs[b] = row[token] - row.max() - np.log(np.sum(np.exp(row - row.max())))
    return {"tokens": None, "logprobs": torch.from_numpy(logprobs)}
