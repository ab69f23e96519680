"""Cases of the operators that serve many requests at once over one paged cache.

Beside the sharded linears, the paged attentions and the draw, a server's step needs
  plan     block tables, positions and slots of a step's tokens, built on the GPU
           from the requests' lengths and a shared pool of pages (tp_paged_plan),
           and the grouping of the tokens by adapter (tp_lora_plan);
  lora     low-rank adapters of many requests beside a shared projection: the
           column-parallel form (tp_lora_all_to_sharded) and the row-parallel one
           (tp_lora_sharded_to_all);
  verify   drafted tokens checked against the target's probabilities with given
           random numbers, and the token that follows them (tp_verify).

The N ranks' buffers are the slices [r] of one tensor with N as its first
dimension.  ``run`` computes the operators in plain torch operations (32-bit, or
whole numbers), or with the library's entry points where ``own`` is true.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "none": 0}
FMAX = float(np.finfo(np.float32).max)


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # four chats, one token each: the smallest step (latency)
        dict(name="plan_step", op="plan", B=4, page=16, hi=2000, clo=1, chi=1, ends=0.0, rejected=False, adapters=0,
             short=False),
        # a decode batch that drafts: 1 to 8 tokens each, some of the last step's refused, some requests done,
        # tokens grouped by 64 adapters
        dict(name="plan_drafts", op="plan", B=256, page=16, hi=16384, clo=1, chi=8, ends=0.1, rejected=True,
             adapters=64, short=False),
        # prompts admitted together, chunked prefill beside them
        dict(name="plan_prompts", op="plan", B=96, page=64, hi=4096, clo=1, chi=4096, ends=0.05, rejected=False,
             adapters=16, short=False),
        # one chat turn on the 4096-wide fused QKV layer's 8 ranks (latency)
        dict(name="lora_one", op="lora", form="column", T=1, B=1, N=8, K=4096, O=12288, R=16, n=32, none=0.0, dt="bf16",
             out="bf16"),
        # a decode batch in which nearly every request has its own adapter, the same layer
        dict(name="lora_decode", op="lora", form="column", T=64, B=64, N=8, K=4096, O=12288, R=16, n=128, none=0.1,
             dt="bf16", out="bf16"),
        # prompts of eight requests through the MLP's 4096 x 11008 layer
        dict(name="lora_prompt", op="lora", form="column", T=8192, B=8, N=4, K=4096, O=11008, R=64, n=8, none=0.1,
             dt="bf16", out="bf16"),
        # the row-parallel W_o of the same decode batch, float32 out
        dict(name="lora_row_decode", op="lora", form="row", T=97, B=97, N=8, K=4096, O=4096, R=32, n=40, none=0.2,
             dt="f16", out="f32"),
        # ragged prompts through the MLP's row-parallel 11008 x 4096 layer
        dict(name="lora_row_prompt", op="lora", form="row", T=5003, B=13, N=4, K=11008, O=4096, R=16, n=64, none=0.0,
             dt="bf16", out="f32"),
        # one request, four drafted tokens (latency)
        dict(name="verify_one", op="verify", B=1, mlo=4, mhi=4, V=50272, dt="f32", q="f32", plain=False),
        # a batch whose drafts come from a lookup (no probabilities of their own), each request with its settings
        dict(name="verify_lookup", op="verify", B=32, mlo=0, mhi=7, V=50272, dt="bf16", q="none", plain=False),
        # a large batch with a draft model, temperatures only
        dict(name="verify_free", op="verify", B=96, mlo=3, mhi=3, V=50272, dt="f32", q="bf16", plain=True),
        # a large batch with a draft model, each request with its settings
        dict(name="verify_batch", op="verify", B=96, mlo=1, mhi=5, V=50272, dt="f32", q="f32", plain=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _drawn(rng):
    op = rng.choice(["plan", "lora", "lora", "verify"])
    if op == "plan":
        chi = rng.choice([1, 1, 8, _spread(rng, 8, 4096)])
        return dict(op=op, B=_spread(rng, 1, 1024), page=rng.choice([16, 32, 64, 128]), hi=_spread(rng, 16, 16384),
                    clo=rng.choice([0, 1, chi]), chi=chi, ends=rng.choice([0.0, 0.0, 0.1]),
                    rejected=rng.choice([True, False]), adapters=rng.choice([0, _spread(rng, 1, 512)]),
                    short=rng.random() < 0.1)
    if op == "verify":
        mhi = rng.choice([0, 1, 2, 3, 4, 5, 8])
        return dict(op=op, B=_spread(rng, 1, 256), mlo=rng.randint(0, mhi), mhi=mhi, V=_spread(rng, 1000, 200000),
                    dt=rng.choice(["f32", "bf16", "f16"]), q=rng.choice(["f32", "f32", "bf16", "f16", "none"]),
                    plain=rng.choice([True, False]))
    N = rng.choice([1, 2, 4, 8])
    form = rng.choice(["column", "row"])
    T = _spread(rng, 1, 8192)
    K, O = _spread(rng, 64, 8192), _spread(rng, 64, 12288)
    if rng.random() < 0.75:  # otherwise rows that begin at any element
        K, O = -(-K // (8 * N)) * 8 * N, -(-O // (8 * N)) * 8 * N
    else:
        K, O = (-(-K // N) * N, O) if form == "row" else (K, -(-O // N) * N)
    return dict(op=op, form=form, T=T, B=_spread(rng, 1, T), N=N, K=K, O=O, R=rng.choice([4, 8, 16, 16, 32, 64, 128]),
                n=_spread(rng, 1, 256), none=rng.choice([0.0, 0.0, 0.2]), dt=rng.choice(["bf16", "bf16", "f16"]),
                out=rng.choice(["bf16", "f16", "f32"]))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = {k: max(w[k], most.get(c["op"], w)[k]) for k in w}
    while True:
        c = _drawn(rng)
        if c["op"] == "lora" and c["T"] * c["n"] * c["R"] > 1 << 26:  # the plain form's products hold every adapter
            continue
        if all(v <= most[c["op"]][k] for k, v in work(c).items()):
            return c


def _lens(lo, hi, n):
    """n lengths spread over lo..hi, hi among them."""
    return [hi - int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _tokens(case):
    """The rows that a plan is made for: all of its requests', and some more of a padded step."""
    return sum(_lens(case["clo"], case["chi"], case["B"])) + case["B"] % 7


def _adapters(case):
    """The adapter of each request, -1: none."""
    rng = np.random.default_rng(case["B"] * 1000 + case["n"])
    ids = rng.integers(0, case["n"], case["B"])
    return np.where(rng.random(case["B"]) < case["none"], -1, ids).astype(np.int32)


def _offsets(case):
    """Where each request's tokens begin: ragged, one token at least."""
    B, T = case["B"], case["T"]
    rng = np.random.default_rng(T * 1000 + B)
    cuts = np.sort(rng.choice(T - 1, B - 1, replace=False)) + 1 if B > 1 else []
    return np.concatenate([[0], cuts, [T]]).astype(np.int32)


def work(case):
    if case["op"] == "plan":
        T, B = _tokens(case), case["B"]
        pages = T // case["page"] + B
        return {"bytes": float(T * (12 + (4 if case["adapters"] else 0)) + B * 36 + pages * 8), "flops": float(4 * T)}
    if case["op"] == "verify":
        rows = sum(_lens(case["mlo"], case["mhi"], case["B"])) + case["B"]
        row = case["V"] * BYTES[case["dt"]]
        return {"bytes": float(rows * (row + 24) + (case["B"] if case["mhi"] else 0) * case["V"] * BYTES[case["q"]]),
                "flops": float(4 * rows * case["V"])}
    T, K, O, R = (case[k] for k in ("T", "K", "O", "R"))
    ids, cu = _adapters(case), _offsets(case)
    with_one = int(((cu[1:] - cu[:-1]) * (ids >= 0)).sum())
    used = len(np.unique(ids[ids >= 0]))
    return {"bytes": float(2 * with_one * K + 2 * used * R * (K + O) + 2 * T * O * BYTES[case["out"]]),
            "flops": float(2 * with_one * R * (K + O))}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    st = {"case": case}

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()

    if case["op"] == "plan":
        B, page, hi = case["B"], case["page"], case["hi"]
        order = rng.permutation(B)
        counts = np.array(_lens(case["clo"], case["chi"], B))[order]
        lens = rng.integers(0, hi + 1, B)
        if case["chi"] > 64:  # most prompts are new
            lens = np.where(rng.random(B) < 0.7, 0, lens)
        back = np.minimum(rng.integers(0, 5, B), lens) if case["rejected"] else np.zeros(B, np.int64)
        held = -(-lens // page)
        ended = rng.random(B) < case["ends"]
        need = np.where(ended, 0, np.maximum(0, -(-(lens - back + counts) // page) - held))
        width = -(-(hi + case["chi"]) // page)
        pages = B * width + 8
        spare = int(need.sum()) // 2 if case["short"] else pages - int(held.sum())
        names = rng.permutation(pages).astype(np.int32)
        table = np.full((B, width), -1, np.int32)
        table[np.arange(width)[None, :] < held[:, None]] = names[:int(held.sum())]
        free = np.full(pages, -1, np.int32)
        free[:spare] = names[int(held.sum()):][:spare]
        st |= dict(counts=dev(np.where(ended, -1, counts).astype(np.int32)), seq_lens=dev(lens.astype(np.int32)),
                   owned=dev(held.astype(np.int32)), block_table=dev(table), free_pages=dev(free),
                   free_count=dev(np.array([spare], np.int32)), tokens=_tokens(case),
                   rejected=dev(back.astype(np.int32)) if case["rejected"] else None)
        n = case["adapters"]
        st["adapters"] = dev(rng.integers(-1, n, B).astype(np.int32)) if n else None
        # what a program writes each step into: lengths, pages, pool, what lacks, offsets, positions, slots
        T = st["tokens"]
        st["step"] = [torch.empty(m, dtype=torch.int32, device="cuda") for m in (B, B, 1, 1, B + 1, T)]
        st["step"] += [torch.empty(T, dtype=torch.int64, device="cuda")]
        st["groups"] = torch.empty(4 + 4 * min(T, n + 1) + T, dtype=torch.int32, device="cuda") if n else None
        return st

    if case["op"] == "lora":
        T, N, K, O, R, n = (case[k] for k in ("T", "N", "K", "O", "R", "n"))
        ids = _adapters(case)
        rng.shuffle(ids)
        st["plan"] = _grouped(dev(ids), dev(_offsets(case)), T, n)
        st["token_ids"] = dev(np.repeat(ids, np.diff(_offsets(case))).astype(np.int64))
        st["scales"] = dev(rng.choice(np.float32([0.5, 1, 2]), n).astype(np.float32))

        def normal(shape, std, dt):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(DT[dt])
        # Weights of a layer: outputs of the adapters about as large as the projection's
        nx, ny = (N, 1) if case["form"] == "row" else (1, N)
        st["x"] = normal((nx, T, K // nx), 1.0, case["dt"])
        st["a"] = normal((nx, n, R, K // nx), K ** -0.5, case["dt"])
        st["b"] = normal((ny, n, O // ny, R), R ** -0.5, case["dt"])
        st["y"] = normal((ny, T, O // ny), 1.0, case["out"])
        st["out"] = torch.empty_like(st["y"])
        return st

    B, V = case["B"], case["V"]
    drafted = np.array(_lens(case["mlo"], case["mhi"], B))[rng.permutation(B)]
    cu = np.concatenate([[0], np.cumsum(drafted + 1)])
    T = int(cu[-1])
    seq = np.repeat(np.arange(B), drafted + 1)
    if case["plain"]:
        t = rng.choice(np.float32([0.7, 1, 1, 1.3]), B)
        st |= dict(top_k=None, top_p=None, min_p=None)
    else:
        t = rng.choice(np.float32([0, 0.5, 0.7, 1, 1, 1.3]), B)
        st["top_k"] = dev(rng.choice([0, 0, 1, 20, 50, 1000], B).astype(np.int32))
        st["top_p"] = dev(rng.choice(np.float32([1, 1, 0.5, 0.9, 0.95, 0.999]), B).astype(np.float32))
        st["min_p"] = dev(rng.choice(np.float32([0, 0, 0, 0.02, 0.1]), B).astype(np.float32))
    st["temperature"] = dev(t.astype(np.float32))
    logits = torch.randn((T, V), generator=g, device="cuda").mul_(2.5)
    # what the draft model thinks of the same places: near the target, a token of each row drawn from it
    near = logits + 0.7 * torch.randn((T, V), generator=g, device="cuda")
    sharp = dev((1 / np.maximum(t[seq], 0.3)).astype(np.float32))
    q = torch.softmax(near * sharp[:, None], 1)
    del near
    u = torch.rand((T, 1), generator=g, device="cuda", dtype=torch.float64)
    st["drafts"] = (q.double().cumsum(1) < u).sum(1).clamp(max=V - 1)
    st["draft_probs"] = None if case["q"] == "none" else q.to(DT[case["q"]])
    st["logits"] = logits.to(DT[case["dt"]])
    st["u"] = dev(rng.random(T, dtype=np.float32))
    st["cu_rows"] = dev(cu.astype(np.int32))
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    c = st["case"]
    if own:
        import sharded_gemm_gb300 as tp
        if c["op"] == "plan":
            p = tp.tp_paged_plan(st["counts"], st["seq_lens"], st["owned"], st["block_table"], st["free_pages"],
                                 st["free_count"], c["page"], st["tokens"], rejected=st["rejected"], out=st["step"])
            out = {"seq_lens": p.seq_lens, "owned": p.owned, "free_count": p.free_count, "missing": p.missing,
                   "cu_seqlens": p.cu_seqlens, "positions": p.positions, "slots": p.slots,
                   "block_table": st["block_table"], "free_pages": st["free_pages"]}
            if st["adapters"] is not None:
                out["groups"] = tp.tp_lora_plan(st["adapters"], st["tokens"], c["adapters"], cu_seqlens=p.cu_seqlens,
                                                out=st["groups"])
            return out
        if c["op"] == "lora":
            if c["form"] == "column":
                y = tp.tp_lora_all_to_sharded(st["x"][0], st["a"][0], st["b"], st["plan"], st["y"],
                                              scales=st["scales"], out=st["out"])
            else:
                y = tp.tp_lora_sharded_to_all(st["x"], st["a"], st["b"][0], st["plan"], st["y"][0],
                                              scales=st["scales"], out=st["out"][0])[None]
            return {"y": y}
        tokens, logprobs, accepted, rejected = tp.tp_verify(
            st["logits"], st["drafts"], st["cu_rows"], st["u"], draft_probs=st["draft_probs"],
            temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"], min_p=st["min_p"])
        return {"tokens": tokens, "logprobs": logprobs, "accepted": accepted, "rejected": rejected}
    return {"plan": _plan, "lora": _lora, "verify": _verify}[c["op"]](st)


def _before(x):
    """The sum of the elements before each."""
    return x.cumsum(0) - x


def _plan(st):
    c = st["case"]
    page, T = c["page"], st["tokens"]
    table, pool, counts, held = st["block_table"], st["free_pages"], st["counts"].long(), st["owned"].long()
    B, width = table.shape
    lens = st["seq_lens"].long() - (0 if st["rejected"] is None else st["rejected"].long())
    ends, new = counts < 0, counts.clamp(min=0)
    after = torch.where(ends, 0, lens + new)
    need = torch.where(ends, 0, (-(-after // page) - held).clamp(min=0))
    back = torch.where(ends, held, 0)
    top = st["free_count"].long() + back.sum()
    lack = (need.sum() - top).clamp(min=0)
    fits = (lack == 0) & (new.sum() <= T)
    j = torch.arange(width, device="cuda")
    # pages of the requests that ended go on top of the pool, then what is needed is taken from there
    where = st["free_count"] + _before(back)[:, None] + j
    where = torch.where((j < back[:, None]) & fits, where, len(pool)).flatten()
    grown = torch.cat([pool, pool.new_zeros(1)]).scatter(0, where, table.flatten())[:-1]
    pool.copy_(grown)
    taken = top - 1 - (_before(need)[:, None] + j - held[:, None])
    fresh = (j >= held[:, None]) & (j < (held + need)[:, None]) & fits
    table.copy_(torch.where(fresh, pool[taken.clamp(0, len(pool) - 1)], table))
    cu = torch.cat([new.new_zeros(1), torch.where(fits, new, 0).cumsum(0)])
    row = torch.arange(T, device="cuda")
    b = (torch.searchsorted(cu, row, right=True) - 1).clamp(max=B - 1)
    live = row < cu[-1]
    pos = torch.where(live, after[b] - new[b] + row - cu[b], 0)
    at = table[b, (pos // page).clamp(0, width - 1)].long() * page + pos % page
    i32 = torch.int32
    out = {"seq_lens": torch.where(fits, after, st["seq_lens"]).to(i32),
           "owned": torch.where(fits, torch.where(ends, 0, held + need), held).to(i32),
           "free_count": torch.where(fits, top - need.sum(), st["free_count"]).to(i32),
           "missing": lack.to(i32).reshape(1), "cu_seqlens": cu.to(i32), "positions": pos.to(i32),
           "slots": torch.where(live, at, -1), "block_table": table, "free_pages": pool}
    if st["adapters"] is not None:
        out["groups"] = _grouped(st["adapters"], out["cu_seqlens"], T, c["adapters"])
    return out


def _grouped(adapters, cu, T, n):
    """The plan of a step's adapters: [groups, tokens with an adapter, 0, 0], then min(T, n + 1) groups of (adapter,
    first place, tokens, 0), -1 where there is none, then the T tokens in the order of their adapters, -1 for the
    rows of no request.  Tokens without an adapter (-1) are the last group."""
    B, most = len(adapters), min(T, n + 1)
    row = torch.arange(T, device="cuda")
    b = (torch.searchsorted(cu.long(), row, right=True) - 1).clamp(max=B - 1)
    live = row < cu[-1]
    kind = torch.where(live, torch.where(adapters < 0, n, adapters).long()[b], n + 1)
    order = torch.sort(kind, stable=True)[1]
    tokens = torch.zeros(n + 2, dtype=torch.int64, device="cuda").scatter_add(0, kind, torch.ones_like(kind))
    first, tokens = _before(tokens)[:n + 1], tokens[:n + 1]
    some = tokens > 0
    place = torch.where(some, _before(some.long()), most)  # the groups without tokens behind the end
    ids = torch.arange(n + 1, device="cuda")
    rows = torch.stack([torch.where(ids < n, ids, -1), first, tokens, torch.zeros_like(ids)], 1)
    groups = torch.full((most + 1, 4), -1, dtype=torch.int64, device="cuda")
    groups = groups.scatter(0, place[:, None].expand(-1, 4), torch.where(some[:, None], rows, -1))[:most]
    zero = torch.zeros_like(first[0])
    head = torch.stack([some.sum(), tokens[:n].sum(), zero, zero])
    order = torch.where(row < tokens.sum(), order, -1)
    return torch.cat([head, groups.flatten(), order]).to(torch.int32)


def _lora(st):
    c = st["case"]
    T, R, n, ids = c["T"], c["R"], c["n"], st["token_ids"]
    x, a, b = st["x"].float(), st["a"].float(), st["b"].float()
    h = torch.matmul(x, a.flatten(1, 2).transpose(1, 2)).sum(0).view(T, n, R)  # every adapter's, the ranks added up
    mine = (torch.arange(n, device="cuda") == ids[:, None]) * st["scales"]
    h = (h * mine[:, :, None]).view(T, n * R)
    delta = torch.matmul(h, b.transpose(2, 3).flatten(1, 2))
    return {"y": (st["y"].float() + delta).to(DT[c["out"]])}


def _part(total, share):
    """floor(total * share / 2^24) for whole totals up to 2^62 and shares of 2^24, without leaving 64 bits."""
    return (total >> 24) * share + (((total & 0xFFFFFF) * share) >> 24)


def _verify(st):
    x = st["logits"].float()
    T, V = x.shape
    cu, row = st["cu_rows"].long(), torch.arange(T, device="cuda")
    B = len(cu) - 1
    seq = torch.searchsorted(cu, row, right=True) - 1
    last = cu[seq + 1] - 1
    x = torch.where(torch.isnan(x), -math.inf, x).clamp(max=FMAX) + 0.0

    def setting(name, missing):
        return st[name][seq][:, None] if st[name] is not None else torch.full_like(x[:, :1], missing)
    t, k, p = setting("temperature", 1.0), setting("top_k", 0).long(), setting("top_p", 1.0)
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
    keep = torch.zeros_like(keep).scatter(1, order, keep) & (e >= setting("min_p", 0.0).clamp(max=1))
    w = torch.where(keep, w, 0)
    share = 1.0 / (w.sum(1, keepdim=True).float() * 2.0 ** -40)
    prob = torch.where(keep, e * share, 0.0)
    d, own_place = st["drafts"][:, None], torch.arange(V, device="cuda")
    if st["draft_probs"] is not None:
        q = st["draft_probs"].float().clamp(0, 1)
    else:
        q = (own_place == d).float()
    taken = (st["u"][:, None] * q.gather(1, d) < prob.gather(1, d))[:, 0] & (row < last)
    # a request's drafts up to its first refused one; then a token of what the target has left over the draft
    stop = torch.full((B,), T, device="cuda").scatter_reduce(0, seq, torch.where(taken, T, row), "amin")
    rest = ((prob - q).clamp(min=0) * 2.0 ** 40).long()
    rest = torch.where((row < last)[:, None] & (rest.sum(1, keepdim=True) > 0), rest, w).cumsum(1)
    r = _part(rest[:, -1:], (st["u"][last][:, None] * 2.0 ** 24).long())
    drawn = (rest <= r).sum(1)
    token = torch.where(row < stop[seq], st["drafts"], drawn)
    logz = torch.log(torch.exp(x - top).sum(1))
    logprob = x.gather(1, token[:, None])[:, 0] - top[:, 0] - logz
    behind = row > stop[seq]
    accepted = stop - cu[:-1]
    return {"tokens": torch.where(behind, -1, token), "logprobs": torch.where(behind, 0.0, logprob),
            "accepted": accepted.to(torch.int32), "rejected": (cu[1:] - cu[:-1] - 1 - accepted).to(torch.int32)}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    st = prepare(case, seed)
    with torch.no_grad():
        return _exact_lora(case, st) if case["op"] == "lora" else _exact_verify(case, st)


def _exact_lora(c, st):
    y = st["y"].double()
    for i in range(c["n"]):
        rows = (st["token_ids"] == i).nonzero()[:, 0]
        if len(rows):
            h = sum(torch.einsum("tk,rk->tr", x[rows].double(), a[i].double()) for x, a in zip(st["x"], st["a"]))
            for r, b in enumerate(st["b"]):
                y[r, rows] += torch.einsum("tr,or->to", h, b[i].double()) * float(st["scales"][i])
    return {"y": y}


def _exact_verify(c, st):
    get = {n: st[n].double().cpu().numpy() for n in ("logits", "u", "temperature", "top_k", "top_p", "min_p")
           if st[n] is not None}
    cu, drafts = st["cu_rows"].tolist(), st["drafts"].tolist()
    q = None if st["draft_probs"] is None else st["draft_probs"].double().cpu().numpy()
    logprobs = np.zeros(cu[-1])
    for b in range(c["B"]):
        t, k, p, m = (float(get[n][b]) if n in get else v for n, v in
                      (("temperature", 1), ("top_k", 0), ("top_p", 1), ("min_p", 0)))
        for i in range(cu[b], cu[b + 1]):
            x = get["logits"][i]
            order = np.argsort(-x, kind="stable")
            w = np.exp((x[order] - x[order[0]]) / t) if t > 0 else np.ones(1)
            n = 1 if t == 0 else int(k) if 0 < k < len(x) else len(x)
            w = w[:n]
            if p < 1 and t > 0:
                w = w[:max(1, int(np.sum(np.cumsum(w) - w < p * w.sum())))]
            w = np.where(w >= m, w, 0.0)
            prob = np.zeros(len(x))
            prob[order[:len(w)]] = w / w.sum()
            if i < cu[b + 1] - 1:
                d = drafts[i]
                theirs = q[i] if q is not None else np.bincount([d], minlength=len(x))
                if get["u"][i] * theirs[d] < prob[d]:
                    logprobs[i] = x[d] - x.max() - np.log(np.sum(np.exp(x - x.max())))
                    continue
                left = np.maximum(prob - theirs, 0)
                prob = left if left.sum() > 0 else prob
            run = np.cumsum(prob)
            token = min(len(x) - 1, int(np.searchsorted(run, get["u"][cu[b + 1] - 1] * run[-1], side="right")))
            logprobs[i] = x[token] - x.max() - np.log(np.sum(np.exp(x - x.max())))
            break
    return {"tokens": None, "logprobs": logprobs, "accepted": None, "rejected": None}
