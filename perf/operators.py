"""The operators of the target model's verification step over a paged K/V cache, as cases to measure.

A speculative round ends with the target model checking the drafted block. Around the target's own
matrix products that step takes four operators of this package:

* ``page_slots``       lengths -> pages taken from the free list, block table, slot and position per token;
* ``norm_rope_paged``  per-head RMS norms of q and k, the rotation, and the write of k and v into the pages;
* ``attend_paged``     attention of each request's new tokens over its pages;
* ``sample``           temperature, top-k, top-p, min-p and the draw from given uniform numbers.

Each case runs one of them: in the plain form (``own`` false, elementary torch operations) or through
the package's calls (``own`` true). ``exact`` computes the same from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one request's verification step: the anchor and 16 drafted tokens after 4096 cached ones
        dict(name="slots 1 request", op="slots", B=1, new_lo=17, new_hi=17, ctx_lo=4096, ctx_hi=4096, page=64, pad=0, lens=1),
        # a serving step of 512 requests, decode rows among prompt chunks, padded to a graph's token count
        dict(name="slots 512 requests", op="slots", B=512, new_lo=1, new_hi=255, ctx_lo=0, ctx_hi=32768, page=16, pad=1000, lens=2),
        # q, k, v heads of 32 requests x 17 tokens, this repository's head layout, fp32 products into an fp16 cache
        dict(name="norm rope 544 tokens", op="norm", T=544, nH=16, nKv=2, hd=256, x="fp32", kv="fp16", page=64, pos_hi=8192, v_norm=True, pad=0),
        # a prompt chunk of 16384 tokens at far positions, bf16 throughout, an odd number of padding rows
        dict(name="norm rope 16384 tokens", op="norm", T=16384, nH=32, nKv=8, hd=128, x="bf16", kv="bf16", page=16, pos_hi=1000000, v_norm=False, pad=37),
        # verification of one request: latency
        dict(name="attend verify 1x17", op="attend", B=1, new_lo=17, new_hi=17, ctx_lo=4096, ctx_hi=4096, nH=16, nKv=2, hd=256, kv="fp16", page=64, causal=True, window=0, lse=False, lens=3),
        # verification of 32 ragged requests, small pages
        dict(name="attend verify 32 ragged", op="attend", B=32, new_lo=1, new_hi=17, ctx_lo=512, ctx_hi=4096, nH=16, nKv=2, hd=256, kv="fp16", page=16, causal=True, window=0, lse=False, lens=4),
        # single-token decoding of 64 long requests: the cache's bytes
        dict(name="attend decode 64 long", op="attend", B=64, new_lo=1, new_hi=1, ctx_lo=8192, ctx_hi=32768, nH=32, nKv=8, hd=128, kv="bf16", page=16, causal=True, window=0, lse=True, lens=5),
        # prompt chunks of four requests after up to 6144 cached tokens: the tensor cores
        dict(name="attend chunk 4x2048", op="attend", B=4, new_lo=1900, new_hi=2048, ctx_lo=0, ctx_hi=6144, nH=32, nKv=8, hd=128, kv="bf16", page=64, causal=True, window=0, lse=False, lens=6),
        # a long prompt chunk of a sliding-window layer with wide heads
        dict(name="attend window 1x8191", op="attend", B=1, new_lo=8191, new_hi=8191, ctx_lo=1000, ctx_hi=1000, nH=16, nKv=2, hd=256, kv="fp16", page=32, causal=True, window=1024, lse=False, lens=7),
        # one token of one request
        dict(name="sample 1 row", op="sample", rows=1, V=262144, x="fp32", filters="mixed"),
        # the verified positions of 32 requests, mixed settings, the draft round's fp32 logits
        dict(name="sample 512 rows", op="sample", rows=512, V=262144, x="fp32", filters="mixed"),
        # an odd vocabulary in bf16, temperature alone
        dict(name="sample 77 rows", op="sample", rows=77, V=50257, x="bf16", filters="none"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["slots", "norm", "attend", "attend", "attend", "sample"])
    page = rng.choice([16, 32, 64, 128])
    lens = rng.randrange(1 << 30)
    if op == "slots":
        B = _log(rng, 1, 1024)
        hi = _log(rng, 1, max(1, 131072 // B))
        return dict(op="slots", B=B, new_lo=rng.choice([0, 1]) if B >= 8 and hi >= 4 else 1, new_hi=min(hi, 8192), ctx_lo=0, ctx_hi=_log(rng, 1, 32768), page=page,
                    pad=rng.choice([0, rng.randrange(1, 500)]), lens=lens)
    if op == "norm":
        nKv = rng.choice([1, 2, 4, 8])
        return dict(op="norm", T=_log(rng, 1, 12000), nH=nKv * rng.choice([1, 2, 3, 4]), nKv=nKv, hd=rng.choice([64, 128, 192, 256] if nKv < 8 else [64, 128]),
                    x=rng.choice(["fp32", "bf16", "fp16"]), kv=rng.choice(["fp16", "bf16"]), page=page, pos_hi=_log(rng, 100, 1000000),
                    v_norm=rng.choice([True, False]), pad=rng.choice([0, 5]))
    if op == "sample":
        V = _log(rng, 1000, 262144)
        return dict(op="sample", rows=_log(rng, 1, max(1, min(512, 100_000_000 // V))), V=V, x=rng.choice(["fp32", "bf16"]), filters=rng.choice(["mixed", "none"]))
    nKv, grp = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8])
    hd = rng.choice([64, 128, 128, 192, 256])
    new = rng.choice([1, _log(rng, 2, 32), _log(rng, 33, 4096)])
    ctx = _log(rng, 1, 32768)
    # the plain form's padded scores stay within 2^31 values, the cache within 2^29 a side
    B = _log(rng, 1, max(1, min(128, (1 << 31) // (nKv * grp * new * (ctx + new)), (1 << 29) // ((ctx + new) * nKv * hd))))
    while new > 1 and nKv * grp * B * new * (ctx + new) > 1 << 31:
        new //= 2
    return dict(op="attend", B=B, new_lo=rng.choice([1, new]), new_hi=new, ctx_lo=rng.choice([0, ctx]), ctx_hi=ctx, nH=nKv * grp, nKv=nKv, hd=hd,
                kv=rng.choice(["fp16", "bf16"]), page=page, causal=rng.choice([True, True, False]), window=rng.choice([0, 0, _log(rng, 16, 4096)]),
                lse=rng.choice([True, False]), lens=lens)


def _lengths(case):
    """(cached length, new tokens) of each request: a case's own, whatever the seed."""
    r = random.Random(case["lens"])
    return [(r.randint(case["ctx_lo"], case["ctx_hi"]), r.randint(case["new_lo"], case["new_hi"])) for _ in range(case["B"])]


def _ceil(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    ints = lambda v, dt=torch.int32: torch.tensor(v, dtype=dt, device="cuda")  # noqa: E731
    perm = lambda n: torch.randperm(n, generator=gen, device="cuda")  # noqa: E731
    empty = lambda *s, dt=torch.int32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    s, op = dict(case), case["op"]
    if op == "slots":
        ln, ps, B = _lengths(case), case["page"], case["B"]
        ctx, new = [c for c, _ in ln], [n for _, n in ln]
        held = [_ceil(c, ps) for c in ctx]                       # pages the requests hold already
        need = sum(_ceil(c + n, ps) - h for c, n, h in zip(ctx, new, held))
        pages, width = sum(held) + need + 64, max(_ceil(c + n, ps) for c, n in ln)
        order = perm(pages).to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        at = torch.arange(width, device="cuda")[None] < ints(held)[:, None]
        table[at] = order[:sum(held)]
        s.update(ctx_len=ints(ctx), n_new=ints(new), block_table=table, n_pages=ints(held), free_pages=order[sum(held):].contiguous(),
                 free_count=ints([pages - sum(held)]), tokens=max(1, sum(new)) + case["pad"], pages=pages)
        if own:  # the handle and the output buffers that a serving loop keeps
            import block_draft_model_dspark_b200 as dsp
            s["cache"] = dsp.PagedKvCache(pages, ps, 1, 64, block_table=table, k=empty(1, pages, ps, 1, 64, dt=torch.float16), v=empty(1, pages, ps, 1, 64, dt=torch.float16))
            s["out"] = dict(n_pages_out=empty(B), free_count_out=empty(1), cu_new=empty(B + 1), kv_len=empty(B), slots=empty(s["tokens"], dt=torch.int64), positions=empty(s["tokens"]))
    elif op == "norm":
        T, nH, nKv, hd, ps, dt = case["T"], case["nH"], case["nKv"], case["hd"], case["page"], _DT[case["kv"]]
        x = (rnd(T, (nH + 2 * nKv) * hd) * 1.7).to(_DT[case["x"]])      # one product's rows: [q ; k ; v]
        s["q"], s["k"], s["v"] = (t.unflatten(1, (-1, hd)) for t in x.split([nH * hd, nKv * hd, nKv * hd], 1))
        s["q_norm"], s["k_norm"] = ((1 + 0.1 * rnd(hd)).to(_DT[case["x"]]) for _ in range(2))
        s["inv_freq"] = 1e6 ** (-torch.arange(hd // 2, dtype=torch.float64, device="cuda") * 2 / hd)
        s["positions"] = torch.randint(0, case["pos_hi"], (T,), generator=gen, device="cuda").to(torch.int32)
        pages = _ceil(T, ps) + 3
        s["slots"] = perm(pages * ps)[:T].clone()
        if case["pad"]:
            s["slots"][-min(case["pad"], T):] = -1                       # a graph's padding rows
        s["k_cache"], s["v_cache"] = (rnd(1, pages, ps, nKv, hd).to(dt) for _ in range(2))
        s["q_out"] = torch.zeros(T, nH, hd, dtype=dt, device="cuda")
        if own:
            import block_draft_model_dspark_b200 as dsp
            s["cache"] = dsp.PagedKvCache(pages, ps, nKv, hd, block_table=empty(1, 1), k=s["k_cache"], v=s["v_cache"])
    elif op == "attend":
        ln, ps, B, nH, nKv, hd, dt = _lengths(case), case["page"], case["B"], case["nH"], case["nKv"], case["hd"], _DT[case["kv"]]
        kv, new = [c + n for c, n in ln], [n for _, n in ln]
        need = [_ceil(n, ps) for n in kv]
        pages, T = sum(need) + 2, sum(new)
        table = torch.full((B, max(need)), -1, dtype=torch.int32, device="cuda")
        table[torch.arange(max(need), device="cuda")[None] < ints(need)[:, None]] = perm(pages)[:sum(need)].to(torch.int32)
        # normed queries and keys: scores of unit variance at the scale below, as a trained layer has
        s["q"] = (rnd(T, nH, hd) * 1.2).to(dt)
        s["k_cache"], s["v_cache"] = rnd(1, pages, ps, nKv, hd).to(dt), rnd(1, pages, ps, nKv, hd).to(dt)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s.update(block_table=table, cu_new=ints(cu), kv_len=ints(kv), scale=hd ** -0.5, max_new=max(new), max_kv=max(kv), pages=pages)
        s["o"] = torch.zeros(T, nH, hd, dtype=dt, device="cuda")
        if own:
            import block_draft_model_dspark_b200 as dsp
            s["cache"] = dsp.PagedKvCache(pages, ps, nKv, hd, block_table=table, k=s["k_cache"], v=s["v_cache"])
            s["ws"] = dsp.attend_paged_workspace(s["cache"], T, nH, B)
            s["lse_out"] = empty(T, nH, dt=torch.float32) if case["lse"] else None
    else:
        R, V = case["rows"], case["V"]
        x = rnd(R, V) * 2.5
        top = torch.randint(0, V, (R, 24), generator=gen, device="cuda")
        x.scatter_add_(1, top, 9 + 3 * rnd(R, 24))                        # a few likely tokens above the rest
        s["logits"] = (30 * torch.tanh(x / 30)).to(_DT[case["x"]])        # softcapped, as the round's logits are
        del x
        uni = lambda lo, hi: torch.rand(R, generator=gen, device="cuda") * (hi - lo) + lo  # noqa: E731
        s["u"] = uni(0, 1)
        some = lambda t, off, share: torch.where(torch.rand(R, generator=gen, device="cuda") < share, t, torch.full_like(t, off))  # noqa: E731
        s["temperature"] = some(uni(0.5, 1.3), 0.0 if case["filters"] == "mixed" else 1.0, 0.85)
        s["top_k"] = s["top_p"] = s["min_p"] = None
        if case["filters"] == "mixed":
            s["top_k"] = some(torch.randint(1, 200, (R,), generator=gen, device="cuda").to(torch.int32), 0, 0.5)
            s["top_p"], s["min_p"] = some(uni(0.7, 1.0), 1.0, 0.6), some(uni(0.0, 0.1), 0.0, 0.4)
        s["tokens"], s["probs"] = empty(R), empty(R, dt=torch.float32)
        if own:
            import block_draft_model_dspark_b200 as dsp
            s["ws"] = dsp.sample_workspace(R, V, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return {"slots": _slots, "norm": _norm, "attend": _attend, "sample": _sample}[s["op"]](s)


def _slots(s):
    if own:
        import block_draft_model_dspark_b200 as dsp
        o = s["out"]
        dsp.page_slots(s["cache"], s["ctx_len"], s["n_new"], s["n_pages"], s["free_pages"], s["free_count"], s["tokens"], **o)
        return dict(o, block_table=s["block_table"])
    ps, table, dev = s["page"], s["block_table"], s["ctx_len"].device
    kv = s["ctx_len"] + s["n_new"]
    want = torch.maximum((kv + ps - 1) // ps, s["n_pages"])
    take = want - s["n_pages"]                                            # pages each request takes
    first = torch.cumsum(take, 0) - take
    col = torch.arange(table.shape[1], device=dev)[None]
    fresh = (col >= s["n_pages"][:, None]) & (col < want[:, None])
    rank = first[:, None] + col - s["n_pages"][:, None]
    pick = s["free_pages"][(s["free_count"] - 1 - rank).clamp(0, s["free_pages"].numel() - 1).long()]
    table.copy_(torch.where(fresh, pick, table))
    cu = torch.nn.functional.pad(torch.cumsum(s["n_new"], 0), (1, 0)).to(torch.int32)
    t = torch.arange(s["tokens"], device=dev)
    b = torch.searchsorted(cu[1:], t.to(torch.int32), right=True).clamp(max=kv.numel() - 1)
    p = s["ctx_len"][b].long() + t - cu[b]
    real = t < cu[-1]
    p = torch.where(real, p, torch.zeros_like(p))
    slot = table[b, p // ps].long() * ps + p % ps
    return {"n_pages_out": want, "free_count_out": s["free_count"] - take.sum().to(torch.int32), "cu_new": cu, "kv_len": kv,
            "slots": torch.where(real, slot, torch.full_like(slot, -1)), "positions": p.to(torch.int32), "block_table": table}


def _norm(s):
    if own:
        import block_draft_model_dspark_b200 as dsp
        dsp.norm_rope_paged(s["q"], s["k"], s["v"], s["q_norm"], s["k_norm"], s["inv_freq"], s["positions"], s["slots"], s["cache"], 0,
                            eps=1e-6, v_norm=s["v_norm"], q_out=s["q_out"])
        return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}
    half = s["hd"] // 2
    rms = lambda x: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    turn = s["positions"].double()[:, None] * s["inv_freq"][None]
    cos, sin = turn.cos().float()[:, None], turn.sin().float()[:, None]

    def rope(x):
        a, b = x[..., :half], x[..., half:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    q = rope(rms(s["q"].float()) * s["q_norm"].float())
    k = rope(rms(s["k"].float()) * s["k_norm"].float())
    v = rms(s["v"].float()) if s["v_norm"] else s["v"].float()
    real = s["slots"] >= 0
    at = s["slots"][real]
    dt = s["q_out"].dtype
    s["q_out"].copy_(torch.where(real[:, None, None], q.to(dt), s["q_out"]))
    s["k_cache"].view(-1, s["nKv"], s["hd"])[at] = k[real].to(dt)
    s["v_cache"].view(-1, s["nKv"], s["hd"])[at] = v[real].to(dt)
    return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}


def _attend(s):
    if own:
        import block_draft_model_dspark_b200 as dsp
        dsp.attend_paged(s["q"], s["cache"], 0, s["cu_new"], s["kv_len"], s["max_new"], scale=s["scale"], causal=s["causal"], window=s["window"],
                         out=s["o"], lse=s["lse_out"], ws=s["ws"])
        return {"o": s["o"], "lse": s["lse_out"]} if s["lse"] else {"o": s["o"]}
    T, nH, hd = s["q"].shape
    B, nKv, N, L, ps, dev = s["B"], s["nKv"], s["max_new"], s["max_kv"], s["page"], s["q"].device
    cu, kv = s["cu_new"].long(), s["kv_len"].long()
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cu[1:], t, right=True)
    i = t - cu[b]
    q = torch.zeros(B, N, nH, hd, device=dev)
    q[b, i] = s["q"].float()
    key = torch.arange(L, device=dev)
    page = s["block_table"][:, key // ps].long()                           # [B, L]
    held = key[None] < kv[:, None]
    rows = torch.where(held, page * ps + key % ps, torch.zeros_like(page))
    k = s["k_cache"].view(-1, nKv, hd)[rows].float()                       # [B, L, nKv, hd]
    sc = q.view(B, N, nKv, nH // nKv, hd).permute(0, 2, 3, 1, 4).reshape(B, nKv, -1, hd) @ k.permute(0, 2, 3, 1)
    del k
    sc = (sc * s["scale"]).view(B, nH, N, L)
    pos = (kv - (cu[1:] - cu[:-1]))[:, None] + torch.arange(N, device=dev)  # [B, N] key position of each query
    see = held[:, None].expand(B, N, L)
    if s["causal"]:
        see = see & (key <= pos[..., None])
    if s["window"]:
        see = see & (key > pos[..., None] - s["window"])
    sc.masked_fill_(~see[:, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp_(sc.sub_(top))
    total = p.sum(-1, keepdim=True)
    v = torch.where(held[..., None, None], s["v_cache"].view(-1, nKv, hd)[rows].float(), torch.zeros((), device=dev))
    o = (p.view(B, nKv, -1, L) @ v.permute(0, 2, 1, 3)).view(B, nH, N, hd)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).permute(0, 2, 1, 3)[b, i]
    s["o"].copy_(o.to(s["o"].dtype))
    if not s["lse"]:
        return {"o": s["o"]}
    return {"o": s["o"], "lse": (top + torch.log(total)).squeeze(-1).permute(0, 2, 1)[b, i].contiguous()}


def _sample(s):
    if own:
        import block_draft_model_dspark_b200 as dsp
        dsp.sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], tokens=s["tokens"], probs=s["probs"], ws=s["ws"])
        return {"tokens": s["tokens"], "probs": s["probs"]}
    R, V = s["logits"].shape
    x, order = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)   # equal ones: the lowest index first
    temp = s["temperature"].double()[:, None]
    greedy = temp <= 0
    z = (x.double() - x[:, :1].double()) / torch.where(greedy, torch.ones_like(temp), temp)
    w = torch.exp_(z)
    rank = torch.arange(V, device=x.device)[None]
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        w = torch.where((rank < k) | (k <= 0), w, torch.zeros_like(w))
    low = torch.zeros_like(temp) if s["min_p"] is None else s["min_p"].double()[:, None]
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        cum = torch.cumsum(w, 1)
        w = torch.where((cum - w < p * cum[:, -1:]) | (p >= 1) | (rank == 0), w, torch.zeros_like(w))
        del cum
    w = torch.where(((w >= low) & (~greedy)) | (rank == 0), w, torch.zeros_like(w))
    w = torch.zeros_like(w).scatter_(1, order, w)                          # back in the order of the vocabulary
    cum = torch.cumsum(w, 1)
    at = (cum <= s["u"].double()[:, None] * cum[:, -1:]).sum(1)
    prob = (w.gather(1, at[:, None]) / cum[:, -1:]).squeeze(1)
    return {"tokens": at.to(torch.int32), "probs": prob.float()}


# ------------------------------------------------------------------ the work
def _pairs(case):
    """(query, key) pairs that see each other, and the keys that some query of their request sees."""
    pairs = keys = 0
    for c, n in _lengths(case):
        L, W = c + n, case["window"]
        lo = [max(0, c + i - W + 1) if W else 0 for i in range(n)]
        hi = [c + i + 1 if case["causal"] else L for i in range(n)]
        pairs += sum(max(0, h - l) for h, l in zip(hi, lo))
        keys += max(hi) - min(lo) if n else 0
    return pairs, keys


def work(case):
    op = case["op"]
    if op == "slots":
        ln = _lengths(case)
        taken = sum(_ceil(c + n, case["page"]) - _ceil(c, case["page"]) for c, n in ln)
        return {"bytes": 4 * case["B"] * 6 + 12 * (max(1, sum(n for _, n in ln)) + case["pad"]) + 8 * taken, "flops": 0}
    if op == "norm":
        es, T = (4 if case["x"] == "fp32" else 2), case["T"] - min(case["pad"], case["T"])
        heads = case["nH"] + 2 * case["nKv"]
        return {"bytes": T * heads * case["hd"] * (es + 2) + 12 * case["T"], "flops": T * (heads * 10.0 * case["hd"])}
    if op == "attend":
        pairs, keys = _pairs(case)
        T = sum(n for _, n in _lengths(case))
        return {"bytes": 4 * T * case["nH"] * case["hd"] + 4 * keys * case["nKv"] * case["hd"], "flops": 4.0 * pairs * case["nH"] * case["hd"]}
    return {"bytes": case["rows"] * case["V"] * (4 if case["x"] == "fp32" else 2), "flops": 4.0 * case["rows"] * case["V"]}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    op = case["op"]
    if op == "slots":
        return None
    s = prepare(case, seed)
    if op == "norm":
        T, hd = case["T"], case["hd"]
        angle = torch.outer(s["positions"].double(), s["inv_freq"])
        unit = torch.polar(torch.ones_like(angle), angle)[:, None]         # e^(i angle)
        out = {"q": s["q_out"].double(), "k": s["k_cache"].double(), "v": s["v_cache"].double()}
        keep = torch.nonzero(s["slots"] >= 0).squeeze(1)
        page, row = s["slots"][keep] // case["page"], s["slots"][keep] % case["page"]
        for name, gain in (("q", "q_norm"), ("k", "k_norm"), ("v", None)):
            x = s[name].double()
            if gain or case["v_norm"]:
                x = x / (x.pow(2).sum(-1, keepdim=True) / hd + 1e-6).sqrt()
            if gain:
                x = x * s[gain].double()
                z = torch.complex(x[..., : hd // 2].contiguous(), x[..., hd // 2:].contiguous()) * unit
                x = torch.cat([z.real, z.imag], -1)
            if name == "q":
                out["q"][keep] = x[keep]
            else:
                out[name][0, page, row] = x[keep]
        return out
    if op == "attend":
        T, nH, hd = s["q"].shape
        grp, ps = nH // case["nKv"], case["page"]
        out, lse = torch.zeros(T, nH, hd, dtype=torch.float64, device="cuda"), torch.full((T, nH), -math.inf, dtype=torch.float64, device="cuda")
        t0 = 0
        for b, (c, n) in enumerate(_lengths(case)):
            at = s["block_table"][b, : _ceil(c + n, ps)].long()
            K, V = (s[x][0, at].flatten(0, 1)[: c + n].double() for x in ("k_cache", "v_cache"))
            j = torch.arange(c + n, device="cuda")
            for i0 in range(0, n, 1024):
                i = torch.arange(i0, min(n, i0 + 1024), device="cuda")[:, None] + c
                bias = torch.zeros(i.shape[0], c + n, dtype=torch.float64, device="cuda")
                if case["causal"]:
                    bias[j > i] = -math.inf
                if case["window"]:
                    bias[j <= i - case["window"]] = -math.inf
                for h in range(nH):
                    a = s["q"][t0 + i0: t0 + i0 + i.shape[0], h].double() @ K[:, h // grp].T * s["scale"] + bias
                    z = torch.logsumexp(a, -1)
                    some = z > -math.inf
                    out[t0 + i0: t0 + i0 + i.shape[0], h][some] = torch.exp(a[some] - z[some, None]) @ V[:, h // grp]
                    lse[t0 + i0: t0 + i0 + i.shape[0], h] = z
            t0 += n
        return {"o": out, "lse": lse} if case["lse"] else {"o": out}
    R, V = case["rows"], case["V"]
    probs = torch.empty(R, dtype=torch.float64, device="cuda")
    for r in range(R):
        x = s["logits"][r].double()
        T = s["temperature"][r].item()
        if T <= 0:
            probs[r] = 1.0
            continue
        p = torch.softmax(x / T, 0)
        # by falling probability, then by index, over the kept candidates only
        order = torch.argsort(x, descending=True, stable=True)
        k = V if s["top_k"] is None or s["top_k"][r].item() <= 0 else min(V, s["top_k"][r].item())
        kept = order[:k]
        if s["top_p"] is not None and s["top_p"][r].item() < 1:
            c = torch.cumsum(p[kept], 0)
            n = int((c < s["top_p"][r].double() * c[-1]).sum().item()) + 1
            kept = kept[:n]
        if s["min_p"] is not None:
            kept = kept[p[kept] >= s["min_p"][r].double() * p[kept[0]]]
        kept = torch.sort(kept).values
        c = torch.cumsum(p[kept], 0)
        n = min(int(torch.searchsorted(c, s["u"][r].double() * c[-1], right=True).item()), kept.numel() - 1)
        probs[r] = p[kept[n]] / c[-1]
    return {"tokens": None, "probs": probs}
