"""The operators of a verification step of several requests, as they are measured.

Four operators run in this order around the expert engines: the batch plan
(block tables, slots and positions from request lengths), the append of new
keys and values to a paged cache, the attention of every request's new tokens
over that cache, and the routing of tokens to experts with scores, bias and
groups. Each has a plain form here, made of elementary torch operations.

Sizes: head counts are d / 128 of the layer shapes in configs.py (16, 32 and
56 heads), expert counts and top-k are those shapes' own, and pass sizes are
1..16 tokens per request as in their workloads; page sizes, cache lengths and
batch sizes are generic.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
WIDTH = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one stream's verification pass: what a single user waits for each step
        {"name": "plan_step", "op": "plan", "requests": 1, "page": 64, "q_lo": 5, "q_hi": 5,
         "kv_hi": 2000, "chunks": 0, "chunk_hi": 0, "spare": 1.0, "len_seed": 1},
        # a full serving batch: verification passes beside a few prompts that enter in chunks,
        # with too few free pages for the last requests
        {"name": "plan_batch", "op": "plan", "requests": 1000, "page": 16, "q_lo": 1, "q_hi": 9,
         "kv_hi": 30000, "chunks": 20, "chunk_hi": 2048, "spare": 0.9, "len_seed": 2},
        # new keys and values of four requests' passes
        {"name": "append_step", "op": "append", "tokens": 36, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "src": "bf16", "page": 64, "heads_first": False, "dropped": 0.0},
        # a prompt chunk's keys and values, rounded from fp32 on the way, heads before tokens
        # within a page; some tokens belong to refused requests
        {"name": "append_chunk", "op": "append", "tokens": 12345, "kv_heads": 8, "dim": 128,
         "dtype": "f16", "src": "f32", "page": 32, "heads_first": True, "dropped": 0.02},
        # the routing of one pass of nine tokens: 64 experts, top 6, softmax, renormalised
        {"name": "route_step", "op": "route", "tokens": 9, "experts": 64, "topk": 6, "groups": 1,
         "top_groups": 1, "group_top": 1, "score": "softmax", "bias": False, "renorm": True,
         "scale": 1.0, "dtype": "f32", "masked": 0.0},
        # four streams of sixteen tokens: 256 experts in 8 groups, 4 groups kept, top 8
        {"name": "route_streams", "op": "route", "tokens": 64, "experts": 256, "topk": 8,
         "groups": 8, "top_groups": 4, "group_top": 2, "score": "sigmoid", "bias": True,
         "renorm": True, "scale": 2.5, "dtype": "f32", "masked": 0.0},
        # a prompt chunk's tokens, logits in bf16 with a few experts masked off
        {"name": "route_chunk", "op": "route", "tokens": 20011, "experts": 256, "topk": 8,
         "groups": 8, "top_groups": 4, "group_top": 2, "score": "sigmoid", "bias": True,
         "renorm": True, "scale": 2.5, "dtype": "bf16", "masked": 0.01},
        # one stream's pass of five tokens over a short cache, every head with its own keys:
        # the smallest call, all latency
        {"name": "attend_step", "op": "attend", "requests": 1, "q_lo": 5, "q_hi": 5, "kv_lo": 777,
         "kv_hi": 777, "chunks": 0, "chunk_hi": 0, "empty": 0, "heads": 16, "kv_heads": 16,
         "dim": 128, "dtype": "bf16", "page": 64, "heads_first": False, "window": 0, "sinks": 0,
         "pool": 0, "len_seed": 3},
        # a serving batch's verification passes over long ragged caches: bound by reading them
        {"name": "attend_verify", "op": "attend", "requests": 64, "q_lo": 1, "q_hi": 9,
         "kv_lo": 200, "kv_hi": 16000, "chunks": 0, "chunk_hi": 0, "empty": 0, "heads": 32,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "page": 64, "heads_first": False,
         "window": 0, "sinks": 0, "pool": 0, "len_seed": 4},
        # prompt chunks and verification passes in one call, seven heads per key head, small
        # pages, one refused request whose rows see nothing
        {"name": "attend_mixed", "op": "attend", "requests": 24, "q_lo": 1, "q_hi": 16,
         "kv_lo": 20, "kv_hi": 5000, "chunks": 3, "chunk_hi": 700, "empty": 1, "heads": 56,
         "kv_heads": 8, "dim": 64, "dtype": "f16", "page": 16, "heads_first": True, "window": 0,
         "sinks": 0, "pool": 0, "len_seed": 5},
        # long prompts entering in large chunks: bound by the products
        {"name": "attend_chunk", "op": "attend", "requests": 3, "q_lo": 1500, "q_hi": 4001,
         "kv_lo": 6000, "kv_hi": 12000, "chunks": 0, "chunk_hi": 0, "empty": 0, "heads": 32,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "page": 128, "heads_first": False,
         "window": 0, "sinks": 0, "pool": 0, "len_seed": 6},
        # windowed passes over very long caches whose pool of pages spans more than 2^31
        # elements; pages behind the window are given back
        {"name": "attend_window", "op": "attend", "requests": 48, "q_lo": 1, "q_hi": 9,
         "kv_lo": 3000, "kv_hi": 120000, "chunks": 0, "chunk_hi": 0, "empty": 0, "heads": 56,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "page": 256, "heads_first": False,
         "window": 4096, "sinks": 4, "pool": 2200000, "len_seed": 7},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "route", "attend", "attend"])
    if op == "plan":
        requests = _log(rng, 1, 1024)
        chunks = rng.randint(0, max(0, min(20, requests // 4)))
        return {"op": "plan", "requests": requests, "page": rng.choice([16, 32, 64, 128, 256]),
                "q_lo": rng.randint(0, 1), "q_hi": rng.randint(1, 16), "kv_hi": _log(rng, 10, 30000),
                "chunks": chunks, "chunk_hi": _log(rng, 20, 2048) if chunks else 0,
                "spare": rng.choice([1.0, 1.0, 0.9, 0.5]), "len_seed": rng.randrange(1 << 30)}
    if op == "append":
        dtype = rng.choice(["bf16", "f16"])
        return {"op": "append", "tokens": _log(rng, 1, 12345), "kv_heads": rng.choice([1, 2, 4, 8]),
                "dim": rng.choice([64, 128]), "dtype": dtype, "src": rng.choice([dtype, "f32"]),
                "page": rng.choice([16, 32, 64, 128, 256]), "heads_first": rng.random() < 0.5,
                "dropped": rng.choice([0.0, 0.02, 0.5])}
    if op == "route":
        experts, groups = rng.choice([(8, 1), (16, 4), (60, 1), (64, 1), (64, 8), (128, 1),
                                      (160, 8), (251, 1), (256, 8), (256, 16), (256, 1)])
        size = experts // groups
        top_groups = rng.randint(1, groups)
        dtype = rng.choice(["f32", "bf16", "f16"])
        return {"op": "route", "tokens": _log(rng, 1, 20011 // (WIDTH[dtype] // 2)), "experts": experts,
                "topk": rng.randint(1, min(12, top_groups * size)), "groups": groups,
                "top_groups": top_groups, "group_top": rng.choice([1, 2]) if size > 1 else 1,
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5,
                "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5, 16.0]),
                "dtype": dtype, "masked": rng.choice([0.0, 0.01, 0.3])}
    while True:
        case = _draw_attend(rng)
        if work(case)["bytes"] <= 900e6:
            return case


def _draw_attend(rng):
    kv_heads, per = rng.choice([(16, 1), (8, 4), (8, 7), (4, 8), (1, 16), (2, 3), (8, 2), (1, 1)])
    windowed = rng.random() < 0.35
    if rng.random() < 0.35:   # prompts in large chunks
        requests, chunks = rng.randint(1, 3), 0
        q_lo, q_hi = 1, _log(rng, 64, 3500)
        kv_hi = q_hi + _log(rng, 1, 6000)
        kv_lo = rng.randint(1, kv_hi)
        chunk_hi = 0
    else:                     # verification passes, some with prompts among them
        requests = _log(rng, 1, 64)
        q_lo, q_hi = 1, rng.randint(1, 16)
        kv_hi = _log(rng, 16, 12000)
        kv_lo = rng.randint(1, kv_hi)
        chunks = rng.randint(1, min(3, requests)) if rng.random() < 0.4 else 0
        chunk_hi = _log(rng, 16, 700) if chunks else 0
    return {"op": "attend", "requests": requests, "q_lo": q_lo, "q_hi": q_hi, "kv_lo": kv_lo,
            "kv_hi": kv_hi, "chunks": chunks, "chunk_hi": chunk_hi,
            "empty": 1 if requests > 2 and rng.random() < 0.3 else 0, "heads": kv_heads * per,
            "kv_heads": kv_heads, "dim": rng.choice([64, 128]), "dtype": rng.choice(["bf16", "f16"]),
            "page": rng.choice([16, 32, 64, 128, 256]), "heads_first": rng.random() < 0.5,
            "window": _log(rng, 1, 5000) if windowed else 0,
            "sinks": rng.choice([0, 1, 4, 130]) if windowed else 0, "pool": 0,
            "len_seed": rng.randrange(1 << 30)}


# ---------------------------------------------------- lengths from a case --
def _plan_lengths(case):
    """q_len, cached, held and the number of free pages: whole numbers of the case alone."""
    rng = random.Random(case["len_seed"])
    B, p = case["requests"], case["page"]
    q = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(B)]
    cached = [rng.randint(0, case["kv_hi"]) for _ in range(B)]
    for b in rng.sample(range(B), case["chunks"]):
        q[b] = _log(rng, 1, case["chunk_hi"])
    # a request may still hold pages of drafted tokens that were turned down
    held = [-(-c // p) + (1 if rng.random() < 0.1 else 0) for c in cached]
    need = sum(max(0, -(-(c + n) // p) - h) for c, n, h in zip(cached, q, held))
    free = max(0, int(need * case["spare"]) if case["spare"] < 1.0 else need + 7)
    return q, cached, held, free


def _attend_lengths(case):
    """New tokens and visible cache length of every request (the new tokens included)."""
    rng = random.Random(case["len_seed"])
    B = case["requests"]
    q = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(B)]
    kv = [_log(rng, case["kv_lo"], case["kv_hi"]) for _ in range(B)]
    for b in rng.sample(range(B), case["chunks"]):
        q[b] = _log(rng, max(1, case["chunk_hi"] // 4), case["chunk_hi"])
    kv = [max(n, m) for n, m in zip(q, kv)]
    for b in rng.sample(range(B), case["empty"]):
        kv[b] = 0
    return q, kv


# ---------------------------------------------------------------- prepare --
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((seed * 1000003 + salt) & 0x7FFFFFFF)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pool(case, n_pages, seed):
    """Key and value pages, [pages][tokens][heads][dim] whatever their order in memory."""
    p, H, D, dt = case["page"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    shape = (n_pages, H, p, D) if case["heads_first"] else (n_pages, p, H, D)
    out = []
    for salt in (11, 12):
        t = torch.empty(shape, dtype=dt, device="cuda")
        t.normal_(generator=_gen(seed, salt))
        out.append(t.transpose(1, 2) if case["heads_first"] else t)
    return out


def _prepare_plan(case, seed):
    q, cached, held, n_free = _plan_lengths(case)
    B, p = case["requests"], case["page"]
    M = max(-(-(c + n) // p) for c, n in zip(cached, q)) + 2
    M = max(M, max(held))
    g = _gen(seed, 1)
    pages = torch.randperm(sum(held) + n_free + 3, generator=g, device="cuda").int()
    table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    rows = torch.arange(M, device="cuda")[None, :] < _i32(held)[:, None]
    table[rows] = pages[: sum(held)]
    head = 3
    state = {"case": case, "q_len": _i32(q), "cached": _i32(cached), "held": _i32(held),
             "free": pages[sum(held):].contiguous(), "range": _i32([head, head + n_free]),
             "table": table, "tokens": sum(q) + 5}   # five rows of padding behind the batch
    if own:
        from moe_expert_layer_warp_gb300 import batch
        state["planner"] = batch.BatchPlanner(p, max_requests=B, max_tokens=state["tokens"])
    return state


def _prepare_append(case, seed):
    T, H, D, p = case["tokens"], case["kv_heads"], case["dim"], case["page"]
    n_pages = -(-T // p) + 9
    kc, vc = _pool(case, n_pages, seed)
    src = DTYPES[case["src"]]
    # keys and values as a joint projection leaves them: one row [keys | values] per token
    kv = torch.empty((T, 2, H, D), dtype=src, device="cuda").normal_(generator=_gen(seed, 21))
    g = _gen(seed, 22)
    slots = torch.randperm(n_pages * p, generator=g, device="cuda")[:T].contiguous()
    slots[torch.rand(T, generator=g, device="cuda") < case["dropped"]] = -1
    state = {"case": case, "k": kv[:, 0], "v": kv[:, 1], "slots": slots, "kc": kc, "vc": vc}
    if own:
        from moe_expert_layer_warp_gb300 import batch
        state["cache"] = batch.PagedCache(kc, vc)
    return state


def _prepare_route(case, seed):
    T, E = case["tokens"], case["experts"]
    g = _gen(seed, 31)
    # logits of a trained gate: a spread of about two, some experts liked more than others
    logits = torch.randn((T, E), generator=g, device="cuda") * 1.5
    logits += torch.randn((1, E), generator=g, device="cuda")
    off = torch.rand((T, E), generator=g, device="cuda") < case["masked"]
    logits = logits.masked_fill(off, -math.inf).to(DTYPES[case["dtype"]])
    bias = None
    if case["bias"]:
        bias = torch.randn(E, generator=g, device="cuda") * 0.1
    state = {"case": case, "logits": logits, "bias": bias}
    if own:
        from moe_expert_layer_warp_gb300 import batch
        state["router"] = batch.GroupedRouter(
            E, case["topk"], max_tokens=T, n_groups=case["groups"], top_groups=case["top_groups"],
            group_top=case["group_top"], score=case["score"], bias=bias, renorm=case["renorm"],
            scale=case["scale"])
    return state


def _prepare_attend(case, seed):
    q_len, kv_len = _attend_lengths(case)
    p, H, D = case["page"], case["kv_heads"], case["dim"]
    blocks = [-(-n // p) for n in kv_len]
    n_pages = max(sum(blocks) + 5, -(-case["pool"] // p))
    kc, vc = _pool(case, n_pages, seed)
    g = _gen(seed, 41)
    pages = torch.randperm(n_pages, generator=g, device="cuda").int()
    M = max(max(blocks), 1) + 1
    table = torch.full((case["requests"], M), -1, dtype=torch.int32, device="cuda")
    rows = torch.arange(M, device="cuda")[None, :] < _i32(blocks)[:, None]
    table[rows] = pages[: sum(blocks)]
    if case["window"]:
        # pages that no new token can see any more have gone to other requests
        block = torch.arange(M, device="cuda")[None, :]
        first = (_i32(kv_len) - _i32(q_len) - (case["window"] - 1))[:, None]
        gone = ((block + 1) * p <= first) & (block * p >= case["sinks"])
        table[gone] = -1
    T = sum(q_len)
    q = torch.empty((T, case["heads"], D), dtype=DTYPES[case["dtype"]], device="cuda")
    q.normal_(generator=g)
    # some heads look almost evenly over the cache, others at a few keys
    q *= torch.linspace(0.5, 3.0, case["heads"], device="cuda")[None, :, None].to(q.dtype)
    start = [0]
    for n in q_len:
        start.append(start[-1] + n)
    state = {"case": case, "q": q, "kc": kc, "vc": vc, "table": table, "q_start": _i32(start),
             "kv_len": _i32(kv_len), "host": (q_len, kv_len), "scale": 1.0 / math.sqrt(D)}
    if own:
        from moe_expert_layer_warp_gb300 import batch
        state["attention"] = batch.PagedAttention(
            batch.PagedCache(kc, vc), case["heads"], max_tokens=T, scale=state["scale"],
            window=case["window"], sinks=case["sinks"])
    return state


def prepare(case, seed):
    return {"plan": _prepare_plan, "append": _prepare_append, "route": _prepare_route,
            "attend": _prepare_attend}[case["op"]](case, seed)


# -------------------------------------------------------------------- run --
def _plain_plan(s):
    p, T, table = s["case"]["page"], s["tokens"], s["table"].clone()
    q, cached, held = s["q_len"].long(), s["cached"].long(), s["held"].long()
    M = table.shape[1]
    total = cached + q
    blocks = (total + p - 1) // p
    fits = blocks <= M
    need = torch.where(fits, (blocks - held).clamp_min(0), 0)
    upto = need.cumsum(0)
    head, end = s["range"][0].long(), s["range"][1].long()
    ok = fits & ((need == 0) | (head + upto <= end))
    given = torch.where(ok, need, 0)
    # the table's new entries
    i = torch.arange(M, device="cuda")[None, :] - held[:, None]
    fresh = (i >= 0) & (i < given[:, None])
    take = (head + (upto - need)[:, None] + i).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][take], table)
    q_start = torch.cat([q.new_zeros(1), q.cumsum(0)])
    # every new token's request, position and slot
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(q_start[1:].contiguous(), t, right=True)
    real = b < q.numel()
    b = b.clamp_max(q.numel() - 1)
    pos = cached[b] + t - q_start[b]
    live = real & ok[b]
    page = table[b, (pos // p).clamp(0, M - 1)].long()
    slots = torch.where(live, page * p + pos % p, -1)
    pos = torch.where(real, pos, -1)
    return {"q_start": q_start.int(), "kv_len": torch.where(ok, total, 0).int(),
            "held": (held + given).int(), "free_head": (head + given.sum()).int().reshape(1),
            "slots": slots, "positions": pos.int(), "table": table}


def _plain_append(s):
    p, live = s["case"]["page"], (s["slots"] >= 0).nonzero().flatten()
    page, off = s["slots"][live] // p, s["slots"][live] % p
    s["kc"][page, off] = s["k"][live].to(s["kc"].dtype)
    s["vc"][page, off] = s["v"][live].to(s["vc"].dtype)
    return {"k": s["kc"], "v": s["vc"]}


def _plain_route(s):
    c = s["case"]
    logits = s["logits"]
    T, E = logits.shape
    k, G = c["topk"], c["groups"]
    size = E // G
    masked = logits <= torch.finfo(logits.dtype).min
    z = logits.double().masked_fill(masked, -math.inf)   # next to a border 32 bits would choose
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + (-z).exp())
    else:
        top = z.amax(1, keepdim=True)
        e = (z - torch.where(top.isinf(), 0.0, top)).exp()
        total = e.sum(1, keepdim=True)
        score = e / torch.where(total == 0, 1.0, total)
    score = score.masked_fill(masked, 0.0)
    choice = score if s["bias"] is None else score + s["bias"].double()
    choice = choice.masked_fill(masked, -math.inf)
    if c["top_groups"] < G:
        best = choice.view(T, G, size).sort(dim=2, descending=True, stable=True).values
        group = best[:, :, : c["group_top"]].sum(2)
        kept = group.sort(dim=1, descending=True, stable=True).indices[:, : c["top_groups"]]
        # experts of kept groups come first, whatever their score, then the others
        rank = torch.zeros((T, G), device="cuda", dtype=torch.bool).scatter_(1, kept, True)
        allowed = rank[:, :, None].expand(T, G, size).reshape(T, E)
        order = choice.sort(dim=1, descending=True, stable=True).indices
        first = allowed.gather(1, order).int().sort(dim=1, descending=True, stable=True).indices
        idx = order.gather(1, first)[:, :k]
    else:
        idx = choice.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, idx)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total == 0, 1.0, total)
    return {"idx": idx.int(), "weights": (w * c["scale"]).float()}


def _visible_keys(length, first_pos, window, sinks):
    """Positions that some new token of the request sees, ascending."""
    lo = max(0, first_pos - window + 1) if window else 0
    j = torch.arange(lo, length, device="cuda")
    if window and sinks and lo > 0:
        j = torch.cat([torch.arange(0, min(sinks, lo), device="cuda"), j])
    return j


def _plain_attend(s):
    c = s["case"]
    p, H, D, W, S = c["page"], c["kv_heads"], c["dim"], c["window"], c["sinks"]
    per = c["heads"] // H
    out = torch.zeros_like(s["q"])
    at = 0
    for b, (n, m) in enumerate(zip(*s["host"])):
        q = s["q"][at:at + n].float()
        at += n
        if n == 0 or m == 0:
            continue
        j = _visible_keys(m, m - n, W, S)
        page = s["table"][b][j // p].long()
        k = s["kc"][page, j % p].float()                      # [keys][H][D]
        v = s["vc"][page, j % p].float()
        pos = torch.arange(m - n, m, device="cuda")[:, None]
        see = j[None, :] <= pos
        if W:
            see &= (pos - j[None, :] < W) | (j[None, :] < S)
        for h in range(H):
            x = q[:, h * per:(h + 1) * per].reshape(n * per, D) * s["scale"]
            a = (x @ k[:, h].t()).view(n, per, -1)
            a = a.masked_fill(~see[:, None, :], -math.inf)
            a = (a - a.amax(2, keepdim=True)).exp()
            y = (a.view(n * per, -1) @ v[:, h]).view(n, per, D) / a.sum(2, keepdim=True)
            out[at - n:at, h * per:(h + 1) * per] = y.to(out.dtype)
    return out


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "append": _plain_append, "route": _plain_route,
                "attend": _plain_attend}[op](state)
    if op == "plan":
        r = state["planner"].plan(state["q_len"], state["cached"], state["held"], state["free"],
                                  state["range"], state["table"], state["tokens"])
        return {"q_start": r.q_start, "kv_len": r.kv_len, "held": r.held,
                "free_head": r.free_head, "slots": r.slots, "positions": r.positions,
                "table": state["table"]}
    if op == "append":
        state["cache"].append(state["k"], state["v"], state["slots"])
        return {"k": state["kc"], "v": state["vc"]}
    if op == "route":
        idx, weights = state["router"].route(state["logits"])
        return {"idx": idx, "weights": weights}
    return state["attention"].attend(state["q"], state["q_start"], state["kv_len"], state["table"])


# ------------------------------------------------------------------- work --
def _seen(q, m, W, S):
    """(pairs of a new token and a key it sees, keys that some new token sees) of one request."""
    if q == 0 or m == 0:
        return 0, 0
    pairs = 0
    for pos in range(m - q, m):
        lo = max(0, pos - W + 1) if W else 0
        pairs += pos - lo + 1 + (min(S, lo) if W else 0)
    lo = max(0, m - q - W + 1) if W else 0
    return pairs, m - lo + (min(S, lo) if W else 0)


def work(case):
    op = case["op"]
    if op == "plan":
        q, cached, held, _ = _plan_lengths(case)
        p, B, T = case["page"], case["requests"], sum(q) + 5
        new = sum(max(0, -(-(c + n) // p) - h) for c, n, h in zip(cached, q, held))
        # lengths in, tables and prefix out; pages read and written; slots and positions
        return {"bytes": B * 12 + (3 * B + 2) * 4 + 8 * new + 4 * B + 12 * T,
                "flops": 2 * T + 4 * B}
    if op == "append":
        n = case["tokens"] * case["kv_heads"] * case["dim"] * 2
        return {"bytes": int(n * (WIDTH[case["src"]] + WIDTH[case["dtype"]]) *
                             (1.0 - case["dropped"])) + 8 * case["tokens"], "flops": n}
    if op == "route":
        T, E = case["tokens"], case["experts"]
        return {"bytes": T * E * WIDTH[case["dtype"]] + T * case["topk"] * 8 + 4 * E,
                "flops": 8 * T * E}
    q, kv = _attend_lengths(case)
    pairs = keys = 0
    for n, m in zip(q, kv):
        a, b = _seen(n, m, case["window"], case["sinks"])
        pairs, keys = pairs + a, keys + b
    width = WIDTH[case["dtype"]]
    return {"bytes": 2 * sum(q) * case["heads"] * case["dim"] * width +
            2 * keys * case["kv_heads"] * case["dim"] * width,
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# ------------------------------------------------------------------ exact --
def _exact_plan(case, s):
    p = case["page"]
    q, cached, held, n_free = _plan_lengths(case)
    free, (head, end) = s["free"].tolist(), s["range"].tolist()
    table = s["table"].cpu().numpy().copy()
    M = table.shape[1]
    slots, pos, kv, out_held, start, cursor, taken = [], [], [], [], [0], head, 0
    for b in range(case["requests"]):
        want = -(-(cached[b] + q[b]) // p)
        need = max(0, want - held[b]) if want <= M else 0
        ok = want <= M and (need == 0 or cursor + need <= end)
        if ok:
            for i in range(need):
                table[b, held[b] + i] = free[cursor + i]
            taken += need
        cursor += need
        for i in range(q[b]):
            at = cached[b] + i
            pos.append(at)
            slots.append(int(table[b, at // p]) * p + at % p if ok else -1)
        kv.append(cached[b] + q[b] if ok else 0)
        out_held.append(held[b] + (need if ok else 0))
        start.append(start[-1] + q[b])
    rest = s["tokens"] - len(slots)
    return {"q_start": np.array(start, np.int32), "kv_len": np.array(kv, np.int32),
            "held": np.array(out_held, np.int32), "free_head": np.array([head + taken], np.int32),
            "slots": np.array(slots + [-1] * rest, np.int64),
            "positions": np.array(pos + [-1] * rest, np.int32), "table": table}


def _exact_append(case, s):
    # a page's rows by their slot number, in 64 bits, then back to the pool's order
    n, p = s["kc"].shape[0], case["page"]
    out = {}
    live = s["slots"] >= 0
    for name, pool, src in (("k", s["kc"], s["k"]), ("v", s["vc"], s["v"])):
        rows = pool.double().reshape(n * p, case["kv_heads"], case["dim"])
        rows.index_copy_(0, s["slots"][live], src.double()[live])
        out[name] = rows.view(n, p, case["kv_heads"], case["dim"])
    return out


def _exact_route(case, s):
    x = s["logits"].double().cpu().numpy()
    low = torch.finfo(s["logits"].dtype).min
    bias = np.zeros(x.shape[1]) if s["bias"] is None else s["bias"].double().cpu().numpy()
    T, E = x.shape
    k, G = case["topk"], case["groups"]
    size = E // G
    off = x <= low
    with np.errstate(over="ignore", invalid="ignore"):
        if case["score"] == "sigmoid":
            score = np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))),
                             np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))
        else:
            y = np.where(off, -np.inf, x)
            m = np.max(y, axis=1, keepdims=True)
            e = np.where(off, 0.0, np.exp(y - np.where(np.isinf(m), 0.0, m)))
            score = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
    score = np.where(off, 0.0, score)
    choice = np.where(off, -np.inf, score + bias)
    keep = np.ones((T, G), bool)
    if case["top_groups"] < G:
        part = -np.sort(-choice.reshape(T, G, size), axis=2)[:, :, :case["group_top"]].sum(2)
        order = np.argsort(-part, axis=1, kind="stable")[:, :case["top_groups"]]
        keep = np.zeros((T, G), bool)
        np.put_along_axis(keep, order, True, 1)
    idx = np.empty((T, k), np.int32)
    allowed = np.repeat(keep, size, axis=1)
    for t in range(T):
        inside = np.nonzero(allowed[t])[0]
        idx[t] = inside[np.argsort(-choice[t, inside], kind="stable")[:k]]
    w = np.take_along_axis(score, idx.astype(np.int64), 1)
    if case["renorm"]:
        total = w.sum(1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1.0), 0.0)
    return {"idx": idx, "weights": w * case["scale"]}


def _exact_attend(case, s):
    p, H, D = case["page"], case["kv_heads"], case["dim"]
    per, W, S = case["heads"] // H, case["window"], case["sinks"]
    q_len, kv_len = _attend_lengths(case)
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["requests"]):
        first, last = int(s["q_start"][b]), int(s["q_start"][b + 1])
        n, m = last - first, kv_len[b]
        if n == 0 or m == 0:
            continue
        # one block of new tokens at a time, over the keys that block sees
        for a in range(0, n, 512):
            z = min(n, a + 512)
            pos = torch.arange(m - n + a, m - n + z, device="cuda")
            end = m - n + z
            keep = torch.arange(end, device="cuda")
            if W:
                keep = keep[(keep > m - n + a - W) | (keep < S)]
            page = s["table"][b].long().gather(0, keep // p)
            dist = pos[:, None] - keep[None, :]
            hidden = dist < 0
            if W:
                hidden |= (dist >= W) & (keep[None, :] >= S)
            for h in range(H):
                k = s["kc"][page, keep % p, h].double()
                v = s["vc"][page, keep % p, h].double()
                x = s["q"][first + a:first + z, h * per:(h + 1) * per].double()
                score = torch.einsum("ngd,md->gnm", x, k) * s["scale"]
                score.masked_fill_(hidden[None], -math.inf)
                score = torch.softmax(score, dim=-1)
                y[first + a:first + z, h * per:(h + 1) * per] = torch.einsum(
                    "gnm,md->ngd", score, v)
    return y


def exact(case, seed):
    global own
    was, own = own, False     # the inputs alone: no handle of this repository's
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"plan": _exact_plan, "append": _exact_append, "route": _exact_route,
            "attend": _exact_attend}[case["op"]](case, s)
