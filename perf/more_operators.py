"""Operators around a paged cache held in 8 bits, as they are measured.

In the order a verification step calls them: rotary positions of the new
tokens' queries and keys, their keys and values into a cache of e4m3 codes
with one scale for each block of tokens and head, attention over that cache,
and reading rows of it back. Each has a plain form here, made of elementary
torch operations.

Sizes: head counts are d / 128 of the layer shapes in configs.py (16, 32 and
56 heads), pass sizes are 1..16 tokens per request as in their workloads; page
sizes, blocks, cache lengths and batch sizes are generic.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
WIDTH = {"f32": 4, "bf16": 2, "f16": 2}
LIMIT = 50        # exponents of scales are in [-50, 50]
CODE = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # queries and keys of four requests' verification passes, whole heads, halves of a head
        # paired: the smallest call, all latency
        {"name": "rotate_step", "op": "rotate", "tokens": 36, "heads": 32, "kv_heads": 8,
         "dim": 128, "rotated": 128, "first": 0, "interleaved": False, "scaling": "none",
         "factor": 1.0, "dtype": "bf16", "far": 16000, "padding": 0},
        # a long prompt's chunk at far positions, frequencies stretched by bands of wavelengths,
        # neighbours of the last half of each head paired, some rows of padding
        {"name": "rotate_chunk", "op": "rotate", "tokens": 12345, "heads": 56, "kv_heads": 8,
         "dim": 128, "rotated": 64, "first": 64, "interleaved": True, "scaling": "bands",
         "factor": 8.0, "dtype": "bf16", "far": 900000, "padding": 57},
        # new keys and values of four requests' passes into blocks that are partly filled
        {"name": "store_step", "op": "store", "requests": 4, "q_lo": 9, "q_hi": 9, "kv_hi": 2000,
         "kv_heads": 8, "dim": 128, "src": "bf16", "page": 64, "block": 16, "heads_first": False,
         "dropped": 0, "len_seed": 1},
        # a serving batch's passes beside prompt chunks, rounded from fp32, one scale for each
        # page, heads before tokens within a page; some requests were refused
        {"name": "store_batch", "op": "store", "requests": 40, "q_lo": 1, "q_hi": 613,
         "kv_hi": 5000, "kv_heads": 8, "dim": 128, "src": "f32", "page": 32, "block": 32,
         "heads_first": True, "dropped": 2, "len_seed": 2},
        # one request's last tokens, to look at or to move
        {"name": "read_step", "op": "read", "tokens": 131, "kv_heads": 8, "dim": 128, "out": "f32",
         "page": 64, "block": 64, "heads_first": False, "missing": 0.0},
        # a shared prefix into 16 bits, a few of whose rows are gone
        {"name": "read_prefix", "op": "read", "tokens": 32001, "kv_heads": 8, "dim": 128,
         "out": "bf16", "page": 128, "block": 16, "heads_first": True, "missing": 0.01},
        # one stream's pass of five tokens over a short cache, every head with its own keys
        {"name": "attend8_step", "op": "attend", "requests": 1, "q_lo": 5, "q_hi": 5, "kv_lo": 777,
         "kv_hi": 777, "chunks": 0, "chunk_hi": 0, "empty": 0, "heads": 16, "kv_heads": 16,
         "dim": 128, "dtype": "bf16", "page": 64, "block": 16, "heads_first": False, "window": 0,
         "sinks": 0, "pool": 0, "len_seed": 3},
        # single tokens of many requests over long ragged caches: bound by reading them
        {"name": "attend8_decode", "op": "attend", "requests": 128, "q_lo": 1, "q_hi": 1,
         "kv_lo": 100, "kv_hi": 24000, "chunks": 0, "chunk_hi": 0, "empty": 2, "heads": 32,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "page": 64, "block": 64,
         "heads_first": False, "window": 0, "sinks": 0, "pool": 0, "len_seed": 8},
        # a serving batch's verification passes, a scale for sixteen tokens
        {"name": "attend8_verify", "op": "attend", "requests": 64, "q_lo": 1, "q_hi": 9,
         "kv_lo": 200, "kv_hi": 16000, "chunks": 0, "chunk_hi": 0, "empty": 0, "heads": 32,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "page": 64, "block": 16,
         "heads_first": False, "window": 0, "sinks": 0, "pool": 0, "len_seed": 4},
        # prompt chunks and verification passes in one call, seven heads per key head, small
        # pages, fp16 queries, one refused request whose rows see nothing
        {"name": "attend8_mixed", "op": "attend", "requests": 24, "q_lo": 1, "q_hi": 16,
         "kv_lo": 20, "kv_hi": 5000, "chunks": 3, "chunk_hi": 700, "empty": 1, "heads": 56,
         "kv_heads": 8, "dim": 64, "dtype": "f16", "page": 16, "block": 16, "heads_first": True,
         "window": 0, "sinks": 0, "pool": 0, "len_seed": 5},
        # long prompts entering in large chunks: bound by the products
        {"name": "attend8_chunk", "op": "attend", "requests": 2, "q_lo": 900, "q_hi": 3001,
         "kv_lo": 4000, "kv_hi": 9000, "chunks": 0, "chunk_hi": 0, "empty": 0, "heads": 32,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "page": 128, "block": 32,
         "heads_first": False, "window": 0, "sinks": 0, "pool": 0, "len_seed": 6},
        # windowed passes over very long caches whose pool of pages spans more than 2^31
        # codes; pages behind the window are given back
        {"name": "attend8_window", "op": "attend", "requests": 48, "q_lo": 1, "q_hi": 9,
         "kv_lo": 3000, "kv_hi": 120000, "chunks": 0, "chunk_hi": 0, "empty": 0, "heads": 56,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "page": 256, "block": 128,
         "heads_first": False, "window": 4096, "sinks": 4, "pool": 2200000, "len_seed": 7},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rotate", "store", "read", "attend", "attend", "attend"])
    page = rng.choice([16, 32, 64, 128, 256])
    block = rng.choice([b for b in (16, 32, 64, 128, 256) if b <= page])
    if op == "rotate":
        dtype = rng.choice(["f32", "bf16", "f16"])
        dim = rng.choice([64, 80, 96, 128, 192])
        rotated = rng.choice([dim, dim, 16 * rng.randint(1, dim // 16)])
        heads, kv_heads = rng.choice([(16, 16), (32, 8), (56, 8), (5, 1), (6, 2), (32, 0)])
        scaling = rng.choice(["none", "linear", "base", "ramp", "bands"])
        tokens = _log(rng, 1, 8000 // (WIDTH[dtype] // 2))
        return {"op": "rotate", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "rotated": rotated, "first": rng.choice([0, dim - rotated]),
                "interleaved": rng.random() < 0.5, "scaling": scaling,
                "factor": 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]),
                "dtype": dtype, "far": _log(rng, 10, 1000000),
                "padding": rng.choice([0, 0, min(3, tokens - 1)])}
    if op == "store":
        requests = _log(rng, 1, 64)
        return {"op": "store", "requests": requests, "q_lo": 1,
                "q_hi": _log(rng, 1, min(2000, 10000 // requests)), "kv_hi": _log(rng, 1, 5000),
                "kv_heads": rng.choice([1, 2, 4, 8, 16]), "dim": rng.choice([64, 128]),
                "src": rng.choice(["f32", "bf16", "f16"]), "page": page, "block": block,
                "heads_first": rng.random() < 0.5, "dropped": rng.choice([0, 0, 1]),
                "len_seed": rng.randrange(1 << 30)}
    if op == "read":
        return {"op": "read", "tokens": _log(rng, 1, 16000), "kv_heads": rng.choice([1, 2, 4, 8]),
                "dim": rng.choice([64, 128]), "out": rng.choice(["f32", "bf16", "f16"]),
                "page": page, "block": block, "heads_first": rng.random() < 0.5,
                "missing": rng.choice([0.0, 0.01, 0.5])}
    while True:
        case = _draw_attend(rng)
        w = work(case)
        if w["bytes"] <= 400e6 and w["flops"] <= 250e9:
            return case


def _draw_attend(rng):
    kv_heads, per = rng.choice([(16, 1), (8, 4), (8, 7), (4, 8), (1, 16), (2, 3), (8, 2), (1, 1)])
    page = rng.choice([16, 32, 64, 128, 256])
    windowed = rng.random() < 0.35
    if rng.random() < 0.35:   # prompts in large chunks
        requests, chunks = rng.randint(1, 3), 0
        q_lo, q_hi = 1, _log(rng, 64, 3001)
        kv_hi = q_hi + _log(rng, 1, 6000)
        kv_lo = rng.randint(1, kv_hi)
        chunk_hi = 0
    else:                     # single tokens or verification passes, some with prompts among them
        requests = _log(rng, 1, 128)
        q_lo, q_hi = 1, rng.choice([1, rng.randint(1, 16)])
        kv_hi = _log(rng, 16, 12000)
        kv_lo = rng.randint(1, kv_hi)
        chunks = rng.randint(1, min(3, requests)) if rng.random() < 0.4 else 0
        chunk_hi = _log(rng, 16, 700) if chunks else 0
    return {"op": "attend", "requests": requests, "q_lo": q_lo, "q_hi": q_hi, "kv_lo": kv_lo,
            "kv_hi": kv_hi, "chunks": chunks, "chunk_hi": chunk_hi,
            "empty": 1 if requests > 2 and rng.random() < 0.3 else 0, "heads": kv_heads * per,
            "kv_heads": kv_heads, "dim": rng.choice([64, 128]), "dtype": rng.choice(["bf16", "f16"]),
            "page": page, "block": rng.choice([b for b in (16, 32, 64, 128, 256) if b <= page]),
            "heads_first": rng.random() < 0.5, "window": _log(rng, 1, 5000) if windowed else 0,
            "sinks": rng.choice([0, 1, 4, 130]) if windowed else 0, "pool": 0,
            "len_seed": rng.randrange(1 << 30)}


# ---------------------------------------------------- lengths from a case --
def _store_lengths(case):
    """New tokens and tokens cached before of every request, and which were refused."""
    rng = random.Random(case["len_seed"])
    B = case["requests"]
    q = [_log(rng, case["q_lo"], case["q_hi"]) for _ in range(B)]
    cached = [rng.randint(0, case["kv_hi"]) for _ in range(B)]
    return q, cached, set(rng.sample(range(B), min(case["dropped"], B - 1)))


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


def _frequencies(case):
    """Angles per position in radians of the rotated pairs."""
    n, base, factor, kind = case["rotated"], 10000.0, case["factor"], case["scaling"]
    original = 4096.0
    if kind == "base":          # a larger base: the slowest pair is stretched by the factor
        base *= factor ** (n / (n - 2.0))
    f = [base ** (-2.0 * i / n) for i in range(n // 2)]
    if kind == "linear":
        return [v / factor for v in f]
    if kind == "bands":         # long wavelengths are stretched, short ones stay
        out = []
        for v in f:
            turns = original * v / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - 1.0) / (4.0 - 1.0)))
            out.append(keep * v + (1.0 - keep) * v / factor)
        return out
    if kind == "ramp":          # the same over the pairs' indices
        def at(turns):
            return n * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(0.0, math.floor(at(32.0))), min(n - 1.0, math.ceil(at(1.0)))
        out = []
        for i, v in enumerate(f):
            gone = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            out.append(v * (1.0 - gone) + v / factor * gone)
        return out
    return f


def _amplitude(case):
    """What long contexts' scaling multiplies rotated queries and keys by."""
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "ramp" else 1.0


# ---------------------------------------------------------------- prepare --
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((seed * 1000003 + salt) & 0x7FFFFFFF)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _exponent(amax):
    """The smallest e with amax <= 448 * 2^e, in [-LIMIT, LIMIT]."""
    part, e = torch.frexp(amax)
    e = e - 9 + (part > 0.875).int()
    return torch.where(amax > 0, e.clamp(-LIMIT, LIMIT), -LIMIT)


def _encode(x, e):
    """Codes of x with scales 2^e: rounded to e4m3, what is beyond its range held at 448."""
    y = torch.ldexp(x.float(), -e)
    return torch.where(y.isfinite(), y.clamp(-448.0, 448.0), math.nan).to(CODE)


def _pool(case, n_pages, seed):
    """A pool of codes [pages][tokens][heads][dim], whatever their order in memory, and its
    scales [pages][heads][blocks], keys then values."""
    p, H, D, c = case["page"], case["kv_heads"], case["dim"], case["block"]
    out = []
    for salt in (11, 12):
        shape = (n_pages, H, p, D) if case["heads_first"] else (n_pages, p, H, D)
        codes = torch.empty(shape, dtype=CODE, device="cuda")
        if case["heads_first"]:
            codes = codes.transpose(1, 2)
        scales = torch.empty((n_pages, H, p // c), dtype=torch.float32, device="cuda")
        g = _gen(seed, salt)
        # keys have a few columns much larger than the others
        column = torch.ones(D, device="cuda")
        if salt == 11:
            column[torch.randperm(D, generator=g, device="cuda")[:3]] = 4.0
        step = max(1, (1 << 26) // (p * H * D))
        for a in range(0, n_pages, step):
            n = min(step, n_pages - a)
            x = torch.randn((n, p // c, c, H, D), generator=g, device="cuda") * column
            # tokens differ in size
            x *= torch.exp2(torch.randn((n, p // c, c, H, 1), generator=g, device="cuda") * 0.7)
            e = _exponent(x.abs().amax(dim=(2, 4)))                    # [n][blocks][H]
            codes[a:a + n] = _encode(x, e[:, :, None, :, None]).view(n, p, H, D)
            scales[a:a + n] = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e).transpose(1, 2)
        out += [codes, scales]
    return out


def _bytes(codes):
    return codes.view(torch.uint8)    # rows are taken and put as bytes


def _cache(state):
    from moe_expert_layer_warp_gb300 import batch
    return batch.PagedCache8(state["kc"], state["vc"], state["ks"], state["vs"])


def _prepare_rotate(case, seed):
    T, H, K, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    # queries, keys and values as a joint projection leaves them
    x = torch.empty((T, H + 2 * K, D), dtype=DTYPES[case["dtype"]], device="cuda")
    x.normal_(generator=_gen(seed, 1))
    # verification passes and chunks: runs of consecutive positions
    rng = random.Random(seed)
    pos = []
    while len(pos) < T - case["padding"]:
        first = rng.randint(0, case["far"])
        pos += range(first, first + min(_log(rng, 1, 4000), T - case["padding"] - len(pos)))
    pos += [-1] * (T - len(pos))
    state = {"case": case, "q": x[:, :H], "k": x[:, H:H + K] if K else None, "pos": _i32(pos),
             "q_out": torch.empty((T, H, D), dtype=x.dtype, device="cuda"),
             "k_out": torch.empty((T, K, D), dtype=x.dtype, device="cuda") if K else None}
    if own:
        from moe_expert_layer_warp_gb300 import batch
        state["rotary"] = batch.Rotary(D, case["rotated"], frequencies=_frequencies(case),
                                       first=case["first"], interleaved=case["interleaved"],
                                       amplitude=_amplitude(case))
    return state


def _prepare_store(case, seed):
    q, cached, dropped = _store_lengths(case)
    p, H, D, c = case["page"], case["kv_heads"], case["dim"], case["block"]
    blocks = [-(-(a + n) // p) for a, n in zip(cached, q)]
    kc, ks, vc, vs = _pool(case, sum(blocks) + 3, seed)
    g = _gen(seed, 22)
    pages = torch.randperm(sum(blocks) + 3, generator=g, device="cuda").tolist()
    slots, rows, at = [], [], 0
    for b, (n, m) in enumerate(zip(q, cached)):
        mine = pages[at:at + blocks[b]]
        at += blocks[b]
        if b in dropped:
            slots += [-1] * n
            continue
        slots += [mine[i // p] * p + i % p for i in range(m, m + n)]
        # the tokens that share a block with new ones, and the new ones
        rows += [mine[i // p] * p + i % p for i in range(m // c * c, m + n)]
    T = len(slots)
    x = torch.empty((T, 2, H, D), device="cuda").normal_(generator=_gen(seed, 21))
    # some tokens are larger than what their block holds
    x *= torch.exp2(torch.randn((T, 2, H, 1), generator=g, device="cuda") * 1.5)
    x = x.to(DTYPES[case["src"]])
    state = {"case": case, "k": x[:, 0], "v": x[:, 1], "kc": kc, "ks": ks, "vc": vc, "vs": vs,
             "slots": torch.tensor(slots, dtype=torch.int64, device="cuda"),
             "rows": torch.tensor(rows, dtype=torch.int64, device="cuda")}
    if own:
        state["cache"] = _cache(state)
    return state


def _prepare_read(case, seed):
    T, p = case["tokens"], case["page"]
    n_pages = -(-T // p) + 5
    kc, ks, vc, vs = _pool(case, n_pages, seed)
    g = _gen(seed, 31)
    pages = torch.randperm(n_pages, generator=g, device="cuda")
    i = torch.arange(T, device="cuda")
    slots = pages[i // p] * p + i % p
    slots[torch.rand(T, generator=g, device="cuda") < case["missing"]] = -1
    state = {"case": case, "kc": kc, "ks": ks, "vc": vc, "vs": vs, "slots": slots}
    if own:
        state["cache"] = _cache(state)
    return state


def _prepare_attend(case, seed):
    q_len, kv_len = _attend_lengths(case)
    p, D = case["page"], case["dim"]
    blocks = [-(-n // p) for n in kv_len]
    n_pages = max(sum(blocks) + 5, -(-case["pool"] // p))
    kc, ks, vc, vs = _pool(case, n_pages, seed)
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
    q *= torch.linspace(0.25, 1.5, case["heads"], device="cuda")[None, :, None].to(q.dtype)
    start = [0]
    for n in q_len:
        start.append(start[-1] + n)
    state = {"case": case, "q": q, "kc": kc, "ks": ks, "vc": vc, "vs": vs, "table": table,
             "q_start": _i32(start), "kv_len": _i32(kv_len), "host": (q_len, kv_len),
             "scale": 1.0 / math.sqrt(D)}
    if own:
        from moe_expert_layer_warp_gb300 import batch
        state["attention"] = batch.PagedAttention8(
            _cache(state), case["heads"], max_tokens=T, dtype=q.dtype, scale=state["scale"],
            window=case["window"], sinks=case["sinks"])
    return state


def prepare(case, seed):
    return {"rotate": _prepare_rotate, "store": _prepare_store, "read": _prepare_read,
            "attend": _prepare_attend}[case["op"]](case, seed)


# -------------------------------------------------------------------- run --
def _plain_rotate(s):
    c = s["case"]
    r, a = c["rotated"], c["first"]
    # far positions' angles lose their meaning in 32 bits
    f = torch.tensor(_frequencies(c), dtype=torch.float64, device="cuda")
    angle = s["pos"].clamp_min(0).double()[:, None] * f
    cos = (angle.cos() * _amplitude(c)).float()[:, None]
    sin = (angle.sin() * _amplitude(c)).float()[:, None]
    idle = (s["pos"] < 0)[:, None, None]
    out = {}
    for name in ("q", "k"):
        if s[name] is None:
            continue
        y = s[name].clone()
        x = s[name][:, :, a:a + r].float()
        if c["interleaved"]:
            u, v = x[..., 0::2], x[..., 1::2]
            z = torch.stack((u * cos - v * sin, u * sin + v * cos), dim=-1).flatten(2)
        else:
            u, v = x[..., : r // 2], x[..., r // 2:]
            z = torch.cat((u * cos - v * sin, u * sin + v * cos), dim=-1)
        y[:, :, a:a + r] = torch.where(idle, x, z).to(y.dtype)
        out[name] = y
    return out


def _plain_values(codes, scales, slots, page, block, dtype):
    """Rows of a pool as the values they stand for; zeros for slot -1."""
    at = slots.clamp_min(0)
    x = _bytes(codes)[at // page, at % page].view(CODE).float()       # [n][H][D]
    x = x * scales[at // page, :, at % page // block][:, :, None]
    return torch.where((slots < 0)[:, None, None], 0.0, x).to(dtype)


def _plain_store(s):
    c = s["case"]
    p, w, H, D = c["page"], c["block"], c["kv_heads"], c["dim"]
    live = (s["slots"] >= 0).nonzero().flatten()
    slots = s["slots"][live]
    ids, inverse = torch.unique(slots // w, return_inverse=True)       # the blocks written
    page, at = ids * w // p, ids * w % p // w
    anew = torch.zeros(ids.numel(), dtype=torch.bool, device="cuda")
    anew[inverse[slots % w == 0]] = True
    for x, codes, scales in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        x = x[live].float()                                            # [n][H][D]
        size = x.abs().masked_fill(~x.isfinite(), 0.0).amax(2)
        amax = torch.zeros((ids.numel(), H), device="cuda")
        amax.scatter_reduce_(0, inverse[:, None].expand(-1, H), size, "amax")
        was = torch.frexp(scales[page, :, at])[1] - 1                  # exponents of powers of two
        e = torch.maximum(_exponent(amax), torch.where(anew[:, None], -LIMIT, was))
        # what the block holds is rounded again where its scale grows
        rows = torch.arange(w, device="cuda")[None, :] + (at * w)[:, None]
        old = _bytes(codes)[page[:, None], rows].view(CODE).float()    # [blocks][w][H][D]
        shift = torch.where(anew[:, None], 0, e - was)[:, None, :, None]
        _bytes(codes)[page[:, None], rows] = _bytes(_encode(old, shift))
        scales[page, :, at] = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
        _bytes(codes)[slots // p, slots % p] = _bytes(_encode(x, e[inverse][:, :, None]))
    dtype = DTYPES[c["src"]]
    return {"k": _plain_values(s["kc"], s["ks"], s["rows"], p, w, dtype),
            "v": _plain_values(s["vc"], s["vs"], s["rows"], p, w, dtype)}


def _plain_read(s):
    c, dtype = s["case"], DTYPES[s["case"]["out"]]
    return {"k": _plain_values(s["kc"], s["ks"], s["slots"], c["page"], c["block"], dtype),
            "v": _plain_values(s["vc"], s["vs"], s["slots"], c["page"], c["block"], dtype)}


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
        slots = s["table"][b][j // p].long() * p + j % p
        k = _plain_values(s["kc"], s["ks"], slots, p, c["block"], torch.float32)
        v = _plain_values(s["vc"], s["vs"], slots, p, c["block"], torch.float32)
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
    c = state["case"]
    op = c["op"]
    if not own:
        return {"rotate": _plain_rotate, "store": _plain_store, "read": _plain_read,
                "attend": _plain_attend}[op](state)
    if op == "rotate":
        q, k = state["rotary"].rotate(state["q"], state["k"], state["pos"],
                                      q_out=state["q_out"], k_out=state["k_out"])
        return {"q": q} if k is None else {"q": q, "k": k}
    if op == "store":
        state["cache"].append(state["k"], state["v"], state["slots"])
        k, v = state["cache"].read(state["rows"], dtype=DTYPES[c["src"]])
        return {"k": k, "v": v}
    if op == "read":
        k, v = state["cache"].read(state["slots"], dtype=DTYPES[c["out"]])
        return {"k": k, "v": v}
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
    op, D = case["op"], case["dim"]
    if op == "rotate":
        T, H = case["tokens"], case["heads"] + case["kv_heads"]
        return {"bytes": 2 * T * H * D * WIDTH[case["dtype"]] + 4 * T,
                "flops": 3 * T * H * case["rotated"]}
    if op == "store":
        q, cached, dropped = _store_lengths(case)
        row = 2 * case["kv_heads"] * D
        n = m = 0
        for b, (new, old) in enumerate(zip(q, cached)):
            if b not in dropped:
                n += new
                m += new + old % case["block"]
        # sources in, codes out; codes in and values out
        return {"bytes": n * row * (WIDTH[case["src"]] + 1) + m * row * (1 + WIDTH[case["src"]]) +
                8 * (n + m), "flops": 2 * (n + m) * row}
    if op == "read":
        n = case["tokens"] * 2 * case["kv_heads"] * D
        return {"bytes": int(n * (1.0 - case["missing"])) + n * WIDTH[case["out"]] +
                8 * case["tokens"], "flops": n}
    q, kv = _attend_lengths(case)
    pairs = keys = 0
    for n, m in zip(q, kv):
        a, b = _seen(n, m, case["window"], case["sinks"])
        pairs, keys = pairs + a, keys + b
    return {"bytes": 2 * sum(q) * case["heads"] * D * WIDTH[case["dtype"]] +
            2 * keys * case["kv_heads"] * D + 8 * keys * case["kv_heads"] // case["block"],
            "flops": 4 * pairs * case["heads"] * D}


# ------------------------------------------------------------------ exact --
def _exact_rotate(case, s):
    # a pair as a complex number, turned by e^(i·angle)
    f = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
    pos = s["pos"].double()
    turn = torch.polar(torch.full((pos.numel(), f.numel()), _amplitude(case), device="cuda",
                                  dtype=torch.float64), torch.outer(pos, f))
    turn[s["pos"] < 0] = 1.0
    a, b = case["first"], case["first"] + case["rotated"]
    out = {}
    for name in ("q", "k"):
        if s[name] is None:
            continue
        y = s[name].double()
        T, H, _ = y.shape
        if case["interleaved"]:
            z = torch.view_as_complex(y[:, :, a:b].reshape(T, H, -1, 2).contiguous())
            y[:, :, a:b] = torch.view_as_real(z * turn[:, None]).reshape(T, H, -1)
        else:
            z = torch.complex(y[:, :, a:(a + b) // 2], y[:, :, (a + b) // 2:b]) * turn[:, None]
            y[:, :, a:b] = torch.cat((z.real, z.imag), dim=2)
        out[name] = y
    return out


def _exact_e4m3(y):
    """y rounded to 4 significant bits, or to multiples of 2^-9, ties to even; at most 448."""
    e = torch.frexp(y)[1].double()
    step = torch.exp2((e - 4).clamp_min(-9))
    return torch.where(y.abs() <= 448, torch.round(y / step) * step, torch.sign(y) * 448)


def _exact_rows(codes, scales, case):
    """A whole pool's values as [slots][H][D]."""
    n, p, H, D = codes.shape
    x = codes.double().view(n, p // case["block"], case["block"], H, D) if \
        codes.is_contiguous() else codes.double().reshape(n, p // case["block"], case["block"], H, D)
    return (x * scales.double().permute(0, 2, 1)[:, :, None, :, None]).reshape(n * p, H, D)


def _exact_store(case, s):
    w, out = case["block"], {}
    slots = s["slots"].tolist()
    # runs of tokens in one block, in the order of the call
    runs, i = [], 0
    while i < len(slots):
        j = i + 1
        while j < len(slots) and slots[j] >= 0 and slots[j] // w == slots[i] // w:
            j += 1
        if slots[i] >= 0:
            runs.append((i, j))
        i = j
    at = torch.tensor([a for a, _ in runs], device="cuda")
    long = max(b - a for a, b in runs)
    token = at[:, None] + torch.arange(long, device="cuda")
    valid = token < torch.tensor([b for _, b in runs], device="cuda")[:, None]
    token = torch.where(valid, token, at[:, None])
    block = s["slots"][at] // w                                        # [runs]
    anew = ((s["slots"][token] % w == 0) & valid).any(1)
    for name, x, codes, scales in (("k", s["k"], s["kc"], s["ks"]), ("v", s["v"], s["vc"], s["vs"])):
        H = case["kv_heads"]
        unit = scales.double().permute(0, 2, 1).reshape(-1, H)         # [blocks][H]
        pool = codes.double().reshape(unit.shape[0], w, H, case["dim"])
        new = x.double()[token]                                        # [runs][long][H][D]
        amax = (new.abs() * valid[:, :, None, None]).amax(dim=(1, 3))
        e = torch.ceil(torch.log2(amax.clamp_min(1e-300) / 448.0))
        e += (amax > 448.0 * torch.exp2(e)).double()
        e -= (amax <= 448.0 * torch.exp2(e - 1)).double()
        unit_new = torch.exp2(e.clamp(-50, 50))
        unit_new = torch.where(anew[:, None], unit_new, torch.maximum(unit_new, unit[block]))
        ratio = torch.where(anew[:, None], 1.0, unit[block] / unit_new)
        pool[block] = _exact_e4m3(pool[block] * ratio[:, None, :, None])
        unit[block] = unit_new
        run = torch.arange(len(runs), device="cuda")[:, None].expand(-1, long)[valid]
        pool[block[run], s["slots"][token[valid]] % w] = _exact_e4m3(
            x.double()[token[valid]] / unit_new[run][:, :, None])
        value = pool * unit[:, None, :, None]
        out[name] = value.reshape(-1, H, case["dim"])[s["rows"]]
    return out


def _exact_read(case, s):
    out = {}
    for name, codes, scales in (("k", s["kc"], s["ks"]), ("v", s["vc"], s["vs"])):
        rows = _exact_rows(codes, scales, case)
        rows = torch.cat((rows, torch.zeros_like(rows[:1])))           # slot -1: the last one
        out[name] = rows[s["slots"]]
    return out


def _exact_attend(case, s):
    p, H, D, c = case["page"], case["kv_heads"], case["dim"], case["block"]
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
                part = keep % p // c
                k = s["kc"].view(torch.uint8)[page, keep % p, h].view(CODE).double()
                v = s["vc"].view(torch.uint8)[page, keep % p, h].view(CODE).double()
                k = k * s["ks"][page, h, part].double()[:, None]
                v = v * s["vs"][page, h, part].double()[:, None]
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
    return {"rotate": _exact_rotate, "store": _exact_store, "read": _exact_read,
            "attend": _exact_attend}[case["op"]](case, s)
