"""The operators of include/moe_batch.h from their definitions, in 64 bits, with
the error bounds their tests use. Shares no code with the
package."""
from __future__ import annotations

import math

import numpy as np
import torch


def plan(q_len, cached, held, free, head, end, table, page, n_tokens):
    """(q_start, kv_len, held, free_head, slots, positions, table) as lists and an array."""
    table = np.array(table, np.int64)
    M = table.shape[1]
    cursor = taken = 0
    q_start, kv, new_held, slots, pos = [0], [], [], [], []
    for b, (q, c, h) in enumerate(zip(q_len, cached, held)):
        blocks = -(-(c + q) // page)
        fits = blocks <= M
        need = max(0, blocks - h) if fits else 0
        ok = fits and (need == 0 or head + cursor + need <= end)
        for i in range(need if ok else 0):
            table[b, h + i] = free[head + cursor + i]
        cursor += need
        taken += need if ok else 0
        for i in range(q):
            pos.append(c + i)
            slots.append(int(table[b, (c + i) // page]) * page + (c + i) % page if ok else -1)
        kv.append(c + q if ok else 0)
        new_held.append(h + (need if ok else 0))
        q_start.append(q_start[-1] + q)
    pad = n_tokens - len(slots)
    return (q_start, kv, new_held, [head + taken], slots + [-1] * pad, pos + [-1] * pad, table)


def attend(q, k, v, q_start, kv_len, table, scale, window, sinks):
    """(out, bound) for q [T][Hq][D] and page pools k, v [pages][rows][heads][D],
    both float64 [T][Hq][D], on q's device.

    bound: what a kernel may be off by that rounds its softmax weights and its
    result to the type of q (half a step each, of Σ p|v| and of |out|), sums
    in fp32 (a score is off by at most (D + 8)·2^-24·scale·Σ|q k|, which moves
    p by twice that, relatively; statistics and exponentials 2^-20), and, in
    fp16, loses what of a weight falls below half the least step, 2^-25."""
    T, Hq, D = q.shape
    page, H = k.shape[1], k.shape[2]
    per = Hq // H
    eps = torch.finfo(q.dtype).eps / 2
    tiny = 2.0 ** -25 if q.dtype == torch.float16 else 0.0
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=q.device)
    bound = torch.zeros((T, Hq, D), dtype=torch.float64, device=q.device)
    for b in range(len(kv_len)):
        first, n = q_start[b], q_start[b + 1] - q_start[b]
        for t0 in range(0, n, 256):                       # a block of tokens at a time
            pos = torch.arange(t0, min(n, t0 + 256), device=q.device) + kv_len[b] - n
            j = torch.arange(max(0, int(pos[-1]) + 1), device=q.device)
            back = pos[:, None] - j[None, :]
            see = back >= 0
            if window:
                see &= (back < window) | (j[None, :] < sinks)
            j, see = j[see.any(0)], see[:, see.any(0)]
            if not j.numel():
                continue
            rows = slice(first + t0, first + t0 + pos.numel())
            pages = table[b].long()[j // page]
            kk, vv = k[pages, j % page].double(), v[pages, j % page].double()   # [keys][H][D]
            for h in range(H):
                x = q[rows, h * per:(h + 1) * per].double()                      # [rows][per][D]
                s = torch.einsum("rgd,md->rgm", x, kk[:, h]) * scale
                s = s.masked_fill(~see[:, None, :], -math.inf)
                top = s.amax(2, keepdim=True)
                w = torch.where(see[:, None, :], (s - top.clamp_min(-1e300)).exp(), 0.0)
                total = w.sum(2, keepdim=True)
                w = w / torch.where(total > 0, total, 1.0)
                mag = torch.einsum("rgd,md->rgm", x.abs(), kk[:, h].abs()) * scale
                mag = torch.where(see[:, None, :], mag, 0.0)
                ds = (D + 8) * 2.0 ** -24 * mag.amax(2, keepdim=True)
                y = torch.einsum("rgm,md->rgd", w, vv[:, h])
                a = torch.einsum("rgm,md->rgd", w, vv[:, h].abs())
                lost = tiny * (see.double() @ vv[:, h].abs())[:, None, :]
                cut = slice(h * per, (h + 1) * per)
                out[rows, cut] = y
                bound[rows, cut] = (eps * y.abs() + (eps + 2 * ds + 2.0 ** -20) * a +
                                    lost) * 1.01 + tiny
    return out, bound


def route(logits, bias, topk, groups, top_groups, group_top, score, renorm, scale):
    """(idx, weights, bound): numpy, float64. bound: exp and the divisions a few
    steps each, l - max rounded once (|l - max| steps through the exponential),
    sums over lanes and over the k weights: (64 + max|l - max|)·2^-24 of the
    weight."""
    low = torch.finfo(logits.dtype).min
    x = logits.double().numpy()
    n, E = x.shape
    b = np.zeros(E) if bias is None else bias.double().numpy()
    off = x <= low
    idx = np.zeros((n, topk), np.int64)
    wts = np.zeros((n, topk))
    bound = np.zeros((n, topk))
    for t in range(n):
        if score == "sigmoid":
            s = [0.0 if off[t, e] else 1.0 / (1.0 + math.exp(-x[t, e])) if x[t, e] > -700 else 0.0
                 for e in range(E)]
            spread = 0.0
        else:
            live = x[t][~off[t]]
            m = live.max() if live.size else 0.0
            ex = [0.0 if off[t, e] else math.exp(x[t, e] - m) for e in range(E)]
            s = [v / math.fsum(ex) if live.size else 0.0 for v in ex]
            spread = float(np.ptp(live)) if live.size else 0.0
        c = [-math.inf if off[t, e] else s[e] + b[e] for e in range(E)]
        size = E // groups
        # (so for groups of one choice each)
        value = c if bias is not None or group_top == 2 else np.where(off[t], -np.inf, x[t]).tolist()
        best = [sum(sorted(value[g * size:(g + 1) * size], reverse=True)[:group_top])
                for g in range(groups)]
        kept = sorted(range(groups), key=lambda g: (-best[g], g))[:top_groups]
        pool = [e for g in kept for e in range(g * size, (g + 1) * size)]
        # without a bias the order of the choices is that of the logits, which
        # no exponential's underflow can hide
        order = (lambda e: (-c[e], e)) if bias is not None else (
            lambda e: (off[t, e], -x[t, e] if not off[t, e] else 0.0, e))
        chosen = sorted(pool, key=order)[:topk]
        w = np.array([s[e] for e in chosen])
        if renorm:
            w = w / w.sum() if w.sum() > 0 else 0 * w
        idx[t], wts[t] = chosen, w * scale
        bound[t] = np.abs(w * scale) * (64 + spread) * 2.0 ** -24 + 1e-37
    return idx, wts, bound
