"""The operators of include/moe_kv8.h from their definitions, in 64 bits, with
the error bounds their tests use. Shares no code with the package."""
from __future__ import annotations

import math

import torch

CODE = torch.float8_e4m3fn
LIMIT = 50


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ rotary --
def rotate(x, positions, radians, first, interleaved, amplitude):
    """(out, bound) of rows x [T][H][D], float64.

    bound: the angle is off by at most 2^-28 turns (a quarter turn's rest in
    fp32, and its conversion), sine and cosine by another 2^-23 of themselves with
    the amplitude's product; products and their sum are rounded in fp32, the
    result to the type of x."""
    T, H, D = x.shape
    r = 2 * len(radians)
    f = torch.tensor(radians, dtype=torch.float64, device=x.device)
    p = positions.to(x.device).double()
    angle = p[:, None] * f
    c, s = (angle.cos() * amplitude)[:, None], (angle.sin() * amplitude)[:, None]
    y = x.double().clone()
    bound = torch.zeros_like(y)
    cols = torch.arange(r // 2, device=x.device)
    a = first + (2 * cols if interleaved else cols)
    b = a + 1 if interleaved else a + r // 2
    u, v = x[:, :, a].double(), x[:, :, b].double()
    live = (positions.to(x.device) >= 0)[:, None, None]
    size = (u.abs() + v.abs()) * abs(amplitude)
    # 64-bit angles of far positions are off themselves: p · 2^-53 of a radian
    da = 2 * math.pi * 2.0 ** -28 + (p.abs()[:, None] * f.abs() * 2.0 ** -52)[:, None]
    off = size * (da + 2.0 ** -23 + 2.0 ** -23)
    y[:, :, a] = torch.where(live, u * c - v * s, u)
    y[:, :, b] = torch.where(live, u * s + v * c, v)
    tiny = torch.finfo(x.dtype).smallest_normal * torch.finfo(x.dtype).eps
    for at in (a, b):
        bound[:, :, at] = torch.where(live, off + half_step(x.dtype) * (y[:, :, at].abs() + off) +
                                      tiny, torch.zeros_like(off))
    return y, bound


# ------------------------------------------------------------------- codes --
def e4m3(y):
    """float64 rounded to e4m3, ties to even, held at 448; NaN of what is not finite."""
    e = torch.frexp(y)[1].double()
    step = torch.exp2((e - 4).clamp_min(-9.0))
    z = torch.round(y / step) * step
    z = torch.where(z.abs() > 448, torch.sign(y) * 448.0, z)
    return torch.where(torch.isfinite(y), z, math.nan)


def exponent(a):
    """The smallest e in [-50, 50] with a <= 448 · 2^e (50 if none)."""
    if a == 0:
        return -LIMIT
    e = -LIMIT
    while e < LIMIT and a > 448.0 * 2.0 ** e:
        e += 1
    return e


class Pool:
    """A pool of codes' values [pages][rows][heads][dim] in float64 and scales'
    exponents [pages][heads][blocks]; NaN where a row holds nothing yet."""

    def __init__(self, pages, page, heads, dim, block):
        self.page, self.block = page, block
        self.code = torch.full((pages, page, heads, dim), math.nan, dtype=torch.float64)
        self.exp = torch.zeros((pages, heads, page // block), dtype=torch.int64)

    @classmethod
    def of(cls, codes, scales, block):
        p = cls(codes.shape[0], codes.shape[1], codes.shape[2], codes.shape[3], block)
        p.code = codes.cpu().float().double()
        p.exp = torch.frexp(scales.cpu())[1].long() - 1
        return p

    def append(self, x, slots):
        """x [T][heads][dim], slots a list: token after token's definition, a block
        at a time."""
        x = x.cpu().double()
        blocks = {}
        for t, s in enumerate(slots):
            if s >= 0:
                blocks.setdefault(s // self.block, []).append(t)
        for b, tokens in blocks.items():
            page, at = b * self.block // self.page, b * self.block % self.page // self.block
            rows = [slots[t] % self.page for t in tokens]
            anew = any(r % self.block == 0 for r in rows)
            for h in range(x.shape[1]):
                new = x[tokens, h]
                size = new[torch.isfinite(new)].abs()
                e = exponent(float(size.max()) if size.numel() else 0.0)
                was = int(self.exp[page, h, at])
                if not anew:
                    e = max(e, was)
                    first = at * self.block
                    old = self.code[page, first:first + self.block, h]
                    old = e4m3(old * 2.0 ** (was - e)) if e > was else old
                    self.code[page, first:first + self.block, h] = old
                self.exp[page, h, at] = e
                self.code[page, rows, h] = e4m3(new * 2.0 ** -e)

    def values(self, slots):
        """[n][heads][dim] for slots, zeros for -1."""
        out = torch.zeros((len(slots), *self.code.shape[2:]), dtype=torch.float64)
        for i, s in enumerate(slots):
            if s >= 0:
                page, row = s // self.page, s % self.page
                e = self.exp[page, :, row // self.block].double()
                out[i] = self.code[page, row] * torch.exp2(e)[:, None]
        return out

    def all_values(self):
        e = self.exp.double().permute(0, 2, 1).repeat_interleave(self.block, dim=1)
        return self.code * torch.exp2(e)[..., None]


# --------------------------------------------------------------- attention --
def attend(q, k, v, vs, q_start, kv_len, table, scale, window, sinks):
    """(out, bound) for q [T][Hq][D] and pools of values k, v (float64)
    [pages][rows][heads][D] with vs [pages][rows][heads] the scale of each row's
    values, both float64 [T][Hq][D], on q's device.

    bound: a kernel may hold a query, and its weights, as sums of two (bf16) or three
    (fp16) e4m3 numbers, each 16 times what the ones before it left, rounded. A
    number above 2^-6 is off by at most 2^-4 of itself, one below by 2^-10.
    Queries are scaled so that their row's largest is above 224: 8 (11) bits are
    exact, but for what is below 2^-10 · 16^-1 (16^-2), 2^-21.8 (2^-25.8) of the largest.
    Weights are scaled so that the largest w · vs is 2^4 or more, and rounded to
    fp16 before (2^-11 of themselves): off by 2^-8 + 2^-11 (2^-11 + 2^-12) of themselves
    and, where they are below 2^-6, by 2^-10 · 16^-1 = 2^-14 (2^-10 · 16^-2 = 2^-18), which is
    2^-14 · 2^-4 (2^-18 · 2^-4) of the largest.
    The result is rounded to the type of q. Sums are fp32 (a score is off by at most
    (D + 8)·2^-22·scale·Σ|q k|: the tensor cores add e4m3 products with 2^-22 of
    the sum of their sizes, which was measured; that moves a weight by as much,
    twice; statistics and exponentials 2^-20; sums over keys 2^-20)."""
    T, Hq, D = q.shape
    page, H = k.shape[1], k.shape[2]
    per = Hq // H
    f16 = q.dtype == torch.float16
    eps, w_rel, w_abs, q_abs = half_step(q.dtype), 2.0 ** -8 + 2.0 ** -11, 2.0 ** -18, 2.0 ** -21.8
    if f16:
        w_rel, w_abs, q_abs = 2.0 ** -11 + 2.0 ** -12, 2.0 ** -22, 2.0 ** -25.8
    tiny = 2.0 ** -25 if f16 else 2.0 ** -134
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
            kk, vv, unit = k[pages, j % page], v[pages, j % page], vs[pages, j % page]
            for h in range(H):
                x = q[rows, h * per:(h + 1) * per].double()                      # [rows][per][D]
                s = torch.einsum("rgd,md->rgm", x, kk[:, h]) * scale
                s = s.masked_fill(~see[:, None, :], -math.inf)
                top = s.amax(2, keepdim=True)
                w = torch.where(see[:, None, :], (s - top.clamp_min(-1e300)).exp(), 0.0)
                total = w.sum(2, keepdim=True)
                w = w / torch.where(total > 0, total, 1.0)
                mag = torch.einsum("rgd,md->rgm", x.abs(), kk[:, h].abs()) * scale
                lost = x.abs().amax(2, keepdim=True) * q_abs * kk[:, h].abs().sum(1) * scale
                ds = torch.where(see[:, None, :], mag * (D + 8) * 2.0 ** -22 + lost, 0.0)
                ds = ds.amax(2, keepdim=True)
                y = torch.einsum("rgm,md->rgd", w, vv[:, h])
                a = torch.einsum("rgm,md->rgd", w, vv[:, h].abs())
                # what weights far below the largest one lose
                code = vv[:, h].abs() / unit[:, h, None]
                most = (w * unit[:, h]).amax(2, keepdim=True)
                far = most * (see.double() @ code)[:, None, :]
                cut = slice(h * per, (h + 1) * per)
                out[rows, cut] = y
                bound[rows, cut] = (eps * y.abs() + (w_rel + 2 * ds + 2.0 ** -19) * a +
                                    w_abs * far) * 1.02 + tiny
    return out, bound
