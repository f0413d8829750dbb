"""A verification step of several requests, through the C ABI of
include/moe_batch.h.

``BatchPlanner`` turns request lengths into block tables, slots and
positions; ``PagedCache`` holds pages of keys and values and takes new ones;
``PagedAttention`` lets every new token attend over its request's pages;
``GroupedRouter`` picks experts from router logits. A decoder block calls
them in that order, then an expert engine (``layer.PassRunner``):

    plan = planner.plan(q_len, cached, held, free_pages, free_range, table, n)
    cache.append(k, v, plan.slots)
    y = attention.attend(q, plan.q_start, plan.kv_len, table)
    idx, w = router.route(logits)

Each object allocates its buffers once, through torch, at construction; a
call only checks and marshals its arguments, returns views of those buffers
(overwritten by the object's next call) and is asynchronous on ``stream``
(None: torch's current stream). Values that only the device sees are checked
there, see ``api.moe_last_device_error``. There are no gradients.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional

import torch

from . import api


def _need(t, name, dtype, shape, device):
    """The device pointer of `t`, a contiguous tensor of the given kind."""
    if (t.dtype != dtype or t.device != device or not t.is_contiguous() or
            tuple(t.shape) != tuple(shape)):
        raise ValueError("%s must be a contiguous %s %s tensor on %s, got %s %s on %s"
                         % (name, str(dtype)[6:], list(shape), device, str(t.dtype)[6:],
                            list(t.shape), t.device))
    return t.data_ptr()


def _cuda(device) -> torch.device:
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError("a CUDA device is needed, got %s" % device)
    return torch.device("cuda", torch.cuda.current_device() if device.index is None
                        else device.index)


class BatchPlan(NamedTuple):
    q_start: torch.Tensor    # [B+1] int32: first packed row of each request, then the total
    kv_len: torch.Tensor     # [B] int32: visible cache length, the new tokens included; 0: refused
    held: torch.Tensor       # [B] int32: pages held now
    free_head: torch.Tensor  # [1] int32: the free list's new head
    slots: torch.Tensor      # [n_tokens] int64: cache slot of each new token, -1: none
    positions: torch.Tensor  # [n_tokens] int32: position in its request, -1: padding


class BatchPlanner:
    """Block tables, slots and positions of a step's new tokens
    (moe_plan_batch) for up to max_requests requests and max_tokens tokens."""

    def __init__(self, page_size: int, max_requests: int, max_tokens: int, device="cuda"):
        if not 1 <= max_requests <= api.MOE_MAX_REQUESTS or max_tokens < 0:
            raise ValueError("max_requests must be 1..%d and max_tokens not negative"
                             % api.MOE_MAX_REQUESTS)
        self.device = _cuda(device)
        self.page_size, self.max_requests, self.max_tokens = page_size, max_requests, max_tokens
        i32 = dict(dtype=torch.int32, device=self.device)
        self._q_start = torch.empty(max_requests + 1, **i32)
        self._kv_len = torch.empty(max_requests, **i32)
        self._held = torch.empty(max_requests, **i32)
        self._free_head = torch.empty(1, **i32)
        self._positions = torch.empty(max_tokens, **i32)
        self._slots = torch.empty(max_tokens, dtype=torch.int64, device=self.device)
        self._lib = api.load()

    def plan(self, q_len, cached, held, free_pages, free_range, block_table, n_tokens: int,
             stream=None) -> BatchPlan:
        """q_len, cached, held: [B] int32; free_pages: [F] int32; free_range:
        [2] int32 {head, end}; block_table: [B][M] int32, written in place
        from entry held[b] on. The returned buffers are the planner's own: to
        feed `held` or `free_head` to the next plan, copy them into the
        caller's first."""
        B, dev, i32 = q_len.shape[0], self.device, torch.int32
        if not 1 <= B <= self.max_requests or not 0 <= n_tokens <= self.max_tokens:
            raise ValueError("a plan holds 1..%d requests and 0..%d tokens, got %d and %d"
                             % (self.max_requests, self.max_tokens, B, n_tokens))
        if block_table.dim() != 2:
            raise ValueError("block_table must be [requests][blocks]")
        F, M = free_pages.numel(), block_table.shape[1]
        b = api.BatchC(B, M, self.page_size, F, _need(q_len, "q_len", i32, [B], dev),
                       _need(cached, "cached", i32, [B], dev), _need(held, "held", i32, [B], dev),
                       _need(free_pages, "free_pages", i32, [F], dev),
                       _need(free_range, "free_range", i32, [2], dev),
                       _need(block_table, "block_table", i32, [B, M], dev),
                       self._q_start.data_ptr(), self._kv_len.data_ptr(), self._held.data_ptr(),
                       self._free_head.data_ptr())
        slots, positions = self._slots[:n_tokens], self._positions[:n_tokens]
        api._check(self._lib.moe_plan_batch(ctypes.byref(b), n_tokens, slots.data_ptr(),
                                            positions.data_ptr(), api._stream(stream)),
                   "moe_plan_batch")
        return BatchPlan(self._q_start[:B + 1], self._kv_len[:B], self._held[:B], self._free_head,
                         slots, positions)


class PagedCache:
    """Pages of keys and values: k, v [n_pages][page_size][n_kv_heads][head_dim]
    in bfloat16 or float16, in any order in memory that keeps head_dim
    contiguous (a transposed [page][head][row] pool, say)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        if not k.is_cuda or k.device != v.device:
            raise ValueError("k and v must live on one CUDA device")
        self.k, self.v, self.device = k, v, k.device
        self.c = api.make_cache(k, v)
        self.page_size, self.n_kv_heads, self.head_dim = k.shape[1:]
        self.dtype = k.dtype
        self._lib = api.load()

    @classmethod
    def allocate(cls, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int,
                 dtype=torch.bfloat16, device="cuda", heads_first: bool = False) -> "PagedCache":
        """A pool of its own, not initialised; heads_first: heads before rows
        within a page."""
        shape = ((n_pages, n_kv_heads, page_size, head_dim) if heads_first else
                 (n_pages, page_size, n_kv_heads, head_dim))
        k, v = (torch.empty(shape, dtype=dtype, device=_cuda(device)) for _ in range(2))
        return cls(k.transpose(1, 2), v.transpose(1, 2)) if heads_first else cls(k, v)

    def append(self, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
        """New keys and values [n][n_kv_heads][head_dim] (of the cache's type
        or float32, rounded once) to their slots (moe_kv_append). Rows must be
        contiguous; token and head strides may be any multiple of 16 bytes."""
        n = k.shape[0]
        if (k.dim() != 3 or k.shape != v.shape or k.dtype != v.dtype or
                any(api._stride(k, i) != api._stride(v, i) for i in range(2)) or
                tuple(k.shape[1:]) != (self.n_kv_heads, self.head_dim) or k.stride(2) != 1 or
                v.stride(2) != 1 or
                k.dtype not in (self.dtype, torch.float32) or
                k.device != self.device or v.device != self.device):
            raise ValueError("k and v must be [n][%d][%d] %s or float32 tensors on %s with "
                             "contiguous rows and equal strides"
                             % (self.n_kv_heads, self.head_dim, str(self.dtype)[6:], self.device))
        sp = _need(slots, "slots", torch.int64, [n], self.device)
        api._check(self._lib.moe_kv_append(ctypes.byref(self.c), k.data_ptr(), v.data_ptr(),
                                           api.DTYPES[k.dtype], api._stride(k, 0),
                                           api._stride(k, 1), n, sp, api._stream(stream)),
                   "moe_kv_append")


class PagedAttention:
    """Attention of packed new tokens over a paged cache (moe_attend) for up
    to max_tokens tokens: causal; with window > 0 a token sees the `window`
    newest keys, its own included, and the request's first `sinks` keys.
    scale None: 1/sqrt(head_dim)."""

    def __init__(self, cache: PagedCache, n_heads: int, max_tokens: int,
                 scale: Optional[float] = None, window: int = 0, sinks: int = 0):
        self.cache, self.n_heads, self.max_tokens = cache, n_heads, max_tokens
        self.desc = api.AttnDesc(n_heads, window, sinks, 1.0 / math.sqrt(cache.head_dim)
                                 if scale is None else scale)
        nbytes = api.moe_attend_workspace_bytes(cache.c, self.desc)
        if nbytes == 0:
            raise ValueError("cache or attention shape not covered by this library: %d heads over "
                             "%d of %d, pages of %d, %s, window %d, sinks %d"
                             % (n_heads, cache.n_kv_heads, cache.head_dim, cache.page_size,
                                str(cache.dtype)[6:], window, sinks))
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=cache.device)
        self._out = torch.empty((max_tokens, n_heads, cache.head_dim), dtype=cache.dtype,
                                device=cache.device)
        self._lib = api.load()

    def attend(self, q: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor,
               block_table: torch.Tensor, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
        """q: [n][n_heads][head_dim] of the cache's type; q_start [B+1], kv_len
        [B] and block_table [B][M] int32 as BatchPlanner.plan leaves them.
        Returns `out` (same shape and type, rows contiguous), or the object's
        own buffer. Rows of no request keep what `out` held."""
        c, n = self.cache, q.shape[0]
        shape = (n, self.n_heads, c.head_dim)
        if out is None:
            if n > self.max_tokens:
                raise ValueError("%d tokens, more than max_tokens %d" % (n, self.max_tokens))
            out = self._out[:n]
        for name, t in (("q", q), ("out", out)):
            if (tuple(t.shape) != shape or t.dtype != c.dtype or t.device != c.device or
                    t.stride(2) != 1):
                raise ValueError("%s must be a %s %s tensor on %s with contiguous rows"
                                 % (name, str(c.dtype)[6:], list(shape), c.device))
        if block_table.dim() != 2:
            raise ValueError("block_table must be [requests][blocks]")
        B, M = block_table.shape
        i32 = torch.int32
        api._check(self._lib.moe_attend(
            ctypes.byref(c.c), ctypes.byref(self.desc), q.data_ptr(), api._stride(q, 0),
            api._stride(q, 1), n,
            _need(q_start, "q_start", i32, [B + 1], c.device),
            _need(kv_len, "kv_len", i32, [B], c.device),
            _need(block_table, "block_table", i32, [B, M], c.device), M, B,
            self.workspace.data_ptr(), self.workspace.numel(), out.data_ptr(),
            api._stride(out, 0), api._stride(out, 1), api._stream(stream)), "moe_attend")
        return out


class GroupedRouter:
    """Experts of up to max_tokens tokens from router logits
    (moe_route_grouped): softmax or sigmoid scores, an optional bias that only
    selects, group-limited top-k, weights renormalised (renorm) and scaled."""

    def __init__(self, n_experts: int, top_k: int, max_tokens: int, n_groups: int = 1,
                 top_groups: int = 1, group_top: int = 1, score: str = "softmax",
                 bias: Optional[torch.Tensor] = None, renorm: bool = True, scale: float = 1.0,
                 device="cuda"):
        if score not in ("softmax", "sigmoid"):
            raise ValueError("score must be 'softmax' or 'sigmoid'")
        self.device = _cuda(device if bias is None else bias.device)
        if bias is not None:
            _need(bias, "bias", torch.float32, [n_experts], self.device)
        self.n_experts, self.top_k, self.max_tokens, self.bias = n_experts, top_k, max_tokens, bias
        self.desc = api.RouterDesc(
            n_experts, top_k, n_groups, top_groups, group_top,
            api.MOE_SCORE_SIGMOID if score == "sigmoid" else api.MOE_SCORE_SOFTMAX,
            1 if renorm else 0, scale)
        self._idx = torch.empty(max_tokens * top_k, dtype=torch.int32, device=self.device)
        self._w = torch.empty(max_tokens * top_k, dtype=torch.float32, device=self.device)
        self._lib = api.load()
        # the descriptor's own checks, before the first pass
        api._check(self._lib.moe_route_grouped(ctypes.byref(self.desc), None, api.MOE_F32,
                                               n_experts, None, 0, None, None, None),
                   "GroupedRouter")

    def route(self, logits: torch.Tensor, idx: Optional[torch.Tensor] = None,
              weights: Optional[torch.Tensor] = None, stream=None):
        """(idx [n][k] int32, weights [n][k] float32) for logits [n][E] in
        float32, bfloat16 or float16 with contiguous rows; written to idx and
        weights if given (n·k contiguous elements), else to the router's own."""
        if (logits.dim() != 2 or logits.shape[1] != self.n_experts or logits.stride(1) != 1 or
                logits.dtype not in api.DTYPES or logits.device != self.device):
            raise ValueError("logits must be a [n][%d] float32, bfloat16 or float16 tensor on %s "
                             "with contiguous rows" % (self.n_experts, self.device))
        n, k = logits.shape[0], self.top_k
        if (idx is None or weights is None) and n > self.max_tokens:
            raise ValueError("%d tokens, more than max_tokens %d" % (n, self.max_tokens))
        idx = self._idx[:n * k] if idx is None else idx.view(-1)
        weights = self._w[:n * k] if weights is None else weights.view(-1)
        ip = _need(idx, "idx", torch.int32, [n * k], self.device)
        wp = _need(weights, "weights", torch.float32, [n * k], self.device)
        api._check(self._lib.moe_route_grouped(
            ctypes.byref(self.desc), logits.data_ptr(), api.DTYPES[logits.dtype],
            api._stride(logits, 0), None if self.bias is None else self.bias.data_ptr(), n, ip, wp,
            api._stream(stream)), "moe_route_grouped")
        return idx.view(n, k), weights.view(n, k)
