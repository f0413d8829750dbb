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
(None: torch's current stream). An object's device must be the current one when
it is called. Values that only the device sees are checked
there, see ``api.moe_last_device_error``. There are no gradients.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional

import torch

from . import api


# A call here takes a few microseconds of the GPU at its smallest, so what it
# does on the host is kept short: checks read each attribute once, C structs
# and views of the buffers are kept, and the stream is fetched as a handle.
# (The current device is asked for only where there are others: 0.15 us of a
# call's 4 to 6, and 0.45 through torch.cuda.)
_several_devices = torch.cuda.device_count() > 1
_current_device = torch._C._cuda_getDevice


def _need(t, name, dtype, shape, index):
    """The device pointer of `t`, a contiguous tensor of the given kind."""
    if (t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous()):
        return t.data_ptr()
    raise ValueError("%s must be a contiguous %s %s tensor on cuda:%d, got %s %s on %s"
                     % (name, str(dtype)[6:], list(shape), index, str(t.dtype)[6:],
                        list(t.shape), t.device))


def _handle(stream, index):
    """The handle of `stream`, or of torch's current stream on the device, which
    must be the current one: the library launches there."""
    if _several_devices and _current_device() != index:
        raise ValueError("the object lives on cuda:%d, but cuda:%d is the current device"
                         % (index, _current_device()))
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return api._stream(stream)


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
        self._index = self.device.index
        self._c = api.BatchC(page_size=page_size, q_start=self._q_start.data_ptr(),
                             kv_len=self._kv_len.data_ptr(), held_out=self._held.data_ptr(),
                             free_head=self._free_head.data_ptr())
        self._cref = ctypes.byref(self._c)
        self._slots_ptr, self._pos_ptr = self._slots.data_ptr(), self._positions.data_ptr()
        self._size, self._plan = None, None

    def plan(self, q_len, cached, held, free_pages, free_range, block_table, n_tokens: int,
             stream=None) -> BatchPlan:
        """q_len, cached, held: [B] int32; free_pages: [F] int32; free_range:
        [2] int32 {head, end}; block_table: [B][M] int32, written in place
        from entry held[b] on. The returned buffers are the planner's own: to
        feed `held` or `free_head` to the next plan, copy them into the
        caller's first."""
        c, at, i32 = self._c, self._index, torch.int32
        if block_table.dim() != 2 or free_pages.dim() != 1:
            raise ValueError("block_table must be [requests][blocks], free_pages [pages]")
        (B, M), F = block_table.shape, free_pages.shape[0]
        if (B, n_tokens) != self._size:
            if not 1 <= B <= self.max_requests or not 0 <= n_tokens <= self.max_tokens:
                raise ValueError("a plan holds 1..%d requests and 0..%d tokens, got %d and %d"
                                 % (self.max_requests, self.max_tokens, B, n_tokens))
            self._plan = BatchPlan(self._q_start[:B + 1], self._kv_len[:B], self._held[:B],
                                   self._free_head, self._slots[:n_tokens],
                                   self._positions[:n_tokens])
            self._size = (B, n_tokens)
        c.n_requests, c.max_blocks, c.free_capacity = B, M, F
        c.q_len = _need(q_len, "q_len", i32, (B,), at)
        c.cached = _need(cached, "cached", i32, (B,), at)
        c.held = _need(held, "held", i32, (B,), at)
        c.free_pages = _need(free_pages, "free_pages", i32, (F,), at)
        c.free_range = _need(free_range, "free_range", i32, (2,), at)
        c.block_table = _need(block_table, "block_table", i32, (B, M), at)
        st = self._lib.moe_plan_batch(self._cref, n_tokens, self._slots_ptr, self._pos_ptr,
                                      _handle(stream, at))
        if st:
            api._check(st, "moe_plan_batch")
        return self._plan


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
        self._index, self._cref = self.device.index, ctypes.byref(self.c)
        self._row = (self.n_kv_heads, self.head_dim)

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
        n, dt, at = k.shape[0], k.dtype, self._index
        sk, sv = k.stride(), v.stride()
        if (k.shape != (n, *self._row) or v.shape != k.shape or v.dtype is not dt or
                (dt is not self.dtype and dt is not torch.float32) or k.get_device() != at or
                v.get_device() != at or sk[2] != 1 or sv[2] != 1 or (n > 1 and sk[0] != sv[0]) or
                (self.n_kv_heads > 1 and sk[1] != sv[1])):
            raise ValueError("k and v must be [n][%d][%d] %s or float32 tensors on %s with "
                             "contiguous rows and equal strides"
                             % (*self._row, str(self.dtype)[6:], self.device))
        D = self.head_dim                      # for the stride of a dimension of one entry
        st = self._lib.moe_kv_append(self._cref, k.data_ptr(), v.data_ptr(), api.DTYPES[dt],
                                     sk[0] if n > 1 else D, sk[1] if self.n_kv_heads > 1 else D, n,
                                     _need(slots, "slots", torch.int64, (n,), at),
                                     _handle(stream, at))
        if st:
            api._check(st, "moe_kv_append")


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
        self._dref, self._ws_ptr, self._ws_bytes = (ctypes.byref(self.desc),
                                                    self.workspace.data_ptr(), nbytes)
        self._n, self._view = None, None

    def _check(self, name, t, n):
        """The token and head strides of q or out."""
        c, H = self.cache, self.n_heads
        s = t.stride()
        if (t.shape != (n, H, c.head_dim) or t.dtype is not c.dtype or
                t.get_device() != c._index or s[2] != 1):
            raise ValueError("%s must be a %s %s tensor on %s with contiguous rows"
                             % (name, str(c.dtype)[6:], [n, H, c.head_dim], c.device))
        return s[0] if n > 1 else c.head_dim, s[1] if H > 1 else c.head_dim

    def attend(self, q: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor,
               block_table: torch.Tensor, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
        """q: [n][n_heads][head_dim] of the cache's type; q_start [B+1], kv_len
        [B] and block_table [B][M] int32 as BatchPlanner.plan leaves them.
        Returns `out` (same shape and type, rows contiguous), or the object's
        own buffer. Rows of no request (a padded batch's) keep what `out` held,
        and are zeros in the object's own buffer."""
        c, n, i32 = self.cache, q.shape[0], torch.int32
        at, call = c._index, self._lib.moe_attend
        if out is None:
            if n != self._n:
                if n > self.max_tokens:
                    raise ValueError("%d tokens, more than max_tokens %d" % (n, self.max_tokens))
                self._n, self._view = n, self._out[:n]
            out, call = self._view, self._lib.moe_attend_padded
        q_token, q_head = self._check("q", q, n)
        out_token, out_head = self._check("out", out, n)
        if block_table.dim() != 2:
            raise ValueError("block_table must be [requests][blocks]")
        B, M = block_table.shape
        st = call(
            c._cref, self._dref, q.data_ptr(), q_token, q_head, n,
            _need(q_start, "q_start", i32, (B + 1,), at), _need(kv_len, "kv_len", i32, (B,), at),
            _need(block_table, "block_table", i32, (B, M), at), M, B, self._ws_ptr,
            self._ws_bytes, out.data_ptr(), out_token, out_head, _handle(stream, at))
        if st:
            api._check(st, "moe_attend")
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
        self._index = self.device.index
        self._bias_ptr = None if bias is None else _need(bias, "bias", torch.float32,
                                                         (n_experts,), self._index)
        self.n_experts, self.top_k, self.max_tokens, self.bias = n_experts, top_k, max_tokens, bias
        self.desc = api.RouterDesc(
            n_experts, top_k, n_groups, top_groups, group_top,
            api.MOE_SCORE_SIGMOID if score == "sigmoid" else api.MOE_SCORE_SOFTMAX,
            1 if renorm else 0, scale)
        self._idx = torch.empty((max_tokens, top_k), dtype=torch.int32, device=self.device)
        self._w = torch.empty((max_tokens, top_k), dtype=torch.float32, device=self.device)
        self._n, self._views = None, None
        self._lib = api.load()
        self._dref = ctypes.byref(self.desc)
        # the descriptor's own checks, before the first pass
        api._check(self._lib.moe_route_grouped(ctypes.byref(self.desc), None, api.MOE_F32,
                                               n_experts, None, 0, None, None, None),
                   "GroupedRouter")

    def route(self, logits: torch.Tensor, idx: Optional[torch.Tensor] = None,
              weights: Optional[torch.Tensor] = None, stream=None):
        """(idx [n][k] int32, weights [n][k] float32) for logits [n][E] in
        float32, bfloat16 or float16 with contiguous rows; written to idx and
        weights if given (n·k contiguous elements), else to the router's own."""
        E, k, at = self.n_experts, self.top_k, self._index
        dt = api.DTYPES.get(logits.dtype)
        s = logits.stride()
        if (logits.dim() != 2 or logits.shape[1] != E or s[1] != 1 or dt is None or
                logits.get_device() != at):
            raise ValueError("logits must be a [n][%d] float32, bfloat16 or float16 tensor on %s "
                             "with contiguous rows" % (E, self.device))
        n = logits.shape[0]
        if idx is None and weights is None:
            if n != self._n:
                if n > self.max_tokens:
                    raise ValueError("%d tokens, more than max_tokens %d" % (n, self.max_tokens))
                self._n, self._views = n, (self._idx[:n], self._w[:n])
            idx, weights = self._views
            ip, wp = idx.data_ptr(), weights.data_ptr()
        elif idx is None or weights is None:
            raise ValueError("give both idx and weights, or neither")
        else:
            idx, weights = idx.view(n, k), weights.view(n, k)
            ip = _need(idx, "idx", torch.int32, (n, k), at)
            wp = _need(weights, "weights", torch.float32, (n, k), at)
        st = self._lib.moe_route_grouped(self._dref, logits.data_ptr(), dt, s[0] if n > 1 else E,
                                         self._bias_ptr, n, ip, wp, _handle(stream, at))
        if st:
            api._check(st, "moe_route_grouped")
        return idx, weights
