"""A verification step of several requests, through the C ABI of
include/moe_batch.h and include/moe_kv8.h.

``BatchPlanner`` turns request lengths into block tables, slots and
positions; ``PagedCache`` holds pages of keys and values and takes new ones;
``PagedAttention`` lets every new token attend over its request's pages;
``GroupedRouter`` picks experts from router logits. A decoder block calls
them in that order, then an expert engine (``layer.PassRunner``):

    plan = planner.plan(q_len, cached, held, free_pages, free_range, table, n)
    cache.append(k, v, plan.slots)
    y = attention.attend(q, plan.q_start, plan.kv_len, table)
    idx, w = router.route(logits)

``Rotary`` gives queries and keys their positions before that, and
``PagedCache8`` with ``PagedAttention8`` is the same cache and attention with
keys and values held in 8 bits:

    rotary.rotate(q, k, plan.positions)

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


def _empty(shape, dtype, device, stream):
    """A new tensor that a call on `stream` writes: of that stream's memory. (Memory of
    torch's current stream may be in use by what that one still has to do.)"""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = api._stream(stream).value
        stream = (torch.cuda.ExternalStream(handle, device) if handle else
                  torch.cuda.default_stream(device))
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


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


def rotary_frequencies(n_rotated: int, base: float = 10000.0, scaling: str = "none",
                       factor: float = 1.0, original: int = 4096, fast: Optional[float] = None,
                       slow: float = 1.0) -> list:
    """Angles per position in radians of n_rotated / 2 pairs, base^(-2i/n_rotated),
    stretched for contexts `factor` times as long as the `original` positions that
    the unstretched angles were made for (these and the others are a checkpoint's):

      "linear"  every angle divided by factor;
      "base"    the base times factor^(n/(n-2)): the slowest pair is stretched by
                the factor, the fastest not at all;
      "ramp"    pairs that turn less than `slow` times within `original` positions
                divided, those that turn more than `fast` times kept, the pairs
                between by their index (usual with an amplitude of
                0.1 ln(factor) + 1); fast is 32 if not given;
      "bands"   the same by the number of turns itself; fast is 4 if not given.
    """
    n = n_rotated
    if fast is None:
        fast = 4.0 if scaling == "bands" else 32.0
    if n < 2 or n % 2 or not base > 0 or not factor > 0 or original < 1 or not 0 < slow < fast:
        raise ValueError("n_rotated must be even and positive, base, factor and original positive, "
                         "and slow below fast")
    if scaling == "base":
        if n < 4:
            raise ValueError("scaling the base takes two pairs at least")
        base *= factor ** (n / (n - 2))
    f = [base ** (-2.0 * i / n) for i in range(n // 2)]
    if scaling in ("none", "base"):
        return f
    if scaling == "linear":
        return [v / factor for v in f]
    if scaling == "bands":
        keep = [(original * v / (2 * math.pi) - slow) / (fast - slow) for v in f]
    elif scaling == "ramp":
        if base == 1.0:
            raise ValueError("a ramp takes a base other than 1")

        def index(turns):
            return n * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(0.0, math.floor(index(fast))), min(n - 1.0, math.ceil(index(slow)))
        keep = [1.0 - (i - lo) / max(hi - lo, 0.001) for i in range(n // 2)]
    else:
        raise ValueError("scaling must be 'none', 'linear', 'base', 'ramp' or 'bands'")
    keep = [min(1.0, max(0.0, v)) for v in keep]
    return [v * w + v / factor * (1.0 - w) for v, w in zip(f, keep)]


class Rotary:
    """Rotary positions of queries and keys (moe_rotary): of every head the
    n_rotated columns from `first` on (None: all) are turned in pairs, halves of
    them or neighbours (interleaved). frequencies: angles per position in radians,
    n_rotated / 2 of them (None: rotary_frequencies(n_rotated))."""

    def __init__(self, head_dim: int, n_rotated: Optional[int] = None, frequencies=None,
                 first: int = 0, interleaved: bool = False, amplitude: float = 1.0, device="cuda"):
        n = head_dim if n_rotated is None else n_rotated
        if frequencies is None:
            frequencies = rotary_frequencies(n)
        frequencies = [float(v) for v in frequencies]
        if len(frequencies) * 2 != n:
            raise ValueError("%d rotated columns need %d frequencies, got %d"
                             % (n, n // 2, len(frequencies)))
        turns = api.moe_rotary_turns(frequencies)
        self.device = _cuda(device)
        self.head_dim, self.n_rotated, self.frequencies = head_dim, n, frequencies
        self._turns = turns.to(self.device)
        self.desc = api.RotaryDesc(head_dim, n, first, 1 if interleaved else 0, amplitude,
                                   self._turns.data_ptr())
        self._lib, self._index, self._dref = api.load(), self.device.index, ctypes.byref(self.desc)
        # the descriptor's own checks, before the first step
        api._check(self._lib.moe_rotary(self._dref, api.MOE_F32, None, None, None, 0, None),
                   "Rotary")

    def _rows(self, name, x, out, n):
        """The C rows of q or k (a struct of its own for each call: host threads may
        share the object), and the tensor that they are written to."""
        D = self.head_dim
        s = x.stride()
        if x.dim() != 3 or x.shape[0] != n or x.shape[2] != D or x.get_device() != self._index or (
                s[2] != 1):
            raise ValueError("%s must be a [%d][heads][%d] tensor on %s with contiguous rows"
                             % (name, n, D, self.device))
        H = x.shape[1]
        if out is None:
            out, t = x, s
        elif out.shape != x.shape or out.dtype is not x.dtype or (
                out.get_device() != self._index or out.stride(2) != 1):
            raise ValueError("%s_out must be a %s %s tensor on %s with contiguous rows"
                             % (name, str(x.dtype)[6:], list(x.shape), self.device))
        else:
            t = out.stride()
        return api.RotaryRows(
            x.data_ptr(), out.data_ptr(), H, s[0] if n > 1 else D, s[1] if H > 1 else D,
            t[0] if n > 1 else D, t[1] if H > 1 else D), out

    def rotate(self, q: Optional[torch.Tensor], k: Optional[torch.Tensor],
               positions: torch.Tensor, q_out: Optional[torch.Tensor] = None,
               k_out: Optional[torch.Tensor] = None, stream=None):
        """q, k: [n][heads][head_dim] float32, bfloat16 or float16 with contiguous
        rows, either may be None; positions [n] int32, as BatchPlanner.plan leaves
        them. In place, or into q_out and k_out. Returns (q, k) rotated."""
        n, x = positions.shape[0], k if q is None else q
        if x is None or (q is not None and k is not None and q.dtype is not k.dtype) or (
                x.dtype not in api.DTYPES):
            raise ValueError("give q or k, of one type: float32, bfloat16 or float16")
        if (q is None and q_out is not None) or (k is None and k_out is not None):
            raise ValueError("q_out and k_out take what q and k give: one is there without the other")
        q_rows = k_rows = None
        if q is not None:
            q_rows, q = self._rows("q", q, q_out, n)
        if k is not None:
            k_rows, k = self._rows("k", k, k_out, n)
        st = self._lib.moe_rotary(
            self._dref, api.DTYPES[x.dtype], q_rows, k_rows,
            _need(positions, "positions", torch.int32, (n,), self._index), n,
            _handle(stream, self._index))
        if st:
            api._check(st, "moe_rotary")
        return q, k


class PagedCache8:
    """Pages of keys and values in 8 bits: codes k, v
    [n_pages][page_size][n_kv_heads][head_dim] in float8_e4m3fn, in any order in
    memory that keeps head_dim contiguous, and scales k_scale, v_scale
    [n_pages][n_kv_heads][page_size / block] in float32, one for each `block`
    tokens of a page and head. An element stands for code · scale."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor):
        if not k.is_cuda or any(t.device != k.device for t in (v, k_scale, v_scale)):
            raise ValueError("codes and scales must live on one CUDA device")
        self.k, self.v, self.k_scale, self.v_scale, self.device = k, v, k_scale, v_scale, k.device
        self.c = api.make_cache8(k, v, k_scale, v_scale)
        self.page_size, self.n_kv_heads, self.head_dim = k.shape[1:]
        self.block = self.c.block
        self._lib = api.load()
        self._index, self._cref = self.device.index, ctypes.byref(self.c)
        self._row = (self.n_kv_heads, self.head_dim)

    @classmethod
    def allocate(cls, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int,
                 block: int = 16, device="cuda", heads_first: bool = False) -> "PagedCache8":
        """A pool of its own, not initialised; heads_first: heads before rows
        within a page."""
        if block < 1 or page_size % block:
            raise ValueError("block must divide page_size")
        shape = ((n_pages, n_kv_heads, page_size, head_dim) if heads_first else
                 (n_pages, page_size, n_kv_heads, head_dim))
        device = _cuda(device)
        k, v = (torch.empty(shape, dtype=torch.float8_e4m3fn, device=device) for _ in range(2))
        ks, vs = (torch.empty((n_pages, n_kv_heads, page_size // block), device=device)
                  for _ in range(2))
        return cls(k.transpose(1, 2), v.transpose(1, 2), ks, vs) if heads_first else cls(k, v, ks,
                                                                                          vs)

    def append(self, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
        """New keys and values [n][n_kv_heads][head_dim] (float32, bfloat16 or
        float16) to their slots, rounded to codes (moe_kv8_append). A block's
        scale grows with what comes into it, and starts anew when its first row
        is written; the tokens of a block are consecutive rows of the call, with no
        skipped one (slot -1) between them. Rows must be contiguous; token and head strides may be any multiple of 16
        bytes."""
        n, dt, at = k.shape[0], k.dtype, self._index
        sk, sv = k.stride(), v.stride()
        if (k.shape != (n, *self._row) or v.shape != k.shape or v.dtype is not dt or
                dt not in api.DTYPES or k.get_device() != at or v.get_device() != at or
                sk[2] != 1 or sv[2] != 1 or (n > 1 and sk[0] != sv[0]) or
                (self.n_kv_heads > 1 and sk[1] != sv[1])):
            raise ValueError("k and v must be [n][%d][%d] float32, bfloat16 or float16 tensors on "
                             "%s with contiguous rows and equal strides" % (*self._row, self.device))
        D = self.head_dim                      # for the stride of a dimension of one entry
        st = self._lib.moe_kv8_append(self._cref, k.data_ptr(), v.data_ptr(), api.DTYPES[dt],
                                      sk[0] if n > 1 else D, sk[1] if self.n_kv_heads > 1 else D, n,
                                      _need(slots, "slots", torch.int64, (n,), at),
                                      _handle(stream, at))
        if st:
            api._check(st, "moe_kv8_append")

    def read(self, slots: torch.Tensor, dtype=torch.bfloat16, k: Optional[torch.Tensor] = None,
             v: Optional[torch.Tensor] = None, stream=None):
        """(keys, values) [n][n_kv_heads][head_dim] that the rows of slots [n] int64
        stand for (moe_kv8_read), zeros for slot -1, written to k and v if given
        (of one type and strides), else to new tensors of `dtype`, which are
        `stream`'s as torch counts them."""
        n, at = slots.shape[0], self._index
        if k is None and v is None:
            k, v = (_empty((n, *self._row), dtype, self.device, stream) for _ in range(2))
        elif k is None or v is None:
            raise ValueError("give both k and v, or neither")
        sk, sv = k.stride(), v.stride()
        if (k.shape != (n, *self._row) or v.shape != k.shape or v.dtype is not k.dtype or
                k.dtype not in api.DTYPES or k.get_device() != at or v.get_device() != at or
                sk[2] != 1 or sv[2] != 1 or (n > 1 and sk[0] != sv[0]) or
                (self.n_kv_heads > 1 and sk[1] != sv[1])):
            raise ValueError("k and v must be [%d][%d][%d] float32, bfloat16 or float16 tensors on "
                             "%s with contiguous rows and equal strides"
                             % (n, *self._row, self.device))
        D = self.head_dim
        st = self._lib.moe_kv8_read(self._cref, _need(slots, "slots", torch.int64, (n,), at), n,
                                    api.DTYPES[k.dtype], k.data_ptr(), v.data_ptr(),
                                    sk[0] if n > 1 else D, sk[1] if self.n_kv_heads > 1 else D,
                                    _handle(stream, at))
        if st:
            api._check(st, "moe_kv8_read")
        return k, v


class PagedAttention8:
    """PagedAttention over a cache in 8 bits (moe_attend8): queries and results
    are of `dtype`, bfloat16 or float16."""

    def __init__(self, cache: PagedCache8, n_heads: int, max_tokens: int, dtype=torch.bfloat16,
                 scale: Optional[float] = None, window: int = 0, sinks: int = 0):
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("dtype must be bfloat16 or float16")
        self.cache, self.n_heads, self.max_tokens, self.dtype = cache, n_heads, max_tokens, dtype
        self.desc = api.AttnDesc(n_heads, window, sinks, 1.0 / math.sqrt(cache.head_dim)
                                 if scale is None else scale)
        nbytes = api.moe_attend8_workspace_bytes(cache.c, self.desc)
        if nbytes == 0:
            raise ValueError("cache or attention shape not covered by this library: %d heads over "
                             "%d of %d, pages of %d, blocks of %d, window %d, sinks %d"
                             % (n_heads, cache.n_kv_heads, cache.head_dim, cache.page_size,
                                cache.block, window, sinks))
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=cache.device)
        self._out = torch.empty((max_tokens, n_heads, cache.head_dim), dtype=dtype,
                                device=cache.device)
        self._lib = api.load()
        self._dref, self._ws_ptr, self._ws_bytes = (ctypes.byref(self.desc),
                                                    self.workspace.data_ptr(), nbytes)
        self._type = api.DTYPES[dtype]
        self._n, self._view = None, None

    def _check(self, name, t, n):
        """The token and head strides of q or out."""
        c, H = self.cache, self.n_heads
        s = t.stride()
        if (t.shape != (n, H, c.head_dim) or t.dtype is not self.dtype or
                t.get_device() != c._index or s[2] != 1):
            raise ValueError("%s must be a %s %s tensor on %s with contiguous rows"
                             % (name, str(self.dtype)[6:], [n, H, c.head_dim], c.device))
        return s[0] if n > 1 else c.head_dim, s[1] if H > 1 else c.head_dim

    def attend(self, q: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor,
               block_table: torch.Tensor, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
        """As PagedAttention.attend."""
        c, n, i32 = self.cache, q.shape[0], torch.int32
        at, call = c._index, self._lib.moe_attend8
        if out is None:
            if n != self._n:
                if n > self.max_tokens:
                    raise ValueError("%d tokens, more than max_tokens %d" % (n, self.max_tokens))
                self._n, self._view = n, self._out[:n]
            out, call = self._view, self._lib.moe_attend8_padded
        q_token, q_head = self._check("q", q, n)
        out_token, out_head = self._check("out", out, n)
        if block_table.dim() != 2:
            raise ValueError("block_table must be [requests][blocks]")
        B, M = block_table.shape
        st = call(
            c._cref, self._dref, self._type, q.data_ptr(), q_token, q_head, n,
            _need(q_start, "q_start", i32, (B + 1,), at), _need(kv_len, "kv_len", i32, (B,), at),
            _need(block_table, "block_table", i32, (B, M), at), M, B, self._ws_ptr,
            self._ws_bytes, out.data_ptr(), out_token, out_head, _handle(stream, at))
        if st:
            api._check(st, "moe_attend8")
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
