"""Thin ctypes binding of libmoewarp.so — the same entry points as the C ABI
in include/moe_warp.h and include/moe_batch.h, taking torch CUDA tensors for
the device pointers.

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels. If the library has not been built, or no CUDA device is present,
every call raises; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from .configs import LayerShape

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoewarp.so")

MOE_OK, MOE_EINVAL, MOE_ECUDA, MOE_ETIMEOUT, MOE_EUNSUPPORTED, MOE_EDEVICE = range(6)
MOE_MAX_TOKENS, MOE_MAX_PAIRS, MOE_MAX_EXPERTS, MOE_MAX_TOPK, MOE_MAX_SHARED = 128, 512, 256, 16, 4

EXPORTED = ("moe_workspace_bytes", "moe_route", "moe_build_union", "moe_verify_perslot",
            "moe_verify_dedup", "moe_combine", "moe_last_device_error", "moe_status_str",
            "moe_last_cuda_error_string", "moe_verify_dedup_noalloc", "moe_noalloc_scratch_limit",
            "moe_diag_bounded_wait", "moe_route_biased", "moe_route_union", "moe_verify_pass",
            "moe_verify_pass_fused", "moe_gate", "moe_plan_batch", "moe_kv_append",
            "moe_attend_workspace_bytes", "moe_attend", "moe_attend_padded", "moe_route_grouped")

MOE_F32, MOE_BF16, MOE_F16 = range(3)
MOE_MAX_REQUESTS, MOE_MAX_GROUPS, MOE_MAX_HEAD_GROUP = 1024, 32, 128
MOE_MAX_CACHE_LEN = 2 ** 31 - 257
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
DTYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.float16: MOE_F16}


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        super().__init__("%s failed: %s%s" % (where, status_str(status) if _lib else status,
                                              (" (" + detail + ")") if detail else ""))


class LayerDesc(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("inter", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("wdtype", ctypes.c_int32)]


class LayerWeightsC(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in
                ("w_router", "w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down")]


class UnionC(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in
                ("union_ids", "union_count", "offsets", "pair_tok", "pair_slot", "bytes")]


class BatchC(ctypes.Structure):
    _fields_ = ([(name, ctypes.c_int32) for name in
                 ("n_requests", "max_blocks", "page_size", "free_capacity")] +
                [(name, ctypes.c_void_p) for name in
                 ("q_len", "cached", "held", "free_pages", "free_range", "block_table",
                  "q_start", "kv_len", "held_out", "free_head")])


class KvCacheC(ctypes.Structure):
    _fields_ = ([("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int64)] +
                [(name, ctypes.c_int32) for name in
                 ("page_size", "n_kv_heads", "head_dim", "dtype")] +
                [(name, ctypes.c_int64) for name in
                 ("page_stride", "token_stride", "head_stride")])


class AttnDesc(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int32), ("window", ctypes.c_int32),
                ("sinks", ctypes.c_int32), ("scale", ctypes.c_float)]


class RouterDesc(ctypes.Structure):
    _fields_ = ([(name, ctypes.c_int32) for name in
                 ("n_experts", "top_k", "n_groups", "top_groups", "group_top", "score",
                  "renorm")] + [("scale", ctypes.c_float)])


_lib = None


def load(path: str = LIB_PATH):
    """Loads libmoewarp.so and declares its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("libmoewarp.so is not built (expected at %s); run "
                           "__graft_entry__.build() or python -m "
                           "moe_expert_layer_warp_gb300.build" % path)
    lib = ctypes.CDLL(path)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    D = ctypes.POINTER(LayerDesc)
    W = ctypes.POINTER(LayerWeightsC)
    U = ctypes.POINTER(UnionC)
    lib.moe_workspace_bytes.argtypes = [D, I32]
    lib.moe_workspace_bytes.restype = SZ
    lib.moe_gate.argtypes = [D, P, P, I32, P, P]
    lib.moe_route.argtypes = [D, P, P, I32, P, P, P, SZ, P]
    lib.moe_route_biased.argtypes = [D, P, P, I32, P, I32, P, P, P, SZ, P]
    lib.moe_build_union.argtypes = [D, P, I32, U, P]
    lib.moe_route_union.argtypes = [D, P, P, I32, P, I32, P, P, U, P, SZ, P]
    lib.moe_verify_pass.argtypes = [D, W, P, I32, P, I32, I32, P, P, U, P, SZ, P, P, P]
    lib.moe_verify_pass_fused.argtypes = [D, W, P, I32, P, I32, I32, P, P, U, P, SZ, P, P, P]
    lib.moe_verify_perslot.argtypes = [D, W, P, I32, P, P, P, SZ, P, P]
    lib.moe_verify_dedup.argtypes = [D, W, P, I32, U, P, P, SZ, P, P]
    lib.moe_combine.argtypes = [D, P, I32, P, P]
    lib.moe_verify_dedup_noalloc.argtypes = [D, W, P, I32, U, P, P, P]
    lib.moe_noalloc_scratch_limit.argtypes = []
    lib.moe_noalloc_scratch_limit.restype = SZ
    lib.moe_last_device_error.argtypes = [P]
    lib.moe_diag_bounded_wait.argtypes = [I32, P]
    lib.moe_status_str.argtypes = [ctypes.c_int]
    lib.moe_status_str.restype = ctypes.c_char_p
    lib.moe_last_cuda_error_string.argtypes = []
    lib.moe_last_cuda_error_string.restype = ctypes.c_char_p
    I64 = ctypes.c_int64
    C, A = ctypes.POINTER(KvCacheC), ctypes.POINTER(AttnDesc)
    lib.moe_plan_batch.argtypes = [ctypes.POINTER(BatchC), I32, P, P, P]
    lib.moe_kv_append.argtypes = [C, P, P, I32, I64, I64, I32, P, P]
    lib.moe_attend_workspace_bytes.argtypes = [C, A]
    lib.moe_attend_workspace_bytes.restype = SZ
    lib.moe_attend.argtypes = [C, A, P, I64, I64, I32, P, P, P, I32, I32, P, SZ, P, I64, I64, P]
    lib.moe_attend_padded.argtypes = lib.moe_attend.argtypes
    lib.moe_route_grouped.argtypes = [ctypes.POINTER(RouterDesc), P, I32, I64, P, I32, P, P, P]
    for f in ("moe_plan_batch", "moe_kv_append", "moe_attend", "moe_attend_padded",
              "moe_route_grouped"):
        getattr(lib, f).restype = ctypes.c_int
    for f in ("moe_route", "moe_build_union", "moe_verify_perslot", "moe_verify_dedup",
              "moe_combine", "moe_last_device_error", "moe_verify_dedup_noalloc",
              "moe_diag_bounded_wait", "moe_route_biased", "moe_route_union", "moe_verify_pass",
              "moe_verify_pass_fused", "moe_gate"):
        getattr(lib, f).restype = ctypes.c_int
    _lib = lib
    return lib


def status_str(status: int) -> str:
    return load().moe_status_str(status).decode()


def _check(status: int, where: str):
    if status != MOE_OK:
        detail = load().moe_last_cuda_error_string().decode()
        raise MoeError(status, where, detail)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor, got one on %s" % t.device)
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if isinstance(stream, ctypes.c_void_p):
        return stream
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def make_desc(shape: LayerShape) -> LayerDesc:
    return LayerDesc(shape.d, shape.n_experts, shape.top_k, shape.inter, shape.n_shared,
                     shape.wdtype)


def make_weights(w) -> LayerWeightsC:
    """From a synth.LayerWeights on a CUDA device."""
    return LayerWeightsC(_ptr(w.w_router), _ptr(w.w_gate), _ptr(w.w_up), _ptr(w.w_down),
                         _ptr(w.ws_gate), _ptr(w.ws_up), _ptr(w.ws_down))


def moe_workspace_bytes(desc: LayerDesc, n_max: int) -> int:
    return int(load().moe_workspace_bytes(ctypes.byref(desc), n_max))


def moe_gate(desc, w_router, x, n, logits, stream=None):
    _check(load().moe_gate(ctypes.byref(desc), _ptr(w_router), _ptr(x), n, _ptr(logits),
                           _stream(stream)), "moe_gate")


def moe_route(desc, w_router, x, n, topk_idx, topk_w, workspace, stream=None):
    _check(load().moe_route(ctypes.byref(desc), _ptr(w_router), _ptr(x), n, _ptr(topk_idx),
                            _ptr(topk_w), _ptr(workspace), workspace.numel() *
                            workspace.element_size(), _stream(stream)), "moe_route")


def moe_route_biased(desc, w_router, bias, bias_in_weights, x, n, topk_idx, topk_w, workspace,
                     stream=None):
    _check(load().moe_route_biased(ctypes.byref(desc), _ptr(w_router), _ptr(bias),
                                   1 if bias_in_weights else 0, _ptr(x), n, _ptr(topk_idx),
                                   _ptr(topk_w), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream)),
           "moe_route_biased")


def moe_build_union(desc, topk_idx, n, u: UnionC, stream=None):
    _check(load().moe_build_union(ctypes.byref(desc), _ptr(topk_idx), n, ctypes.byref(u),
                                  _stream(stream)), "moe_build_union")


def moe_route_union(desc, w_router, bias, bias_in_weights, x, n, topk_idx, topk_w, u: UnionC,
                    workspace, stream=None):
    _check(load().moe_route_union(ctypes.byref(desc), _ptr(w_router), _ptr(bias),
                                  1 if bias_in_weights else 0, _ptr(x), n, _ptr(topk_idx),
                                  _ptr(topk_w), ctypes.byref(u), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream)),
           "moe_route_union")


MOE_ENGINE_PERSLOT, MOE_ENGINE_DEDUP = 0, 1


def moe_verify_pass(desc, weights: LayerWeightsC, bias, bias_in_weights, x, n, engine, topk_idx,
                    topk_w, u: UnionC, workspace, y_slot, y, stream=None):
    _check(load().moe_verify_pass(ctypes.byref(desc), ctypes.byref(weights), _ptr(bias),
                                  1 if bias_in_weights else 0, _ptr(x), n, engine,
                                  _ptr(topk_idx), _ptr(topk_w), ctypes.byref(u), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _ptr(y_slot),
                                  _ptr(y), _stream(stream)), "moe_verify_pass")


def moe_verify_pass_fused(desc, weights: LayerWeightsC, bias, bias_in_weights, x, n, engine,
                          topk_idx, topk_w, u: UnionC, workspace, y_slot, y, stream=None):
    _check(load().moe_verify_pass_fused(ctypes.byref(desc), ctypes.byref(weights), _ptr(bias),
                                        1 if bias_in_weights else 0, _ptr(x), n, engine,
                                        _ptr(topk_idx), _ptr(topk_w), ctypes.byref(u),
                                        _ptr(workspace),
                                        workspace.numel() * workspace.element_size(),
                                        _ptr(y_slot), _ptr(y), _stream(stream)),
           "moe_verify_pass_fused")


def moe_verify_perslot(desc, weights: LayerWeightsC, x, n, topk_idx, topk_w, workspace, y_slot,
                       stream=None):
    _check(load().moe_verify_perslot(ctypes.byref(desc), ctypes.byref(weights), _ptr(x), n,
                                     _ptr(topk_idx), _ptr(topk_w), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(),
                                     _ptr(y_slot), _stream(stream)), "moe_verify_perslot")


def moe_verify_dedup(desc, weights: LayerWeightsC, x, n, u: UnionC, topk_w, workspace, y_slot,
                     stream=None):
    _check(load().moe_verify_dedup(ctypes.byref(desc), ctypes.byref(weights), _ptr(x), n,
                                   ctypes.byref(u), _ptr(topk_w), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _ptr(y_slot),
                                   _stream(stream)), "moe_verify_dedup")


def moe_verify_dedup_noalloc(desc, weights: LayerWeightsC, x, n, u: UnionC, topk_w, y_slot,
                             stream=None):
    """moe_verify_dedup without a workspace: scratch lives in the library's
    static device array (see include/moe_warp.h)."""
    _check(load().moe_verify_dedup_noalloc(ctypes.byref(desc), ctypes.byref(weights), _ptr(x), n,
                                           ctypes.byref(u), _ptr(topk_w), _ptr(y_slot),
                                           _stream(stream)), "moe_verify_dedup_noalloc")


def moe_noalloc_scratch_limit() -> int:
    return int(load().moe_noalloc_scratch_limit())


def moe_combine(desc, y_slot, n, y, stream=None):
    _check(load().moe_combine(ctypes.byref(desc), _ptr(y_slot), n, _ptr(y), _stream(stream)),
           "moe_combine")


def moe_diag_bounded_wait(limit_us: int, stream=None):
    _check(load().moe_diag_bounded_wait(limit_us, _stream(stream)), "moe_diag_bounded_wait")


def moe_last_device_error(stream=None) -> int:
    return int(load().moe_last_device_error(_stream(stream)))


# ---- include/moe_batch.h -----------------------------------------------------
def _raw(t: Optional[torch.Tensor]):
    """The device pointer of a tensor whose strides the call takes."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor, got one on %s" % t.device)
    return ctypes.c_void_p(t.data_ptr())


def _stride(t: torch.Tensor, i: int) -> int:
    """The stride of dimension i, or of one contiguous row where the dimension
    has one entry (torch leaves any value there)."""
    return t.stride(i) if t.shape[i] > 1 else t.shape[-1]


def make_cache(k: torch.Tensor, v: torch.Tensor) -> KvCacheC:
    """From page pools [n_pages][page_size][n_kv_heads][head_dim], the last
    dimension contiguous, both with the same strides."""
    if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or any(
            _stride(k, i) != _stride(v, i) for i in range(4)):
        raise ValueError("k and v must be [pages][rows][heads][dim] of one type, shape and strides")
    if k.dtype not in DTYPES or k.stride(3) != 1 or v.stride(3) != 1:
        raise ValueError("cache pages must be float32, bfloat16 or float16 with contiguous rows")
    return KvCacheC(k.data_ptr(), v.data_ptr(), k.shape[0], k.shape[1], k.shape[2], k.shape[3],
                    DTYPES[k.dtype], _stride(k, 0), _stride(k, 1), _stride(k, 2))


def _shaped(name, t, dtype, shape):
    """ValueError unless `t` is of that type and shape (None: any size)."""
    if t.dtype is not dtype or t.dim() != len(shape) or any(
            want is not None and want != got for want, got in zip(shape, t.shape)):
        raise ValueError("%s must be a %s tensor of shape %s, got %s %s"
                         % (name, str(dtype)[6:], ["?" if v is None else v for v in shape],
                            str(t.dtype)[6:], list(t.shape)))


def _holding(name, t, dtype, n):
    """ValueError unless `t` is of that type with n elements at least."""
    if t.dtype is not dtype or t.numel() < n:
        raise ValueError("%s must be a %s tensor of %d elements or more, got %s %s"
                         % (name, str(dtype)[6:], n, str(t.dtype)[6:], list(t.shape)))


def moe_plan_batch(batch: BatchC, n_tokens, slots, positions, stream=None):
    _holding("slots", slots, torch.int64, n_tokens)
    _holding("positions", positions, torch.int32, n_tokens)
    _check(load().moe_plan_batch(ctypes.byref(batch), n_tokens, _ptr(slots), _ptr(positions),
                                 _stream(stream)), "moe_plan_batch")


def moe_kv_append(cache: KvCacheC, k, v, slots, stream=None):
    """k, v: [n_tokens][n_kv_heads][head_dim], last dimension contiguous."""
    row = (cache.n_kv_heads, cache.head_dim)
    _shaped("k", k, k.dtype, (None, *row))
    _shaped("v", v, k.dtype, k.shape)
    _holding("slots", slots, torch.int64, k.shape[0])
    if k.stride(2) != 1 or v.stride(2) != 1 or any(
            _stride(k, i) != _stride(v, i) for i in range(2)):
        raise ValueError("k and v must share their strides, their rows contiguous")
    if k.dtype not in DTYPES:
        raise ValueError("k and v must be float32, bfloat16 or float16")
    _check(load().moe_kv_append(ctypes.byref(cache), _raw(k), _raw(v), DTYPES[k.dtype],
                                _stride(k, 0), _stride(k, 1), k.shape[0], _ptr(slots),
                                _stream(stream)), "moe_kv_append")


def moe_attend_workspace_bytes(cache: KvCacheC, attn: AttnDesc) -> int:
    return int(load().moe_attend_workspace_bytes(ctypes.byref(cache), ctypes.byref(attn)))


def moe_attend(cache: KvCacheC, attn: AttnDesc, q, q_start, kv_len, block_table, workspace, out,
               stream=None, padded: bool = False):
    """q, out: [n_tokens][n_heads][head_dim], last dimension contiguous; padded:
    moe_attend_padded."""
    if DTYPES.get(q.dtype) != cache.dtype:
        raise ValueError("q must be of the cache's type, got %s" % str(q.dtype)[6:])
    _shaped("q", q, q.dtype, (None, attn.n_heads, cache.head_dim))
    _shaped("out", out, q.dtype, q.shape)
    _shaped("kv_len", kv_len, torch.int32, (None,))
    n = kv_len.shape[0]
    _holding("q_start", q_start, torch.int32, n + 1)
    _shaped("block_table", block_table, torch.int32, (None, None))
    _holding("block_table", block_table, torch.int32, n * block_table.shape[1])
    if q.stride(2) != 1 or out.stride(2) != 1:
        raise ValueError("the rows of q and out must be contiguous")
    call = load().moe_attend_padded if padded else load().moe_attend
    _check(call(ctypes.byref(cache), ctypes.byref(attn), _raw(q), _stride(q, 0), _stride(q, 1),
                q.shape[0], _ptr(q_start), _ptr(kv_len), _ptr(block_table), block_table.shape[1],
                n, _ptr(workspace), workspace.numel() * workspace.element_size(),
                _raw(out), _stride(out, 0), _stride(out, 1), _stream(stream)),
           "moe_attend_padded" if padded else "moe_attend")


def moe_route_grouped(router: RouterDesc, logits, bias, topk_idx, topk_w, stream=None):
    """logits: [n][E] float32, bfloat16 or float16, last dimension contiguous."""
    _shaped("logits", logits, logits.dtype, (None, router.n_experts))
    if logits.dtype not in DTYPES or logits.stride(1) != 1:
        raise ValueError("logits must be float32, bfloat16 or float16 with contiguous rows")
    _holding("topk_idx", topk_idx, torch.int32, logits.shape[0] * router.top_k)
    _holding("topk_w", topk_w, torch.float32, logits.shape[0] * router.top_k)
    if bias is not None:
        _holding("bias", bias, torch.float32, router.n_experts)
    _check(load().moe_route_grouped(ctypes.byref(router), _raw(logits), DTYPES[logits.dtype],
                                    _stride(logits, 0), _ptr(bias),
                                    logits.shape[0], _ptr(topk_idx), _ptr(topk_w),
                                    _stream(stream)), "moe_route_grouped")
