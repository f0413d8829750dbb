"""Host-only checks of include/moe_batch.h's entry points: every refusal has
its status and its reason, and nothing is launched (no GPU is touched)."""
import ctypes

import pytest
import torch

from moe_expert_layer_warp_gb300 import api, batch, build

ONE = 1 << 20          # stands for an aligned device pointer; never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load()


def _why():
    return api.load().moe_last_cuda_error_string().decode()


def _batch(**over):
    f = dict(n_requests=2, max_blocks=4, page_size=16, free_capacity=8, q_len=ONE, cached=ONE + 64,
             held=ONE + 128, free_pages=ONE + 192, free_range=ONE + 256, block_table=ONE + 320,
             q_start=ONE + 384, kv_len=ONE + 448, held_out=ONE + 512, free_head=ONE + 576)
    f.update(over)
    return api.BatchC(*[f[n] for n, _ in api.BatchC._fields_])


@pytest.mark.parametrize("over,status,reason", [
    (dict(n_requests=0), api.MOE_EINVAL, "n_requests"),
    (dict(n_requests=1025), api.MOE_EINVAL, "n_requests"),
    (dict(max_blocks=0), api.MOE_EINVAL, "max_blocks"),
    (dict(free_capacity=-1), api.MOE_EINVAL, "free_capacity"),
    (dict(q_len=None), api.MOE_EINVAL, "null array"),
    (dict(free_pages=None), api.MOE_EINVAL, "free_pages"),
    (dict(kv_len=ONE + 2), api.MOE_EINVAL, "misaligned"),
    (dict(held_out=ONE + 128), api.MOE_EINVAL, "one of the inputs"),
    (dict(kv_len=ONE + 64), api.MOE_EINVAL, "one of the inputs"),
    (dict(free_head=ONE + 260), api.MOE_EINVAL, "one of the inputs"),
    (dict(page_size=24), api.MOE_EUNSUPPORTED, "page_size"),
    (dict(page_size=8), api.MOE_EUNSUPPORTED, "page_size"),
])
def test_plan_refusals(lib, over, status, reason):
    b = _batch(**over)
    assert lib.moe_plan_batch(ctypes.byref(b), 4, ONE, ONE, None) == status
    assert reason in _why()


def test_plan_refuses_bad_outputs(lib):
    b = _batch()
    f = lib.moe_plan_batch
    assert f(None, 4, ONE, ONE, None) == api.MOE_EINVAL
    assert f(ctypes.byref(b), -1, ONE, ONE, None) == api.MOE_EINVAL
    assert f(ctypes.byref(b), 4, None, ONE, None) == api.MOE_EINVAL
    assert f(ctypes.byref(b), 4, ONE + 4, ONE, None) == api.MOE_EINVAL
    assert "slots" in _why()


def _cache(**over):
    f = dict(k=ONE, v=ONE, n_pages=10, page_size=16, n_kv_heads=2, head_dim=64,
             dtype=api.MOE_BF16, page_stride=16 * 128, token_stride=128, head_stride=64)
    f.update(over)
    return api.KvCacheC(*[f[n] for n, _ in api.KvCacheC._fields_])


CACHE_FAULTS = [
    (dict(k=None), api.MOE_EINVAL, "aligned"),
    (dict(v=ONE + 8), api.MOE_EINVAL, "aligned"),
    (dict(n_pages=0), api.MOE_EINVAL, "n_pages"),
    (dict(n_kv_heads=0), api.MOE_EINVAL, "sizes"),
    (dict(dtype=7), api.MOE_EINVAL, "type"),
    (dict(token_stride=100), api.MOE_EINVAL, "strides"),
    (dict(head_stride=0), api.MOE_EINVAL, "strides"),
    (dict(page_stride=1 << 40), api.MOE_EINVAL, "stride out of range"),
    (dict(dtype=api.MOE_F32), api.MOE_EUNSUPPORTED, "bf16 or fp16"),
    (dict(page_size=8), api.MOE_EUNSUPPORTED, "page_size"),
    (dict(page_size=512), api.MOE_EUNSUPPORTED, "page_size"),
    (dict(head_dim=96), api.MOE_EUNSUPPORTED, "head_dim"),
]


@pytest.mark.parametrize("over,status,reason", CACHE_FAULTS)
def test_cache_descriptor_refusals(lib, over, status, reason):
    c, a = _cache(**over), api.AttnDesc(8, 0, 0, 0.125)
    assert lib.moe_kv_append(ctypes.byref(c), ONE, ONE, api.MOE_BF16, 128, 64, 4, ONE,
                             None) == status
    assert reason in _why() and "moe_kv_append" in _why()
    assert lib.moe_attend(ctypes.byref(c), ctypes.byref(a), ONE, 512, 64, 4, ONE, ONE, ONE, 4, 2,
                          ONE, 1 << 30, ONE, 512, 64, None) == status
    assert reason in _why() and "moe_attend" in _why()
    assert lib.moe_attend_workspace_bytes(ctypes.byref(c), ctypes.byref(a)) == 0


@pytest.mark.parametrize("args,reason", [
    ((ONE, ONE, api.MOE_F16, 128, 64, 4, ONE), "src_dtype"),
    ((ONE, ONE, api.MOE_BF16, 100, 64, 4, ONE), "strides"),
    ((ONE, ONE, api.MOE_F32, 128, 62, 4, ONE), "strides"),
    ((ONE, ONE, api.MOE_BF16, -128, 64, 4, ONE), "strides"),
    ((ONE, ONE, api.MOE_BF16, 128, 64, -1, ONE), "n_tokens"),
    ((None, ONE, api.MOE_BF16, 128, 64, 4, ONE), "null"),
    ((ONE, ONE + 8, api.MOE_BF16, 128, 64, 4, ONE), "misaligned"),
    ((ONE, ONE, api.MOE_BF16, 128, 64, 4, ONE + 4), "misaligned"),
])
def test_append_refusals(lib, args, reason):
    c = _cache()
    assert lib.moe_kv_append(ctypes.byref(c), *args, None) == api.MOE_EINVAL
    assert reason in _why()


def test_no_tokens_is_no_launch(lib):
    c, a = _cache(), api.AttnDesc(8, 0, 0, 0.125)
    assert lib.moe_kv_append(ctypes.byref(c), None, None, api.MOE_BF16, 128, 64, 0, None,
                             None) == api.MOE_OK
    assert lib.moe_attend(ctypes.byref(c), ctypes.byref(a), None, 512, 64, 0, None, None, None, 4,
                          2, None, 0, None, 512, 64, None) == api.MOE_OK
    r = api.RouterDesc(8, 2, 1, 1, 1, 0, 1, 1.0)
    assert lib.moe_route_grouped(ctypes.byref(r), None, api.MOE_F32, 8, None, 0, None, None,
                                 None) == api.MOE_OK


@pytest.mark.parametrize("desc,status,reason", [
    ((7, 0, 0, 0.1), api.MOE_EINVAL, "multiple of n_kv_heads"),
    ((0, 0, 0, 0.1), api.MOE_EINVAL, "multiple of n_kv_heads"),
    ((8, -1, 0, 0.1), api.MOE_EINVAL, "negative"),
    ((8, 4, -1, 0.1), api.MOE_EINVAL, "negative"),
    ((8, 0, 0, 0.0), api.MOE_EINVAL, "scale"),
    ((8, 0, 0, float("nan")), api.MOE_EINVAL, "scale"),
    ((8, 0, 0, float("inf")), api.MOE_EINVAL, "scale"),
    ((2 * 129, 0, 0, 0.1), api.MOE_EUNSUPPORTED, "128 query heads"),
])
def test_attention_descriptor_refusals(lib, desc, status, reason):
    c, a = _cache(), api.AttnDesc(*desc)
    assert lib.moe_attend(ctypes.byref(c), ctypes.byref(a), ONE, 512, 64, 4, ONE, ONE, ONE, 4, 2,
                          ONE, 1 << 30, ONE, 512, 64, None) == status
    assert reason in _why()
    assert lib.moe_attend_workspace_bytes(ctypes.byref(c), ctypes.byref(a)) == 0


@pytest.mark.parametrize("at,value,reason", [
    (0, ONE + 8, "q or out"), (1, 100, "q strides"), (2, -64, "q strides"), (4, ONE + 2, "q_start"),
    (5, None, "kv_len"), (6, None, "block_table"), (7, 0, "max_blocks"), (8, 0, "n_requests"),
    (8, 1025, "n_requests"), (9, ONE + 64, "workspace"), (10, 16, "workspace"),
    (11, None, "q or out"), (12, 504, "out strides"), (13, 32, "out strides"),
    (12, 500, "out strides")])
def test_attend_refusals(lib, at, value, reason):
    c, a = _cache(), api.AttnDesc(8, 0, 0, 0.125)
    args = [ONE, 512, 64, 4, ONE, ONE, ONE, 4, 2, ONE, 1 << 30, ONE, 512, 64]
    args[at] = value
    assert lib.moe_attend(ctypes.byref(c), ctypes.byref(a), *args, None) == api.MOE_EINVAL
    assert reason in _why()


@pytest.mark.parametrize("desc,reason", [
    ((0, 1, 1, 1, 1, 0, 1, 1.0), "n_experts"), ((257, 1, 1, 1, 1, 0, 1, 1.0), "n_experts"),
    ((64, 6, 7, 1, 1, 0, 1, 1.0), "n_groups"), ((128, 6, 64, 1, 1, 0, 1, 1.0), "n_groups"),
    ((64, 6, 8, 0, 1, 0, 1, 1.0), "top_groups"), ((64, 6, 8, 9, 1, 0, 1, 1.0), "top_groups"),
    ((64, 6, 8, 1, 3, 0, 1, 1.0), "group_top"), ((8, 1, 8, 1, 2, 0, 1, 1.0), "group_top"),
    ((64, 17, 1, 1, 1, 0, 1, 1.0), "top_k"), ((64, 9, 8, 1, 1, 0, 1, 1.0), "top_k"),
    ((64, 0, 1, 1, 1, 0, 1, 1.0), "top_k"), ((64, 6, 1, 1, 1, 2, 1, 1.0), "score"),
    ((64, 6, 1, 1, 1, 0, 2, 1.0), "renorm"), ((64, 6, 1, 1, 1, 0, 1, float("inf")), "scale")])
def test_router_descriptor_refusals(lib, desc, reason):
    r = api.RouterDesc(*desc)
    assert lib.moe_route_grouped(ctypes.byref(r), ONE, api.MOE_F32, 512, None, 4, ONE, ONE,
                                 None) == api.MOE_EINVAL
    assert reason in _why()


@pytest.mark.parametrize("args", [
    (None, api.MOE_F32, 64, None, 4, ONE, ONE), (ONE, 3, 64, None, 4, ONE, ONE),
    (ONE, api.MOE_F32, 63, None, 4, ONE, ONE), (ONE, api.MOE_F32, 64, None, -1, ONE, ONE),
    (ONE + 2, api.MOE_F32, 64, None, 4, ONE, ONE), (ONE, api.MOE_F32, 64, ONE + 2, 4, ONE, ONE),
    (ONE, api.MOE_F32, 64, None, 4, None, ONE), (ONE, api.MOE_F32, 64, None, 4, ONE, ONE + 2)])
def test_route_refusals(lib, args):
    r = api.RouterDesc(64, 6, 1, 1, 1, 0, 1, 1.0)
    assert lib.moe_route_grouped(ctypes.byref(r), *args, None) == api.MOE_EINVAL


def test_wrappers_refuse_cpu_tensors():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        batch.PagedCache(k, k)
    with pytest.raises(ValueError):
        batch.BatchPlanner(16, 0, 4, device="cpu")
    with pytest.raises(ValueError):
        batch.GroupedRouter(8, 2, 4, score="relu")
    with pytest.raises(ValueError):
        api.make_cache(k, k[:, :, :, :32])
    with pytest.raises(ValueError):
        api.make_cache(k.transpose(2, 3), k.transpose(2, 3))
