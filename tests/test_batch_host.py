"""Host-only checks of include/moe_batch.h's entry points and their Python
objects beyond their refusals: nothing is launched (no GPU is touched)."""
import ctypes

import pytest
import torch

from moe_expert_layer_warp_gb300 import api, batch
from tests.test_batch_abi import ONE, _cache, _why, lib  # noqa: F401


@pytest.mark.parametrize("at,value,reason", [
    (0, ONE + 8, "q or out"), (1, 100, "q strides"), (8, 0, "n_requests"), (10, 16, "workspace"),
    (13, 32, "out strides")])
def test_padded_attend_refuses_what_attend_refuses(lib, at, value, reason):
    c, a = _cache(), api.AttnDesc(8, 0, 0, 0.125)
    args = [ONE, 512, 64, 4, ONE, ONE, ONE, 4, 2, ONE, 1 << 30, ONE, 512, 64]
    args[at] = value
    assert lib.moe_attend_padded(ctypes.byref(c), ctypes.byref(a), *args, None) == api.MOE_EINVAL
    assert reason in _why() and "moe_attend_padded" in _why()


def test_objects_of_another_device_than_the_current_one_are_refused(monkeypatch):
    monkeypatch.setattr(batch, "_several_devices", True)
    monkeypatch.setattr(batch, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
        batch._handle(None, 1)
    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
        batch._handle(ctypes.c_void_p(0), 1)
    assert batch._handle(ctypes.c_void_p(5), 0).value == 5


@pytest.mark.parametrize("token,head,ok", [
    (512, 64, True), (504, 64, False),                  # tokens of 8 heads of 64, dense
    (960, 128, True), (952, 128, False),                # every other one of 15 heads
    (64, 256, True), (64, 248, False),                  # heads of 4 tokens, dense
    (128, 448, True), (128, 440, False),                # every other one of 7 tokens
    (512, 1 << 61, True), (1 << 61, 1 << 61, False), (1 << 61, 64, True), (0, 64, False),
    (-512, 64, False)])
def test_attend_out_strides(lib, token, head, ok):
    """Rows apart are taken whatever lies between them, rows that overlap are
    not. (Accepted strides get as far as the missing q.)"""
    c, a = _cache(), api.AttnDesc(8, 0, 0, 0.125)
    assert lib.moe_attend(ctypes.byref(c), ctypes.byref(a), None, 512, 64, 4, ONE, ONE, ONE, 4, 2,
                          ONE, 1 << 30, ONE, token, head, None) == api.MOE_EINVAL
    assert ("q or out null" if ok else "out strides") in _why()


def test_binding_refuses_tensors_of_another_kind(lib):
    """What the calls cannot see: types and shapes behind the pointers. (None of
    these tensors is on a GPU; each refusal comes before that is asked.)"""
    B16, I32 = torch.bfloat16, torch.int32
    c, a = _cache(), api.AttnDesc(8, 0, 0, 0.125)
    q, ws = torch.zeros(4, 8, 64, dtype=B16), torch.zeros(16, dtype=torch.uint8)
    start, length, table = (torch.zeros(n, dtype=I32) for n in (3, 2, 8))
    table = table.view(2, 4)
    good = dict(q=q, q_start=start, kv_len=length, block_table=table, workspace=ws, out=q)
    for over, reason in [
            (dict(q=q.half(), out=q.half()), "cache's type"), (dict(q=q[:, :7], out=q[:, :7]), "q"),
            (dict(out=q[:3]), "out"), (dict(out=q.float()), "out"),
            (dict(q_start=start[:2]), "q_start"), (dict(kv_len=length.long()), "kv_len"),
            (dict(block_table=table[0]), "block_table"),
            (dict(q=q.transpose(0, 2).contiguous().transpose(0, 2)), "contiguous")]:
        for padded in (False, True):
            with pytest.raises(ValueError, match=reason):
                api.moe_attend(c, a, **dict(good, **over), padded=padded)
    k, slots = torch.zeros(4, 2, 64, dtype=B16), torch.zeros(4, dtype=torch.int64)
    for args, reason in [((k[:, :1], k[:, :1], slots), "k must"), ((k, k.float(), slots), "v must"),
                         ((k, k, slots[:3]), "slots"), ((k, k, slots.int()), "slots"),
                         ((k.double(), k.double(), slots), "float32"),
                         ((k, k.transpose(0, 1).contiguous().transpose(0, 1), slots), "strides")]:
        with pytest.raises(ValueError, match=reason):
            api.moe_kv_append(c, *args)
    r = api.RouterDesc(8, 2, 1, 1, 1, 0, 1, 1.0)
    x, idx, w = torch.zeros(3, 8), torch.zeros(3, 2, dtype=I32), torch.zeros(3, 2)
    for args, reason in [((x[:, :7], None, idx, w), "logits"), ((x.double(), None, idx, w), "logits"),
                         ((x, x[0].half(), idx, w), "bias"), ((x, None, idx.long(), w), "topk_idx"),
                         ((x, None, idx, w[:2]), "topk_w")]:
        with pytest.raises(ValueError, match=reason):
            api.moe_route_grouped(r, *args)
    with pytest.raises(ValueError, match="slots"):
        api.moe_plan_batch(api.BatchC(), 4, slots.int(), slots.int())
    with pytest.raises(ValueError, match="positions"):
        api.moe_plan_batch(api.BatchC(), 4, slots, slots)
