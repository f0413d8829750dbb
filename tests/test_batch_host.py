"""Host-only checks of include/moe_batch.h's entry points and their Python
objects beyond their refusals: nothing is launched (no GPU is touched)."""
import ctypes

import pytest

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
