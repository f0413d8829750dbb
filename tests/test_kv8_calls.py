"""Calls of include/moe_kv8.h's Python objects and binding: what is refused before
anything is launched, and (on a GPU) new tensors of calls on other streams."""
import ctypes

import pytest
import torch

from moe_expert_layer_warp_gb300 import api, batch


def test_rotated_results_without_their_rows():
    """q_out is where q goes: given without q it would stay as it was."""
    rotary = batch.Rotary.__new__(batch.Rotary)
    x, positions = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32)
    for args in ((None, x, positions, x, None), (x, None, positions, None, x),
                 (None, x, positions, x, x)):
        with pytest.raises(ValueError, match="q_out and k_out"):
            rotary.rotate(*args)
    desc = api.RotaryDesc(64, 64, 0, 0, 1.0, 1 << 20)
    with pytest.raises(ValueError, match="q_out without q"):
        api.moe_rotary(desc, None, x, positions, q_out=x)
    with pytest.raises(ValueError, match="k_out without k"):
        api.moe_rotary(desc, x, None, positions, k_out=x)


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["stream", "number", "handle"])
def test_read_on_another_stream_takes_no_memory_in_use(how):
    """Tensors that are given up while their stream still has to read them are that
    stream's to use again, and not those of a read on another one."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from moe_expert_layer_warp_gb300 import build
    build.build()
    n, H, D = 8192, 4, 128
    cache = batch.PagedCache8.allocate(n // 64, 64, H, D)
    for x in (cache.k, cache.v):
        x.view(torch.uint8).fill_(0x30)                    # 0.5
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(1.0)
    slots = torch.arange(n, device="cuda")
    side = torch.cuda.Stream()
    stream = {"stream": side, "number": side.cuda_stream,
              "handle": ctypes.c_void_p(side.cuda_stream)}[how]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    kept = [torch.empty(n, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    held = [torch.full((n, H, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                         # some 50 ms before they are read
    for y, x in zip(kept, held):
        y.copy_(x)
    del held, x
    k, v = cache.read(slots, stream=stream)
    side.synchronize()
    assert (k == 0.5).all() and (v == 0.5).all()
    torch.cuda.synchronize()
    assert all((y == 7.0).all() for y in kept)
    assert api.moe_last_device_error() == api.MOE_OK
