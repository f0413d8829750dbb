"""GPU checks of include/moe_batch.h's operators where sizes, values and
neighbouring results come near what their types hold: windows and lengths near
2^31, choices closer than fp32 resolves, values that are not finite, padded
batches, replayed graphs, several streams and threads."""
import math

import numpy as np
import pytest
import torch

from tests import batch_oracle as oracle
from tests.test_batch_ops import B16, F16, Attend, _route, i32, lib  # noqa: F401

pytestmark = pytest.mark.gpu

NO_LIMIT = 2 ** 31 - 1


# ----------------------------------------------- windows and lengths --------
@pytest.mark.parametrize("window", [NO_LIMIT, NO_LIMIT - 100, 2 ** 30])
@pytest.mark.parametrize("q_len,kv_len,Hq,H,D,dtype,page,sinks", [
    ([5], [5], 4, 2, 64, B16, 16, 0),                 # the first tokens of a request
    ([300], [300], 4, 2, 128, B16, 64, 3),            # a fresh prompt
    ([3, 9], [40, 900], 8, 1, 128, F16, 32, 0),
    ([9, 200], [4, 150], 4, 2, 64, B16, 16, 2),       # caches shorter than the pass
    ([700, 3, 650], [700, 30, 2000], 64, 8, 64, F16, 16, 0),
])
def test_window_near_the_types_limit(lib, window, q_len, kv_len, Hq, H, D, dtype, page, sinks):
    a = Attend(q_len, kv_len, Hq, H, D, dtype, page, window=window, sinks=sinks)
    out = torch.full(a.q.shape, float("nan"), dtype=a.q.dtype, device="cuda")
    a.runner().attend(*a.args(), out=out)
    assert lib.moe_last_device_error() == lib.MOE_OK
    a.check(out)


def test_lengths_near_the_limit(lib):
    """A window at the end of the longest cache; a longer one is reported and
    its rows are zeros."""
    from moe_expert_layer_warp_gb300 import api
    page, most = 256, api.MOE_MAX_CACHE_LEN
    a = Attend([5], [512 + most % page], 4, 2, 64, B16, page, window=100)
    shift = most - a.kv_len[0]
    q, qs, kv, table = a.args()
    far = torch.full((1, (2 ** 31) // page), -1, dtype=torch.int32, device="cuda")
    far[0, shift // page:shift // page + table.shape[1] - 2] = table[0, :-2]
    r = a.runner()
    a.check(r.attend(q, qs, kv + shift, far))
    assert lib.moe_last_device_error() == lib.MOE_OK
    for more in (1, 2 ** 31 - 1 - most):
        out = r.attend(q, qs, kv + (shift + more), far)
        assert lib.moe_last_device_error() == lib.MOE_EDEVICE
        assert (out == 0).all()


# ------------------------------------------------------- padded batches -----
@pytest.mark.parametrize("q_len,kv_len,pad", [([3, 5], [40, 300], 7), ([0, 0], [5, 0], 4),
                                              ([400], [600], 300), ([2], [0], 1)])
def test_rows_of_no_request_are_zeros_in_the_objects_buffer(lib, q_len, kv_len, pad):
    """Padding rows of a batch of fixed size: neither what the buffer held at
    first nor an earlier call's results."""
    from moe_expert_layer_warp_gb300 import batch
    a = Attend(q_len, kv_len, 6, 2, 128, B16, 16)
    q, qs, kv, table = a.args()
    n = q.shape[0]
    wide = torch.cat([q, torch.randn(pad, *q.shape[1:], device="cuda").to(q.dtype)])
    r = batch.PagedAttention(batch.PagedCache(a.k, a.v), 6, n + pad)
    r.attend(wide, qs, kv, table).fill_(float("nan"))       # what an earlier call left
    out = r.attend(wide, qs, kv, table)
    assert lib.moe_last_device_error() == lib.MOE_OK
    assert (out[n:] == 0).all()
    a.check(out[:n])
