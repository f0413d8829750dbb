"""The example's decoder block over several verification steps: pages are kept
and taken as planned, rejected drafts are written over, and every stage agrees
with its definition in 64 bits on what the stage before it computed."""
import random

import numpy as np
import pytest
import torch

from oracle import oracle as moe_oracle
from tests import batch_oracle

pytestmark = pytest.mark.gpu


def test_block_over_steps():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from examples import verify_step as ex
    from moe_expert_layer_warp_gb300 import api, build, synth
    build.build()
    B, rng = 6, random.Random(3)
    block = ex.Block(B, max_tokens=60, max_blocks=8, seed=5)
    L = block.moe.weights
    history = [[] for _ in range(B)]         # accepted keys and values, in the cache's type
    for step in range(6):
        q_len = [rng.randint(1, 10) if step == 0 else rng.randint(0, 6) for _ in range(B)]
        x = torch.randn((sum(q_len), ex.SHAPE.d), device="cuda")
        y, got = block.step(x, torch.tensor(q_len, dtype=torch.int32, device="cuda"))
        assert api.moe_last_device_error() == api.MOE_OK
        start = got["plan"].q_start.tolist()
        assert got["plan"].kv_len.tolist() == [len(h) + n for h, n in zip(history, q_len)]
        # attention, against the accepted history and the new tokens themselves
        new = [[(got["k"][start[b] + i].to(torch.bfloat16), got["v"][start[b] + i].to(torch.bfloat16))
                for i in range(q_len[b])] for b in range(B)]
        rows = [history[b] + new[b] for b in range(B)]
        longest = max(1, max(len(r) for r in rows))
        k = torch.zeros((B, longest, ex.KV_HEADS, ex.DIM), dtype=torch.bfloat16, device="cuda")
        v = torch.zeros_like(k)
        for b, r in enumerate(rows):
            for j, (kk, vv) in enumerate(r):
                k[b, j], v[b, j] = kk, vv
        want, bound = batch_oracle.attend(got["q"], k, v, start, [len(r) for r in rows],
                                          torch.arange(B, device="cuda")[:, None], ex.DIM ** -0.5,
                                          0, 0)
        err = (got["attention"].double() - want).abs()
        assert (err <= bound).all(), err.max()
        # routing, on the gate's own logits
        T = sum(q_len)
        logits = block.moe.logits[: T * ex.SHAPE.n_experts].view(T, -1).cpu()
        idx, w, wb = batch_oracle.route(logits, block.router.bias.cpu(), ex.SHAPE.top_k, 4, 2, 2,
                                        "sigmoid", True, 2.0)
        got_idx, got_w = block.moe.routing(T)
        np.testing.assert_array_equal(got_idx.cpu().numpy(), idx)
        assert (np.abs(got_w.cpu().double().numpy() - w) <= wb).all()
        # experts and combine, against the float64 oracle on that routing
        h = got["h"]
        y_moe = moe_oracle.moe_tokens(
            h.cpu().numpy(), got_idx.cpu().numpy(), got_w.cpu().double().numpy(),
            synth.weights_numpy(L.w_gate), synth.weights_numpy(L.w_up),
            synth.weights_numpy(L.w_down), synth.weights_numpy(L.ws_gate),
            synth.weights_numpy(L.ws_up), synth.weights_numpy(L.ws_down))
        out = (y - h).cpu().double().numpy()
        assert np.max(np.abs(out - y_moe)) <= 2e-2 * np.sqrt(np.mean(y_moe ** 2))
        # the verifier keeps some of the new tokens
        kept = [n if step == 0 else rng.randint(0, n) for n in q_len]
        block.accept(torch.tensor(kept, dtype=torch.int32, device="cuda"))
        for b in range(B):
            history[b] += new[b][: kept[b]]
    held = block.held.tolist()
    taken = [p for b in range(B) for p in block.table[b, : held[b]].tolist()]
    assert len(set(taken)) == len(taken), "a page given out twice"
    assert int(block.free_range[0]) == len(taken)


def test_router_of_another_layer_is_refused():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from examples import verify_step as ex
    from moe_expert_layer_warp_gb300.batch import GroupedRouter
    block = ex.Block(2, max_tokens=8, max_blocks=2)
    with pytest.raises(ValueError):
        block.moe.route_grouped(torch.zeros(3, ex.SHAPE.d, device="cuda"),
                                GroupedRouter(ex.SHAPE.n_experts, 2, 8))
