"""A decoder block over verification steps of several requests.

Every step, each request brings its newest accepted token and a few drafted
ones (the first step: its prompt). One step runs, on one stream and without
reading anything back:

  plan    pages, slots and positions of the new tokens (BatchPlanner)
  append  their keys and values into the paged cache (PagedCache)
  attend  their attention over every request's cache (PagedAttention)
  route   gate, then grouped routing with sigmoid scores and a balance bias
          (GroupedRouter) into the expert layer's buffers
  experts the deduplicating engine and the combine (PassRunner)

The projections around the attention are plain matrix products. Weights are
random; a "verifier" accepts a random number of drafted tokens. Rejected
tokens leave their pages to the request: the next plan writes over them.

    python examples/verify_step.py [--requests 12] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import random
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from moe_expert_layer_warp_gb300 import api, synth                      # noqa: E402
from moe_expert_layer_warp_gb300.batch import (BatchPlanner, GroupedRouter,  # noqa: E402
                                               PagedAttention, PagedCache)
from moe_expert_layer_warp_gb300.configs import LayerShape, W_BF16      # noqa: E402
from moe_expert_layer_warp_gb300.layer import DEDUP, PassRunner         # noqa: E402

HEADS, KV_HEADS, DIM, PAGE = 8, 2, 64, 16
SHAPE = LayerShape(512, 32, 4, 256, 1, W_BF16)      # 32 routed experts top-4, 1 shared


class Block:
    """One decoder block's weights, cache and step."""

    def __init__(self, requests: int, max_tokens: int, max_blocks: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        d = SHAPE.d

        def weight(rows, cols):
            return torch.randn((rows, cols), generator=g, device="cuda") / rows ** 0.5

        self.w_qkv = weight(d, (HEADS + 2 * KV_HEADS) * DIM)
        self.w_out = weight(HEADS * DIM, d)
        pages = requests * max_blocks
        self.cache = PagedCache.allocate(pages, PAGE, KV_HEADS, DIM)
        self.planner = BatchPlanner(PAGE, requests, max_tokens)
        self.attention = PagedAttention(self.cache, HEADS, max_tokens)
        self.moe = PassRunner(synth.make_layer(SHAPE, seed + 1, "cuda"), max_tokens)
        bias = torch.randn(SHAPE.n_experts, generator=g, device="cuda") * 0.1
        self.router = GroupedRouter(SHAPE.n_experts, SHAPE.top_k, max_tokens, n_groups=4,
                                    top_groups=2, group_top=2, score="sigmoid", bias=bias,
                                    scale=2.0)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.zeros((requests, max_blocks), **i32)
        self.cached = torch.zeros(requests, **i32)
        self.held = torch.zeros(requests, **i32)
        self.free_pages = torch.randperm(pages, generator=g, device="cuda").int()
        self.free_range = torch.tensor([0, pages], **i32)

    def step(self, x: torch.Tensor, q_len: torch.Tensor):
        """x [T][d]: the new tokens' hidden states, request by request; q_len
        [B] int32 on the device. Returns (y [T][d], what the step computed)."""
        T = x.shape[0]
        plan = self.planner.plan(q_len, self.cached, self.held, self.free_pages, self.free_range,
                                 self.table, T)
        self.held.copy_(plan.held)
        self.free_range[:1].copy_(plan.free_head)
        qkv = (x @ self.w_qkv).view(T, HEADS + 2 * KV_HEADS, DIM)
        q = qkv[:, :HEADS].to(self.cache.dtype)
        k, v = qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
        self.cache.append(k, v, plan.slots)           # rounded from fp32 on the way
        y = self.attention.attend(q, plan.q_start, plan.kv_len, self.table)
        h = x + y.view(T, -1).float() @ self.w_out
        self.moe.route_grouped(h, self.router)
        self.moe.build_union(T)
        self.moe.experts(h, DEDUP)
        self.moe.combine(T)
        out = h + self.moe.y[: T * SHAPE.d].view(T, SHAPE.d)
        return out, {"plan": plan, "q": q, "k": k, "v": v, "attention": y, "h": h}

    def accept(self, n: torch.Tensor):
        """n [B] int32: the verifier keeps this many of each request's new tokens."""
        self.cached += n


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--requests", type=int, default=12)
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args(argv)
    # an expert pass takes 128 tokens at most: every request brings one at least
    if not 1 <= a.requests <= 128 or a.steps < 1:
        p.error("1 to 128 requests and one step at least")
    rng = random.Random(1)
    prompt, draft = min(10, 128 // a.requests), min(5, 128 // a.requests)
    # pages for the longest request: every draft kept
    block = Block(a.requests, max_tokens=min(128, a.requests * 10),
                  max_blocks=(prompt + a.steps * draft - 1) // PAGE + 1)
    total, timed_from = 0, min(2, a.steps - 1)            # the first steps warm up
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for step in range(a.steps):
        longest = prompt if step == 0 else draft
        q = [rng.randint(1, longest) for _ in range(a.requests)]
        x = torch.randn((sum(q), SHAPE.d), device="cuda")
        if step == timed_from:
            start.record()
        y, _ = block.step(x, torch.tensor(q, dtype=torch.int32, device="cuda"))
        kept = [n if step == 0 else rng.randint(1, n) for n in q]
        block.accept(torch.tensor(kept, dtype=torch.int32, device="cuda"))
        total += sum(kept) if step >= timed_from else 0
    end.record()
    status = api.moe_last_device_error()
    if status != api.MOE_OK:
        raise RuntimeError(api.status_str(status))
    ms = start.elapsed_time(end)
    print("%d requests, %d steps: %d tokens kept, %.0f tokens/s through the block, cache lengths %s"
          % (a.requests, a.steps, total, 1e3 * total / ms, block.cached.tolist()))


if __name__ == "__main__":
    main()
