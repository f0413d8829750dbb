"""GPU checks of include/moe_kv8.h's operators against their definitions in 64
bits (tests/kv8_oracle.py), at the sizes and masks where they can go wrong.
Tolerances are the oracle's bounds; codes and scales are exact."""
import functools
import math

import numpy as np
import pytest
import torch

from tests import kv8_oracle as oracle

pytestmark = pytest.mark.gpu

B16, F16, F32, CODE = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from moe_expert_layer_warp_gb300 import api, build
    build.build()
    assert api.moe_last_device_error() == api.MOE_OK
    return api


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def i64(v):
    return torch.tensor(v, dtype=torch.int64, device="cuda")


# ------------------------------------------------------------------ rotary --
def _positions(n, far, seed=0):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, far + 1, (n,), generator=g, dtype=torch.int64)
    p[0] = far
    if n > 3:
        p[1], p[2] = 0, -1                       # the first position, and padding
    return p.int()


ROTARIES = {
    "whole heads": dict(n=7, H=4, K=2, D=128, r=128),
    "one token": dict(n=1, H=1, K=1, D=64, r=64),
    "first half": dict(n=33, H=5, K=1, D=128, r=64),
    "last half": dict(n=9, H=4, K=4, D=128, r=64, first=64),
    "columns inside": dict(n=9, H=3, K=2, D=192, r=48, first=72),
    "narrow": dict(n=20, H=2, K=0, D=80, r=16),
    "wide": dict(n=5, H=2, K=1, D=1024, r=1024),
    "far": dict(n=300, H=2, K=1, D=64, r=64, far=1000000),
    "farthest": dict(n=9, H=2, K=1, D=64, r=64, far=2 ** 31 - 1, base=4.0),
    "amplified": dict(n=9, H=2, K=1, D=64, r=32, far=5000, amplitude=1.25),
    "turned back": dict(n=9, H=2, K=1, D=64, r=64, far=5000, sign=-1.0),
    "many tokens": dict(n=3001, H=3, K=1, D=64, r=64, far=3000),
    # several tokens a CTA: one piece a head, and counts that are no powers of two
    "many tokens, one piece a head": dict(n=8003, H=3, K=1, D=16, r=16, far=9000),
    "many tokens, one head": dict(n=6001, H=1, K=0, D=16, r=16, far=9000),
    "many tokens, odd heads": dict(n=5003, H=7, K=3, D=80, r=48, first=8, far=9000),
    "many heads": dict(n=1300, H=70, K=5, D=192, r=96, first=96, far=9000),
}


@pytest.mark.parametrize("dtype", [F32, B16, F16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("name", ROTARIES)
def test_rotary(lib, name, interleaved, dtype):
    from moe_expert_layer_warp_gb300 import batch
    c = dict(dict(first=0, far=100, amplitude=1.0, base=10000.0, sign=1.0), **ROTARIES[name])
    n, H, K, D = c["n"], c["H"], c["K"], c["D"]
    radians = [c["sign"] * v for v in batch.rotary_frequencies(c["r"], c["base"])]
    r = batch.Rotary(D, c["r"], radians, c["first"], interleaved, c["amplitude"])
    pos = _positions(n, c["far"])
    g = torch.Generator().manual_seed(n)
    joint = torch.randn((n, H + 2 * K + 1, D), generator=g).to(dtype).cuda()
    q, k = joint[:, :H], joint[:, H:H + K]
    want = [oracle.rotate(x, pos, radians, c["first"], interleaved, c["amplitude"])
            for x in (q, k)]
    q_out, k_out = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    got = r.rotate(q, k if K else None, pos.cuda(), q_out=q_out, k_out=k_out if K else None)
    assert got[0] is q_out and lib.moe_last_device_error() == lib.MOE_OK
    for x, (y, bound) in zip((q_out, k_out), want):
        over = (x.double() - y).abs() - bound
        assert x.numel() == 0 or (over <= 0).all(), "off by %.3g" % (x.double() - y).abs().max()
    # in place: the same bits, and what lies between is left
    rest = joint[:, H + K:].clone()
    assert r.rotate(q, k if K else None, pos.cuda())[0] is q
    assert torch.equal(q, q_out) and (K == 0 or torch.equal(k, k_out))
    assert torch.equal(joint[:, H + K:], rest)


def test_rotary_of_keys_alone_and_of_no_token(lib):
    from moe_expert_layer_warp_gb300 import batch
    r = batch.Rotary(64)
    k = torch.randn(3, 2, 64, device="cuda")
    y, bound = oracle.rotate(k, torch.tensor([5, 6, 7]), r.frequencies, 0, False, 1.0)
    assert r.rotate(None, k, i32([5, 6, 7]))[0] is None
    assert ((k.double() - y).abs() <= bound).all()
    r.rotate(torch.empty(0, 2, 64, device="cuda"), None, i32([]))
    with pytest.raises(ValueError):
        r.rotate(None, None, i32([1]))
    with pytest.raises(ValueError):
        r.rotate(k, k.half(), i32([5, 6, 7]))
    with pytest.raises(lib.MoeError):            # rows that share their memory
        r.rotate(k[:1].expand(3, 2, 64), None, i32([5, 6, 7]))


def test_rotary_keeps_scores_of_equal_distances(lib):
    """What rotary positions are for: a score depends on the distance alone."""
    from moe_expert_layer_warp_gb300 import batch
    r = batch.Rotary(128, frequencies=batch.rotary_frequencies(128, scaling="ramp", factor=8.0))
    q, k = (torch.randn(1, 1, 128, device="cuda").expand(40, 1, 128).contiguous() for _ in range(2))
    p = torch.arange(40, device="cuda", dtype=torch.int32) * 25013
    r.rotate(q, k, p)
    r.rotate(None, k, torch.full((40,), 3, dtype=torch.int32, device="cuda"))
    s = (q * k).double().sum((1, 2))
    assert (s - s[0]).abs().max() <= 2.0 ** -18 * (q.norm() ** 2 + k.norm() ** 2) / 40


# ------------------------------------------------------------------ append --
def _pool(pages, page, H, D, block, heads_first, seed=0):
    """Codes of every kind but NaN, and scales in their range."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        shape = (pages, H, page, D) if heads_first else (pages, page, H, D)
        codes = torch.randint(0, 256, shape, generator=g).to(torch.uint8)
        codes[(codes & 127) == 127] = 3
        codes = codes.cuda().view(CODE)
        e = torch.randint(-9, 3, (pages, H, page // block), generator=g).float()
        out += [codes.transpose(1, 2) if heads_first else codes, torch.exp2(e).cuda()]
    return out[0], out[2], out[1], out[3]        # k, v, k_scale, v_scale


def _same(got, want):
    """Equal values, NaN in the same places."""
    got = got.cpu().double()
    return torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(
        torch.nan_to_num(got, nan=0.0), torch.nan_to_num(want, nan=0.0))


def _check_pool(cache, pools):
    for codes, scales, p in ((cache.k, cache.k_scale, pools[0]), (cache.v, cache.v_scale, pools[1])):
        assert torch.equal(torch.frexp(scales.cpu())[1].long() - 1, p.exp)
        assert torch.equal(scales.cpu().double(), torch.exp2(p.exp.double()))
        assert _same(codes.cpu().float(), p.code)


def _slots(pages, page, q_len, cached, seed=0):
    """Slots of requests' new tokens over pages in random places, -1 for a request of -n."""
    ids = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    out, at = [], 0
    for n, m in zip(q_len, cached):
        mine = ids[at:at + -(-(m + abs(n)) // page)]
        at += len(mine)
        out += [mine[i // page] * page + i % page if n > 0 else -1 for i in range(m, m + abs(n))]
    return out


APPENDS = {
    "one token, first of its block": dict(q=[1], cached=[0]),
    "one token inside a block": dict(q=[1], cached=[5]),
    "passes": dict(q=[9, 9, 1, 5], cached=[0, 30, 15, 7], H=3, D=128, page=32),
    "block edges": dict(q=[1, 2, 17, 16, 33], cached=[15, 15, 15, 16, 31], page=64),
    "refused requests": dict(q=[4, -3, 5, -20, 2], cached=[0, 3, 9, 0, 14]),
    "prompt": dict(q=[300], cached=[77], H=2, D=128, page=64, block=32),
    "a block is a page of 256": dict(q=[700, 3], cached=[100, 250], page=256, block=256, H=2),
    "blocks of 128": dict(q=[129, 255], cached=[0, 1], page=128, block=128, D=128),
    "many": dict(q=[1 + i % 70 for i in range(60)], cached=[i * 7 % 130 for i in range(60)], H=8,
                 page=64, block=16),
}


@pytest.mark.parametrize("src", [F32, B16, F16])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("name", APPENDS)
def test_append_and_read(lib, name, heads_first, src):
    from moe_expert_layer_warp_gb300 import batch
    c = dict(dict(H=1, D=64, page=16, block=16), **APPENDS[name])
    H, D, page, block = c["H"], c["D"], c["page"], c["block"]
    pages = sum(-(-(m + abs(n)) // page) for n, m in zip(c["q"], c["cached"])) + 2
    cache = batch.PagedCache8(*_pool(pages, page, H, D, block, heads_first))
    pools = [oracle.Pool.of(cache.k, cache.k_scale, block),
             oracle.Pool.of(cache.v, cache.v_scale, block)]
    slots = _slots(pages, page, c["q"], c["cached"])
    n = len(slots)
    g = torch.Generator().manual_seed(n)
    x = torch.randn((n, 3, H, D), generator=g)
    x *= torch.exp2(torch.randn((n, 3, H, 1), generator=g) * 4)     # scales grow, and do not
    x = x.to(src).cuda()
    for k, v in ((x[:, 0], x[:, 1]), (x[:, 1], x[:, 2])):           # and written over once more
        cache.append(k, v, i64(slots))
        pools[0].append(k, slots)
        pools[1].append(v, slots)
        assert lib.moe_last_device_error() == lib.MOE_OK
        _check_pool(cache, pools)
    # reading back: any rows, some twice, some missing
    rows = slots + [-1, pages * page - 1, 0] + slots[:3]
    for dtype in (F32, B16, F16):
        k, v = cache.read(i64(rows), dtype=dtype)
        assert lib.moe_last_device_error() == lib.MOE_OK and k.dtype is dtype
        for got, p in ((k, pools[0]), (v, pools[1])):
            assert _same(got, p.values(rows).to(dtype).double())


def test_append_values_that_are_not_finite(lib):
    """NaN and infinities become NaN and have no part in the scale; a block of zeros
    has the least one; what is beyond the largest one is held at 448 · 2^50."""
    from moe_expert_layer_warp_gb300 import batch
    cache = batch.PagedCache8(*_pool(4, 32, 1, 64, 16, False))
    pools = [oracle.Pool.of(cache.k, cache.k_scale, 16), oracle.Pool.of(cache.v, cache.v_scale, 16)]
    x = torch.randn(40, 1, 64)
    x[0, 0, :4] = torch.tensor([math.nan, math.inf, -math.inf, -0.0])
    x[5] = 0.0
    x[16:32] = 0.0
    x[33, 0, 0], x[34, 0, 1], x[35, 0, 2] = 3e38, -1e20, 1e-38
    slots = list(range(16, 32)) + list(range(0, 16)) + list(range(64, 72))
    v = torch.flip(x, (2,))
    cache.append(x.cuda(), v.cuda(), i64(slots))
    pools[0].append(x, slots)
    pools[1].append(v, slots)
    _check_pool(cache, pools)
    assert int(pools[0].exp[0, 0, 0]) == -50 and int(pools[0].exp[2, 0, 0]) == 50
    # a part of a block with nothing but such values leaves its scale
    y = torch.full((2, 1, 64), math.inf)
    cache.append(y.cuda(), y.cuda(), i64([18, 19]))
    pools[0].append(y, [18, 19])
    pools[1].append(y, [18, 19])
    _check_pool(cache, pools)


def test_append_largest_sizes_at_the_border(lib):
    """A = 448 · 2^e to the bit, and one step above."""
    from moe_expert_layer_warp_gb300 import batch
    cache = batch.PagedCache8(*_pool(8, 16, 1, 64, 16, False))
    pools = [oracle.Pool.of(cache.k, cache.k_scale, 16), oracle.Pool.of(cache.v, cache.v_scale, 16)]
    x = torch.randn(8, 1, 64) * 0.25
    for i in range(8):
        a = torch.tensor(448.0 * 2.0 ** (i - 8))
        x[i, 0, 3] = a if i % 2 else torch.nextafter(a, torch.tensor(1e9))
    slots = [16 * i for i in range(8)]
    cache.append(x.cuda(), x.cuda(), i64(slots))
    pools[0].append(x, slots)
    pools[1].append(x, slots)
    _check_pool(cache, pools)


def test_slots_out_of_range_are_skipped_and_reported(lib):
    from moe_expert_layer_warp_gb300 import batch
    cache = batch.PagedCache8(*_pool(2, 16, 1, 64, 16, False))
    p = oracle.Pool.of(cache.k, cache.k_scale, 16)
    x = torch.ones(3, 1, 64, device="cuda")
    cache.append(x, x, i64([32, 4, -7]))
    assert lib.moe_last_device_error() == lib.MOE_EDEVICE
    p.append(x, [-1, 4, -1])
    assert _same(cache.k.cpu().float(), p.code)
    k, _ = cache.read(i64([32, 4, -7]), dtype=F32)
    assert lib.moe_last_device_error() == lib.MOE_EDEVICE
    assert _same(k, p.values([-1, 4, -1]))
    cache.append(x[:0], x[:0], i64([]))
    assert cache.read(i64([]))[0].shape == (0, 1, 64)
    assert lib.moe_last_device_error() == lib.MOE_OK


def test_read_into_given_rows(lib):
    """Values inside a wider row, heads apart; what lies between is left."""
    from moe_expert_layer_warp_gb300 import batch
    cache = batch.PagedCache8(*_pool(3, 32, 2, 64, 32, True))
    wide = torch.full((5, 3, 2, 96), 9.0, dtype=B16, device="cuda")
    slots = [40, 3, -1, 95, 3]
    k, v = wide[:, 0, :, 16:80], wide[:, 2, :, 16:80]
    assert cache.read(i64(slots), k=k, v=v)[0] is k
    p = oracle.Pool.of(cache.k, cache.k_scale, 32)
    assert _same(k, p.values(slots).to(B16).double())
    assert (wide[:, 1] == 9).all() and (wide[..., :16] == 9).all() and (wide[..., 80:] == 9).all()
    with pytest.raises(ValueError):
        cache.read(i64(slots), k=k)
    with pytest.raises(lib.MoeError):
        cache.read(i64(slots), k=k[:1].expand(5, 2, 64), v=v[:1].expand(5, 2, 64))


# --------------------------------------------------------------- attention --
class Attend:
    """One attention problem: packed queries over pages of codes in random
    places; NaN in every code that no new token sees."""

    def __init__(self, q_len, kv_len, Hq, H, D, dtype, page, block=16, heads_first=False, window=0,
                 sinks=0, scale=None, spread=1.0, sizes=0.7, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.q_len, self.kv_len, self.page, self.block = q_len, kv_len, page, block
        self.window, self.sinks = window, sinks
        blocks = [-(-m // page) for m in kv_len]
        n_pages, M = sum(blocks) + 3, max(max(blocks), 1) + 2
        ids = torch.randperm(n_pages, generator=g)
        self.table, at = torch.full((len(kv_len), M), -1, dtype=torch.int32), 0
        self.scale = D ** -0.5 if scale is None else scale
        self.pools = [oracle.Pool(n_pages, page, H, D, block) for _ in range(2)]
        for b, m in enumerate(kv_len):
            self.table[b, :blocks[b]] = ids[at:at + blocks[b]]
            at += blocks[b]
            first = m - q_len[b]
            lo = max(0, first - window + 1) if window else 0
            j = torch.arange(m)
            seen = (j >= lo) | (j < sinks) if q_len[b] else j < 0
            pages, rows = self.table[b].long()[j // page][seen], (j % page)[seen]
            # pages without a key that a new token sees are not to be read
            used = torch.zeros(M, dtype=torch.bool)
            used[(j // page)[seen]] = True
            self.table[b][~used] = -1
            for p in self.pools:
                x = torch.randn((pages.numel(), H, D), generator=g, dtype=torch.float64)
                x *= torch.exp2(torch.randn((pages.numel(), H, 1), generator=g) * sizes)
                p.code[pages, rows] = x
        for p in self.pools:                 # from values to codes and scales
            x = p.code.view(n_pages, page // block, block, H, D)
            top = torch.nan_to_num(x, nan=0.0).abs().amax((2, 4))
            e = torch.tensor([[[oracle.exponent(float(v)) for v in w] for w in z] for z in top])
            p.exp = e.permute(0, 2, 1).contiguous()
            p.code = oracle.e4m3(x * torch.exp2(-e.double())[:, :, None, :, None]).view_as(p.code)
        self.q_start = [0]
        for n in q_len:
            self.q_start.append(self.q_start[-1] + n)
        self.q = (torch.randn((self.q_start[-1], Hq, D), generator=g) * spread).to(dtype)
        self.heads_first = heads_first

    def cache(self):
        from moe_expert_layer_warp_gb300 import batch
        out = []
        for p in self.pools:
            c = p.code.float().to(CODE).cuda()
            if self.heads_first:
                c = c.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(CODE)
            out += [c, torch.exp2(p.exp.float()).cuda()]
        return batch.PagedCache8(out[0], out[2], out[1], out[3])

    def runner(self):
        from moe_expert_layer_warp_gb300 import batch
        return batch.PagedAttention8(self.cache(), self.q.shape[1], self.q.shape[0],
                                     dtype=self.q.dtype, scale=self.scale, window=self.window,
                                     sinks=self.sinks)

    def args(self):
        return self.q.cuda(), i32(self.q_start), i32(self.kv_len), self.table.cuda()

    def want(self):
        k, v = (torch.nan_to_num(p.all_values(), nan=0.0).cuda() for p in self.pools)
        vs = torch.exp2(self.pools[1].exp.double()).permute(0, 2, 1)
        vs = vs.repeat_interleave(self.block, dim=1).cuda()
        return oracle.attend(self.q.cuda(), k, v, vs, self.q_start, self.kv_len, self.table.cuda(),
                             self.scale, self.window, self.sinks)

    def check(self, got):
        want, bound = self.want()
        got = got.double()
        assert torch.isfinite(got).all()
        over = (got - want).abs() - bound
        assert (over <= 0).all(), "off by %.3g beyond %.3g at %s" % (
            (got - want).abs().max(), bound.max(), np.unravel_index(int(over.argmax().cpu()),
                                                                    over.shape))


def spec(*args, **kwargs):     # of an Attend, which is built on the GPU
    return args, kwargs


ATTENDS = {
    "one token, one key": spec([1], [1], 1, 1, 64, B16, 16),
    "one token": spec([1], [130], 4, 2, 128, F16, 16),
    "one token, one head": spec([1], [700], 1, 1, 128, B16, 64),
    "pass of five": spec([5], [77], 16, 16, 128, B16, 64),
    "first tokens of a request": spec([9], [9], 8, 2, 64, B16, 16),
    "tile edges": spec([1, 2, 3, 1, 2, 3, 1], [127, 128, 129, 255, 256, 257, 64], 8, 2, 64, F16,
                       64, heads_first=True),
    "ragged passes": spec([1, 9, 5, 3, 16, 2], [700, 33, 5, 1030, 128, 450], 8, 2, 128, B16, 32),
    "ragged passes, a scale for a page": spec([1, 9, 5, 3, 16, 2], [700, 33, 5, 1030, 128, 450], 8,
                                              2, 128, B16, 256, block=256),
    "blocks of 64": spec([3, 40], [300, 500], 8, 2, 64, F16, 128, block=64),
    "blocks of 128": spec([3, 40], [300, 500], 8, 2, 128, F16, 256, block=128, heads_first=True),
    "seven heads per key head": spec([4, 20], [50, 300], 14, 2, 64, F16, 16),
    "three heads per key head": spec([50], [190], 3, 1, 128, B16, 128),
    "sixteen heads, one key head": spec([7, 9], [300, 200], 16, 1, 128, B16, 256),
    "64 heads per key head": spec([3], [150], 64, 1, 64, B16, 64),
    "48 heads per key head": spec([6, 1], [40, 400], 96, 2, 128, F16, 64),
    "33 heads per key head": spec([2, 1], [300, 400], 33, 1, 128, B16, 16),
    "chunk": spec([300], [300], 2, 2, 128, B16, 64),
    "chunk over a cache": spec([200, 77], [520, 500], 4, 1, 64, F16, 16, heads_first=True),
    "chunk beside passes": spec([1, 260, 4], [600, 413, 90], 8, 4, 128, B16, 16),
    "empty requests": spec([3, 0, 2, 0], [0, 0, 40, 70], 4, 2, 64, B16, 16),
    "only empty rows": spec([3, 5], [0, 0], 4, 2, 128, B16, 16),
    "cache shorter than the pass": spec([6, 300], [4, 140], 4, 2, 64, B16, 16),
    "window of one": spec([5, 140], [60, 300], 4, 2, 64, B16, 16, window=1),
    "window": spec([5, 9, 1], [700, 45, 129], 8, 2, 128, F16, 16, window=40),
    "window and sinks": spec([5, 9, 1], [700, 45, 390], 8, 2, 128, B16, 16, window=40, sinks=4),
    "sinks past a tile": spec([5, 200], [900, 700], 4, 2, 64, B16, 64, window=33, sinks=130),
    "sinks alone beside one": spec([3], [400], 4, 1, 64, F16, 128, window=1, sinks=1),
    "window over a chunk": spec([400], [650], 4, 2, 128, B16, 32, window=100, sinks=3),
    "window longer than the cache": spec([5], [200], 4, 2, 64, B16, 16, window=5000, sinks=9),
    "peaked scores": spec([9, 150], [800, 400], 4, 2, 128, B16, 64, spread=12.0),
    "peaked scores in fp16": spec([9, 150], [800, 400], 4, 2, 128, F16, 64, spread=12.0),
    "large scale": spec([4], [300], 4, 2, 64, B16, 16, scale=3.0),
    "tiny scale": spec([4], [300], 4, 2, 64, F16, 16, scale=1e-20),
    "small queries": spec([4], [300], 4, 2, 64, B16, 16, spread=1e-18, scale=1e18),
    "large queries": spec([4], [300], 4, 2, 128, B16, 16, spread=1e18, scale=1e-19),
    "blocks of very different sizes": spec([4, 60], [300, 700], 4, 2, 128, B16, 16, sizes=5.0),
    "blocks of different sizes in fp16": spec([4, 60], [300, 700], 4, 2, 64, F16, 16, sizes=3.0),
    # several tiles and several items per CTA
    "many passes": spec([1 + i % 9 for i in range(40)], [100 + 97 * i for i in range(40)], 16, 4,
                        128, B16, 64),
    "many single tokens": spec([1] * 150, [100 + 37 * i for i in range(150)], 32, 8, 128, B16, 64,
                               block=64),
    "many passes, small pages": spec([1 + i % 5 for i in range(60)], [3000 - 49 * i for i in
                                     range(60)], 12, 4, 64, F16, 16, heads_first=True),
    "long chunks": spec([900, 1100], [2600, 1100], 8, 2, 128, B16, 64),
    "long chunks, odd groups": spec([700, 333, 40], [3000, 333, 2000], 15, 3, 64, F16, 32),
    "mixed batch": spec([500, 3, 9, 0, 260, 1] + [4] * 30, [1500, 0, 2500, 9, 2000, 1] +
                        [600 + 31 * i for i in range(30)], 28, 4, 128, F16, 16),
    "many windows": spec([1 + i % 9 for i in range(40)], [200 + 190 * i for i in range(40)], 16,
                         4, 64, B16, 16, window=700, sinks=5),
    "long windows over chunks": spec([1500, 800], [2500, 4000], 8, 4, 128, B16, 128, block=128,
                                     window=900, sinks=200),
    "peaked long chunks": spec([900, 1100], [2600, 1500], 8, 2, 128, F16, 64, spread=10.0),
    "short items": spec([1 + i % 7 for i in range(120)], [1 + (i * 37) % 300 for i in range(120)],
                        16, 8, 128, B16, 16),
    "short items, odd heads": spec([1 + i % 3 for i in range(200)], [0 if i % 9 == 4 else 200 + i
                                   for i in range(200)], 9, 3, 64, F16, 32, heads_first=True),
    "short items, windows": spec([i % 6 for i in range(150)], [40 + 11 * i for i in range(150)], 28,
                                 4, 64, B16, 256, block=32, window=200, sinks=2),
    "many tokens that see nothing": spec([3, 400, 5, 0, 260, 2, 333], [300, 0, 90, 50, 30, 700, 0],
                                         14, 2, 64, F16, 16),
    "nothing but the last sees": spec([40, 300, 1], [0, 0, 1], 8, 2, 128, B16, 64),
    "nothing behind the first sees": spec([1, 300, 40], [200, 0, 0], 8, 2, 64, B16, 16),
    "chunks longer than their caches": spec([700, 300, 65, 9], [1, 120, 64, 8], 28, 4, 128, B16,
                                            32),
    "widest window and sinks": spec([9, 200, 1], [700, 300, 129], 8, 2, 64, B16, 16,
                                    window=2 ** 31 - 1, sinks=2 ** 31 - 1),
    "window and widest sinks": spec([9, 200, 1], [700, 300, 129], 8, 2, 64, B16, 16, window=20,
                                    sinks=2 ** 31 - 1),
    "requests of different widths": spec([1, 16, 4, 1, 8, 200, 1, 2, 31], [900, 800, 700, 600, 500,
                                         400, 300, 200, 100], 8, 2, 128, B16, 32, block=32),
}


@functools.lru_cache(maxsize=None)
def problem(name):
    args, kwargs = ATTENDS[name]
    return Attend(*args, **kwargs)


@pytest.mark.parametrize("name", ATTENDS)
def test_attend(lib, name):
    a = problem(name)
    r = a.runner()
    out = torch.full(a.q.shape, float("nan"), dtype=a.q.dtype, device="cuda")
    r.attend(*a.args(), out=out)
    assert lib.moe_last_device_error() == lib.MOE_OK
    a.check(out)
    again = r.attend(*a.args())
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


def test_attend_rising_scores(lib):
    """Every key scores above all before it: the running maximum grows at every
    step."""
    a = Attend([3, 130], [700, 400], 2, 1, 64, B16, 16, spread=0.0)
    for b, m in enumerate(a.kv_len):
        for j in range(m):
            page, row = int(a.table[b, j // 16]), j % 16
            a.pools[0].code[page, row] = 0
            a.pools[0].code[page, row, :, 0] = 8 + j // 16 % 8      # an e4m3 number
            a.pools[0].exp[page, :, 0] = j // 128
    a.q[:, :, 0] = 4.0
    a.check(a.runner().attend(*a.args()))


def test_attend_leaves_rows_of_no_request(lib):
    a = problem("ragged passes")
    q, qs, kv, table = a.args()
    wide = torch.cat([q[:1], q, q[:2]])
    out = torch.full(wide.shape, 7.0, dtype=q.dtype, device="cuda")
    r = a.runner()
    r.attend(wide, qs + 1, kv, table, out=out)
    a.check(out[1:-2])
    assert (out[-2:] == 7.0).all() and (out[0] == 7.0).all()
    from moe_expert_layer_warp_gb300 import batch
    r = batch.PagedAttention8(a.cache(), q.shape[1], wide.shape[0], dtype=q.dtype)
    r._out.fill_(7.0)
    own = r.attend(wide, qs + 1, kv, table)
    assert torch.equal(own[1:-2], out[1:-2]) and (own[-2:] == 0).all() and (own[0] == 0).all()


def test_attend_strides(lib):
    """Queries inside a joint projection, results in [heads][tokens] order."""
    a = problem("chunk beside passes")
    q, qs, kv, table = a.args()
    T, H, D = q.shape
    joint = torch.randn(T, H + 8, D, device="cuda").to(q.dtype)
    joint[:, 3:3 + H] = q
    out = torch.empty(H, T, D, dtype=q.dtype, device="cuda").transpose(0, 1)
    a.runner().attend(joint[:, 3:3 + H], qs, kv, table, out=out)
    a.check(out)


def test_attend_other_stream_and_graph(lib):
    a = problem("window and sinks")
    r, args = a.runner(), a.args()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros(a.q.shape, dtype=a.q.dtype, device="cuda")
    torch.cuda.synchronize()
    r.attend(*args, out=out, stream=side)
    side.synchronize()
    a.check(out)
    out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.attend(*args, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        a.check(out)


def test_attend_two_at_once(lib):
    """Two calls in flight at a time, each with its workspace: the bits of one
    after the other."""
    problems = [problem("many passes"), problem("mixed batch")]
    runs = [(a.runner(), a.args(), torch.cuda.Stream()) for a in problems]
    want = [r.attend(*args).clone() for r, args, _ in runs]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for (r, args, stream), out in zip(runs, outs):
            r.attend(*args, out=out, stream=stream)
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert torch.equal(out.view(torch.int16), w.view(torch.int16))
            out.zero_()
        torch.cuda.synchronize()
    assert lib.moe_last_device_error() == lib.MOE_OK


def test_graph_of_steps_while_requests_grow(lib):
    """One captured step of rotate, append, attend and read, replayed with other
    tokens, positions, slots and lengths: the bits of steps without a graph."""
    from moe_expert_layer_warp_gb300 import batch
    B, H, K, D, page, n = 3, 8, 2, 64, 16, 10
    g = torch.Generator().manual_seed(3)
    rotary = batch.Rotary(D)
    sides = []
    for _ in range(2):
        cache = batch.PagedCache8.allocate(60, page, K, D)
        cache.k.view(torch.uint8).zero_()
        cache.v.view(torch.uint8).zero_()
        cache.k_scale.fill_(1.0)
        cache.v_scale.fill_(1.0)
        sides.append((cache, batch.PagedAttention8(cache, H, n)))
    table = torch.randperm(60, generator=g).int().view(B, 20)
    x, pos = torch.zeros(n, H + 2 * K, D, dtype=B16, device="cuda"), i32([-1] * n)
    slots, q_start, kv_len = i64([-1] * n), i32([0] * (B + 1)), i32([0] * B)
    dev_table, out = table.cuda(), torch.zeros(n, H, D, dtype=B16, device="cuda")
    back = [torch.zeros(n, K, D, dtype=B16, device="cuda") for _ in range(2)]

    def step(side, x, out, back):
        cache, attention = side
        q, k, v = x[:, :H], x[:, H:H + K], x[:, H + K:]
        rotary.rotate(q, k, pos)
        cache.append(k, v, slots)
        attention.attend(q, q_start, kv_len, dev_table, out=out)
        cache.read(slots, k=back[0], v=back[1])

    step(sides[0], x, out, back)                   # (nothing: every row is padding)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(sides[0], x, out, back)
    lens = [0, 0, 0]
    for i in range(12):
        q_len = [[3, 5, 2], [1, 0, 7], [4, 4, 1], [0, 1, 0]][i % 4]
        at, p, s, starts = 0, [], [], [0]
        for b, m in enumerate(q_len):
            for j in range(lens[b], lens[b] + m):
                p.append(j)
                s.append(int(table[b, j // page]) * page + j % page)
            lens[b] += m
            at += m
            starts.append(at)
        pos.copy_(i32(p + [-1] * (n - at)))
        slots.copy_(i64(s + [-1] * (n - at)))
        q_start.copy_(i32(starts))
        kv_len.copy_(i32(lens))
        new = torch.randn(x.shape, generator=g).to(B16).cuda() * 2.0 ** (i % 5)
        x.copy_(new)
        out.fill_(7.0)
        graph.replay()
        plain = new.clone()
        out2, back2 = torch.full_like(out, 7.0), [torch.zeros_like(y) for y in back]
        step(sides[1], plain, out2, back2)
        torch.cuda.synchronize()
        for y, z in ((x, plain), (out, out2), (back[0], back2[0]), (back[1], back2[1])):
            assert torch.equal(y.view(torch.int16), z.view(torch.int16))
        assert (out[at:] == 7.0).all() and torch.isfinite(out[:at]).all()
    assert lib.moe_last_device_error() == lib.MOE_OK


def test_rotary_of_several_host_threads(lib):
    """One object, four threads with tensors and streams of their own."""
    from concurrent.futures import ThreadPoolExecutor
    from moe_expert_layer_warp_gb300 import batch
    r = batch.Rotary(64)

    def work(i):
        n, H = 5 + i, 3 + 2 * i
        x = torch.randn(n, H, 64, generator=torch.Generator().manual_seed(i)).cuda()
        pos = torch.arange(100 * i, 100 * i + n).int().cuda()
        y, bound = oracle.rotate(x, pos.cpu(), r.frequencies, 0, False, 1.0)
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        for _ in range(200):
            out = torch.zeros_like(x)
            torch.cuda.current_stream().synchronize()
            r.rotate(x, None, pos, q_out=out, stream=stream)
            stream.synchronize()
            if not ((out.double() - y).abs() <= bound).all():
                return False
        return True

    with ThreadPoolExecutor(4) as pool:
        assert all(pool.map(work, range(4)))


def test_attend_reports_bad_pages_lengths_and_scales(lib):
    """A table entry outside the pool, a cache length past the table, request bounds
    past the rows and scales out of their range are reported; nothing is read
    out of range, and other requests are not touched by it."""
    a = problem("ragged passes")
    q, qs, kv, table = a.args()
    for spoil in ("page", "negative page", "length", "negative length", "bounds", "order", "scale",
                  "scale of NaN"):
        qs2, kv2, t2 = qs.clone(), kv.clone(), table.clone()
        r = a.runner()
        scales = r.cache.v_scale
        kept = scales.clone()
        if spoil == "page":
            t2[0, 1] = a.pools[0].code.shape[0]
        elif spoil == "negative page":
            t2[0, 1] = -5
        elif spoil == "length":
            kv2[0] = t2.shape[1] * a.page + 1
        elif spoil == "negative length":
            kv2[0] = -1
        elif spoil == "bounds":
            qs2[-1] = q.shape[0] + 5
        elif spoil == "order":
            qs2[1] = 12
        elif spoil == "scale":
            scales[table[0, 1].long()] = 0.0
        else:
            scales[table[0, 1].long()] = math.nan
        out = r.attend(q, qs2, kv2, t2).clone()
        assert lib.moe_last_device_error() == lib.MOE_EDEVICE, spoil
        scales.copy_(kept)
        good = r.attend(q, qs, kv, table)
        assert lib.moe_last_device_error() == lib.MOE_OK
        a.check(good)
        if spoil not in ("bounds", "order"):
            n = a.q_len[0]
            assert torch.equal(out[n:].view(torch.int16), good[n:].view(torch.int16)), spoil


def test_attend_scales_of_another_source(lib):
    """Scales that are no powers of two."""
    a = problem("ragged passes")
    r = a.runner()
    g = torch.Generator().manual_seed(3)
    by = [torch.rand(s.shape, generator=g) + 0.5 for s in (r.cache.k_scale, r.cache.v_scale)]
    r.cache.k_scale.mul_(by[0].cuda())
    r.cache.v_scale.mul_(by[1].cuda())
    got = r.attend(*a.args())
    units = [s.double().permute(0, 2, 1).repeat_interleave(a.block, dim=1)
             for s in (r.cache.k_scale, r.cache.v_scale)]
    k, v = (torch.nan_to_num(p.code, nan=0.0).cuda() * u[..., None]
            for p, u in zip(a.pools, units))
    want, bound = oracle.attend(a.q.cuda(), k, v, units[1], a.q_start, a.kv_len, a.table.cuda(),
                                a.scale, 0, 0)
    assert ((got.double() - want).abs() <= bound).all()


def test_attend_values_that_are_not_finite(lib):
    """NaN among a key's or a query's elements makes NaN of the rows that see it,
    one among a value's of that column of those rows, and nothing of the others."""
    for window, sinks, dtype in ((0, 0, B16), (40, 3, F16), (0, 0, F16), (300, 2, B16)):
        a = Attend([5, 150, 1], [300, 400, 150], 4, 2, 128, dtype, 16, window=window, sinks=sinks)
        bad_v = [(0, 297, 5), (0, 299, 127), (0, 270, 7), (1, 1, 0), (1, 260, 64), (1, 395, 1),
                 (1, 300, 126), (2, 149, 50), (2, 111, 51)]
        bad_k = [(0, 298), (1, 340), (1, 2)]
        for b, j, d in bad_v:
            if int(a.table[b, j // 16]) >= 0:
                a.pools[1].code[int(a.table[b, j // 16]), j % 16, 1, d] = math.nan
        for b, j in bad_k:
            if int(a.table[b, j // 16]) >= 0:
                a.pools[0].code[int(a.table[b, j // 16]), j % 16, 0] = math.nan
        a.q[7, 3, 9] = math.nan
        got = a.runner().attend(*a.args())
        assert lib.moe_last_device_error() == lib.MOE_OK
        want, bound = a.want()
        nan = torch.zeros(want.shape, dtype=torch.bool)
        for b in range(3):
            for i in range(a.q_len[b]):
                pos, row = a.kv_len[b] - a.q_len[b] + i, a.q_start[b] + i

                def sees(j):
                    return j <= pos and (not window or pos - j < window or j < sinks)
                for c, j, d in bad_v:
                    if c == b and sees(j):
                        nan[row, 2:, d] = True
                for c, j in bad_k:
                    if c == b and sees(j):
                        nan[row, :2] = True
        nan[7, 3] = True
        assert torch.equal(torch.isnan(got).cpu(), nan)
        fine = ~nan.cuda()
        assert ((got.double() - want).abs() <= bound)[fine].all()


@pytest.mark.parametrize("name", ["ragged passes", "chunk over a cache", "window and sinks"])
def test_attend_queries_that_are_not_finite(lib, name):
    """NaN or an infinity in a query row: NaN in its result, and the others' bits
    as without."""
    a = problem(name)
    r, (q, *rest) = a.runner(), a.args()
    want = r.attend(q, *rest).clone()
    q = q.clone()
    hit = torch.zeros(q.shape[:2], dtype=torch.bool)
    for i, bad in enumerate((math.nan, math.inf, -math.inf)):
        t, h = i * (q.shape[0] - 1) // 2, i % q.shape[1]
        q[t, h, (17 * i + 3) % q.shape[2]] = bad
        hit[t, h] = True
    got = r.attend(q, *rest)
    assert torch.equal(torch.isnan(got).all(-1).cpu(), hit)
    assert torch.equal(got[~hit].view(torch.int16), want[~hit].view(torch.int16))


def test_beyond_32_bit_offsets(lib):
    """Pages past 2^31 codes of the pool."""
    from moe_expert_layer_warp_gb300 import batch
    page, H, D = 256, 8, 128
    pages = (1 << 31) // (page * H * D) + 40
    a = Attend([3, 2], [700, 300], 16, H, D, B16, page, block=32)
    small = a.cache()
    big = batch.PagedCache8.allocate(pages, page, H, D, block=32)
    base = pages - small.k.shape[0]
    for x, y in ((big.k, small.k), (big.v, small.v)):
        x.view(torch.uint8)[base:] = y.view(torch.uint8)
    big.k_scale[base:], big.v_scale[base:] = small.k_scale, small.v_scale
    q, qs, kv, table = a.args()
    r = batch.PagedAttention8(big, 16, q.shape[0])
    out = r.attend(q, qs, kv, torch.where(table >= 0, table + base, table))
    assert lib.moe_last_device_error() == lib.MOE_OK
    a.check(out)
    # and the append writes there
    new = torch.randn(5, H, D, device="cuda").to(B16)
    slots = torch.arange(5, device="cuda") + (pages * page - 32)
    big.append(new, new, slots)
    k, v = big.read(slots, dtype=F32)
    assert (k - new.float()).abs().max() <= 2.0 ** -4 * new.abs().max()
    assert torch.equal(k, v) and lib.moe_last_device_error() == lib.MOE_OK


# ---------------------------------------------------------------- together --
def test_steps_together(lib):
    """Prompts, then passes some of whose tokens are turned down: plan, rotate,
    append, attend, and the cache read back, each against its definition on what
    the one before it left."""
    from moe_expert_layer_warp_gb300 import batch
    B, H, K, D, page = 4, 6, 2, 64, 32
    g = torch.Generator().manual_seed(1)
    cache = batch.PagedCache8.allocate(40, page, K, D, block=16, heads_first=True)
    cache.k.view(torch.uint8).fill_(0x7f)
    cache.v.view(torch.uint8).fill_(0x7f)
    planner = batch.BatchPlanner(page, B, 200)
    attention = batch.PagedAttention8(cache, H, 200, window=90, sinks=2)
    rotary = batch.Rotary(D, 32, first=32, interleaved=True)
    pools = [oracle.Pool.of(cache.k, cache.k_scale.fill_(1.0), 16),
             oracle.Pool.of(cache.v, cache.v_scale.fill_(1.0), 16)]
    table, cached, held = i32([[0] * 10] * B), i32([0] * B), i32([0] * B)
    free, free_range = torch.randperm(40, generator=g).int().cuda(), i32([0, 40])
    for step in range(5):
        q_len = [[50, 7, 16, 33], [1, 9, 5, 3], [0, 4, 4, 2], [6, 1, 16, 9], [1, 1, 1, 1]][step]
        n = sum(q_len) + 3
        plan = planner.plan(i32(q_len), cached, held, free, free_range, table, n)
        held.copy_(plan.held)
        free_range[:1].copy_(plan.free_head)
        x = torch.randn((n, H + 2 * K, D), generator=g).to(B16).cuda()
        x *= 2.0 ** step                          # later tokens are larger: scales grow
        q, k, v = x[:, :H], x[:, H:H + K], x[:, H + K:]
        plain = x.clone()
        rotary.rotate(q, k, plan.positions)
        for y, was in ((q, plain[:, :H]), (k, plain[:, H:H + K])):
            want, bound = oracle.rotate(was, plan.positions, rotary.frequencies, 32, True, 1.0)
            assert ((y.double() - want).abs() <= bound).all()
        slots = plan.slots.tolist()
        cache.append(k, v, plan.slots)
        pools[0].append(k, slots)
        pools[1].append(v, slots)
        got = attention.attend(q, plan.q_start, plan.kv_len, table)
        assert lib.moe_last_device_error() == lib.MOE_OK
        back = cache.read(plan.slots, dtype=F32)
        for y, p in zip(back, pools):
            assert _same(y, p.values(slots))
        kk, vv = (torch.nan_to_num(p.all_values(), nan=0.0).cuda() for p in pools)
        vs = torch.exp2(pools[1].exp.double()).permute(0, 2, 1).repeat_interleave(16, dim=1).cuda()
        want, bound = oracle.attend(q, kk, vv, vs, plan.q_start.tolist(), plan.kv_len.tolist(),
                                    table, D ** -0.5, 90, 2)
        assert ((got.double() - want).abs() <= bound).all()
        cached += i32([n if step == 0 else n - n // 3 for n in q_len])


def test_example_with_a_cache_in_8_bits(lib):
    """The example's block with rotary positions and this cache: attention against
    its definition on what the cache holds, over several steps; and the command."""
    from examples import verify_step as ex
    B, g = 5, torch.Generator().manual_seed(2)
    block = ex.Block(B, max_tokens=50, max_blocks=6, seed=7, cache8=True)
    block.cache.k.view(torch.uint8).zero_()
    block.cache.v.view(torch.uint8).zero_()
    block.cache.k_scale.fill_(1.0)
    block.cache.v_scale.fill_(1.0)
    for step in range(4):
        q_len = torch.randint(1 if step == 0 else 0, 11 if step == 0 else 7, (B,), generator=g)
        n = int(q_len.sum())
        x = torch.randn((n, ex.SHAPE.d), generator=g).cuda()
        _, got = block.step(x, q_len.int().cuda())
        assert lib.moe_last_device_error() == lib.MOE_OK
        plan, c = got["plan"], block.cache
        plain = (x @ block.w_qkv).view(n, -1, ex.DIM)
        for y, was, step_of in ((got["q"], plain[:, :ex.HEADS], 2.0 ** -8),
                                (got["k"], plain[:, ex.HEADS:ex.HEADS + ex.KV_HEADS], 0.0)):
            want, bound = oracle.rotate(was, plan.positions, block.rotary.frequencies, 0, False,
                                        1.0)
            # (queries are rounded once more, to bf16)
            over = (y.double() - want).abs() - bound * (1 + step_of) - step_of * want.abs()
            assert (over <= 0).all()
        pools = [oracle.Pool.of(c.k, c.k_scale, 16), oracle.Pool.of(c.v, c.v_scale, 16)]
        kk, vv = (p.all_values().cuda() for p in pools)
        vs = torch.exp2(pools[1].exp.double()).permute(0, 2, 1).repeat_interleave(16, dim=1).cuda()
        want, bound = oracle.attend(got["q"], kk, vv, vs, plan.q_start.tolist(),
                                    plan.kv_len.tolist(), block.table, ex.DIM ** -0.5, 0, 0)
        assert ((got["attention"].double() - want).abs() <= bound).all()
        block.accept((q_len - q_len // 3).int().cuda())
    ex.main(["--requests", "4", "--steps", "3", "--cache8"])
