"""GPU checks of include/moe_batch.h's operators against their definitions in
64 bits (tests/batch_oracle.py), at the sizes and masks where they can go
wrong. Tolerances are the oracle's bounds."""
import functools
import random

import numpy as np
import pytest
import torch

from tests import batch_oracle as oracle

pytestmark = pytest.mark.gpu


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


# -------------------------------------------------------------------- plan --
def _plan_case(q_len, cached, extra, page, n_free, M, head=2, pad=3, tail=0):
    """extra[b]: pages held beyond those the cached tokens need."""
    B = len(q_len)
    held = [min(M, -(-c // page) + e) for c, e in zip(cached, extra)]
    ids = list(range(1000, 1000 + sum(held) + head + n_free + tail))
    random.Random(5).shuffle(ids)
    table, at = -np.ones((B, M), np.int64), 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    return dict(q_len=q_len, cached=cached, held=held, free=ids[at:], head=head,
                end=head + n_free, table=table, page=page, n_tokens=sum(q_len) + pad)


PLANS = {
    "one": _plan_case([5], [100], [0], 16, 4, 9),
    "nothing": _plan_case([0], [0], [0], 16, 0, 1, pad=0),
    "zero-length requests": _plan_case([0, 3, 0, 0, 7, 0], [5, 0, 64, 0, 63, 16], [0] * 6, 64, 9, 4),
    "page edges": _plan_case([1, 1, 1, 16, 17], [15, 16, 17, 0, 31], [0] * 5, 16, 20, 6),
    "pages held for drafts": _plan_case([9, 9, 9], [10, 30, 47], [1, 2, 0], 16, 5, 8),
    "out of pages": _plan_case([40, 40, 1, 40, 0, 2], [0, 10, 3, 0, 9, 0], [0] * 6, 32, 3, 8),
    "last page exactly": _plan_case([32, 32], [0, 0], [0, 0], 32, 2, 8, tail=0),
    "one page short": _plan_case([32, 32], [0, 0], [0, 0], 32, 1, 8, tail=0),
    "does not fit the table": _plan_case([10, 100, 10], [0, 40, 5], [0] * 3, 16, 40, 4),
    "long chunk": _plan_case([5000, 3], [77, 9000], [0, 0], 256, 60, 40),
}


def _run_plan(api, c, stream=None):
    from moe_expert_layer_warp_gb300 import batch
    P = batch.BatchPlanner(c["page"], len(c["q_len"]), c["n_tokens"])
    table = i32(c["table"])
    free = i32(c["free"])
    r = P.plan(i32(c["q_len"]), i32(c["cached"]), i32(c["held"]), free,
               i32([c["head"], c["end"]]), table, c["n_tokens"], stream)
    return r, table


def _check_plan(c, r, table):
    want = oracle.plan(**c)
    names = ("q_start", "kv_len", "held", "free_head", "slots", "positions")
    for name, w in zip(names, want):
        assert getattr(r, name).tolist() == [int(x) for x in w], name
    np.testing.assert_array_equal(table.cpu().numpy(), want[6])


@pytest.mark.parametrize("name", PLANS)
def test_plan(lib, name):
    c = PLANS[name]
    r, table = _run_plan(lib, c)
    assert lib.moe_last_device_error() == lib.MOE_OK
    _check_plan(c, r, table)


@pytest.mark.parametrize("B,page,seed", [(31, 16, 0), (256, 64, 1), (257, 32, 2), (1024, 16, 3),
                                         (1024, 256, 4)])
def test_plan_random_batches(lib, B, page, seed):
    g = random.Random(seed)
    q = [g.choice([0, 1, 5, 9, 300]) for _ in range(B)]
    cached = [g.randint(0, 2000) for _ in range(B)]
    extra = [g.choice([0, 0, 0, 1]) for _ in range(B)]
    c = _plan_case(q, cached, extra, page, g.randint(0, B), 2304 // page)
    r, table = _run_plan(lib, c)
    _check_plan(c, r, table)
    # calling it again on what it wrote gives the same
    from moe_expert_layer_warp_gb300 import batch
    P = batch.BatchPlanner(page, B, c["n_tokens"])
    r2 = P.plan(i32(q), i32(cached), i32(c["held"]), i32(c["free"]), i32([c["head"], c["end"]]),
                table, c["n_tokens"])
    _check_plan(c, r2, table)
    assert lib.moe_last_device_error() == lib.MOE_OK


@pytest.mark.parametrize("change", [dict(q_len=[5, -1]), dict(cached=[-3, 0]), dict(held=[-1, 0]),
                                    dict(n_tokens=7), dict(end=99), dict(head=-1)])
def test_plan_reports_bad_values(lib, change):
    """Values only the device sees: reported, and everything stays in range."""
    c = dict(_plan_case([5, 4], [10, 20], [0, 0], 16, 4, 4, pad=0), **change)
    r, _ = _run_plan(lib, c)
    assert lib.moe_last_device_error() == lib.MOE_EDEVICE
    assert lib.moe_last_device_error() == lib.MOE_OK
    ok = _plan_case([5, 4], [10, 20], [0, 0], 16, 4, 4)
    _check_plan(ok, *_run_plan(lib, ok))


def test_plan_refuses_its_own_buffers_as_input(lib):
    from moe_expert_layer_warp_gb300 import batch
    P = batch.BatchPlanner(16, 2, 8)
    table, free = i32([[-1] * 4] * 2), i32(list(range(8)))
    r = P.plan(i32([3, 4]), i32([0, 0]), i32([0, 0]), free, i32([0, 8]), table, 7)
    with pytest.raises(lib.MoeError):
        P.plan(i32([3, 4]), i32([0, 0]), r.held, free, i32([0, 8]), table, 7)


# ------------------------------------------------------------------ append --
def _pools(pages, page, H, D, dtype, heads_first, fill=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    shape = (pages, H, page, D) if heads_first else (pages, page, H, D)
    out = []
    for _ in range(2):
        t = (torch.randn(shape, generator=g) if fill is None else
             torch.full(shape, fill)).to(dtype).cuda()
        out.append(t.transpose(1, 2) if heads_first else t)
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("src32", [False, True])
@pytest.mark.parametrize("H,D,page,heads_first,n", [(1, 64, 16, False, 1), (3, 128, 64, True, 37),
                                                    (8, 64, 256, False, 300)])
def test_append(lib, dtype, src32, H, D, page, heads_first, n):
    from moe_expert_layer_warp_gb300 import batch
    pages = -(-n // page) + 2
    k, v = _pools(pages, page, H, D, dtype, heads_first)
    want = [k.cpu().clone(), v.cpu().clone()]
    g = torch.Generator().manual_seed(n)
    slots = torch.randperm(pages * page, generator=g)[:n]
    if n > 1:
        slots[::5] = -1
    # a slice of a joint projection: token stride 3·H·D
    src = torch.randn((n, 3, H, D), generator=g).to(torch.float32 if src32 else dtype).cuda()
    batch.PagedCache(k, v).append(src[:, 1], src[:, 2], slots.cuda())
    assert lib.moe_last_device_error() == lib.MOE_OK
    for i, w in enumerate(want):
        for t in range(n):
            s = int(slots[t])
            if s >= 0:
                w[s // page, s % page] = src[t, 1 + i].cpu().to(dtype)
        got = (k, v)[i].cpu()
        assert torch.equal(got.view(torch.int16), w.contiguous().view_as(got).view(torch.int16)
                           if got.is_contiguous() else w.view(torch.int16))


def test_append_skips_and_reports_slots_out_of_range(lib):
    from moe_expert_layer_warp_gb300 import batch
    k, v = _pools(2, 16, 1, 64, torch.bfloat16, False)
    before = k.clone()
    src = torch.ones(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    batch.PagedCache(k, v).append(src, src, torch.tensor([32, 4, -7], device="cuda"))
    assert lib.moe_last_device_error() == lib.MOE_EDEVICE
    before[0, 4] = 1
    assert torch.equal(k, before)


# --------------------------------------------------------------- attention --
class Attend:
    """One attention problem: packed queries over pages in random places."""

    def __init__(self, q_len, kv_len, Hq, H, D, dtype, page, heads_first=False, window=0, sinks=0,
                 scale=None, spread=1.0, seed=0, unseen=float("nan")):
        g = torch.Generator().manual_seed(seed)
        self.q_len, self.kv_len, self.page, self.window, self.sinks = (q_len, kv_len, page, window,
                                                                       sinks)
        blocks = [-(-m // page) for m in kv_len]
        n_pages, M = sum(blocks) + 3, max(max(blocks), 1) + 2
        k, v = _pools(n_pages, page, H, D, dtype, heads_first, fill=unseen)
        ids = torch.randperm(n_pages, generator=g)
        table, at = torch.full((len(kv_len), M), -1, dtype=torch.int32), 0
        self.scale = D ** -0.5 if scale is None else scale
        kc, vc = k.cpu(), v.cpu()
        for b, m in enumerate(kv_len):
            table[b, :blocks[b]] = ids[at:at + blocks[b]]
            at += blocks[b]
            first = m - q_len[b]
            lo = max(0, first - window + 1) if window else 0
            j = torch.arange(m)
            seen = (j >= lo) | (j < sinks) if q_len[b] else j < 0
            for pool in (kc, vc):
                pool[table[b].long()[j // page][seen], (j % page)[seen]] = torch.randn(
                    (int(seen.sum()), H, D), generator=g).to(dtype)
            # pages without a key that a new token sees are not to be read
            used = torch.zeros(M, dtype=torch.bool)
            used[(j // page)[seen]] = True
            table[b][~used] = -1
        k.copy_(kc)
        v.copy_(vc)
        self.k, self.v, self.kc, self.vc, self.table = k, v, kc, vc, table
        self.q_start = [0]
        for n in q_len:
            self.q_start.append(self.q_start[-1] + n)
        self.q = (torch.randn((self.q_start[-1], Hq, D), generator=g) * spread).to(dtype)

    def runner(self):
        from moe_expert_layer_warp_gb300 import batch
        return batch.PagedAttention(batch.PagedCache(self.k, self.v), self.q.shape[1],
                                    self.q.shape[0], scale=self.scale, window=self.window,
                                    sinks=self.sinks)

    def args(self):
        return self.q.cuda(), i32(self.q_start), i32(self.kv_len), self.table.cuda()

    def check(self, got):
        kc = torch.nan_to_num(self.kc.cuda(), nan=0.0)     # unseen places, not used below
        vc = torch.nan_to_num(self.vc.cuda(), nan=0.0)
        want, bound = oracle.attend(self.q.cuda(), kc, vc, self.q_start, self.kv_len,
                                    self.table.cuda(), self.scale, self.window, self.sinks)
        got = got.double()
        assert torch.isfinite(got).all()
        over = (got - want).abs() - bound
        assert (over <= 0).all(), "off by %.3g beyond %.3g at %s" % (
            (got - want).abs().max(), bound.max(), np.unravel_index(int(over.argmax()), over.shape))


B16, F16 = torch.bfloat16, torch.float16
def spec(*args, **kwargs):     # of an Attend, which is built on the GPU
    return args, kwargs


ATTENDS = {
    "one token, one key": spec([1], [1], 1, 1, 64, B16, 16),
    "one token": spec([1], [130], 4, 2, 128, F16, 16),
    "pass of five": spec([5], [77], 16, 16, 128, B16, 64),
    "first tokens of a request": spec([9], [9], 8, 2, 64, B16, 16),
    "tile edges": spec([1, 2, 3, 1, 2, 3, 1], [127, 128, 129, 255, 256, 257, 64], 8, 2, 64, F16,
                         64, heads_first=True),
    "ragged passes": spec([1, 9, 5, 3, 16, 2], [700, 33, 5, 1030, 128, 450], 8, 2, 128, B16, 32),
    "seven heads per key head": spec([4, 20], [50, 300], 14, 2, 64, F16, 16),
    "three heads per key head": spec([50], [190], 3, 1, 128, B16, 128),
    "sixteen heads, one key head": spec([7, 9], [300, 200], 16, 1, 128, B16, 256),
    "128 heads per key head": spec([3], [150], 128, 1, 64, B16, 64),
    "48 heads per key head": spec([6, 1], [40, 400], 96, 2, 128, F16, 64),
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
    # several tiles and several items per CTA
    "many passes": spec([1 + i % 9 for i in range(40)], [100 + 97 * i for i in range(40)], 16, 4,
                          128, B16, 64),
    "many passes, small pages": spec([1 + i % 5 for i in range(60)], [3000 - 49 * i for i in
                                       range(60)], 12, 4, 64, F16, 16, heads_first=True),
    "long chunks": spec([900, 1100], [2600, 1100], 8, 2, 128, B16, 64),
    "long chunks, odd groups": spec([700, 333, 40], [3000, 333, 2000], 15, 3, 64, F16, 32),
    "mixed batch": spec([500, 3, 9, 0, 260, 1] + [4] * 30, [1500, 0, 2500, 9, 2000, 1] +
                          [600 + 31 * i for i in range(30)], 28, 4, 128, F16, 16),
    "many windows": spec([1 + i % 9 for i in range(40)], [200 + 190 * i for i in range(40)], 16,
                           4, 64, B16, 16, window=700, sinks=5),
    "long windows over chunks": spec([1500, 800], [2500, 4000], 8, 4, 128, B16, 128, window=900,
                                       sinks=200),
    "peaked long chunks": spec([900, 1100], [2600, 1500], 8, 2, 128, F16, 64, spread=10.0),
    "tiny scale": spec([4], [300], 4, 2, 64, F16, 16, scale=1e-20),
    # more blocks of two query tiles than SMs
    "blocks of two": spec([700, 333], [900, 333], 64, 4, 64, B16, 64),
    "blocks of two, odd groups, windows": spec([611, 40, 290], [700, 1000, 1300], 56, 8, 128, F16,
                                               16, heads_first=True, window=150, sinks=3),
    "blocks of two beside passes": spec([600, 3, 9, 0, 160, 1, 33, 17, 16], [1500, 0, 2500, 9, 100,
                                          1, 600, 17, 900], 64, 8, 64, B16, 32),
    "blocks of two, peaked": spec([1250], [2100], 32, 8, 128, B16, 256, spread=12.0),
    # more whole items than SMs: a CTA's go in pairs
    "short items": spec([1 + i % 7 for i in range(120)], [1 + (i * 37) % 300 for i in range(120)],
                        16, 8, 128, B16, 16),
    "short items, odd heads": spec([1 + i % 3 for i in range(200)], [0 if i % 9 == 4 else 200 + i
                                     for i in range(200)], 9, 3, 64, F16, 32, heads_first=True),
    "short items, windows": spec([i % 6 for i in range(150)], [40 + 11 * i for i in range(150)], 28,
                                 4, 64, B16, 256, window=200, sinks=2),
    "blocks of two, one key head": spec([640, 9], [640, 3000], 128, 1, 64, F16, 128),
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
    """Every key scores above all before it: the running maximum grows at
    every step, by little and by much."""
    a = Attend([3, 130], [700, 400], 2, 1, 64, B16, 16, spread=0.0)
    for step, pool in ((1, a.kc),):
        for b, m in enumerate(a.kv_len):
            for j in range(m):
                pool[int(a.table[b, j // 16]), j % 16] = 0
                pool[int(a.table[b, j // 16]), j % 16, :, 0] = j * step / 8
    a.q[:, :, 0] = 4.0
    a.k.copy_(a.kc)
    a.check(a.runner().attend(*a.args()))


def test_attend_leaves_rows_of_no_request(lib):
    a = problem("ragged passes")
    q, qs, kv, table = a.args()
    wide = torch.cat([q, q[:2]])
    out = torch.full(wide.shape, 7.0, dtype=q.dtype, device="cuda")
    a.runner().attend(wide, qs, kv, table, out=out)
    a.check(out[:-2])
    assert (out[-2:] == 7.0).all()


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
    g.replay()
    torch.cuda.synchronize()
    a.check(out)


def test_attend_reports_bad_pages_and_lengths(lib):
    """A table entry outside the pool, a cache length past the table and
    request bounds past the rows are reported; nothing is read out of range,
    and other requests are not touched by it."""
    a = problem("ragged passes")
    q, qs, kv, table = a.args()
    for spoil in ("page", "negative page", "length", "negative length", "bounds", "order"):
        qs2, kv2, t2 = qs.clone(), kv.clone(), table.clone()
        if spoil == "page":
            t2[0, 1] = a.k.shape[0]
        elif spoil == "negative page":
            t2[0, 1] = -5
        elif spoil == "length":
            kv2[0] = t2.shape[1] * a.page + 1
        elif spoil == "negative length":
            kv2[0] = -1
        elif spoil == "bounds":
            qs2[-1] = q.shape[0] + 5
        else:
            qs2[1] = 12
        r = a.runner()
        out = r.attend(q, qs2, kv2, t2).clone()
        assert lib.moe_last_device_error() == lib.MOE_EDEVICE, spoil
        good = r.attend(q, qs, kv, table)
        assert lib.moe_last_device_error() == lib.MOE_OK
        a.check(good)
        if spoil not in ("bounds", "order"):
            n = a.q_len[0]
            assert torch.equal(out[n:].view(torch.int16), good[n:].view(torch.int16)), spoil


def test_attend_beyond_32_bit_offsets(lib):
    """Pages past 2^31 elements of the pool."""
    from moe_expert_layer_warp_gb300 import batch
    page, H, D = 256, 8, 128
    pages = (1 << 31) // (page * H * D) + 40
    small = Attend([3, 2], [700, 300], 16, H, D, B16, page)
    k = torch.empty(pages, page, H, D, dtype=B16, device="cuda")
    v = torch.empty_like(k)
    base = pages - small.k.shape[0]
    k[base:], v[base:] = small.k, small.v
    q, qs, kv, table = small.args()
    r = batch.PagedAttention(batch.PagedCache(k, v), 16, q.shape[0])
    out = r.attend(q, qs, kv, torch.where(table >= 0, table + base, table))
    assert lib.moe_last_device_error() == lib.MOE_OK
    small.check(out)
    # and the append writes there
    new = torch.randn(5, H, D, device="cuda").to(B16)
    slots = torch.arange(5, device="cuda") + (pages * page - 9)
    batch.PagedCache(k, v).append(new, new, slots)
    assert torch.equal(k[-1, page - 9:page - 4], new) and torch.equal(v[-1, page - 9:page - 4], new)


# ----------------------------------------------------------------- routing --
ROUTERS = {
    "plain": dict(E=64, k=6),
    "one expert": dict(E=1, k=1, score="sigmoid", renorm=False, scale=3.0),
    "odd": dict(E=251, k=16, score="sigmoid", bias=True),
    "all kept": dict(E=8, k=8, renorm=False),
    "softmax and bias": dict(E=60, k=4, bias=True, renorm=False),
    "groups by sums of two": dict(E=256, k=8, G=8, tg=4, top=2, score="sigmoid", bias=True,
                                  scale=2.5),
    "groups by maxima": dict(E=160, k=6, G=8, tg=3, top=1, renorm=False, scale=16.0),
    "groups of one": dict(E=32, k=5, G=32, tg=9, score="sigmoid", bias=True),
    "uneven lanes": dict(E=120, k=12, G=24, tg=11, top=2, score="softmax", bias=True),
    "one group of many": dict(E=256, k=12, G=8, tg=1, top=2, score="sigmoid", bias=True),
    "two groups, few lanes": dict(E=256, k=16, G=8, tg=2, top=2, score="softmax", bias=True),
    "every group": dict(E=64, k=3, G=8, tg=8, top=2, score="sigmoid"),
}


def _route(lib, logits, k, G, tg, top, score, bias, renorm, scale):
    from moe_expert_layer_warp_gb300 import batch
    r = batch.GroupedRouter(logits.shape[1], k, logits.shape[0], G, tg, top, score,
                            None if bias is None else bias.cuda(), renorm, scale)
    idx, w = r.route(logits.cuda())
    assert lib.moe_last_device_error() == lib.MOE_OK
    want_idx, want_w, bound = oracle.route(logits, bias, k, G, tg, top, score, renorm, scale)
    np.testing.assert_array_equal(idx.cpu().numpy(), want_idx)
    err = np.abs(w.cpu().double().numpy() - want_w)
    assert (err <= bound).all(), "off by %.3g" % (err - bound).max()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kind", ["spread", "ties", "masked", "all masked", "near ties"])
@pytest.mark.parametrize("name", ROUTERS)
def test_route(lib, name, kind, dtype):
    p = dict(dict(G=1, tg=1, top=1, score="softmax", bias=False, renorm=True, scale=1.0),
             **ROUTERS[name])
    g = torch.Generator().manual_seed(len(name))
    n, E = 67, p["E"]
    x = torch.randn((n, E), generator=g) * 2
    bias = torch.randn(E, generator=g) * 0.2 if p["bias"] else None
    if kind == "ties":
        x = (x * 1.5).round()
        if bias is not None:
            bias = (bias * 4).round() / 4
    elif kind == "masked":
        off = torch.rand((n, E), generator=g) < 0.6
        x[off] = -float("inf")
        x[::2] = x[::2].clamp_min(torch.finfo(dtype).min)
    elif kind == "all masked":
        x[:] = -float("inf")
        x[1::2] = torch.finfo(dtype).min
        x[2::3, 0] = 1.0
    elif kind == "near ties":
        # choices a few fp32 roundings apart: the bias cancels what the score
        # adds, as far as fp32 can hold it
        x = (torch.randn((n, 1), generator=g) + torch.randn((n, E), generator=g) * 1e-6)
        if bias is not None:
            bias = torch.randn(E, generator=g) * 2.0 ** -24
    _route(lib, x.to(dtype), p["k"], p["G"], p["tg"], p["top"], p["score"], bias, p["renorm"],
           p["scale"])


@pytest.mark.parametrize("name", ROUTERS)
def test_route_equal_logits(lib, name):
    """Rows of one value (padding) and rows with many equal best ones."""
    p = dict(dict(G=1, tg=1, top=1, score="softmax", bias=False, renorm=True, scale=1.0),
             **ROUTERS[name])
    x = torch.zeros(6, p["E"])
    x[1] = -3.5
    x[2:, ::2] = 0.25
    x[4:, 1::3] = 7.0
    bias = torch.zeros(p["E"]) if p["bias"] else None
    _route(lib, x, p["k"], p["G"], p["tg"], p["top"], p["score"], bias, p["renorm"], p["scale"])
    if p["bias"]:
        bias[::5] = 0.5
        _route(lib, x, p["k"], p["G"], p["tg"], p["top"], p["score"], bias, p["renorm"],
               p["scale"])


@pytest.mark.parametrize("n", [1, 2, 1000])
def test_route_rows(lib, n):
    g = torch.Generator().manual_seed(n)
    _route(lib, torch.randn((n, 256), generator=g), 8, 8, 4, 2, "sigmoid",
           torch.randn(256, generator=g) * 0.1, True, 2.5)


def test_route_extreme_logits(lib):
    """Scores that under- and overflow on the way stay ordered."""
    x = torch.tensor([[-120.0, -110.0, -130.0, -115.0, -600.0, -100.5, -104.0, -103.0],
                      [80.0, 30.0, 90.0, -80.0, 0.0, 100.0, 1e30, -1e30]])
    _route(lib, x, 3, 1, 1, 1, "softmax", None, True, 1.0)
    _route(lib, x[:1], 3, 1, 1, 1, "sigmoid", None, True, 1.0)
    _route(lib, x[:, :6].contiguous(), 2, 2, 1, 2, "softmax", torch.zeros(6), True, 1.0)


def test_route_scores_below_fp32(lib):
    """Scores that fp32 flushes to zero, of which the quotients are asked for;
    below fp64 too, the logits still order the experts."""
    x = -100 - 0.25 * torch.arange(64, dtype=torch.float32)
    x = x[(torch.arange(64) * 29) % 64].repeat(3, 1)
    x[1, 40] = 0.0
    x[2] *= 9
    _route(lib, x, 4, 1, 1, 1, "sigmoid", None, True, 1.0)
    _route(lib, x, 4, 8, 2, 1, "sigmoid", None, True, 2.5)
    _route(lib, x[:2], 4, 8, 2, 2, "sigmoid", None, True, 1.0)
    bias = torch.zeros(64)
    bias[:16] = 2.0
    _route(lib, x[:2], 5, 1, 1, 1, "softmax", bias, True, 1.0)
    _route(lib, x[:2], 5, 8, 2, 2, "softmax", bias, True, 1.0)


def test_route_row_stride_and_buffers(lib):
    from moe_expert_layer_warp_gb300 import batch
    g = torch.Generator().manual_seed(1)
    wide = torch.randn((9, 100), generator=g).cuda()
    r = batch.GroupedRouter(64, 6, 9)
    idx = torch.empty(9 * 6, dtype=torch.int32, device="cuda")
    w = torch.empty(9 * 6, device="cuda")
    r.route(wide[:, 11:75], idx=idx, weights=w)
    i2, w2 = r.route(wide[:, 11:75].contiguous())
    assert torch.equal(idx.view(9, 6), i2) and torch.equal(w.view(9, 6), w2)
    with pytest.raises(lib.MoeError):
        r.route(wide[:1, :64].expand(9, 64))      # rows that share their memory
