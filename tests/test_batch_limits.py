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


# ------------------------------------------------------------- near ties ----
def test_route_near_tie_past_its_neighbour(lib):
    """The three best choices lie within 3e-8: the second's bound is small, the
    third's, a large score beside a negative bias, is not, and the third is the
    largest of the three."""
    x = torch.tensor([[-25.0, -25.0, 1.1229205131530762]])
    bias = torch.tensor([0.05000002682209015, 0.050000011920928955, -0.7045300006866455])
    _route(lib, x, 1, 1, 1, 1, "sigmoid", bias, False, 1.0)
    _route(lib, x, 2, 1, 1, 1, "sigmoid", bias, True, 1.0)


def _near_ties(score, E, n, seed):
    """Rows whose choices lie within some 1e-7 of each other: half of the
    experts by their bias alone, the others by a large score beside a bias that
    takes it back, their logits a few roundings away from a tie."""
    g = torch.Generator().manual_seed(seed)
    half = E // 2
    x = torch.full((n, E), -25.0)
    x[:, half:] = (torch.rand(E - half, generator=g) * 2).expand(n, -1)
    step = 2.0 ** -23 * torch.randint(-6, 7, (n, E - half), generator=g)
    x[:, half:] += step.float() * x[:, half:]
    s = torch.sigmoid(x[0].double()) if score == "sigmoid" else torch.softmax(x[0].double(), 0)
    near = 0.05 + (torch.rand(E, generator=g).double() - 0.5) * 6e-8
    order = torch.randperm(E, generator=g)
    return x[:, order].contiguous(), (near - s).float()[order].contiguous()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,G,tg,top", [(8, 1, 1, 1, 1), (16, 3, 1, 1, 1), (32, 8, 1, 1, 1),
                                          (64, 6, 1, 1, 1), (24, 2, 4, 2, 1), (64, 8, 8, 3, 2),
                                          (256, 16, 8, 4, 2)])
def test_route_near_ties_of_unequal_bounds(lib, score, E, k, G, tg, top):
    x, bias = _near_ties(score, E, 300, E + k)
    _route(lib, x, k, G, tg, top, score, bias, False, 1.0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_near_ties_among_many_equal_choices(lib, score):
    """Forty experts of one logit and one bias, and others whose choices lie a
    few roundings above or below theirs."""
    x, bias = _near_ties(score, 64, 300, 1)
    low = x[0] == -25.0
    few = low.nonzero().flatten()
    x[:, few[20:]] = -30.0
    bias[few[20:]] = -1.0
    more = (~low).nonzero().flatten()[:20]
    x[:, more] = -25.0
    s = torch.sigmoid(x.double()) if score == "sigmoid" else torch.softmax(x.double(), 1)
    bias[~low] -= (s[0] + bias.double() - 0.05)[~low].float()
    bias[more] = bias[few[:20]] = 0.05
    for k in (1, 5, 16):
        _route(lib, x, k, 1, 1, 1, score, bias, False, 1.0)


# ------------------------------------------------ tiles of one loader's boxes
@pytest.mark.parametrize("page", [128, 256])
@pytest.mark.parametrize("q_len,kv_len,Hq,H,window", [
    ([3], [30000], 4, 1, 0), ([2] * 40, [4000 + 900 * i for i in range(40)], 8, 4, 0),
    ([600, 5, 900], [6000, 9000, 900], 16, 8, 0), ([9] * 12, [20000] * 12, 4, 2, 9000)])
def test_items_longer_than_the_ring_in_one_box_a_tile(lib, page, q_len, kv_len, Hq, H, window):
    """Heads of 64 columns in pages of a tile or two: a tile is one box, and the
    second loader has none of its own for more tiles than the ring holds."""
    a = Attend(q_len, kv_len, Hq, H, 64, B16, page, window=window)
    r = a.runner()
    for _ in range(3):
        out = r.attend(*a.args())
        assert lib.moe_last_device_error() == lib.MOE_OK
    a.check(out)


# --------------------------------------------------------- padded plans -----
def test_plan_padded_to_the_types_limit(lib):
    """Rows of padding up to 2^31 - 1: all written, none beside them."""
    from moe_expert_layer_warp_gb300 import batch
    n = 2 ** 31 - 1
    P = batch.BatchPlanner(16, 2, n)
    P._slots.fill_(7)
    P._positions.fill_(7)
    table = i32([[3, -1], [5, 6]])
    r = P.plan(i32([4, 3]), i32([14, 15]), i32([1, 2]), i32([9, 8]), i32([0, 2]), table, n)
    assert lib.moe_last_device_error() == lib.MOE_OK
    assert r.slots[:7].tolist() == [62, 63, 144, 145, 95, 96, 97]
    assert r.positions[:7].tolist() == [14, 15, 16, 17, 15, 16, 17]
    for t in (r.slots, r.positions):
        for part in t[7:].split(2 ** 28):
            assert bool((part == -1).all())


# ------------------------------------------------- values that are not finite
def _by_definition(a, kc, vc):
    """out [T][Hq][D] in 64 bits, every row over the keys that it sees alone."""
    q, out = a.q.double().cuda(), torch.zeros(a.q.shape, dtype=torch.float64, device="cuda")
    H = kc.shape[2]
    per = q.shape[1] // H
    for b, m in enumerate(a.kv_len):
        for i in range(a.q_len[b]):
            t, pos = a.q_start[b] + i, m - a.q_len[b] + i
            j = torch.arange(max(0, pos + 1), device="cuda")
            if a.window:
                j = j[(pos - j < a.window) | (j < a.sinks)]
            if not j.numel():
                continue
            page = a.table[b].long().cuda()[j // a.page]
            k, v = kc[page, j % a.page].double(), vc[page, j % a.page].double()
            s = torch.einsum("hpd,jhd->hpj", q[t].view(H, per, -1), k) * a.scale
            y = (torch.softmax(s, 2)[..., None] * v.permute(1, 0, 2)[:, None]).sum(2)
            out[t] = y.reshape(-1, y.shape[-1])
    return out


def _check_not_finite(a, got):
    """Rows that see nothing but numbers as ever; the others by the definition:
    NaN, or the infinity of one sign."""
    want = _by_definition(a, a.kc.cuda(), a.vc.cuda())
    plain = [torch.nan_to_num(p.cuda(), nan=0.0, posinf=0.0, neginf=0.0) for p in (a.kc, a.vc)]
    q = torch.nan_to_num(a.q.cuda(), nan=0.0, posinf=0.0, neginf=0.0)
    _, bound = oracle.attend(q, *plain, a.q_start, a.kv_len, a.table.cuda(), a.scale, a.window,
                             a.sinks)
    got, fine = got.double(), torch.isfinite(want)
    assert torch.isfinite(got[fine]).all(), "%d numbers lost" % (~torch.isfinite(got[fine])).sum()
    assert ((got - want).abs() <= bound)[fine].all()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])


def _place(a, pool, b, j):
    return pool[int(a.table[b, j // a.page]), j % a.page]


NOT_FINITE = {
    "pass": dict(q_len=[5, 1, 9], kv_len=[77, 40, 300], Hq=16, H=4, D=128, dtype=F16, page=16),
    "pass at a tile's edge": dict(q_len=[6], kv_len=[131], Hq=8, H=2, D=64, dtype=B16, page=64),
    "chunk": dict(q_len=[300], kv_len=[420], Hq=8, H=2, D=128, dtype=B16, page=64),
    "chunk, heads of their own": dict(q_len=[500], kv_len=[520], Hq=2, H=2, D=64, dtype=F16,
                                      page=32, heads_first=True),
    "window": dict(q_len=[9, 130], kv_len=[700, 400], Hq=4, H=2, D=128, dtype=B16, page=16,
                   window=50, sinks=3),
    "sinks past a tile": dict(q_len=[40], kv_len=[600], Hq=4, H=1, D=64, dtype=F16, page=16,
                              window=20, sinks=140),
    "odd groups": dict(q_len=[61, 9], kv_len=[100, 400], Hq=56, H=8, D=128, dtype=F16, page=16,
                       window=50, sinks=3),
    "blocks of two": dict(q_len=[700, 9], kv_len=[900, 60], Hq=64, H=8, D=64, dtype=B16, page=64),
    "short items": dict(q_len=[1 + i % 5 for i in range(80)], kv_len=[9 + 7 * i for i in range(80)],
                        Hq=8, H=4, D=128, dtype=B16, page=16),
}


@pytest.mark.parametrize("name", NOT_FINITE)
def test_scores_not_finite(lib, name):
    """A query of NaN, and a key of NaN, give NaN to the rows they belong to
    and to those that see them, not zeros."""
    a = Attend(**NOT_FINITE[name])
    last = len(a.q_len) - 1
    _place(a, a.kc, last, a.kv_len[last] - 1)[0, 3] = float("nan")
    a.k.copy_(a.kc)
    a.q[0, 1, 2] = float("nan")
    a.q[a.q_start[-1] // 2, 0] = float("nan")
    out = a.runner().attend(*a.args())
    assert lib.moe_last_device_error() == lib.MOE_OK
    _check_not_finite(a, out)


@pytest.mark.parametrize("name", NOT_FINITE)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_values_not_finite_reach_only_rows_that_see_them(lib, name, value):
    """A drafted token whose value overflowed; one that a window leaves behind
    in the middle of a pass."""
    a = Attend(**NOT_FINITE[name])
    for b, (n, m) in enumerate(zip(a.q_len, a.kv_len)):
        if len(a.q_len) > 9 and b % 3:
            continue
        _place(a, a.vc, b, m - 1)[0, 5] = value                    # the newest token's
        _place(a, a.vc, b, m - 1 - n // 2)[-1, a.q.shape[2] - 1] = value
        if a.window and m - n - a.window + 1 > 0:                  # the first to leave the window
            _place(a, a.vc, b, m - n - a.window + 1)[0, 7] = value
        if a.sinks:
            _place(a, a.vc, b, a.sinks - 1)[-1, 2] = -value        # seen by every row
    a.v.copy_(a.vc)
    out = a.runner().attend(*a.args())
    assert lib.moe_last_device_error() == lib.MOE_OK
    _check_not_finite(a, out)


# ---------------------------------------------------------------- devices ---
def test_calls_beside_another_current_device_are_refused(lib, monkeypatch):
    from moe_expert_layer_warp_gb300 import batch
    a = Attend([3], [20], 4, 2, 64, B16, 16)
    cache = batch.PagedCache(a.k, a.v)
    planner, attention = batch.BatchPlanner(16, 1, 4), a.runner()
    router = batch.GroupedRouter(8, 2, 4)
    args, new = a.args(), torch.zeros(3, 2, 64, dtype=B16, device="cuda")
    calls = [lambda: planner.plan(i32([3]), i32([0]), i32([0]), i32([1]), i32([0, 1]), i32([[0]]), 3),
             lambda: cache.append(new, new, torch.arange(3, device="cuda")),
             lambda: attention.attend(*args),
             lambda: router.route(torch.zeros(4, 8, device="cuda"))]
    current = torch.cuda.current_device()
    for call in calls:
        call()
        with monkeypatch.context() as m:
            m.setattr(batch, "_several_devices", True)
            m.setattr(batch, "_current_device", lambda: current + 1)
            with pytest.raises(ValueError, match="current device"):
                call()
    assert lib.moe_last_device_error() == lib.MOE_OK


# ------------------------------------------------ graphs, streams, threads --
CUT = {     # items cut among several CTAs, whose parts are joined
    "one pass": dict(q_len=[5], kv_len=[777], Hq=16, H=16, D=128, dtype=B16, page=64),
    "passes": dict(q_len=[3, 9, 1, 5], kv_len=[6000, 900, 20, 9000], Hq=8, H=2, D=64, dtype=F16,
                   page=16),
    "chunk beside passes": dict(q_len=[300, 4, 260], kv_len=[1500, 5000, 300], Hq=32, H=8, D=128,
                                dtype=B16, page=32),
}


@pytest.mark.parametrize("name", CUT)
def test_a_graph_replayed_over_changing_inputs(lib, name):
    """Every replay has the same call number: parts of the replay before must
    not pass for its own."""
    a = Attend(**CUT[name], unseen=0.0)
    r, (q, qs, kv, table) = a.runner(), a.args()
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    r.attend(q, qs, kv, table, out=out)
    with torch.cuda.graph(graph):
        r.attend(q, qs, kv, table, out=out)
    lengths = list(a.kv_len)
    g = torch.Generator().manual_seed(1)
    for i in range(8):
        a.q = (torch.randn(a.q.shape, generator=g) * (0.5 + i)).to(a.q.dtype)
        a.kv_len = [max(n, m - 97 * i if i % 2 else m // (i + 1)) for n, m in
                    zip(a.q_len, lengths)]
        a.vc = torch.randn(a.vc.shape, generator=g).to(a.vc.dtype)
        q.copy_(a.q), kv.copy_(i32(a.kv_len)), a.v.copy_(a.vc), out.fill_(float("nan"))
        graph.replay()
        assert lib.moe_last_device_error() == lib.MOE_OK
        a.check(out)
        again = out.clone()
        graph.replay()
        graph.replay()
        assert torch.equal(again, out)
    assert lib.moe_last_device_error() == lib.MOE_OK


def test_two_objects_on_two_streams(lib):
    """Calls that overlap, each with its object's workspace."""
    problems = [Attend(**CUT["passes"]), Attend(**CUT["chunk beside passes"], seed=3)]
    runners, args = [a.runner() for a in problems], [a.args() for a in problems]
    streams = [torch.cuda.Stream() for _ in problems]
    outs = [torch.empty_like(a[0]) for a in args]
    torch.cuda.synchronize()
    for _ in range(50):
        for r, x, out, s in zip(runners, args, outs, streams):
            r.attend(*x, out=out, stream=s)
    torch.cuda.synchronize()
    assert lib.moe_last_device_error() == lib.MOE_OK
    for a, out in zip(problems, outs):
        a.check(out)


def test_two_host_threads(lib):
    """First calls of each kernel from two threads at once, an object each."""
    import threading
    problems = [Attend(**dict(CUT["passes"], D=D, dtype=dtype), seed=i)
                for i, (D, dtype) in enumerate([(64, B16), (128, F16), (64, B16), (128, F16)])]
    runners, args = [a.runner() for a in problems], [a.args() for a in problems]
    streams = [torch.cuda.Stream() for _ in problems]
    outs, faults = [torch.empty_like(a[0]) for a in args], []
    start = threading.Barrier(len(problems))
    torch.cuda.synchronize()

    def work(i):
        try:
            start.wait(30)
            for _ in range(100):
                runners[i].attend(*args[i], out=outs[i], stream=streams[i])
        except Exception as e:                                # reported below
            faults.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(problems))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    torch.cuda.synchronize()
    assert not faults
    assert lib.moe_last_device_error() == lib.MOE_OK
    for a, out in zip(problems, outs):
        a.check(out)


def test_first_call_of_a_host_thread(lib):
    """A thread that has made no CUDA call before."""
    import threading
    a = Attend(**CUT["passes"])
    r, args = a.runner(), a.args()
    out, faults, stream = torch.empty_like(args[0]), [], torch.cuda.Stream()
    torch.cuda.synchronize()

    def work():
        try:
            r.attend(*args, out=out, stream=stream)
        except Exception as e:                                # reported below
            faults.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join(60)
    stream.synchronize()
    assert not faults
    a.check(out)


# ---------------------------------------------------------------- strides ---
def test_results_with_gaps_between_heads_and_tokens(lib):
    """Every other one of an odd number of heads, or of tokens."""
    a = Attend(**CUT["chunk beside passes"])
    q, qs, kv, table = a.args()
    T, H, D = q.shape
    for shape, order in (((T, 2 * H - 1, D), lambda t: t[:, ::2]),
                         ((H, 2 * T - 1, D), lambda t: t[:, ::2].transpose(0, 1))):
        whole = torch.full(shape, 7.0, dtype=q.dtype, device="cuda")
        a.runner().attend(q, qs, kv, table, out=order(whole))
        assert lib.moe_last_device_error() == lib.MOE_OK
        a.check(order(whole))
        assert (whole[:, 1::2] == 7.0).all()


# ---------------------------------------------------------------- example ---
@pytest.mark.parametrize("requests,steps", [(2, 1), (3, 2), (128, 4), (2, 200)])
def test_example_runs_at_any_size(lib, capsys, monkeypatch, requests, steps):
    """Fewer steps than it warms up with, as many requests as a pass holds, and
    caches longer than a few pages: no request is refused."""
    from examples import verify_step as ex
    step = ex.Block.step

    def checked(self, x, q_len):
        out = step(self, x, q_len)
        assert (out[1]["plan"].kv_len == self.cached + q_len).all()
        return out

    monkeypatch.setattr(ex.Block, "step", checked)
    ex.main(["--requests", str(requests), "--steps", str(steps)])
    assert "%d requests, %d steps" % (requests, steps) in capsys.readouterr().out


def test_example_refuses_what_a_pass_cannot_hold(lib):
    from examples import verify_step as ex
    for args in (["--requests", "129"], ["--requests", "0"], ["--steps", "0"]):
        with pytest.raises(SystemExit):
            ex.main(args)


# ---------------------------------------------------------------- binding ---
def test_binding_calls_agree_with_the_objects(lib):
    from moe_expert_layer_warp_gb300 import batch
    a = Attend(**CUT["passes"])
    q, qs, kv, table = a.args()
    want = a.runner().attend(q, qs, kv, table)
    cache, attn = lib.make_cache(a.k, a.v), lib.AttnDesc(8, 0, 0, a.scale)
    ws = torch.empty(lib.moe_attend_workspace_bytes(cache, attn), dtype=torch.uint8, device="cuda")
    for padded in (False, True):
        out = torch.full_like(q, 7.0)
        lib.moe_attend(cache, attn, q, qs, kv, table, ws, out, padded=padded)
        assert torch.equal(out, want)
    x = torch.randn(9, 64, device="cuda")
    idx, w = torch.empty(9, 6, dtype=torch.int32, device="cuda"), torch.empty(9, 6, device="cuda")
    lib.moe_route_grouped(lib.RouterDesc(64, 6, 1, 1, 1, 0, 1, 1.0), x, None, idx, w)
    want_idx, want_w = batch.GroupedRouter(64, 6, 9).route(x)
    assert torch.equal(idx, want_idx) and torch.equal(w, want_w)
    # plan and append, one request of 20 tokens into 2 pages
    q_len, cached, held, free, ends = i32([20]), i32([0]), i32([0]), i32([4, 1, 2]), i32([0, 3])
    outs = [i32([-1, -1]), i32([0]), i32([0]), i32([0]), i32([[-1, -1]])]
    slots = torch.empty(20, dtype=torch.int64, device="cuda")
    pos = torch.empty(20, dtype=torch.int32, device="cuda")
    p = [t.data_ptr() for t in (q_len, cached, held, free, ends, outs[4], *outs[:4])]
    lib.moe_plan_batch(lib.BatchC(1, 2, 16, 3, *p), 20, slots, pos)
    assert slots.tolist() == list(range(64, 80)) + list(range(16, 20))
    k = torch.randn(20, 2, 64, device="cuda").half()
    lib.moe_kv_append(cache, k, -k, slots)
    assert torch.equal(a.k[4, :16], k[:16]) and torch.equal(a.v[1, :4], -k[16:])
    assert lib.moe_last_device_error() == lib.MOE_OK


@pytest.mark.parametrize("name", NOT_FINITE)
def test_values_not_finite_change_no_other_bit(lib, name):
    """What is finite is the same, bit for bit, whatever stands where it is not
    seen; and a call after one with such values is as ever."""
    a = Attend(**NOT_FINITE[name])
    r, args = a.runner(), a.args()
    clean = r.attend(*args).clone()
    for b, (n, m) in enumerate(zip(a.q_len, a.kv_len)):
        _place(a, a.vc, b, m - 1)[0, 5] = float("inf")
        _place(a, a.vc, b, m - 1 - n // 2)[-1, 11] = float("nan")
    a.v.copy_(a.vc)
    spoilt = r.attend(*args).clone()
    again = r.attend(*args).clone()
    assert torch.equal(spoilt.view(torch.int16), again.view(torch.int16))
    fine = torch.isfinite(_by_definition(a, a.kc.cuda(), a.vc.cuda()))
    assert not fine.all()
    assert torch.equal(spoilt[fine], clean[fine])
    a.v.copy_(torch.nan_to_num(a.vc, nan=0.0, posinf=0.0))
    a.vc.copy_(a.v.cpu())
    a.check(r.attend(*args))
    assert lib.moe_last_device_error() == lib.MOE_OK
