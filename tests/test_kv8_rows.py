"""GPU checks of moe_attend8 on rows of which one key takes most, and on blocks of
values whose scales differ widely: what the other keys bring must stay.

A row's error is held against that of its result with weights rounded to 16 bits
(and nothing else), and every element against a bound in which no term grows with
the number of keys to a size that matters. Weights are rounded to fp16, 2^4 (bf16) or
2^10 (fp16) times larger or more than they are relative to the row's largest product
of a weight and its block's scale, and held as three e5m2 numbers of 3 bits, each the
rounding of 8 times what the ones before left: 11 bits for fp16, off by 2^-11 for the
rounding to fp16, and for bf16, whose first number is cut and not rounded, by 2^-10
more. Where they are small they are off by half a step of the last number, 2^-16 · 8^-2
/ 2 = 2^-23, and of fp16, 2^-25: 2^-27 + 2^-29 of the largest one, or 2^-33 + 2^-35. A
product takes 32 keys at a time, and the tensor cores cut each sum to the 24 bits of
its fp32 accumulator: off by 2^-23 of the sum, so that n keys add n/32 · 2^-23 of the
sum of their sizes at most (2^-11 of it for 131072)."""
import math

import pytest
import torch

from tests.kv8_oracle import half_step

pytestmark = pytest.mark.gpu

B16, F16, CODE = torch.bfloat16, torch.float16, torch.float8_e4m3fn
GROUP = 3                       # query heads of a key head: shares of the large key
SHARES = (0.5, 0.75, 0.9)
VALUES = (1.0, 0.05)            # its values beside the others', by key head


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from moe_expert_layer_warp_gb300 import api, build
    build.build()
    assert api.moe_last_device_error() == api.MOE_OK
    return api


def e4m3(x):
    """x to the nearest code's value (sizes within the codes' range)."""
    return x.float().to(CODE)


class Rows:
    """`requests` requests of q_len new tokens over the same n keys, in pages in
    random places, two key heads of GROUP query heads each. Key `at` has a score of
    its own with every query, and values of another size."""

    def __init__(self, n, q_len, D, dtype, at, requests, window=0, sinks=0, page=128, block=16,
                 spread=1.0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, generator=g, device="cuda")
        H, self.n, self.q_len, self.D, self.dtype = len(VALUES), n, q_len, D, dtype
        self.at = at
        self.window, self.sinks, self.scale, self.requests = window, sinks, D ** -0.5, requests
        pages = -(-n // page)
        k, v = normal(pages * page, H, D), normal(pages * page, H, D) + 0.5
        k[..., 0] = 0
        k[at] = 0
        k[at, :, 0] = 16
        v[at] *= torch.tensor(VALUES, device="cuda")[:, None]
        self.k, self.v = e4m3(k), e4m3(v)
        self.k_exp, self.v_exp = (torch.zeros(pages, H, page // block, device="cuda")
                                  for _ in range(2))
        self.page, self.block = page, block
        self.order = torch.randperm(pages, generator=g, device="cuda")
        self.q = normal(requests * q_len, H * GROUP, D) * spread
        self.q[..., 0] = 0
        self.q = self.q.to(dtype)
        self.checked = sorted({0, 1, requests // 3, requests // 2, requests - 1} &
                              set(range(requests)))
        # the score that gives the key its share of every row
        for b in self.checked:
            s, see = self.scores(b)
            others = s.masked_fill(~see | (torch.arange(n, device="cuda") == at), -math.inf)
            others = torch.logsumexp(others, -1)                      # [q_len][H][GROUP]
            share = torch.tensor(SHARES, device="cuda", dtype=torch.float64)
            want = (torch.log(share / (1 - share)) + others) / (16 * self.scale)
            self.q[b * q_len:(b + 1) * q_len, :, 0] = want.view(q_len, -1).to(dtype)

    def values(self, x, exp):
        """[n][H][D] in float64, and each key's scale [n][H]."""
        unit = torch.exp2(exp).permute(0, 2, 1).repeat_interleave(self.block, dim=1)
        unit = unit.reshape(-1, unit.shape[2])[:self.n].double()
        return x[:self.n].double() * unit[..., None], unit

    def scores(self, b):
        """[q_len][H][GROUP][n] and what is seen [q_len][1][1][n], for request b."""
        k, _ = self.values(self.k, self.k_exp)
        q = self.q[b * self.q_len:(b + 1) * self.q_len].double()
        q = q.view(self.q_len, -1, GROUP, self.D)
        s = torch.einsum("thgd,nhd->thgn", q, k) * self.scale
        back = (torch.arange(self.q_len, device="cuda")[:, None] + self.n - self.q_len -
                torch.arange(self.n, device="cuda"))
        see = back >= 0
        if self.window:
            see &= (back < self.window) | (torch.arange(self.n, device="cuda") < self.sinks)
        return s, see[:, None, None, :]

    def want(self, b):
        """The rows of request b, their bounds, the rows with weights in 16 bits, and
        what small weights and long sums may lose beside."""
        s, see = self.scores(b)
        k, _ = self.values(self.k, self.k_exp)
        v, unit = self.values(self.v, self.v_exp)
        q = self.q[b * self.q_len:(b + 1) * self.q_len].double()
        q = q.view(self.q_len, -1, GROUP, self.D)
        s = s.masked_fill(~see, -math.inf)
        w = (s - s.amax(-1, keepdim=True)).exp()
        # scores: fp32 sums, and elements of a query below 2^-10 of its largest times
        # 16^-1 (16^-2), as in tests/kv8_oracle.py
        f16 = self.dtype is F16
        size = torch.einsum("thgd,nhd->thgn", q.abs(), k.abs()) * self.scale
        lost = (q.abs().amax(-1) * (2.0 ** -25.8 if f16 else 2.0 ** -21.8))[..., None] * (
            k.abs().sum(-1).t()[None, :, None]) * self.scale
        ds = torch.where(see, size * (self.D + 8) * 2.0 ** -22 + lost, 0.0).amax(-1)[..., None]
        total = w.sum(-1, keepdim=True)
        rel, far = (2.0 ** -11, 2.0 ** -33 + 2.0 ** -35) if f16 else (
            2.0 ** -10 + 2.0 ** -11, 2.0 ** -27 + 2.0 ** -29)
        y = torch.einsum("thgn,nhd->thgd", w, v) / total
        a = torch.einsum("thgn,nhd->thgd", w, v.abs()) / total
        most = (w * unit.t()[None, :, None]).amax(-1, keepdim=True) / total
        codes = torch.einsum("thgn,nhd->thgd", see.double().expand(s.shape),
                             v.abs() / unit[..., None])
        eps = half_step(self.dtype)
        lost = far * most * codes + see.sum(-1)[..., None] / 32 * 2.0 ** -23 * a
        # a row's reference need not be the large key's (it follows growth beyond 2^10.5
        # or 2^4.5),
        # and then its weight is rounded as any other, where that in 16 bits is exactly 1
        lost += rel * (w[..., self.at] / total[..., 0])[..., None] * v[self.at].abs()[:, None]
        bound = (eps * y.abs() + (rel * (1 + eps) + 2 * ds + 2.0 ** -19) * a + lost) * (
            1 + 2 * eps) + (2.0 ** -25 if f16 else 2.0 ** -134)
        short = w.to(self.dtype).double()
        if f16:                  # (11 bits at every size)
            e = torch.frexp(w)[1]
            short = torch.ldexp(torch.ldexp(w, -e).half().double(), e)
        short = torch.einsum("thgn,nhd->thgd", short, v) / total
        shape = (self.q_len, -1, self.D)
        return [x.reshape(shape) for x in (y, bound, short, lost)]

    def runner(self):
        from moe_expert_layer_warp_gb300 import batch
        pages, H = self.order.numel(), len(VALUES)
        out = []
        for x, exp in ((self.k, self.k_exp), (self.v, self.v_exp)):
            codes = torch.empty(pages, self.page, H, self.D, dtype=CODE, device="cuda")
            codes.view(torch.uint8)[self.order] = x.view(torch.uint8).view(codes.shape)
            scales = torch.empty(exp.shape, device="cuda")
            scales[self.order] = torch.exp2(exp)
            out += [codes, scales]
        return batch.PagedAttention8(batch.PagedCache8(out[0], out[2], out[1], out[3]), H * GROUP,
                                     self.q.shape[0], dtype=self.dtype, window=self.window,
                                     sinks=self.sinks)

    def check(self, lib):
        q_start = torch.arange(self.requests + 1, device="cuda", dtype=torch.int32) * self.q_len
        kv_len = torch.full((self.requests,), self.n, dtype=torch.int32, device="cuda")
        table = self.order.int()[None].repeat(self.requests, 1)
        out = self.runner().attend(self.q, q_start, kv_len, table)
        assert lib.moe_last_device_error() == lib.MOE_OK
        error = 0.0
        for b in self.checked:
            got = out[b * self.q_len:(b + 1) * self.q_len].double()
            y, bound, short, lost = self.want(b)
            rounded = y.to(self.dtype).double()
            # (rounding errors of 64 elements and more: their norm varies by a tenth)
            row = (got - y).norm(dim=-1) / y.norm(dim=-1)
            limit = (2 * (short - y).norm(dim=-1) + 1.5 * (rounded - y).norm(dim=-1) +
                     lost.norm(dim=-1)) / y.norm(dim=-1)
            error = max(error, float(row.max()))
            assert (row <= limit).all(), "a row is off by %.3g of its norm, not %.3g" % (
                row.max(), limit[row > limit].min())
            over = (got - y).abs() - bound
            assert (over <= 0).all(), "off by %.3g beyond its bound" % over.max()
        return error


@pytest.mark.parametrize("dtype", [B16, F16])
@pytest.mark.parametrize("place", ["first", "middle", "last"])
@pytest.mark.parametrize("q_len, D", [(1, 128), (12, 64), (21, 128)])
@pytest.mark.parametrize("n", [4100, 16384, 65536, 131072])
def test_one_key_takes_most(lib, n, q_len, D, place, dtype):
    """Items of 3, 36 and 63 rows, enough of them that a CTA has whole caches."""
    at = {"first": 0, "middle": n // 2 - 5, "last": n - q_len}[place]
    Rows(n, q_len, D, dtype, at, requests=77, page=256 if n > 100000 else 128).check(lib)


@pytest.mark.parametrize("dtype", [B16, F16])
@pytest.mark.parametrize("q_len, D", [(1, 64), (21, 128)])
def test_sinks_beside_a_window(lib, q_len, D, dtype):
    Rows(70001, q_len, D, dtype, 0, requests=90, window=30011, sinks=4).check(lib)


@pytest.mark.parametrize("dtype", [B16, F16])
@pytest.mark.parametrize("q_len", [1, 21])
def test_one_key_takes_most_of_a_peaked_row(lib, q_len, dtype):
    """Scores of the others that spread over 2^20 and more."""
    Rows(16384, q_len, 128, dtype, 777, requests=77, spread=2.5).check(lib)


@pytest.mark.parametrize("at", [3, 40])
@pytest.mark.parametrize("more", [8, 16, 20])
@pytest.mark.parametrize("dtype", [B16, F16])
@pytest.mark.parametrize("q_len", [1, 21])
def test_blocks_with_larger_scales(lib, q_len, dtype, more, at):
    """Blocks whose scale is 2^8 to 2^20 times the others', for a value that no row
    gives weight, and all but whose other codes are zeros. at 3: the key with most of
    the weight is among them, and then others' weights are 2^-36 of its product with
    its scale, below what is kept."""
    r = Rows(6000, q_len, 128, dtype, at, requests=77, block=16)
    for block in (0, 3, 9, 100):
        r.v_exp[block // 8, :, block % 8] = more
        rows = slice(block * 16, block * 16 + 16)
        r.v[rows] = e4m3(torch.zeros(16, *r.v.shape[1:], device="cuda"))
        r.v[rows.start + 5] = e4m3(torch.full(r.v.shape[1:], 300.0, device="cuda"))
        r.k[rows.start + 5] = e4m3(torch.zeros(r.k.shape[1:], device="cuda"))
        r.k[rows.start + 5, :, 0] = e4m3(torch.full((2,), -200.0, device="cuda"))
    r.check(lib)
