// attend_range.cuh — what the attention kernels share: how a batch's keys are
// cut into equal ranges, one per CTA, from lengths that only the device has
// (items, their units, the start of a CTA's range); waits that end; and small
// arithmetic. The argument structs (AttendArgs, Attend8Args) and the kernels'
// parameters are template arguments: they name their members alike.
#pragma once

#include <limits.h>
#include <math.h>

#include <atomic>
#include <chrono>

#include "batch_launch.h"
#include "common.cuh"

namespace moe {

constexpr int kTile = 128;        // keys of a key tile
constexpr int kPlanThreads = 256;

// A block of new tokens of one request for one key head.
struct Item {
  int row0, ntok;     // packed rows of the block
  int pos0;           // position of its first token
  int lo, hi, sk;     // keys its rows see: [lo, hi) and [0, sk), sk ≤ lo
  int lo_tile, ns;    // first tile of [lo, hi); tiles of [0, sk) before it
  int n;              // tiles in all, at least 1
};

MOE_DEV int tile_of(const Item& it, int j) { return j < it.ns ? j : it.lo_tile + j - it.ns; }

struct Request {
  int first, q, len;
};

// Row range and cache length of request b, cut to what exists.
template <class Args>
MOE_DEV Request request(const Args& a, int page_shift, int b, bool* bad) {
  const int f = a.q_start[b], l = a.q_start[b + 1], len = a.kv_len[b];
  Request r;
  r.first = min(max(f, 0), a.n_tokens);
  const int last = min(max(l, r.first), a.n_tokens);
  r.q = last - r.first;
  r.len = len;
  *bad = f != r.first || l != last;
  if (len < 0 || len > MOE_MAX_CACHE_LEN || len > ((int64_t)a.max_blocks << page_shift)) {
    r.len = 0;
    *bad = true;
  }
  return r;
}

// The first key that a token at position `pos` sees, or below 0. (A cache shorter
// than the pass has negative positions, and a window may be as long as the
// longest cache: their difference passes 32 bits, and says no more than 0's.)
MOE_DEV int window_from(int pos, int window) { return max(pos, 0) - window + 1; }

// `fixed`: the tokens of a block.
template <class Args>
MOE_DEV Item make_item(const Args& a, const Request& r, int block, int fixed) {
  Item it;
  const int tok0 = block * fixed;
  it.row0 = r.first + tok0;
  it.ntok = min(fixed, r.q - tok0);
  it.pos0 = r.len - r.q + tok0;
  it.hi = max(0, it.pos0 + it.ntok);
  it.lo = a.window > 0 ? min(it.hi, max(0, window_from(it.pos0, a.window))) : 0;
  it.sk = min(a.sinks, it.lo);
  it.lo_tile = it.lo / kTile;
  it.ns = min((it.sk + kTile - 1) / kTile, it.lo_tile);
  it.n = max(1, it.ns + (it.hi + kTile - 1) / kTile - it.lo_tile);
  return it;
}

// Whether some rows of the item see `key` and others do not (for a key that no
// row sees it may be either), and whether a tile that begins at key0 has such.
template <class Args>
MOE_DEV bool some_see(const Args& a, int pos0, int hi, int key) {
  return key > pos0 || (a.window > 0 && key >= a.sinks && key < window_from(hi - 1, a.window));
}
template <class Args>
MOE_DEV bool tile_some_see(const Args& a, const Item& it, int key0) {
  return key0 + kTile - 1 > it.pos0 ||
         (a.window > 0 && key0 + kTile > a.sinks && key0 < window_from(it.hi - 1, a.window));
}

// Where a CTA is in its range; every role walks it by itself.
struct Walk {
  int b, h, block, u0, left;
};

struct Start {
  Walk w;
  Request r;       // of w.b
  // the CTA has the last tile of an item that began in an earlier range: the
  // item's rows, and the unit of its first tile
  int joins, row0, ntok, head0;
  long long unit;
  long long each, more;  // units per CTA; the first `more` have one more
};

// a / b of non-negative numbers below 2^62, b > 0; short for 32 bits, and small
// for more (64-bit division is 350 instructions at every place it stands).
MOE_DEV long long divide(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  unsigned long long q = 0, r = 0;
#pragma unroll 1
  for (int i = 61; i >= 0; --i) {
    r = 2 * r + (a >> i & 1);
    q *= 2;
    if (r >= (unsigned long long)b) {
      r -= b;
      ++q;
    }
  }
  return q;
}

// The CTA's range: prefix sums over the requests' units (units_of(p, item): how
// many there are, and which tiles begin before one), then the place of its first
// one. most_ranges(p, total, two): how many ranges that many units are cut into at
// most, `two` when a request has more rows than a query tile. The first
// kPlanThreads threads call it, warps converged; `count` [MOE_MAX_REQUESTS] and
// `part` [8] are shared memory. (Every loop stays a loop: unrolled, this took a
// quarter of the kernel's instructions, which are fetched anew by every launch.)
template <class Params>
MOE_DEV void find_start(const Params& p, long long* count, long long* part, Start* out) {
  const auto& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int fixed = p.block, H = a.cache.n_kv_heads, B = a.n_requests;
  constexpr uint32_t kAll = 0xffffffffu;
  // units of every request for one key head: a request of one block by its
  // own thread, longer ones by the warp (every eighth its, so that a few are shared)
  int any_two = 0;
#pragma unroll 1
  for (int b0 = warp; b0 < B; b0 += kPlanThreads) {
    const int b = b0 + lane * (kPlanThreads / 32);
    Request mine = {0, 0, 0};
    bool bad = false;
    if (b < B) mine = request(a, p.page_shift, b, &bad);
    if (bad && blockIdx.x == 0) report_error(a.err, ERR_CHECK, 0xA20);
    long long units = 0;
    any_two |= mine.q > p.tpt;  // query tiles
    uint32_t todo = __ballot_sync(kAll, mine.q > 0);
    const uint32_t longer = __ballot_sync(kAll, mine.q > fixed);
    // first all short ones together (a turn of their own threads), then the
    // long ones one after the other
#pragma unroll 1
    while (todo) {
      const bool together = (todo & ~longer) != 0;
      const int from = together ? lane : __ffs(todo) - 1;
      todo &= together ? longer : todo - 1;
      Request r;
      r.first = 0;
      r.q = __shfl_sync(kAll, mine.q, from);
      r.len = __shfl_sync(kAll, mine.len, from);
      const bool skip = together && (r.q == 0 || r.q > fixed);
      long long n = 0;
#pragma unroll 1
      for (int q = together ? 0 : lane; !skip && q * fixed < r.q; q += 32)
        n += units_of(p, make_item(a, r, q, fixed)).all;
      if (!together) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(kAll, n, o);
      }
      if (together ? !skip : lane == from) units = n;
    }
    if (b < B) count[b] = units;
  }
  asm volatile("bar.sync 1, 256;" ::: "memory");
  const int per = (B + kPlanThreads - 1) / kPlanThreads, mine0 = tid * per;
  long long sum = 0;
#pragma unroll 1
  for (int b = mine0; b < min(mine0 + per, B); ++b) sum += count[b];
  long long incl = sum;
#pragma unroll 1
  for (int o = 1; o < min(B, 32); o <<= 1) {
    const long long t = __shfl_up_sync(kAll, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == min(B, 32) - 1) part[warp] = incl;
  // whether a request has more rows than a query tile
  int two = any_two;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 p, %0, 0;\n\t"
      "bar.red.or.pred q, 1, 256, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "+r"(two)::"memory");
  long long before = incl - sum, total = 0;
#pragma unroll 1
  for (int w = 0; w < kPlanThreads / 32 && w * 32 * per < B; ++w) {
    if (w < warp) before += part[w];
    total += part[w];
  }
  total *= H;
  before *= H;
  sum *= H;
  // the first `more` ranges are one unit longer than the others
  const long long C = min((long long)gridDim.x, most_ranges(p, total, two)), c = blockIdx.x;
  const long long each = C > 0 ? divide(total, C) : 0, more = total - each * C;
  const long long w0 = c * each + min(c, more), w1 = c < C ? w0 + each + (c < more ? 1 : 0) : w0;
  if (tid == 0) {
    out->w.b = 0;
    out->w.left = (int)(w1 - w0);
    out->each = each;
    out->more = more;
  }
  // the warp with the request whose units hold w0 looks through its blocks
  const uint32_t here = __ballot_sync(kAll, w1 > w0 && w0 >= before && w0 < before + sum);
  if (here == 0) return;
  const int from = __ffs(here) - 1;
  int b = __shfl_sync(kAll, mine0, from);
  long long rem = w0 - __shfl_sync(kAll, before, from);
#pragma unroll 1
  while (rem >= count[b] * H) rem -= count[b++] * H;
  const int h = (int)divide(rem, count[b]);
  rem -= h * count[b];
  bool bad;
  const Request r = request(a, p.page_shift, b, &bad);
#pragma unroll 1
  for (int q0 = 0; q0 * fixed < r.q; q0 += 32) {
    const int q = q0 + lane;
    Item it;
    decltype(units_of(p, it)) units;
    long long n = 0, upto;
    if (q * fixed < r.q) {
      it = make_item(a, r, q, fixed);
      units = units_of(p, it);
      n = units.all;
    }
    upto = n;
#pragma unroll 1
    for (int o = 1; o < 32 && (q0 + o) * fixed < r.q; o <<= 1) {
      const long long t = __shfl_up_sync(kAll, upto, o);
      if (lane >= o) upto += t;
    }
    if (rem < upto && rem >= upto - n) {
      const long long u0 = rem - (upto - n);
      out->w.b = b;
      out->w.h = h;
      out->w.block = q;
      out->w.u0 = (int)u0;
      out->r = r;
      const int t0 = units.tiles((int)u0);
      out->joins = t0 > 0 && t0 < it.n && units.tiles((int)min(n, u0 + w1 - w0)) == it.n;
      out->row0 = it.row0;
      out->ntok = it.ntok;
      out->head0 = h * a.group;
      out->unit = w0 - u0 + units.cost;
    }
    const long long block_sum = __shfl_sync(kAll, upto, 31);
    if (rem < block_sum) return;
    rem -= block_sum;
  }
}

// Bounded wait that gives up at once when any role of the CTA has: `lost`
// then holds the site of the first wait given up, which is reported at the
// kernel's end. Kept short, for it stands in twenty places: the kernel's warps
// run four different programs, and what does not fit the SM's instruction
// cache is fetched again at every turn of an item. A try suspends the warp for
// up to kTryNs; the limit is about half a second of them.
constexpr uint32_t kTryNs = 2000u;
constexpr int kTries = 1 << 18;
MOE_DEV bool try_longer(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity), "r"(kTryNs)
      : "memory");
  return done != 0;
}
MOE_DEV bool try_now(uint64_t* bar, uint32_t parity) {  // without suspending
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
MOE_DEV bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* lost, int site) {
  bool done = mbar_try_wait(bar, parity);
#pragma unroll 1
  for (int i = 0; !done && i < kTries && *lost == 0; ++i) done = try_longer(bar, parity);
  if (!done && *lost == 0) *lost = site;
  return done;
}

MOE_DEV void mbar_inval(uint64_t* bar) {
  asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
MOE_DEV void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

MOE_DEV uint32_t low_bits(int n) {  // the n lowest bits; none for n ≤ 0, all for n ≥ 32
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

MOE_DEV float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

MOE_DEV float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Two fp32 operations in one instruction.
MOE_DEV uint64_t pair(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
MOE_DEV uint64_t pair_f(float lo, float hi) {
  return pair(__float_as_uint(lo), __float_as_uint(hi));
}
MOE_DEV void split(uint64_t v, float* lo, float* hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(v));
}
MOE_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
MOE_DEV uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
MOE_DEV uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 1 / Σ of a row's weights; 0 for a row that sees no key. NaN among the scores a
// row sees makes its Σ, and so its result, NaN.
MOE_DEV float inverse(float sum) { return sum == 0.f ? 0.f : 1.f / sum; }

// A part is waited for this long: ranges take equal times, but one that is gone
// through again (see Misc::bad) five times as long as the others, and a prompt
// of 128 k tokens takes 0.1 s.
constexpr unsigned long long kJoinLimitNs = 2000ull * 1000ull * 1000ull;
// What stands in `left` for a part that is no longer waited for (calls' numbers
// are odd).
MOE_DEV unsigned long long given_up(unsigned long long call) { return call ^ 1ull; }
MOE_DEV unsigned long long exchange(unsigned long long* word, unsigned long long v) {
  unsigned long long old;
  asm volatile("atom.exch.release.gpu.global.b64 %0, [%1], %2;"
               : "=l"(old)
               : "l"(word), "l"(v)
               : "memory");
  return old;
}

// Rows before the first request's and behind the last one's become zeros; the
// softmax threads of all CTAs share them.
template <int kDim, class Args>
__device__ __noinline__ void clear_rows(const Args& a) {
  const int first = min(max(a.q_start[0], 0), a.n_tokens);
  const int last = min(max(a.q_start[a.n_requests], first), a.n_tokens);
  const int64_t n = (int64_t)(first + (a.n_tokens - last)) * a.n_heads * (kDim / 8);
  for (int64_t i = (int64_t)blockIdx.x * 512 + threadIdx.x - 128; i < n; i += gridDim.x * 512) {
    const int64_t row = i / (kDim / 8);
    const int64_t t = row / a.n_heads, token = t < first ? t : t - first + last;
    uint16_t* to = static_cast<uint16_t*>(a.out) + token * a.out_token_stride +
                   (row - t * a.n_heads) * a.out_head_stride;
    reinterpret_cast<uint4*>(to)[i % (kDim / 8)] = make_uint4(0, 0, 0, 0);
  }
}

// A number that no other call of the process, and no leftover word in a
// workspace, has but by a chance of 2^-64: a count from a start taken from
// the clock and an address, its bits mixed by multiplications and shifts.
inline unsigned long long call_number() {
  static std::atomic<unsigned long long> next{
      (unsigned long long)std::chrono::steady_clock::now().time_since_epoch().count() * 4096ull ^
      (unsigned long long)reinterpret_cast<uintptr_t>(&next)};
  unsigned long long v = next.fetch_add(1, std::memory_order_relaxed) * 0x9e3779b97f4a7c15ull;
  v = (v ^ (v >> 31)) * 0xd6e8feb86659fd93ull;
  return (v ^ (v >> 32)) | 1ull;
}

}  // namespace moe
