// attend.cu — attention of every request's new tokens over its paged cache:
// causal, optionally within a sliding window beside a few first keys that
// stay visible.
//
// For a query row q at position p, with s_j = scale·(q·k_j) over the keys it
// sees, out = Σ_j e^(s_j − m) v_j / Σ_j e^(s_j − m), m = max_j s_j. The
// reference m and the two sums are carried along in one pass over the keys:
// when the maximum grows from m to m', what has been summed so far is
// multiplied by e^(m − m'). Partial results over disjoint sets of keys join
// in the same way, so the keys of one row may be cut among CTAs.
//
// Tiles. The query heads that share a key head read the same keys, so their
// rows go together: a tile is 128 rows, (token, head of the group), and the
// scores of 128 keys are one 128 × 128 product S = Q·Kᵀ on the tensor cores
// (tcgen05, Q and K from shared memory), the result O += P·V another one (P
// from tensor memory). Each CTA runs two such streams against each other —
// while the tensor cores work for one, the other's softmax runs — on
//   two query tiles of the same keys, when a block of tokens fills more than
//   one tile (each key tile is then read once for 256 rows), or
//   the even and the odd key tiles of one query tile (verification passes of
//   a few tokens: bound by reading the cache), joined at the end, or
//   two whole items of a request that differ in their key head only, where the
//   CTA has both: nothing is joined, and an item's turn is one for both.
//
// Work. An item is (request, key head, block of tokens); its length is the
// number of 128-key tiles its rows see, weighted by what they cost. All items'
// tiles in a row are cut into equal ranges, one per CTA, wherever the cuts
// fall: every SM has the same work whatever the mix of long and short
// requests. The lengths are on the device: every CTA works out the cuts from
// them by itself. A CTA whose range ends inside an item leaves (O, m, Σ) of
// the item's rows in the workspace, and the CTA with the item's last tile
// joins the parts in key order, so results do not depend on scheduling. It
// waits (bounded) for lower-numbered CTAs only, which leave their parts
// before they wait themselves.
//
// Warps (one CTA per SM):
//   0, 2   TMA: key and value tiles into a ring, a box per page and 64 columns,
//          every other box each; warp 2 also query tiles into two slots, the
//          next as soon as one is free
//   1, 3   MMA issue of stream 0 and of stream 1; they also clear value rows
//          that no row of the item sees
//   4-7    softmax of stream 0 over the first 64 keys of a tile, one thread per
//          row, and a share of its results out
//   8-11   the same over the last 64 keys; the two halves agree on a row's
//          maximum through shared memory
//   12-19  the same for stream 1
//
// What bounds it; 32 query heads on 8 key heads of 128 bf16 columns where nothing
// else is said:
//   verification passes (64 requests of 1 to 9 tokens, caches up to 16000 keys,
//   906 MB): 153 us, 5.9 TB/s, 87 % of a copy's rate. The rest is the start
//   (plan 2 us, first loads 3), turns between items, during which the ring
//   holds only 2.5 tiles, and the joins (2 us). Windows of 4096 keys of 56
//   heads: 144 us for 804 MB; tiles at the windows' ends cost 7 % more bytes.
//   Long prompt chunks (957 GFLOP): 670 us cold and 720 us under the power
//   cap, 1.43 and 1.33 PFLOP/s. A stream's chain of softmax (1450 cycles a
//   tile) and products (1024, and 475 of hand-overs) runs beside the other
//   stream's: the tensor cores work 70 % of a period. Tensor memory is full, so
//   a stream's next scores cannot be computed beside its weights.
//   A mixed batch (3 prompt chunks, 20 passes, 56 heads of 64 columns, pages of
//   16, 69 MB): 33 us, of which 25 are the longest range's item turns and
//   small boxes, the others the start and one join.
//   A prompt of 512 tokens: 18 us; 200 passes within windows of 512 keys: 122 us,
//   for an item's turn (products, results out, the next item's place: 3 us)
//   stands against 5 tiles' loads, or a pair's against 10. Without pairs this took
//   125 us, and 40 passes of 16 heads over 8 to 71 keys 21.1 for 19.
//   One pass of 5 tokens over 777 keys: 12 to 13 us by the card, one chain of
//   plan (2), loads and products (5), a part's hand-over (2), join (1.2) and the
//   launch.
#include <limits.h>
#include <math.h>
#include <string.h>

#include <atomic>
#include <chrono>

#include "attend_mma.cuh"
#include "batch_launch.h"
#include "common.cuh"
#include "round16.cuh"
#include "tmap.h"

namespace moe {
namespace {

constexpr int kTile = 128;        // rows of a query tile, keys of a key tile
constexpr int kThreads = 640;
constexpr int kHalf = kTile / 2;  // keys of one softmax thread
constexpr int kMaxCtas = 160;     // workspace slots are sized for this many
constexpr int kPlanThreads = 256;
// What an item costs beside its tiles when the work is cut, in units: a key
// tile is one unit for a block of one query tile, and two for a block of two,
// which are gone through beside each other but by all of the CTA's warps.
// (Three prompt chunks among 20 passes, 8 key heads of 64 columns: 33.4 us; with
// 1 and 3 units for an item 36.5 and 35.2; with one unit for either kind of tile
// 38.0. 200 passes over caches of up to 6000 keys: 243 us, with 3 units 248.)
constexpr int kItemUnits = 2;
// The reference m follows the row's maximum only when that has grown by more
// than this (in powers of two): until then weights are up to 2^8 instead of
// 1, which fp32 sums and both 16-bit types hold, and O needs no rescaling.
constexpr float kGrow = 8.f;
// Registers per thread: launched with 96, the 16 softmax warps take 104 and
// the 4 others leave 64 (4·104 + 64 = 5·96).
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 104, kOtherRegs = 64;

template <int kDim>
struct Sizes {
  static constexpr int kTileBytes = kTile * kDim * 2;
  static constexpr int kStages = kDim == 128 ? 5 : 10;
  static constexpr int kOffRing = 2 * kTileBytes;  // behind the query slots
  static constexpr int kOffMisc = kOffRing + kStages * kTileBytes;
  static constexpr int kMiscBytes = 512 + 2048;  // Misc, then the streams' row statistics
  static constexpr int kSmem = kOffMisc + kMiscBytes;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // one slot of the workspace: O as [kDim/4][256 rows] float4, then m and Σ
  static constexpr size_t kSlotFloats = size_t(2 * kTile) * (kDim + 2);
};

struct Params {
  CUtensorMap kmap, vmap, qmap;
  AttendArgs a;
  int page_shift;
  int tpt;       // tokens per query tile, 128 / group
  int block;     // tokens per block, tpt or 2·tpt
  float* part;   // [2 per CTA][kSlotFloats]
  // [CTAs]: `call` when the CTA has left the part of its last item. The CTA
  // that reads it sets it to 0, for a replayed graph's call has its number
  // again; what an unused workspace holds is not `call`, a number of 64 mixed
  // bits that no two calls share.
  unsigned long long* left;
  unsigned long long call;
};

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
MOE_DEV Request request(const AttendArgs& a, int page_shift, int b, bool* bad) {
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
MOE_DEV Item make_item(const AttendArgs& a, const Request& r, int block, int fixed) {
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
MOE_DEV bool some_see(const AttendArgs& a, int pos0, int hi, int key) {
  return key > pos0 || (a.window > 0 && key >= a.sinks && key < window_from(hi - 1, a.window));
}
MOE_DEV bool tile_some_see(const AttendArgs& a, const Item& it, int key0) {
  return key0 + kTile - 1 > it.pos0 ||
         (a.window > 0 && key0 + kTile > a.sinks && key0 < window_from(it.hi - 1, a.window));
}

// An item's units: first `cost`, then one for every key tile of a block of one
// query tile, two for one of a block of two. A tile belongs to the CTA whose
// range has its first unit.
struct Units {
  int cost, each, all;
  MOE_DEV int tiles(int u) const {  // that begin before unit u
    return (max(0, u - cost) + each - 1) >> (each - 1);
  }
};
MOE_DEV Units units_of(const Params& p, const Item& it) {
  Units u;
  u.cost = it.hi > 0 ? kItemUnits : 0;  // (rows that see nothing are only cleared)
  u.each = it.ntok > p.tpt ? 2 : 1;
  u.all = u.cost + it.n * u.each;
  return u;
}

// Where a CTA is in its range; every role walks it by itself.
struct Walk {
  int b, h, block, u0, left;
};

// The CTA's part of an item: tiles [t0, t1). Or two whole items of one request
// that differ in their key head only (`pair`), a stream for each: the ring's
// tile j is then tile j / 2 of head h + j % 2.
struct Part {
  Item it;
  int t0, t1;
  int n;     // tiles of the ring
  bool two;  // the block's tokens fill more than one query tile
  int pair;  // 0 or 1
  MOE_DEV int tile(int j) const { return tile_of(it, t0 + (j >> pair)); }
};

// The next part of the walk with tiles in it, which is then behind the walk;
// false when there is none. w keeps the part's request and key head in b, h
// until the next call moves on.
struct Walker {
  const Params& p;
  Walk w;
  Request r;
  int b, h;  // of the present part

  MOE_DEV Walker(const Params& prm, const Walk& start, const Request& first)
      : p(prm), w(start), r(first), b(start.b), h(start.h) {}

  MOE_DEV bool next(Part* out) {
    const int fixed = p.block;
    while (w.left > 0) {
      const Item it = make_item(p.a, r, w.block, fixed);
      const Units units = units_of(p, it);
      const int u1 = min(w.u0 + w.left, units.all);
      out->it = it;
      out->t0 = units.tiles(w.u0);
      out->t1 = units.tiles(u1);
      out->two = it.ntok > p.tpt;
      b = w.b;
      h = w.h;
      const bool whole = out->t0 == 0 && out->t1 == it.n;
      w.left -= u1 - w.u0;
      w.u0 = 0;
      out->pair = 0;
      if (whole && !out->two && r.q <= fixed && w.h + 1 < p.a.cache.n_kv_heads &&
          units.tiles(w.left) >= it.n) {
        out->pair = 1;
        w.left -= min(w.left, units.all);
        ++w.h;
      }
      out->n = (out->t1 - out->t0) << out->pair;
      if (w.left > 0 && ++w.block * fixed >= r.q) {
        w.block = 0;
        if (++w.h == p.a.cache.n_kv_heads) {
          w.h = 0;
          bool bad;
          do {
            r = request(p.a, p.page_shift, ++w.b, &bad);
          } while (r.q == 0 && w.b + 1 < p.a.n_requests);
        }
      }
      if (out->t1 > out->t0) return true;
    }
    return false;
  }
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

// The CTA's range: prefix sums over the requests' units, then the place of
// its first one. The first kPlanThreads threads call it, warps converged;
// `count` [MOE_MAX_REQUESTS] and `part` [8] are shared memory. (Every loop
// stays a loop: unrolled, this took a quarter of the kernel's instructions,
// which are fetched anew by every launch.)
MOE_DEV void find_start(const Params& p, long long* count, long long* part, Start* out) {
  const AttendArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int fixed = p.block, H = a.cache.n_kv_heads, B = a.n_requests;
  constexpr uint32_t kAll = 0xffffffffu;
  // units of every request for one key head: a request of one block by its
  // own thread, longer ones by the warp
  int any_two = 0;
#pragma unroll 1
  for (int b0 = warp * 32; b0 < B; b0 += kPlanThreads) {
    const int b = b0 + lane;
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
  // Units of a range, at least: 2 where a request has more rows than a query
  // tile. In blocks of two every range inside an item then begins a tile; in
  // blocks of one, ranges of one tile would save less than their joins cost
  // (three short prompts among three passes, 13.5 us for 11.7).
  int least = any_two;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 p, %0, 0;\n\t"
      "bar.red.or.pred q, 1, 256, p;\n\t"
      "selp.s32 %0, 2, 1, q;\n\t}"
      : "+r"(least)::"memory");
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
  const long long C = min((long long)gridDim.x, total >> (least - 1)), c = blockIdx.x;
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
    Units units;
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
MOE_DEV uint64_t pair_f(float lo, float hi) { return pair(__float_as_uint(lo), __float_as_uint(hi)); }
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

// 1 / Σ of a row's weights; 0 for a row that sees no key. NaN among the scores a
// row sees makes its Σ, and so its result, NaN.
MOE_DEV float inverse(float sum) { return sum == 0.f ? 0.f : 1.f / sum; }

// Of two values of V, which are not finite: bit 15 of the lower, 31 of the upper.
template <bool kF16>
MOE_DEV uint32_t not_finite(uint32_t w) {
  return ((w & (kF16 ? 0x7c007c00u : 0x7f807f80u)) + (kF16 ? 0x04000400u : 0x00800080u)) &
         0x80008000u;
}
template <bool kF16>
MOE_DEV uint32_t only_finite(uint32_t w) {  // zeros in their place
  return w & ~((not_finite<kF16>(w) >> 15) * 0xffffu);
}
template <bool kF16>
MOE_DEV float widen(uint32_t v16) {
  return kF16 ? __half2float(__ushort_as_half((unsigned short)v16)) : __uint_as_float(v16 << 16);
}

// v[i] of lane 4q + j  <->  v[j] of lane 4q + i.
MOE_DEV uint4 shfl_xor4(uint4 v, int mask) {
  return make_uint4(__shfl_xor_sync(0xffffffffu, v.x, mask), __shfl_xor_sync(0xffffffffu, v.y, mask),
                    __shfl_xor_sync(0xffffffffu, v.z, mask), __shfl_xor_sync(0xffffffffu, v.w, mask));
}
MOE_DEV void quad_transpose(uint4 (&v)[4], int lane) {
#pragma unroll
  for (int bit = 1; bit <= 2; bit <<= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & bit) continue;
      // the lane without the bit sends v[i | bit], the lane with it v[i]
      const uint4 got = shfl_xor4(up ? v[i] : v[i | bit], bit);
      if (up) {
        v[i] = got;
      } else {
        v[i | bit] = got;
      }
    }
  }
}

// The rows of `out` of an item's rows.
struct OutRows {
  uint16_t* first;
  int64_t token, head;
  int group;
  MOE_DEV OutRows(const AttendArgs& a, const Start& st)
      : first(static_cast<uint16_t*>(a.out) + (int64_t)st.row0 * a.out_token_stride +
              (int64_t)st.head0 * a.out_head_stride),
        token(a.out_token_stride), head(a.out_head_stride), group(a.group) {}
  MOE_DEV uint16_t* operator[](int r) const {
    const int t = r / group;
    return first + t * token + (r - t * group) * head;
  }
};

// Where a part of the CTA's row `prow` stands: its slot, and behind O the
// statistics.
template <int kDim>
MOE_DEV const float* part_of(const Params& p, int cta, bool ends) {
  return p.part + (size_t)(2 * cta + (ends ? 0 : 1)) * Sizes<kDim>::kSlotFloats;
}
template <int kDim>
constexpr size_t kStats = size_t(2 * kTile) * kDim;

// The parts of an item joined in key order, those of CTAs `first` to this one.
// Few rows, all of the first tile: a thread has 4 columns of one and loads 8
// parts at once.
template <int kDim, bool kF16>
MOE_DEV void join_few(const Params& p, const Start& st, int first, int rows) {
  const OutRows out(p.a, st);
  const int last = blockIdx.x;
#pragma unroll 1
  for (int i = threadIdx.x - 128; i < rows * (kDim / 4); i += 512) {
    const int c4 = i / rows, row = i - c4 * rows;
    float m = -INFINITY, sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int c0 = first; c0 <= last; c0 += 8) {
      float mc[8], sc[8];
      float4 oc[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        mc[j] = -INFINITY;
        sc[j] = 0.f;
        oc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c0 + j <= last) {
          const float* part = part_of<kDim>(p, c0 + j, c0 + j == last);
          mc[j] = __ldcg(part + kStats<kDim> + row);
          sc[j] = __ldcg(part + kStats<kDim> + 2 * kTile + row);
          oc[j] = __ldcg(reinterpret_cast<const float4*>(part) + c4 * (2 * kTile) + row);
        }
      }
      float top = m;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, mc[j]);
      if (top == -INFINITY) {                      // (the parts hold zeros, or sums of NaN)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += sc[j];
        continue;
      }
      const float keep = exp2_approx(m - top);
      m = top;
      sum *= keep;
      o = make_float4(o.x * keep, o.y * keep, o.z * keep, o.w * keep);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float add = exp2_approx(mc[j] - top);
        sum = fmaf(sc[j], add, sum);
        o.x = fmaf(oc[j].x, add, o.x);
        o.y = fmaf(oc[j].y, add, o.y);
        o.z = fmaf(oc[j].z, add, o.z);
        o.w = fmaf(oc[j].w, add, o.w);
      }
    }
    const float inv = inverse(sum);
    *reinterpret_cast<uint2*>(out[row] + c4 * 4) =
        make_uint2(round16<kF16>(o.x * inv, o.y * inv), round16<kF16>(o.z * inv, o.w * inv));
  }
}

// Many rows: a thread has 32 columns of one, and a warp's stores cover 64 bytes
// of 8 rows each, as where an item ends. (With 16 columns, two parts at once
// and stores of 8 bytes, a prompt of 512 tokens took 19.4 us for 17.9.)
template <int kDim, bool kF16>
MOE_DEV void join_many(const Params& p, const Start& st, int first, int rows) {
  const OutRows out(p.a, st);
  const int last = blockIdx.x, lane = threadIdx.x & 31;
  const int per_tile = p.tpt * p.a.group, padded = (rows + 31) & ~31;
#pragma unroll 1
  for (int i = threadIdx.x - 128; i < padded * (kDim / 32); i += 512) {
    const int c = i / padded * 32, row = i % padded;
    // rows of the second tile start at 128
    const int prow = row < per_tile ? row : kTile + row - per_tile;
    float m = -INFINITY, sum = 0.f;
    float o[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) o[k] = 0.f;
#pragma unroll 1
    for (int cta = first; row < rows && cta <= last; ++cta) {
      const float* part = part_of<kDim>(p, cta, cta == last);
      const float mc = __ldcg(part + kStats<kDim> + prow);
      const float sc = __ldcg(part + kStats<kDim> + 2 * kTile + prow);
      float4 oc[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        oc[k] = __ldcg(reinterpret_cast<const float4*>(part) + (c / 4 + k) * (2 * kTile) + prow);
      const float top = fmaxf(m, mc);
      if (top == -INFINITY) {                      // (the part holds zeros, or a sum of NaN)
        sum += sc;
        continue;
      }
      const float keep = exp2_approx(m - top), add = exp2_approx(mc - top);
      m = top;
      sum = fmaf(sc, add, sum * keep);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        o[4 * k] = fmaf(oc[k].x, add, o[4 * k] * keep);
        o[4 * k + 1] = fmaf(oc[k].y, add, o[4 * k + 1] * keep);
        o[4 * k + 2] = fmaf(oc[k].z, add, o[4 * k + 2] * keep);
        o[4 * k + 3] = fmaf(oc[k].w, add, o[4 * k + 3] * keep);
      }
    }
    __syncwarp();
    const float inv = inverse(sum);
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k].x = round16<kF16>(o[8 * k] * inv, o[8 * k + 1] * inv);
      v[k].y = round16<kF16>(o[8 * k + 2] * inv, o[8 * k + 3] * inv);
      v[k].z = round16<kF16>(o[8 * k + 4] * inv, o[8 * k + 5] * inv);
      v[k].w = round16<kF16>(o[8 * k + 6] * inv, o[8 * k + 7] * inv);
    }
    quad_transpose(v, lane);
    const uint64_t dst = reinterpret_cast<uint64_t>(out[row] + c);
    const int quad = lane & ~3;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint64_t to = __shfl_sync(0xffffffffu, dst, quad + k);
      if (row - (lane & 3) + k < rows)
        reinterpret_cast<uint4*>(to)[lane & 3] = v[k];
    }
  }
}

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

// All softmax threads of the CTA that has the item's last tile call it. (What
// the other CTAs' threads left is ordered before their flags' releases by
// their barrier, and before this CTA's reads by the acquires and this one.)
template <int kDim, bool kF16>
MOE_DEV void join_parts(const Params& p, const Start& st, volatile int* lost) {
  const AttendArgs& a = p.a;
  // the CTA with the item's first tile
  const long long head = st.more * (st.each + 1);
  const int first = (int)(st.unit < head ? divide(st.unit, st.each + 1)
                                         : st.more + divide(st.unit - head, st.each));
  const int last = blockIdx.x;
  const int tid = threadIdx.x - 128;
  if (first + tid < last) {
    unsigned long long* word = p.left + first + tid;
    const unsigned long long t0 = global_ns();
    for (unsigned int i = 0;; ++i) {
      unsigned long long v;
      asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(word) : "memory");
      if (v == p.call) break;
      if ((i & 63u) == 63u && (*lost || global_ns() - t0 > kJoinLimitNs)) {
        *lost = 0xA70;
        // a part that comes later is not to be taken for a replayed graph's,
        // whose call has the same number: its CTA finds this and clears the word
        if (exchange(word, given_up(p.call)) == p.call) break;
        word = nullptr;
        break;
      }
    }
    if (word) *word = 0ull;
  }
  asm volatile("bar.sync 2, 512;" ::: "memory");
  const int rows = st.ntok * a.group;
  if (rows * (kDim / 4) <= 1024)
    join_few<kDim, kF16>(p, st, first, rows);
  else
    join_many<kDim, kF16>(p, st, first, rows);
}

// Rows before the first request's and behind the last one's become zeros; the
// softmax threads of all CTAs share them.
template <int kDim>
__device__ __noinline__ void clear_rows(const AttendArgs& a) {
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

// The second time through the range (see Misc::bad), by one warp: of a tile of
// V, what is not finite in rows that some rows of the item see and others do
// not becomes zeros.
template <int kDim, bool kF16>
__device__ __noinline__ void take_out(const AttendArgs& a, int v_at, int key0, int pos0, int lo,
                                      int hi, int sk) {
  extern __shared__ __align__(1024) unsigned char smem[];
#pragma unroll 1
  for (int i = threadIdx.x & 31; i < kTile * (kDim / 64) * 8; i += 32) {
    const int key = key0 + ((i >> 3) & (kTile - 1));
    if (!some_see(a, pos0, hi, key) || key >= hi || (key < lo && key >= sk)) continue;
    uint4* at = reinterpret_cast<uint4*>(smem + v_at + i * 16);
    const uint4 x = *at;
    *at = make_uint4(only_finite<kF16>(x.x), only_finite<kF16>(x.y), only_finite<kF16>(x.z),
                     only_finite<kF16>(x.w));
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// And what take_out took is added to the O of the rows that see its key (their
// weight of it is not 0), in this thread's columns [c0, c1).
template <int kDim, bool kF16>
__device__ __noinline__ void add_not_finite(const Params& p, const Part& pt, int b, int kv_head,
                                            int first, int step, int hi, int lo, uint32_t o_addr,
                                            int c0, int c1) {
  const AttendArgs& a = p.a;
  const moe_kv_cache& cache = a.cache;
  const int32_t* table = a.block_table + (size_t)b * a.max_blocks;
#pragma unroll 1
  for (int c = c0; c < c1; c += 32) {
    uint32_t o[32];
    umma::ld_x32(o_addr + c, o);
    umma::wait_ld();
#pragma unroll 1
    for (int j = first; j < pt.n; j += step) {
      const int key0 = pt.tile(j) * kTile;
      if (!tile_some_see(a, pt.it, key0)) continue;
      const int end = min(key0 + kTile, pt.it.hi);
#pragma unroll 1
      for (int key = key0; key < end; ++key) {
        if (!some_see(a, pt.it.pos0, pt.it.hi, key) || (key < pt.it.lo && key >= pt.it.sk)) continue;
        const int page = table[key >> p.page_shift];
        if (page < 0 || page >= cache.n_pages) continue;
        const uint4* v = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(cache.v) + page * cache.page_stride +
            (key & ((1 << p.page_shift) - 1)) * cache.token_stride + kv_head * cache.head_stride +
            c);
        const bool seen = key < hi && (key >= lo || key < a.sinks);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 x = v[i];
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t bad = not_finite<kF16>(w[k]);
            const int at = 8 * i + 2 * k;
            if (seen && (bad & 0x8000u))
              o[at] = __float_as_uint(__uint_as_float(o[at]) + widen<kF16>(w[k] & 0xffffu));
            if (seen && (bad >> 31))
              o[at + 1] = __float_as_uint(__uint_as_float(o[at + 1]) + widen<kF16>(w[k] >> 16));
          }
        }
      }
    }
    umma::st_x32(o_addr + c, o);
    umma::wait_st();
  }
  umma::fence_before_sync();
}

// Barriers and words behind the ring.
struct Misc {
  uint64_t full[10], empty[10];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t turn[2], drain[2];
  Start start;
  long long part[8];
  uint32_t tmem;
  int lost;
  // Some result is not finite: the CTA goes through its range once more. A value
  // that is not finite makes NaN of rows that do not see its key: their weight is
  // 0, and 0 times it is not. Looking for such values beforehand takes a warp
  // 3000 cycles a tile, twice what a tile's softmax takes (a prompt of 8192
  // tokens 418 -> 434 us); so it is left to their effect, in the results, where
  // it costs one operation for two of them. The second time such values are
  // taken out of the tiles that not all rows see, and given to the rows that see
  // them. (One in every request: verification batch 434 us for 154, chunks 3670.)
  int bad;
};
static_assert(sizeof(Misc) <= 512, "misc words");
constexpr int kOffStat = 512;  // then [2 streams][2][128 rows] floats

// The CTA's range, by all its roles; `warp`: of the softmax warps, the others'
// are negative. kSecond: see Misc::bad.
template <int kDim, bool kF16, bool kSecond>
MOE_DEV void run_range(const Params& p, unsigned char* smem, int warp, uint32_t tmem) {
  using Z = Sizes<kDim>;
  constexpr int kHalves = kDim / 64;           // 64-column halves of a row
  constexpr int kHalfBytes = kTile * 128;
  constexpr int kStages = Z::kStages;
  const AttendArgs& a = p.a;
  Misc& m = *reinterpret_cast<Misc*>(smem + Z::kOffMisc);
  volatile int* lost = &m.lost;
  const int lane = threadIdx.x & 31;
  bool ok = true;  // no wait of this role has been lost
  auto wait = [&](uint64_t* bar, uint32_t parity, int site) {
    ok = __all_sync(0xffffffffu, ok && wait_or_abort(bar, parity, lost, site));
  };
  Part pt;

  if (!kSecond && warp < 0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  }
  if (warp == -4 || warp == -2) {
    // ------------------------------------------------------------ loaders --
    // A box takes its issuing lane 75 to 100 cycles, one lane after the other:
    // 16 boxes of a tile in small pages took one warp longer than the tile
    // took to arrive. So two warps go through the same tiles, each with every
    // other box.
    const int which = warp == -2;
    const int page = 1 << p.page_shift;
    const int rows = min(page, kTile);          // rows of a box
    const int n_pages = kTile / rows;           // pages of a tile (1 if a page spans tiles)
    const uint64_t policy = l2_evict_normal_policy();
    // this lane's boxes in the ring
    const uint32_t ring = smem_addr(smem) + Z::kOffRing + lane * rows * 128;
    constexpr uint32_t kEven = 0x55555555u;     // even lanes
    int stage = 0, slot = 0, queries = 0, q_row = 0, q_head = 0;
    uint32_t phase = 0, q_phase = 0;
    // the next query tile, if its slot is free: a box is the 128 / group
    // tokens of a tile, times the group's heads, in the order of the tile's rows
    auto try_queries = [&]() {
      if (!__all_sync(0xffffffffu, try_now(&m.q_empty[slot], q_phase ^ 1u))) return;
      if (lane == 0) {
        mbar_arrive_expect_tx(&m.q_full[slot], p.tpt * a.group * kDim * 2);
#pragma unroll
        for (int half = 0; half < kHalves; ++half)
          tma_load_3d(smem + slot * Z::kTileBytes + half * kHalfBytes, &p.qmap, half * 64, q_head,
                      q_row, &m.q_full[slot], policy);
      }
      __syncwarp();
      --queries;
      if (pt.pair) {
        q_head += a.group;
      } else {
        q_row += p.tpt;
      }
      if (slot) q_phase ^= 1u;
      slot ^= 1;
    };
    Walker walk(p, m.start.w, m.start.r);
    while (walk.next(&pt)) {
      const Item& it = pt.it;
      const int n = pt.n;
      const int lead = pt.two ? 1 : 2;          // key tiles ahead of the value tiles
      if (which) {
        queries = pt.two || pt.pair ? 2 : 1;
        q_row = it.row0;
        q_head = walk.h * a.group;
      }
      const int32_t* table = a.block_table + (size_t)walk.b * a.max_blocks;
      // this lane's page of tile j (−1: it has none, or no row of it is seen)
      auto page_of = [&](int j) {
        const int r0 = pt.tile(j) * kTile + lane * rows;
        const bool want =
            j < n && lane < n_pages && r0 < it.hi && (r0 + rows > it.lo || r0 < it.sk);
        int pg = -1;
        if (want) {
          pg = table[r0 >> p.page_shift];
          if (pg < 0 || pg >= a.cache.n_pages) {
            report_error(a.err, ERR_CHECK, 0xA21);
            pg = (int)a.cache.n_pages;          // out of the map: the box reads zeros
          }
        }
        return pg;
      };
      // Keys 0..lead-1, then values j, keys j + lead, for j = 0..n-1; and at the
      // end the queries that are still to load.
      int jk = 0, jv = 0, fetched = 0;
      int pg0 = -1, pg1 = -1, pg2 = -1, pg3 = -1;  // pages of tiles jv .. jv + 3
      while (ok && (jv < n || queries > 0)) {
#pragma unroll 1
        for (; fetched < jv + 4; ++fetched) {
          pg0 = pg1;
          pg1 = pg2;
          pg2 = pg3;
          pg3 = page_of(fetched);
        }
        const bool is_k = jk < n && jk < jv + lead, tiles = jv < n;
        const int j = is_k ? jk : jv, pg = is_k && jk != jv ? pg1 : pg0;
        const uint32_t wanted = __ballot_sync(0xffffffffu, pg >= 0);
        // a free stage of the ring, and meanwhile free slots for the queries
        bool free = false;
#pragma unroll 1
        for (int i = 0; ok && i < 64 * kTries; ++i) {
          if (queries > 0) try_queries();
          free = tiles && __all_sync(0xffffffffu, queries > 0
                                                      ? try_now(&m.empty[stage], phase ^ 1u)
                                                      : try_longer(&m.empty[stage], phase ^ 1u));
          if (free || (!tiles && queries == 0)) break;
          ok = i + 1 < 64 * kTries && __all_sync(0xffffffffu, *lost == 0);
        }
        if (!ok && *lost == 0) *lost = 0xA30;
        if (!free) continue;
        // Either loader arrives, boxes or none: a stage can then not be filled
        // and emptied twice past one of them, which would take the older phase
        // of `empty` for the one it waits for.
        if (lane == 0) {
          int mine = 0;
#pragma unroll
          for (int half = 0; half < kHalves; ++half)
            mine += __popc(wanted & (((half * n_pages) & 1) == which ? kEven : ~kEven));
          mbar_arrive_expect_tx(&m.full[stage], mine * rows * 128);
        }
        __syncwarp();
        const CUtensorMap* map = is_k ? &p.kmap : &p.vmap;
        const int row = page > kTile ? pt.tile(j) * kTile & (page - 1) : 0;
        const int head = walk.h + (j & pt.pair);
#pragma unroll
        for (int half = 0; half < kHalves; ++half)
          if (pg >= 0 && ((half * n_pages + lane) & 1) == which)
            tma_load_4d_at(ring + stage * Z::kTileBytes + half * kHalfBytes, map, half * 64, head,
                           row, pg, &m.full[stage], policy);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
        if (is_k) {
          ++jk;
        } else {
          ++jv;
        }
      }
    }
    // After a lost wait the tiles still in flight must land before the CTA
    // ends; without one, every tile has been waited for by the MMA warps.
    if (!ok) {
#pragma unroll 1
      for (int i = 0; i < 2 * 500 * (kStages + 2); ++i) {      // a millisecond for each, or two
        const int b = i / 1000;
        try_longer(b < kStages ? &m.full[b] : &m.q_full[b - kStages], i & 1);
      }
    }
  } else if (warp < 0) {
    // ---------------------------------------------------------------- MMA --
    // Both warps follow every tile of the ring and of the query slots, in
    // order: a barrier tells only the parity of its phase, so a warp that
    // passed over a tile could take an older phase for the one it wants. A
    // tile that is the other stream's alone is released as soon as it is there.
    const int s = (warp + 3) >> 1;                     // stream
    const uint32_t id_s = umma::idesc_f16(kTile, kTile, kF16, false);
    const uint32_t id_o = umma::idesc_f16(kTile, kDim, kF16, true);
    const uint32_t q_lo = umma::desc_lo(smem_addr(smem), 0);
    const uint32_t k_lo = umma::desc_lo(smem_addr(smem) + Z::kOffRing, 0);
    const uint32_t v_lo = umma::desc_lo(smem_addr(smem) + Z::kOffRing, kHalfBytes);
    const uint32_t d_s = tmem + s * 128, d_o = tmem + 256 + s * 128;
    int stage = 0;
    uint32_t phase = 0, n_q = 0, p_phase = 0, turn = s ^ 1u;
    auto next_tile = [&]() {                           // waits for the ring's next tile
      const int st = stage;
      wait(&m.full[st], phase, 0xA40);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
      return st;
    };
    auto commit = [&](uint64_t* bar) {                 // arrives when the MMAs so far are done
      if (ok) umma::commit_elect(bar);
    };
    auto pass = [&](uint64_t* bar) {                   // arrives now
      if (ok && lane == 0) mbar_arrive(bar);
      __syncwarp();
    };
    auto scores = [&](uint32_t slot, int st) {         // S = Q · Kᵀ
      if (!ok) return;
      const uint32_t q = q_lo + slot * (Z::kTileBytes >> 4), k = k_lo + st * (Z::kTileBytes >> 4);
      umma::mma4_ss(d_s, q, k, id_s, 0u);
      if (kHalves == 2) umma::mma4_ss(d_s, q + (kHalfBytes >> 4), k + (kHalfBytes >> 4), id_s, 1u);
      umma::commit_elect(&m.s_full[s]);
    };
    Walker walk(p, m.start.w, m.start.r);
    while (walk.next(&pt)) {
      const Item& it = pt.it;
      const int n = pt.n;
      const bool two = pt.two;
      // the stream sees something of a tile that begins at key0
      const int t_first = two ? s * p.tpt : 0, t_last = two && s == 0 ? p.tpt : it.ntok;
      const int hi = it.pos0 + t_last;
      const int lo =
          a.window > 0 ? window_from(it.pos0 + t_first, a.window) - (kTile - 1) : INT_MIN;
      auto sees = [&](int j) {
        const int key0 = pt.tile(j) * kTile;
        return (two || (j & 1) == s) && key0 < hi && (key0 >= lo || key0 < a.sinks);
      };
      // the query tiles: the stream's own, and the other one's
      uint32_t slot = 0;
      const bool own = two || pt.pair;                 // a query tile for either stream
      for (int q = 0; q < (own ? 2 : 1); ++q, ++n_q) {
        wait(&m.q_full[n_q & 1u], n_q >> 1 & 1u, 0xA42);
        if (!own || q == s) {
          slot = n_q & 1u;
        } else {
          pass(&m.q_empty[n_q & 1u]);
        }
      }
      const int lead = two ? 1 : 2;                    // the next key tile of the stream
      const int last = two ? n - 1 : ((n - 1 - s) & ~1) + s;  // its last tile (< s: it has none)
      bool first = true;
      if (last < 0) pass(&m.q_empty[slot]);            // no tile of its own at all
      for (int j = -lead; j < n; ++j) {
        // V_j and K_{j+lead}, in the ring's order
        const bool has_v = j >= 0, more = j + lead < n;
        const bool mine = two || (j & 1) == s;         // (lead is even where that matters)
        if (!has_v && !more) continue;
        const int vt = has_v ? next_tile() : 0;
        const int kt = more ? next_tile() : 0;
        if (!mine) {
          if (has_v) pass(&m.empty[vt]);
          if (more) pass(&m.empty[kt]);
          continue;
        }
        // rows of V that no row of the item sees may hold anything: their
        // weights are 0, and 0 · NaN is not
        const int key0 = pt.tile(j) * kTile;
        const bool now = has_v && sees(j);
        if (ok && now && (key0 + kTile > it.hi || (key0 < it.lo && key0 + kTile > it.sk))) {
          unsigned char* v = smem + Z::kOffRing + vt * Z::kTileBytes;
          for (int i = lane; i < kTile * kHalves * 8; i += 32) {
            const int key = key0 + ((i >> 3) & (kTile - 1));
            if (key >= it.hi || (key < it.lo && key >= it.sk))
              *reinterpret_cast<uint4*>(v + (size_t)i * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (kSecond && ok && now && tile_some_see(a, it, key0))
          take_out<kDim, kF16>(a, Z::kOffRing + vt * Z::kTileBytes, key0, it.pos0, it.lo, it.hi,
                               it.sk);
        if (now) wait(&m.p_full[s], p_phase, 0xA41);
        // Two query tiles take turns: a stream's P·V and its next scores are
        // issued in one piece. Were they mixed with the other's, both scores
        // would be ready late and together, both softmaxes would run at the
        // same time, and the tensor cores would wait for them.
        if (two && has_v) {
          wait(&m.turn[s], turn, 0xA44);
          turn ^= 1u;
        }
        if (now) {                                     // O (+)= P · V
          p_phase ^= 1u;
          umma::fence_after_sync();
          if (ok) {
            const uint32_t v = v_lo + vt * (Z::kTileBytes >> 4);
            umma::mma4_ts(d_o, d_s, v, id_o, first ? 0u : 1u);
            umma::mma4_ts(d_o, d_s + 32, v + (4 * 2048 >> 4), id_o, 1u);
          }
          first = false;
        }
        if (more && sees(j + lead)) scores(slot, kt);  // into S, behind the product that reads P
        if (two && has_v) pass(&m.turn[s ^ 1]);
        if (j == last && !first) commit(&m.o_full[s]);
        if (has_v) commit(&m.empty[vt]);
        if (more) commit(&m.empty[kt]);
        if (more && j + lead == last) commit(&m.q_empty[slot]);  // the last scores are issued
      }
    }
    // Every MMA, and every arrival that hangs on one, is done before tensor
    // memory is released.
    umma::commit_elect(&m.drain[s]);
#pragma unroll 1
    for (int i = 0; i < kTries && !try_longer(&m.drain[s], 0); ++i) {
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax --
    if (!kSecond) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    if (!kSecond && a.clear) clear_rows<kDim>(a);    // while the first tiles are on their way
    const int s = warp >> 3, half = warp >> 2 & 1;  // stream, and half of a tile's keys
    const int row = threadIdx.x & 127;               // row of the tile, TMEM lane
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // 32·(warp % 4) in the upper half
    const uint32_t s_addr = lanes + s * 128 + half * kHalf;
    const uint32_t p_addr = lanes + s * 128 + half * (kHalf / 2);
    const uint32_t o_addr = lanes + 256 + s * 128;
    const float to_log2 = a.scale * 1.4426950408889634f;
    const uint64_t to_log2_2 = pair_f(to_log2, to_log2);
    // fp16 weights are held 2^4 larger, so that small ones keep their bits
    const float offset = kF16 ? 4.f : 0.f;
    const int t_in = row / a.group, g_in = row - t_in * a.group;
    float* stat = reinterpret_cast<float*>(smem + Z::kOffMisc + kOffStat);
    float* mine = stat + (2 * s + half) * kTile + row;
    const float* theirs = stat + (2 * s + (half ^ 1)) * kTile + row;
    // the two warps of the same rows
    auto pair_sync = [&]() {
      asm volatile("bar.sync %0, 64;" ::"r"(3 + 4 * s + (warp & 3)) : "memory");
    };
    uint32_t s_phase = 0, o_phase = 0;
    bool open = false;                               // the last part does not end its item
    Walker walk(p, m.start.w, m.start.r);
    while (walk.next(&pt)) {
      const Item& it = pt.it;
      const int n = pt.n;
      const bool two = pt.two, own = two || pt.pair;
      const int t_first = two ? s * p.tpt : 0, t_last = two && s == 0 ? p.tpt : it.ntok;
      const int tok = t_first + t_in;
      const bool valid = t_in < p.tpt && tok < t_last;
      const bool warp_valid = __any_sync(0xffffffffu, valid);
      const int pos = it.pos0 + tok;
      const int hi = valid ? max(0, pos + 1) : 0;
      const int lo = a.window > 0 ? max(0, window_from(pos, a.window)) : 0;
      const int s_hi = it.pos0 + t_last;
      const int s_lo =
          a.window > 0 ? window_from(it.pos0 + t_first, a.window) - (kTile - 1) : INT_MIN;
      float ref = -INFINITY, sum = 0.f;
      bool began = false;
      for (int j = two ? 0 : s; j < n; j += two ? 1 : 2) {
        int key0 = pt.tile(j) * kTile;
        if (!(key0 < s_hi && (key0 >= s_lo || key0 < a.sinks))) continue;
        key0 += half * kHalf;                        // this thread's keys
        wait(&m.s_full[s], s_phase, 0xA51);
        s_phase ^= 1u;
        // (a lost wait leaves the sums wrong, and the barriers in step)
        if (warp_valid) {
          umma::fence_after_sync();
          uint32_t x[kHalf];
          umma::ld_x32(s_addr, x);
          umma::ld_x32(s_addr + 32, x + 32);
          umma::wait_ld();
          const bool whole =
              !valid || (key0 + kHalf <= hi && (key0 >= lo || key0 + kHalf <= a.sinks));
          if (!__all_sync(0xffffffffu, whole)) {
            // bit c of `seen`: key key0 + 32·w + c
#pragma unroll
            for (int w = 0; w < kHalf / 32; ++w) {
              const int at = key0 + 32 * w;
              const uint32_t seen =
                  low_bits(hi - at) & (~low_bits(lo - at) | low_bits(a.sinks - at));
#pragma unroll
              for (int c = 0; c < 32; ++c)
                x[32 * w + c] = seen >> c & 1u ? x[32 * w + c] : 0xff800000u;  // −inf
            }
          }
          float t4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) t4[i] = __uint_as_float(x[i]);
#pragma unroll
          for (int c = 4; c + 8 <= kHalf; c += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              t4[i] = max3(t4[i], __uint_as_float(x[c + 2 * i]), __uint_as_float(x[c + 2 * i + 1]));
#pragma unroll
          for (int i = 0; i < 4; ++i) t4[i] = fmaxf(t4[i], __uint_as_float(x[kHalf - 4 + i]));
          const float own = fmaxf(max3(t4[0], t4[1], t4[2]), t4[3]);
          *mine = own;
          // behind this, the other half's maximum is there, and both halves
          // have read the scores that the weights replace
          pair_sync();
          const float top = fmaxf(own, *theirs) * to_log2;
          const bool grown = top > ref + kGrow;
          if (__any_sync(0xffffffffu, grown)) {      // the same in both warps
            const float keep = grown ? exp2_approx(ref - top) : 1.f;
            if (grown) ref = top;
            sum *= keep;
            if (began) {
#pragma unroll 1
              for (int c = half * (kDim / 2); c < (half + 1) * (kDim / 2); c += 32) {
                uint32_t o[32];
                umma::ld_x32(o_addr + c, o);
                umma::wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
                umma::st_x32(o_addr + c, o);
              }
            }
          }
          const float shift = ref == -INFINITY ? 0.f : offset - ref;
          const uint64_t shift_2 = pair_f(shift, shift);
          uint64_t sums[4] = {0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < kHalf; c += 2) {
            float p0, p1;
            split(fma2(pair(x[c], x[c + 1]), to_log2_2, shift_2), &p0, &p1);
            p0 = exp2_approx(p0);
            p1 = exp2_approx(p1);
            sums[(c >> 1) & 3] = add2(sums[(c >> 1) & 3], pair_f(p0, p1));
            x[c >> 1] = round16<kF16>(p0, p1);
          }
          umma::st_x32(p_addr, x);
          float s0, s1;
          split(add2(add2(sums[0], sums[1]), add2(sums[2], sums[3])), &s0, &s1);
          sum += s0 + s1;
          umma::wait_st();
        }
        began = true;
        umma::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.p_full[s]);
      }
      // ---- results out
      const bool ends = pt.t1 == it.n, whole_item = ends && pt.t0 == 0;
      open = !ends;
      // the results of rows 4·(lane / 4) + i, for i = 0..3, and which of them exist
      const uint64_t dst = reinterpret_cast<uint64_t>(
          static_cast<uint16_t*>(a.out) + (int64_t)(it.row0 + tok) * a.out_token_stride +
          (int64_t)((walk.h + (s & pt.pair)) * a.group + g_in) * a.out_head_stride);
      const uint32_t quad_valid = __ballot_sync(0xffffffffu, valid) >> (lane & ~3) & 15u;
      uint16_t* quad_dst[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        quad_dst[i] = reinterpret_cast<uint16_t*>(__shfl_sync(0xffffffffu, dst, (lane & ~3) + i));
      if (began) {
        wait(&m.o_full[s], o_phase, 0xA52);
        o_phase ^= 1u;
        if (kSecond && ok) {
          umma::fence_after_sync();
          const Part copy = pt;                      // (pt itself stays in registers)
          add_not_finite<kDim, kF16>(p, copy, walk.b, walk.h + (s & pt.pair), two ? 0 : s,
                                     two ? 1 : 2, hi, lo, o_addr, half * (kDim / 2),
                                     (half + 1) * (kDim / 2));
        }
      }
      // the halves' sums, then (one query tile) both streams' statistics; the
      // other half has read the last maximum: O is complete, its weights are in
      *mine = sum;
      pair_sync();
      sum += *theirs;
      pair_sync();
      if (!own) *mine = half == 0 ? ref : sum;
      // factors of the two streams' O, and this thread's columns
      float f0 = 1.f, f1 = 0.f;
      int c_first = half * (kDim / 2), c_end = c_first + kDim / 2;
      if (!own) {
        // both streams hold sums of the same rows: every warp of a row joins
        // its share of the columns, 32 at least
        asm volatile("bar.sync 2, 512;" ::: "memory");
        const float ref0 = stat[row], ref1 = stat[2 * kTile + row];
        ref = fmaxf(ref0, ref1);
        f0 = ref0 == -INFINITY ? 0.f : exp2_approx(ref0 - ref);
        f1 = ref1 == -INFINITY ? 0.f : exp2_approx(ref1 - ref);
        sum = stat[kTile + row] * f0 + stat[3 * kTile + row] * f1;
        c_first = kDim == 128 ? 64 * half + 32 * s : 32 * s;
        c_end = kDim == 128 || half == 0 ? c_first + 32 : c_first;
      }
      umma::fence_after_sync();
      if (ok && warp_valid) {
        if (whole_item) {
          const float inv = inverse(sum);
          f0 *= inv;
          f1 *= inv;
        }
        // a stream that saw no key never wrote its O: what is there is not a
        // number to be scaled. (Factors of NaN are not 0. Where every row is one
        // stream's there is no other O: its place is past tensor memory's end.)
        const bool any0 = f0 != 0.f && sum != 0.f, any1 = !own && f1 != 0.f;
        const bool warp_any1 = __any_sync(0xffffffffu, any1);
        const uint32_t from = lanes + 256 + (own ? s * 128 : 0);
        float* slot = p.part + (size_t)(2 * blockIdx.x + (ends ? 0 : 1)) * Z::kSlotFloats;
        const int prow = (two ? s * kTile : 0) + row;
        uint64_t zero0 = 0, zero1 = 0;               // 0 · o, summed up
#pragma unroll 1
        for (int c = c_first; c < c_end; c += 32) {
          uint32_t o[32];
          umma::ld_x32(from + c, o);
          umma::wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i)
            o[i] = any0 ? __float_as_uint(__uint_as_float(o[i]) * f0) : 0u;
          if (warp_any1) {
            uint32_t o1[32];
            umma::ld_x32(from + 128 + c, o1);
            umma::wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (any1)
                o[i] = __float_as_uint(fmaf(__uint_as_float(o1[i]), f1, __uint_as_float(o[i])));
          }
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            zero0 = fma2(pair(o[i], o[i + 1]), 0ull, zero0);
            zero1 = fma2(pair(o[i + 2], o[i + 3]), 0ull, zero1);
          }
          if (whole_item) {
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[i].x = round16<kF16>(__uint_as_float(o[8 * i]), __uint_as_float(o[8 * i + 1]));
              v[i].y = round16<kF16>(__uint_as_float(o[8 * i + 2]), __uint_as_float(o[8 * i + 3]));
              v[i].z = round16<kF16>(__uint_as_float(o[8 * i + 4]), __uint_as_float(o[8 * i + 5]));
              v[i].w = round16<kF16>(__uint_as_float(o[8 * i + 6]), __uint_as_float(o[8 * i + 7]));
            }
            // four lanes turn their 4 rows × 4 pieces, so that a store covers
            // 64 bytes of 8 rows instead of 16 bytes of 32
            quad_transpose(v, lane);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (quad_valid >> i & 1u)
                *reinterpret_cast<uint4*>(quad_dst[i] + c + (lane & 3) * 8) = v[i];
          } else if (valid) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              reinterpret_cast<uint4*>(slot)[((c + i) >> 2) * (2 * kTile) + prow] =
                  make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
        float z0, z1;
        split(add2(zero0, zero1), &z0, &z1);
        if (valid && z0 + z1 != 0.f) *static_cast<volatile int*>(&m.bad) = 1;
        if (valid && !whole_item && half == 0 && (two || s == 0)) {
          float* st = slot + (size_t)2 * kTile * kDim;
          st[prow] = ref;
          st[2 * kTile + prow] = sum;
        }
      }
      // joined O and statistics have been read before either stream goes on
      umma::fence_before_sync();
      if (own) {
        pair_sync();
      } else {
        asm volatile("bar.sync 2, 512;" ::: "memory");
      }
    }
    // The last part is left to the CTA that ends its item, and an item that began
    // in earlier ranges joined, when all of the range's results are there: but
    // not if the range is gone through again.
    if (open || m.start.joins) {
      asm volatile("bar.sync 2, 512;" ::: "memory");
      if (kSecond || !*static_cast<volatile int*>(&m.bad)) {
        unsigned long long before = 0;               // (used at the end: it takes a while)
        if (open && threadIdx.x == 128) before = exchange(p.left + blockIdx.x, p.call);
        if (m.start.joins) join_parts<kDim, kF16>(p, m.start, lost);
        if (before == given_up(p.call)) p.left[blockIdx.x] = 0ull;
      }
    }
  }
}

template <int kStages>
MOE_DEV void init_barriers(Misc& m) {
  for (int i = 0; i < kStages; ++i) {
    mbar_init(&m.full[i], 2);                  // either loader, with the bytes of its boxes
    mbar_init(&m.empty[i], 2);
  }
  for (int s = 0; s < 2; ++s) {
    mbar_init(&m.q_full[s], 1);
    mbar_init(&m.q_empty[s], 2);
    mbar_init(&m.s_full[s], 1);
    mbar_init(&m.p_full[s], 8);
    mbar_init(&m.o_full[s], 1);
    mbar_init(&m.turn[s], 1);
    mbar_init(&m.drain[s], 1);
  }
  fence_mbar_init();
}

// The range once more, from fresh barriers. Code of its own: with the two steps
// beyond the first time's in one loop with it, registers that they hold slowed
// down every tile (a prompt of 8192 tokens 408 -> 428 us).
template <int kDim, bool kF16>
MOE_DEV void second_time(const Params& p, unsigned char* smem, int warp, uint32_t tmem) {
  using Z = Sizes<kDim>;
  Misc& m = *reinterpret_cast<Misc*>(smem + Z::kOffMisc);
  if (threadIdx.x == 0) {
    for (int i = 0; i < Z::kStages; ++i) {
      mbar_inval(&m.full[i]);
      mbar_inval(&m.empty[i]);
    }
    for (int s = 0; s < 2; ++s)
      for (uint64_t* bar : {m.q_full, m.q_empty, m.s_full, m.p_full, m.o_full, m.turn, m.drain})
        mbar_inval(bar + s);
    init_barriers<Z::kStages>(m);
  }
  __syncthreads();
  umma::fence_after_sync();
  run_range<kDim, kF16, true>(p, smem, warp, tmem);
  umma::fence_before_sync();
  __syncthreads();
}

template <int kDim, bool kF16>
__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const __grid_constant__ Params p) {
  using Z = Sizes<kDim>;
  constexpr uint32_t kCols = 512;              // S0 S1 O0 O1, 128 columns each
  const AttendArgs& a = p.a;
  extern __shared__ __align__(1024) unsigned char smem[];
  if (smem_addr(smem) & 1023u) {               // the tiles' swizzle needs it
    if (threadIdx.x == 0) report_error(a.err, ERR_CHECK, 0xA23);
    return;
  }
  Misc& m = *reinterpret_cast<Misc*>(smem + Z::kOffMisc);
  // the same value in every lane, and known to be
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0) - 4;

  if (threadIdx.x == 0) {
    init_barriers<Z::kStages>(m);
    m.lost = m.bad = 0;
    m.start.joins = 0;
  }
  if (warp == -3) umma::tmem_alloc(&m.tmem, kCols);
  if (threadIdx.x == 0) {
    prefetch_tmap(&p.kmap);
    prefetch_tmap(&p.vmap);
    prefetch_tmap(&p.qmap);
  }
  pdl_wait();
  pdl_trigger();
  // (the ring holds the plan's counts until the first tiles are on their way)
  if (threadIdx.x < kPlanThreads)
    find_start(p, reinterpret_cast<long long*>(smem + Z::kOffRing), m.part, &m.start);
  fence_proxy_async_smem();
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, m.tmem, 0);
  run_range<kDim, kF16, false>(p, smem, warp, tmem);
  umma::fence_before_sync();
  __syncthreads();
  auto finish = [&] {
    if (threadIdx.x == 0 && m.lost) report_error(a.err, ERR_TIMEOUT, m.lost);
    if (warp == -3) umma::tmem_dealloc(tmem, kCols);
  };
  if (__builtin_expect(!*static_cast<volatile int*>(&m.bad), 1)) {
    finish();
    return;
  }
  if (!*static_cast<volatile int*>(&m.lost)) {
    if (warp < 0)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kLaunchRegs));
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLaunchRegs));
    second_time<kDim, kF16>(p, smem, warp, tmem);
  }
  finish();
}

template <int kDim, bool kF16>
cudaError_t launch_t(Params& p, int ctas, cudaStream_t stream) {
  using Z = Sizes<kDim>;
  auto* kernel = attend_kernel<kDim, kF16>;
  // a bit for each device whose kernel may have that much shared memory (two
  // threads that find it missing both ask for it, to the same effect)
  static std::atomic<unsigned long long> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const unsigned long long bit = 1ull << (dev & 63);     // call_device takes devices below 64
  if (e == cudaSuccess && !(configured.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Z::kSmem);
    if (e == cudaSuccess) configured.fetch_or(bit, std::memory_order_release);
  }
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(ctas), dim3(kThreads), Z::kSmem, stream, p);
}

constexpr size_t kLeftBytes = (kMaxCtas * sizeof(unsigned long long) + 255) / 256 * 256;

// A number that no other call of the process, and no leftover word in a
// workspace, has but by a chance of 2^-64: a count from a start taken from
// the clock and an address, its bits mixed by multiplications and shifts.
unsigned long long call_number() {
  static std::atomic<unsigned long long> next{
      (unsigned long long)std::chrono::steady_clock::now().time_since_epoch().count() * 4096ull ^
      (unsigned long long)reinterpret_cast<uintptr_t>(&next)};
  unsigned long long v = next.fetch_add(1, std::memory_order_relaxed) * 0x9e3779b97f4a7c15ull;
  v = (v ^ (v >> 31)) * 0xd6e8feb86659fd93ull;
  return (v ^ (v >> 32)) | 1ull;
}

}  // namespace

size_t attend_workspace_bytes(int head_dim) {
  const size_t slot = head_dim == 128 ? Sizes<128>::kSlotFloats : Sizes<64>::kSlotFloats;
  return kLeftBytes + 2 * kMaxCtas * slot * sizeof(float);
}

cudaError_t launch_attend(const AttendArgs& a, int num_sms, cudaStream_t stream) {
  Params p;
  memset(&p, 0, sizeof p);
  p.a = a;
  p.page_shift = 31 - __builtin_clz(a.cache.page_size);
  p.tpt = kTile / a.group;
  p.left = static_cast<unsigned long long*>(a.workspace);
  p.part = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + kLeftBytes);
  p.call = call_number();
  const moe_kv_cache& c = a.cache;
  // [page][row][head][dim], one 64-column piece of a head's rows per box
  const cuuint64_t dims[4] = {(uint64_t)c.head_dim, (uint64_t)c.n_kv_heads, (uint64_t)c.page_size,
                            (uint64_t)c.n_pages};
  const cuuint64_t strides[3] = {(uint64_t)c.head_stride * 2, (uint64_t)c.token_stride * 2,
                               (uint64_t)c.page_stride * 2};
  const uint32_t box[4] = {64, 1, (uint32_t)(c.page_size < kTile ? c.page_size : kTile), 1};
  const auto type = c.dtype == MOE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                       : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const uint32_t steps[4] = {1, 1, 1, 1};
  const EncodeFn encode = encode_fn();
  if (!encode) return cudaErrorNotSupported;
  // queries as [token][head][dim]: a box is the rows of a query tile
  const cuuint64_t q_dims[3] = {(cuuint64_t)c.head_dim, (cuuint64_t)a.n_heads,
                                (cuuint64_t)a.n_tokens};
  const cuuint64_t q_strides[2] = {(cuuint64_t)a.q_head_stride * 2,
                                   (cuuint64_t)a.q_token_stride * 2};
  const uint32_t q_box[3] = {64, (uint32_t)a.group, (uint32_t)p.tpt};
  auto encode_maps = [&] {
    auto map = [&](CUtensorMap* to, int rank, const void* at, const cuuint64_t* size,
                   const cuuint64_t* stride, const uint32_t* piece) {
      return encode(to, type, rank, const_cast<void*>(at), size, stride, piece, steps,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    return map(&p.kmap, 4, c.k, dims, strides, box) && map(&p.vmap, 4, c.v, dims, strides, box) &&
           map(&p.qmap, 3, a.q, q_dims, q_strides, q_box);
  };
  if (!encode_maps()) {
    // a host thread that has called nothing but this library has no context yet,
    // and encoding, a driver's call, makes none
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaSetDevice(dev);
    if (e != cudaSuccess) return e;
    if (!encode_maps()) return cudaErrorInvalidValue;
  }
  const int ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
  // Blocks of two query tiles halve what is read; but with fewer of them than
  // CTAs most are cut, and their parts' joins take longer than the reads: a
  // prompt of 1024 tokens (32 heads on 8) takes 28.4 us in blocks of two and 26.4
  // in blocks of one, one of 2048 tokens 49.2 and 54.5.
  const long long blocks = (long long)((a.n_tokens - 1) / (2 * p.tpt) + 1) * c.n_kv_heads;
  p.block = blocks < ctas ? p.tpt : 2 * p.tpt;
  const bool f16 = c.dtype == MOE_F16;
  if (c.head_dim == 128)
    return f16 ? launch_t<128, true>(p, ctas, stream) : launch_t<128, false>(p, ctas, stream);
  return f16 ? launch_t<64, true>(p, ctas, stream) : launch_t<64, false>(p, ctas, stream);
}

}  // namespace moe
