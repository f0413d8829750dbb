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
//   a few tokens: bound by reading the cache), joined at the end.
//
// Work. An item is (request, key head, block of tokens); its length is the
// number of 128-key tiles its rows see. All items' tiles in a row are cut
// into equal ranges, one per CTA, wherever the cuts fall: every SM has the
// same number of key tiles to go through whatever the mix of long and short
// requests. Rows of an item that was cut leave (O, m, Σ) in the workspace,
// and a second kernel joins them in key order, so results do not depend on
// scheduling. The lengths are on the device: every CTA works out the cuts
// from them by itself.
//
// Warps (one CTA per SM):
//   0-3   softmax of stream 0, one thread per row; queries in, results out
//   4-7   the same for stream 1
//   8     TMA: key and value tiles into a ring, a box per page and 64 columns
//   9     MMA issue; clears value rows that no row of the item sees
#include <math.h>

#include "batch_launch.h"
#include "common.cuh"
#include "tcgen05.cuh"
#include "tmap.h"

namespace moe {
namespace {

constexpr int kTile = 128;        // rows of a query tile, keys of a key tile
constexpr int kThreads = 320;
constexpr int kMaxCtas = 160;     // workspace slots are sized for this many
constexpr int kPlanThreads = 256;
constexpr int kPerThread = MOE_MAX_REQUESTS / kPlanThreads;
// The reference m follows the row's maximum only when that has grown by more
// than this (in powers of two): until then weights are up to 2^8 instead of
// 1, which fp32 sums and both 16-bit types hold, and O needs no rescaling.
constexpr float kGrow = 8.f;

template <int kDim>
struct Sizes {
  static constexpr int kTileBytes = kTile * kDim * 2;
  static constexpr int kStages = kDim == 128 ? 5 : 10;
  static constexpr int kOffRing = 2 * kTileBytes;
  static constexpr int kOffMisc = kOffRing + kStages * kTileBytes;
  static constexpr int kMiscBytes = 1536;  // Misc, then the streams' row statistics
  static constexpr int kSmem = kOffMisc + kMiscBytes + 1024;  // slack to align the base to 1024
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // one slot of the workspace: O as [kDim/4][256 rows] float4, then m and Σ
  static constexpr size_t kSlotFloats = size_t(2 * kTile) * (kDim + 2);
};

// What a CTA leaves for the join: the item that ends in its range but began
// in an earlier one.
struct JoinRec {
  int valid, row0, ntok, head0, first_cta, pad[3];
};

struct Params {
  CUtensorMap kmap, vmap;
  AttendArgs a;
  int page_shift;
  int tpt;       // tokens per query tile, 128 / group
  float* part;   // [2 per CTA][kSlotFloats]
  JoinRec* rec;  // [CTAs]
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
  if (len < 0 || len > ((int64_t)a.max_blocks << page_shift)) {
    r.len = 0;
    *bad = true;
  }
  return r;
}

// `fixed`: the block's tokens, 2·tpt.
MOE_DEV Item make_item(const AttendArgs& a, const Request& r, int block, int fixed) {
  Item it;
  const int tok0 = block * fixed;
  it.row0 = r.first + tok0;
  it.ntok = min(fixed, r.q - tok0);
  it.pos0 = r.len - r.q + tok0;
  it.hi = max(0, it.pos0 + it.ntok);
  it.lo = a.window > 0 ? min(it.hi, max(0, it.pos0 - a.window + 1)) : 0;
  it.sk = min(a.sinks, it.lo);
  it.lo_tile = it.lo / kTile;
  it.ns = min((it.sk + kTile - 1) / kTile, it.lo_tile);
  it.n = max(1, it.ns + (it.hi + kTile - 1) / kTile - it.lo_tile);
  return it;
}

// Where a CTA is in its range of tiles; every role walks it by itself.
struct Walk {
  int b, h, block, t0, left;
};

// The walk's present item; skips requests without new tokens.
MOE_DEV Item walk_item(const Params& p, Walk& w, Request& r) {
  bool bad;
  r = request(p.a, p.page_shift, w.b, &bad);
  while (r.q == 0 && w.b + 1 < p.a.n_requests) r = request(p.a, p.page_shift, ++w.b, &bad);
  return make_item(p.a, r, w.block, 2 * p.tpt);
}

MOE_DEV void walk_next(const Params& p, Walk& w, const Request& r, int done) {
  w.left -= done;
  w.t0 = 0;
  if (++w.block * 2 * p.tpt >= r.q) {
    w.block = 0;
    if (++w.h == p.a.cache.n_kv_heads) {
      w.h = 0;
      ++w.b;
    }
  }
}

struct Start {
  Walk w;
  int first;  // 1: the range begins inside an item
  int has_rec;
  JoinRec rec;
};

// The CTA's range of tiles: prefix sums over the requests' tile counts, then
// the place of its first tile. Threads 0..kPlanThreads-1 call it.
MOE_DEV void find_start(const Params& p, long long* part, Start* out) {
  const AttendArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int fixed = 2 * p.tpt;
  long long count[kPerThread], sum = 0;
  bool any_bad = false;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = tid * kPerThread + i;
    long long n = 0;
    if (b < a.n_requests) {
      bool bad;
      const Request r = request(a, p.page_shift, b, &bad);
      any_bad |= bad;
      for (int q = 0; q * fixed < r.q; ++q) n += make_item(a, r, q, fixed).n;
    }
    count[i] = n;
    sum += n;
  }
  if (any_bad && blockIdx.x == 0) report_error(a.err, ERR_CHECK, 0xA20);
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) part[warp] = incl;
  asm volatile("bar.sync 1, 256;" ::: "memory");
  long long before = incl - sum, total = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) before += part[w];
    total += part[w];
  }
  const int H = a.cache.n_kv_heads;
  total *= H;
  before *= H;
  // no more CTAs than tiles, so that no range among them is empty
  const long long C = min((long long)gridDim.x, total), c = blockIdx.x;
  const long long w0 = c < C ? c * total / C : 0, w1 = c < C ? (c + 1) * total / C : 0;
  if (tid == 0) {
    out->w.left = (int)(w1 - w0);
    out->has_rec = 0;
  }
  asm volatile("bar.sync 1, 256;" ::: "memory");
  if (w1 == w0) return;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const long long n = count[i] * H;
    if (w0 >= before && w0 < before + n) {
      const int b = tid * kPerThread + i;
      long long rem = w0 - before;
      out->w.b = b;
      out->w.h = (int)(rem / count[i]);
      rem -= out->w.h * count[i];
      bool bad;
      const Request r = request(a, p.page_shift, b, &bad);
      int q = 0;
      Item it = make_item(a, r, 0, fixed);
      while (rem >= it.n) {
        rem -= it.n;
        it = make_item(a, r, ++q, fixed);
      }
      out->w.block = q;
      out->w.t0 = (int)rem;
      // the item ends here and began in an earlier range: this CTA's record
      if (rem > 0 && it.n - rem <= w1 - w0) {
        const long long s = w0 - rem;
        long long c0 = s * C / total;
        while (c0 + 1 < C && (c0 + 1) * total / C <= s) ++c0;
        out->has_rec = 1;
        out->rec = JoinRec{1, it.row0, it.ntok, out->w.h * a.group, (int)c0, {0, 0, 0}};
      }
    }
    before += n;
  }
}

// Bounded wait that gives up at once when any role of the CTA has.
MOE_DEV bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                           unsigned int* err, unsigned int site) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  for (unsigned int i = 0; i < kWaitLimitIters; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if ((i & 63u) == 63u && global_ns() - t0 > kWaitLimitNs) break;
  }
  report_error(err, ERR_TIMEOUT, site);
  *abort_flag = 1;
  return false;
}

MOE_DEV void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

MOE_DEV float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool kF16>
MOE_DEV uint32_t narrow(float lo, float hi) {
  if constexpr (kF16) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    return pack_bf16x2(lo, hi);
  }
}

// Barriers and words behind the ring.
struct Misc {
  uint64_t full[10], empty[10];
  uint64_t q_ready, q_free;
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t drain;
  Start start;
  long long part[8];
  uint32_t tmem;
  int abort_flag;
};
static_assert(sizeof(Misc) <= 512, "misc words");
constexpr int kOffStat = 512;  // then [2][128] floats: row statistics the streams exchange

template <int kDim, bool kF16>
__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const __grid_constant__ Params p) {
  using Z = Sizes<kDim>;
  constexpr int kStages = Z::kStages;
  constexpr int kHalves = kDim / 64;           // 64-column halves of a row
  constexpr int kHalfBytes = kTile * 128;
  constexpr uint32_t kCols = 512;              // S0 S1 O0 O1, 128 columns each
  const AttendArgs& a = p.a;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* ring = smem + Z::kOffRing;
  Misc& m = *reinterpret_cast<Misc*>(smem + Z::kOffMisc);
  volatile int* abort_flag = &m.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&m.full[i], 1);
      mbar_init(&m.empty[i], 1);
    }
    mbar_init(&m.q_ready, 8);
    mbar_init(&m.q_free, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&m.s_full[s], 1);
      mbar_init(&m.p_full[s], 4);
      mbar_init(&m.o_full[s], 1);
    }
    mbar_init(&m.drain, 1);
    m.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) umma::tmem_alloc(&m.tmem, kCols);
  if (threadIdx.x == 8 * 32) {
    prefetch_tmap(&p.kmap);
    prefetch_tmap(&p.vmap);
  }
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < kPlanThreads) find_start(p, m.part, &m.start);
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = m.tmem;
  Walk w = m.start.w;
  if (threadIdx.x == 0) {
    JoinRec& rec = p.rec[blockIdx.x];
    if (m.start.has_rec) {
      rec = m.start.rec;
    } else {
      rec.valid = 0;
    }
  }

  if (warp == 8) {
    // ------------------------------------------------------------- loader --
    const int page = 1 << p.page_shift;
    const int rows = min(page, kTile);          // rows of a box
    const int n_pages = kTile / rows;           // pages of a tile (1 if a page spans tiles)
    const uint64_t policy = l2_evict_normal_policy();
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (w.left > 0) {
      Request r;
      const Item it = walk_item(p, w, r);
      const int n = min(w.left, it.n - w.t0);
      const int lead = it.ntok > p.tpt ? 1 : 2;  // key tiles ahead of the value tiles
      const int32_t* table = a.block_table + (size_t)w.b * a.max_blocks;
      // keys 0..lead-1, then values j, keys j + lead, for j = 0..n-1
      for (int step = 0; step < 2 * n + 2 * lead; ++step) {
        const bool is_v = step >= lead && ((step - lead) & 1) == 0;
        const int j = step < lead ? step : is_v ? (step - lead) >> 1 : ((step - lead) >> 1) + lead;
        if (j >= n) continue;
        const int key0 = tile_of(it, w.t0 + j) * kTile;
        // this lane's page of the tile, if any row of it is seen
        const int r0 = key0 + lane * rows;
        bool want = lane < n_pages && r0 < it.hi && (r0 + rows > it.lo || r0 < it.sk);
        int pg = -1;
        if (want) pg = table[r0 >> p.page_shift];
        if (want && (pg < 0 || pg >= a.cache.n_pages)) {
          report_error(a.err, ERR_CHECK, 0xA21);
          pg = (int)a.cache.n_pages;             // out of the map: the box reads zeros
        }
        const uint32_t wanted = __ballot_sync(0xffffffffu, want);
        ok = ok && wait_or_abort(&m.empty[stage], phase ^ 1u, abort_flag, a.err, 0xA30);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          unsigned char* dst = ring + stage * Z::kTileBytes;
          if (lane == 0)
            mbar_arrive_expect_tx(&m.full[stage], __popc(wanted) * rows * kDim * 2);
          __syncwarp();
          if (want) {
            const CUtensorMap* map = is_v ? &p.vmap : &p.kmap;
#pragma unroll
            for (int half = 0; half < kHalves; ++half)
              tma_load_4d(dst + half * kHalfBytes + lane * rows * 128, map, half * 64, w.h,
                          r0 & (page - 1), pg, &m.full[stage], policy);
          }
        }
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      walk_next(p, w, r, n);
    }
    // After a lost wait the tiles still in flight must land before the CTA
    // ends; without one, every tile has been waited for by the MMA warp.
    if (!ok && lane == 0) {
      for (int i = 0; i < kStages; ++i)
        for (uint32_t ph = 0; ph < 2; ++ph) mbar_wait_for(&m.full[i], ph, a.err, 0xA31, 1000000ull);
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------------- MMA --
    const uint32_t id_s = umma::idesc_f16(kTile, kTile, kF16, false);
    const uint32_t id_o = umma::idesc_f16(kTile, kDim, kF16, true);
    const uint32_t q_addr = smem_addr(smem), ring_addr = smem_addr(ring);
    int stage = 0;
    uint32_t phase = 0, q_phase = 0, p_phase[2] = {0, 0};
    bool ok = true;
    auto next_tile = [&]() {
      const int s = stage;
      ok = ok && wait_or_abort(&m.full[s], phase, abort_flag, a.err, 0xA40);
      ok = __all_sync(0xffffffffu, ok);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
      return s;
    };
    auto scores = [&](int s, int q_tile, int st) {  // S_s = Q · Kᵀ
      if (ok && lane == 0) {
        umma::fence_after_sync();
#pragma unroll
        for (int k = 0; k < kDim / 16; ++k) {
          const uint32_t off = (k >> 2) * kHalfBytes + (k & 3) * 32;
          umma::mma_bf16(tmem + s * 128, umma::desc_sw128(q_addr + q_tile * Z::kTileBytes + off),
                         umma::desc_sw128(ring_addr + st * Z::kTileBytes + off), id_s, k != 0);
        }
        umma::commit(&m.s_full[s]);
      }
    };
    auto values = [&](int s, int st, bool first) {  // O_s (+)= P_s · V
      ok = ok && wait_or_abort(&m.p_full[s], p_phase[s], abort_flag, a.err, 0xA41);
      ok = __all_sync(0xffffffffu, ok);
      p_phase[s] ^= 1u;
      if (ok && lane == 0) {
        umma::fence_after_sync();
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          umma::mma_f16_ts(tmem + 256 + s * 128, tmem + s * 128 + k * 8,
                           umma::desc_sw128_mn(ring_addr + st * Z::kTileBytes + k * 2048,
                                               kHalfBytes),
                           id_o, !first || k != 0);
      }
    };
    auto release = [&](int st) {
      if (ok && lane == 0) umma::commit(&m.empty[st]);
    };
    while (w.left > 0) {
      Request r;
      const Item it = walk_item(p, w, r);
      const int n = min(w.left, it.n - w.t0);
      const bool two = it.ntok > p.tpt;
      // stream s's rows see something of a tile
      auto active = [&](int s, int j) {
        const int key0 = tile_of(it, w.t0 + j) * kTile;
        const int t_first = two ? s * p.tpt : 0;
        const int t_last = two ? min(it.ntok, (s + 1) * p.tpt) : it.ntok;
        const int hi = it.pos0 + t_last, lo = it.pos0 + t_first - a.window + 1;
        return key0 < hi && (a.window == 0 || key0 + kTile > lo || key0 < a.sinks);
      };
      ok = ok && wait_or_abort(&m.q_ready, q_phase, abort_flag, a.err, 0xA42);
      ok = __all_sync(0xffffffffu, ok);
      q_phase ^= 1u;
      bool first[2] = {true, true};
      const int lead = two ? 1 : 2;
      for (int j = 0; j < min(lead, n); ++j) {
        const int st = next_tile();
        if (two) {
          if (active(0, 0)) scores(0, 0, st);
          if (active(1, 0)) scores(1, 1, st);
        } else if (active(0, j)) {
          scores(j, 0, st);
        }
        release(st);
      }
      if (n <= lead && ok && lane == 0) umma::commit(&m.q_free);
      for (int j = 0; j < n; ++j) {
        const int vt = next_tile();
        const int kt = j + lead < n ? next_tile() : -1;
        // rows of V that no row of the item sees may hold anything: their
        // weights are 0, and 0 · NaN is not
        const int key0 = tile_of(it, w.t0 + j) * kTile;
        if (ok && (key0 + kTile > it.hi || (key0 < it.lo && key0 + kTile > it.sk))) {
          unsigned char* v = ring + vt * Z::kTileBytes;
          for (int i = lane; i < kTile * kHalves * 8; i += 32) {
            const int row = (i >> 3) & (kTile - 1), key = key0 + row;
            if (key >= it.hi || (key < it.lo && key >= it.sk))
              *reinterpret_cast<uint4*>(v + (size_t)i * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (two) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (active(s, j)) {
              values(s, vt, first[s]);
              first[s] = false;
            }
            if (s == 1) release(vt);
            if (kt >= 0 && active(s, j + 1)) scores(s, s, kt);
          }
        } else {
          const int s = j & 1;
          if (active(0, j)) {
            values(s, vt, first[s]);
            first[s] = false;
          }
          release(vt);
          if (kt >= 0 && active(0, j + lead)) scores(s, 0, kt);
        }
        if (kt >= 0) release(kt);
        if (j + lead + 1 == n && ok && lane == 0) umma::commit(&m.q_free);
      }
      if (ok && lane == 0) {
        if (!first[0]) umma::commit(&m.o_full[0]);
        if (!first[1]) umma::commit(&m.o_full[1]);
      }
      walk_next(p, w, r, n);
    }
    // Every MMA, and every arrival that hangs on one, is done before tensor
    // memory is released.
    if (lane == 0) {
      umma::commit(&m.drain);
      mbar_wait(&m.drain, 0, a.err, 0xA43);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax --
    const int s = warp >> 2;               // stream
    const int row = threadIdx.x & 127;     // row of the tile, TMEM lane
    const uint32_t lane_base = (uint32_t)(warp & 3) << 21;  // 32·(warp % 4) in the upper half
    const uint32_t s_addr = tmem + lane_base + s * 128;
    const uint32_t o_addr = tmem + lane_base + 256 + s * 128;
    const float to_log2 = a.scale * 1.4426950408889634f;
    // fp16 weights are held 2^4 larger, so that small ones keep their bits
    const float offset = kF16 ? 4.f : 0.f;
    const int G = a.group;
    float* stat = reinterpret_cast<float*>(smem + Z::kOffMisc + kOffStat);
    uint32_t s_phase = 0, o_phase = 0, qf_phase = 0;
    bool ok = true, first_item = true;
    while (w.left > 0) {
      Request r;
      const Item it = walk_item(p, w, r);
      const int n = min(w.left, it.n - w.t0);
      const bool two = it.ntok > p.tpt;
      // ---- queries in: stream s its own tile, or both streams half a tile
      if (!first_item) {
        ok = ok && wait_or_abort(&m.q_free, qf_phase, abort_flag, a.err, 0xA50);
        qf_phase ^= 1u;
      }
      first_item = false;
      {
        constexpr int kChunks = kDim / 8;          // 16-byte pieces of a row
        const int toks = two ? min(it.ntok - s * p.tpt, p.tpt) : it.ntok;
        const int rows = toks * G;
        const int r_first = two ? 0 : s * 64, r_end = two ? rows : min(rows, r_first + 64);
        unsigned char* q_tile = smem + (two ? s : 0) * Z::kTileBytes;
        const int row0 = it.row0 + (two ? s * p.tpt : 0);
        for (int i = row; i < (r_end - r_first) * kChunks; i += 128) {
          const int rr = r_first + i / kChunks, c = i & (kChunks - 1);
          const int tok = rr / G, g = rr - tok * G;
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(
              static_cast<const uint16_t*>(a.q) + (row0 + tok) * a.q_token_stride +
              (w.h * G + g) * a.q_head_stride + c * 8));
          *reinterpret_cast<uint4*>(q_tile + (c >> 3) * kHalfBytes + rr * 128 +
                                    (((c & 7) ^ (rr & 7)) << 4)) = v;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.q_ready);
      }
      // ---- this thread's row
      const int t_in = row / G, tok = (two ? s * p.tpt : 0) + t_in;
      const bool valid = t_in < p.tpt && tok < it.ntok;
      const bool warp_valid = __any_sync(0xffffffffu, valid);
      const int pos = it.pos0 + tok;
      const int hi = valid ? max(0, pos + 1) : 0;
      const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
      const int t_first = two ? s * p.tpt : 0;
      const int t_last = two ? min(it.ntok, (s + 1) * p.tpt) : it.ntok;
      const int s_hi = it.pos0 + t_last, s_lo = it.pos0 + t_first - a.window + 1;
      float ref = -INFINITY, sum = 0.f;
      bool began = false;
      for (int j = two ? 0 : s; j < n; j += two ? 1 : 2) {
        const int key0 = tile_of(it, w.t0 + j) * kTile;
        if (!(key0 < s_hi && (a.window == 0 || key0 + kTile > s_lo || key0 < a.sinks))) continue;
        ok = ok && wait_or_abort(&m.s_full[s], s_phase, abort_flag, a.err, 0xA51);
        ok = __all_sync(0xffffffffu, ok);
        s_phase ^= 1u;
        if (ok && warp_valid) {
          umma::fence_after_sync();
          uint32_t x[kTile];
#pragma unroll
          for (int c = 0; c < kTile; c += 32) umma::ld_x32(s_addr + c, x + c);
          umma::wait_ld();
          const bool whole =
              !valid || (key0 + kTile <= hi && (key0 >= lo || key0 + kTile <= a.sinks));
          if (!__all_sync(0xffffffffu, whole)) {
            const int e_hi = hi - key0, e_lo = lo - key0, e_sk = a.sinks - key0;
#pragma unroll
            for (int c = 0; c < kTile; ++c)
              if (!(c < e_hi && (c >= e_lo || c < e_sk))) x[c] = 0xff800000u;  // −inf
          }
          float top = __uint_as_float(x[0]);
#pragma unroll
          for (int c = 1; c < kTile; ++c) top = fmaxf(top, __uint_as_float(x[c]));
          top *= to_log2;
          const bool grown = top > ref + kGrow || (ref == -INFINITY && top > -INFINITY);
          if (__any_sync(0xffffffffu, grown)) {
            const float keep = grown ? exp2_approx(ref - top) : 1.f;
            if (grown) ref = top;
            sum *= keep;
            if (began) {
#pragma unroll 1
              for (int c = 0; c < kDim; c += 32) {
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
          float s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int c = 0; c < kTile; c += 2) {
            const float p0 = exp2_approx(fmaf(__uint_as_float(x[c]), to_log2, shift));
            const float p1 = exp2_approx(fmaf(__uint_as_float(x[c + 1]), to_log2, shift));
            s0 += p0;
            s1 += p1;
            x[c >> 1] = narrow<kF16>(p0, p1);
          }
          sum += s0 + s1;
          umma::st_x32(s_addr, x);
          umma::st_x32(s_addr + 32, x + 32);
          umma::wait_st();
        }
        began = true;
        umma::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.p_full[s]);
      }
      // ---- results out
      if (began) {
        ok = ok && wait_or_abort(&m.o_full[s], o_phase, abort_flag, a.err, 0xA52);
        o_phase ^= 1u;
      }
      ok = __all_sync(0xffffffffu, ok);
      umma::fence_after_sync();
      const bool ends = w.t0 + n == it.n, whole_item = ends && w.t0 == 0;
      float* slot = p.part + (size_t)(2 * blockIdx.x + (ends ? 0 : 1)) * Z::kSlotFloats;
      // factors of the two streams' O for this thread's columns
      float f0 = 1.f, f1 = 0.f;
      int c_first = 0, c_end = kDim;
      if (!two) {
        // both streams hold sums of the same rows: each joins half the columns
        stat[s * 128 + row] = ref;
        asm volatile("bar.sync 2, 256;" ::: "memory");
        const float other = stat[(s ^ 1) * 128 + row];
        const float top = fmaxf(ref, other);
        const float mine = ref == -INFINITY ? 0.f : exp2_approx(ref - top);
        asm volatile("bar.sync 2, 256;" ::: "memory");
        stat[s * 128 + row] = sum * mine;
        asm volatile("bar.sync 2, 256;" ::: "memory");
        umma::fence_after_sync();
        sum = sum * mine + stat[(s ^ 1) * 128 + row];
        const float theirs = other == -INFINITY ? 0.f : exp2_approx(other - top);
        f0 = s == 0 ? mine : theirs;
        f1 = s == 0 ? theirs : mine;
        ref = top;
        c_first = s * (kDim / 2);
        c_end = c_first + kDim / 2;
      }
      if (ok && warp_valid) {
        const float inv = whole_item ? (sum > 0.f ? 1.f / sum : 0.f) : 1.f;
        f0 *= inv;
        f1 *= inv;
        const int o0 = two ? s : 0;
        const int head = w.h * G + (row - t_in * G);
        uint16_t* dst = static_cast<uint16_t*>(a.out) + (int64_t)(it.row0 + tok) * a.out_token_stride +
                        head * a.out_head_stride;
        const int prow = (two ? s * kTile : 0) + row;
        for (int c = c_first; c < c_end; c += 32) {
          uint32_t o[32];
          umma::ld_x32(tmem + lane_base + 256 + o0 * 128 + c, o);
          umma::wait_ld();
          // a stream that saw no key never wrote its O: what is there is not
          // a number to be scaled
#pragma unroll
          for (int i = 0; i < 32; ++i)
            o[i] = f0 > 0.f && sum > 0.f ? __float_as_uint(__uint_as_float(o[i]) * f0) : 0u;
          if (!two && __any_sync(0xffffffffu, f1 > 0.f)) {
            uint32_t o1[32];
            umma::ld_x32(tmem + lane_base + 384 + c, o1);
            umma::wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (f1 > 0.f)
                o[i] = __float_as_uint(fmaf(__uint_as_float(o1[i]), f1, __uint_as_float(o[i])));
          }
          if (valid) {
            if (whole_item) {
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                uint4 v;
                v.x = narrow<kF16>(__uint_as_float(o[i]), __uint_as_float(o[i + 1]));
                v.y = narrow<kF16>(__uint_as_float(o[i + 2]), __uint_as_float(o[i + 3]));
                v.z = narrow<kF16>(__uint_as_float(o[i + 4]), __uint_as_float(o[i + 5]));
                v.w = narrow<kF16>(__uint_as_float(o[i + 6]), __uint_as_float(o[i + 7]));
                *reinterpret_cast<uint4*>(dst + c + i) = v;
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                reinterpret_cast<uint4*>(slot)[((c + i) >> 2) * (2 * kTile) + prow] =
                    make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            }
          }
        }
        if (valid && !whole_item && (two || s == 0)) {
          float* st = slot + (size_t)2 * kTile * kDim;
          st[prow] = ref;
          st[2 * kTile + prow] = sum;
        }
      }
      // this item's O and statistics have been read before the next item's
      // are written (of both streams, where they were joined)
      umma::fence_before_sync();
      if (!two) asm volatile("bar.sync 2, 256;" ::: "memory");
      walk_next(p, w, r, n);
    }
  }
  umma::fence_before_sync();
  __syncthreads();
  if (warp == 9) umma::tmem_dealloc(tmem, kCols);
}

// ------------------------------------------------------------------ join --
// One CTA per record: the parts of the record's item in key order, a thread
// per (row, 4 columns).
constexpr int kJoinThreads = 256;

template <int kDim, bool kF16>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const __grid_constant__ Params p) {
  using Z = Sizes<kDim>;
  pdl_wait();
  pdl_trigger();
  const JoinRec rec = p.rec[blockIdx.x];
  if (!rec.valid) return;
  const AttendArgs& a = p.a;
  const int G = a.group, rows = rec.ntok * G, per_tile = p.tpt * G;
  const int last = blockIdx.x;
  for (int i = blockIdx.y * kJoinThreads + threadIdx.x; i < rows * (kDim / 4);
       i += gridDim.y * kJoinThreads) {
    const int c4 = i / rows, rr = i - c4 * rows;
    // rows of the second tile start at 128
    const int prow = rr < per_tile ? rr : kTile + rr - per_tile;
    float m = -INFINITY, sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = rec.first_cta; c <= last; ++c) {
      const float* slot = p.part + (size_t)(2 * c + (c == last ? 0 : 1)) * Z::kSlotFloats;
      const float* st = slot + (size_t)2 * kTile * kDim;
      const float mc = st[prow], sc = st[2 * kTile + prow];
      const float4 oc = reinterpret_cast<const float4*>(slot)[c4 * (2 * kTile) + prow];
      if (mc == -INFINITY) continue;
      const float top = fmaxf(m, mc);
      const float keep = m == -INFINITY ? 0.f : exp2_approx(m - top), add = exp2_approx(mc - top);
      m = top;
      sum = sum * keep + sc * add;
      o.x = o.x * keep + oc.x * add;
      o.y = o.y * keep + oc.y * add;
      o.z = o.z * keep + oc.z * add;
      o.w = o.w * keep + oc.w * add;
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const int tok = rr / G, g = rr - tok * G;
    uint16_t* dst = static_cast<uint16_t*>(a.out) + (int64_t)(rec.row0 + tok) * a.out_token_stride +
                    (int64_t)(rec.head0 + g) * a.out_head_stride + c4 * 4;
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(narrow<kF16>(o.x * inv, o.y * inv), narrow<kF16>(o.z * inv, o.w * inv));
  }
}

template <int kDim, bool kF16>
cudaError_t launch_t(Params& p, int ctas, cudaStream_t stream) {
  using Z = Sizes<kDim>;
  auto* kernel = attend_kernel<kDim, kF16>;
  static int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && configured_device != dev) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Z::kSmem);
    if (e == cudaSuccess) configured_device = dev;
  }
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3(ctas), dim3(kThreads), Z::kSmem, stream, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(attend_join_kernel<kDim, kF16>, dim3(ctas, 2), dim3(kJoinThreads), 0, stream, p);
}

}  // namespace

size_t attend_workspace_bytes(int head_dim) {
  const size_t slot = head_dim == 128 ? Sizes<128>::kSlotFloats : Sizes<64>::kSlotFloats;
  return size_t(kMaxCtas) * sizeof(JoinRec) + 2 * kMaxCtas * slot * sizeof(float);
}

cudaError_t launch_attend(const AttendArgs& a, int num_sms, cudaStream_t stream) {
  Params p;
  memset(&p, 0, sizeof p);
  p.a = a;
  p.page_shift = 31 - __builtin_clz(a.cache.page_size);
  p.tpt = kTile / a.group;
  p.rec = static_cast<JoinRec*>(a.workspace);
  p.part = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + kMaxCtas * sizeof(JoinRec));
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
  for (int i = 0; i < 2; ++i)
    if (encode(i ? &p.vmap : &p.kmap, type, 4, i ? c.v : c.k, dims, strides, box, steps,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  const int ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
  const bool f16 = c.dtype == MOE_F16;
  if (c.head_dim == 128)
    return f16 ? launch_t<128, true>(p, ctas, stream) : launch_t<128, false>(p, ctas, stream);
  return f16 ? launch_t<64, true>(p, ctas, stream) : launch_t<64, false>(p, ctas, stream);
}

}  // namespace moe
