// attend8.cu — attention of every request's new tokens over its paged cache of
// e4m3 codes: causal, optionally within a sliding window beside a few first
// keys that stay visible.
//
// For a query row q at position p, over the keys j that it sees, with codes K_j
// and V_j and scales ks_j and vs_j of their blocks,
//   s_j = scale · ks_j · (q · K_j)          (in powers of two: times log2 e)
//   out = Σ_j 2^(s_j + log2 vs_j − m) V_j / Σ_j 2^(s_j − m),
// the reference m and the two sums carried along in one pass over the keys as in
// attend.cu. m follows t_j = s_j + log2 vs_j: the weights w_j = 2^(t_j − m) that
// meet the codes are then largest at 1 whatever the scales, and the second sum is
// that of w_j / vs_j.
//
// Codes go to the tensor cores as they lie in the cache (tcgen05 kind::f8f6f4):
// nothing is widened, and half the bytes of a 16-bit cache are read. Their other
// operands are sums of numbers in 8 bits, columns of one operand beside each other,
// so that a product takes them at once. A query row, divided by a power of two,
// is hi + lo/16 (+ lolo/256), each an e4m3 number, the rounding of 16 times what the
// ones before it left; e4m3 has 4 significant bits, so two numbers hold the 8 of bf16
// exactly, three the 11 of fp16, as long as they are within 2^-14 of the row's
// largest. Weights need range before bits: where one key takes most of a row, what
// the others bring is a sum of many weights that are each far below it. They are
// rounded to fp16, and that becomes three e5m2 numbers, 3 bits each and 8 times what
// the ones before it left (weight_numbers). Weights stay below 2^14.5, and a row's
// largest is 2^4 (bf16) or 2^10 (fp16) at least: m follows growth beyond 2^10.5 (2^4.5)
// only. A weight is then off by 2^-9 (2^-11) of itself, or by 2^-26 (2^-32) of the row's
// largest where that is more, to either side alike. (Two e4m3 numbers, which end at
// 2^-18, left rows of 16384 keys whose first took 0.9 of the weight off by 0.05 of their
// norm. The margin for growth is speed: with 2^9.5 and 2^8.5 prompt chunks in bf16 took 540
// and 548 us for 532. In fp16 it is 2^4.5, 2^6.5 or 2^9.5 for 144, 140 and 136 us, but a
// row's largest weight is exact only where m is its own, and with wider margins
// errors grew from 2.2e-4 to 2.3e-4 and 2.4e-4.)
//
// Tiles. Keys are the rows of both products, query rows their columns:
//   Sᵀ = K · Qᵀ    128 keys × (16 to 64 query rows, times 2 or 3), and
//   Oᵀ += Vᵀ · Pᵀ  head_dim × (the same rows, times 3),
// so that a pass of a few tokens pays for its 16 columns and not for 128 rows
// (an instruction takes 64 cycles for any width up to 128 columns; the second
// product of 64 rows has 192), K and V are read in the order in which they
// lie, and a key's scales are one thread's. A softmax thread has one key and 16 query
// rows. Its rows' references are those of its group of four warps, which hold the
// tile's 128 keys: they change only when some weight passes 2^14.5 (asked by one
// barrier's vote), and then by the exact maximum over the tile.
//
// Work is cut into equal ranges as in attend.cu (attend_range.cuh): an item is
// (request, key head, block of tokens with at most 64 rows), a CTA whose range
// ends inside an item leaves (O, m, Σ) of its rows, and the CTA with the item's
// last tile joins the parts in key order. Within a CTA an item of at most 32 (16)
// rows runs as two (four) streams over every second (fourth) tile, each with its
// own sums, joined at the end.
//
// Warps (one CTA per SM):
//   0      TMA: key and value tiles into a ring each, a box per page
//   1, 2   MMA issue: scores, and results. (An MMA holds the warp that issues it for
//          the 64 cycles that it takes, a wait that ends at once takes 100, a commit
//          50: with both products in one warp that warp was what a tile took.)
//   3      ahead of the others: the parts of the CTA's range, their tiles' pages
//          and scales, the next part's query rows into shared memory
//   4-19   softmax, four groups of four warps: 16 columns of a tile each, or the
//          tiles of a stream; and the next item's queries into e4m3 numbers
//
// What bounds it, beside the rates measured for a copy and a dense product (6.65
// TB/s, 1894 TFLOP/s). Single tokens of 126 requests, 1.3 GB of keys and values: 224
// us, 5.8 TB/s: reading them. 64 requests' passes of 1 to 9 tokens: 96 us for 456 MB
// that a copy moves in 69, and 104 for 61 within a window: a CTA has few tiles, and
// its start (6 us), its joins (4) and its parts of items (4 to 6 us each beside 0.4 to
// 0.8 a tile) are half of its time. Long prompts' chunks: 532 us, 497 TFLOP/s: a
// tile of 64 rows takes 2200 cycles there, half of them the softmax warps' instructions,
// many of those for cutting weights into numbers, and half of them waits, of four
// warps of a sub-partition for each other and for what they load (an instruction
// every other cycle, tensor cores a quarter of the time). One pass of 5 tokens over 777
// keys: 10 us beyond an empty launch, the chain from the plan to a part's end.
//
// Values that are not finite (NaN; e4m3 has no infinities). A weight of 0 times
// NaN is NaN: rows of V that no row of the item sees are cleared, and NaN in rows
// that some see and others do not is taken out of the tile and noted for the rows
// that do see it (in `spoiled`, a bit per column of V and row).
#include <stddef.h>
#include <string.h>

#include "attend8_mma.cuh"
#include "attend_range.cuh"
#include "fp8.cuh"
#include "kv8_launch.h"
#include "round16.cuh"
#include "tmap.h"

namespace moe {
namespace {

constexpr int kThreads = 640;
constexpr int kRows = 64;         // query rows of an item, at most
constexpr int kMaxCtas = 160;     // workspace slots are sized for this many
// What an item costs beside its tiles when the work is cut, and what every 16 rows of
// it add (see Units).
constexpr int kItemUnits = 26, kItemRowUnits = 5;
// Weights are held 2^kBase larger, and m follows growth beyond 2^kGrow (see above).
template <bool kF16>
constexpr float kBase = kF16 ? 10.f : 4.f;
template <bool kF16>
constexpr float kGrow = 14.5f - kBase<kF16>;
constexpr int kWeightNum = 3;     // e5m2 numbers of a weight
// Registers per thread: launched with 96, the 16 softmax warps take 104 and
// the 4 others leave 64 (4·104 + 64 = 5·96).
constexpr int kSoftmaxRegs = 104, kOtherRegs = 64;
constexpr int kSlots = 16;        // tiles whose pages and scales are there
constexpr int kScaleBlocks = kTile / 16;

// kDim: columns of a head; kNum: e4m3 numbers of a query's element.
template <int kDim, int kNum>
struct Sizes {
  static constexpr int kTileBytes = kTile * kDim;
  static constexpr int kQBytes = kRows * kNum * kDim;  // an item's queries as numbers
  static constexpr int kRawBytes = kRows * kDim * 2;   // and the next one's as they come
  // Columns of S, and of O and P (a byte each): a quarter, half or all of them are a
  // stream's. (A stream's P lies within 128 columns, or begins with them.)
  static constexpr int kScoreColumns = kNum == 2 ? 128 : 256, kColumns = 256;
  static constexpr int kPBytes = kTile * kColumns;
  // A ring for keys and one for values, each waited on in order by the one warp that
  // issues its products: with both in one ring, the warp that waits for keys came to
  // a stage whose last tile, values, had not landed yet, and a parity tells only
  // neighbouring fills apart. (tests/test_kv8_rings.py has the roles as a model.)
  static constexpr int kKeyStages = kDim == 64 ? 8 : 4;
  static constexpr int kValueStages = kDim == 64 ? 8 : 5;
  static constexpr int kStages = kKeyStages + kValueStages;
  // (a value tile that a softmax warp waits for is not further behind; see there)
  static_assert(kValueStages >= 4, "a stage for every stream");
  static constexpr int kOffRaw = kQBytes;
  static constexpr int kOffP = kOffRaw + kRawBytes;
  static constexpr int kOffRing = kOffP + kPBytes;
  static constexpr int kOffMisc = kOffRing + kStages * kTileBytes;
  static constexpr int kMiscBytes = 6656;
  static constexpr int kSmem = kOffMisc + kMiscBytes;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kQBytes % 1024 == 0 && kPBytes % 1024 == 0 && kTileBytes % 1024 == 0, "tiles");
  static_assert(kPBytes >= kRows * kDim * 2, "results pass through P");
  // tensor memory: S, then O (a power of two is allocated)
  static constexpr uint32_t kCols = 512, kColO = kScoreColumns;
};
// one slot of the workspace: O as [64 rows][dim] floats, then m and Σ
constexpr size_t slot_floats(int dim) { return size_t(kRows) * (dim + 2); }

struct Params {
  CUtensorMap kmap, vmap;
  Attend8Args a;
  int page_shift;
  int blocks_shift;  // log2 of a page's blocks
  int tpt, block;    // tokens per item, 64 / group (both: see find_start)
  float* part;       // [2 per CTA][slot]
  // [CTAs][128]: see Misc::spoils
  unsigned long long* spoiled;
  // [CTAs]: `call` when the CTA has left the part of its last item; see attend.cu
  unsigned long long* left;
  unsigned long long call;
};

// An item's units, an eighth of what a tile of 64 query rows takes (0.83 us): first
// `cost`, then `each` for every key tile. A tile belongs to the CTA whose range has
// its first unit. Measured with one CTA alone (bf16, pages of 64): tiles of 16, 32, 48
// and 64 rows 0.42, 0.51, 0.74 and 0.83 us, and a part of one tile behind another 4.7,
// 4.9, 5.8 and 6.8. With tiles of 3, 4, 6 and 8 units single tokens took 226 us for 224,
// prompts beside passes 82 for 79 and windows 100 for 103.6; with 4, 5, 6 and 8
// verification passes 102 for 95, windows 107. In pages of 16 a tile of 16 rows takes 0.79
// us (its boxes bound it), in pages of 32 0.53: as 5 units at least where the page is
// of 16, prompts beside passes took 78 us, as 4 81, as 8 79.6.
struct Units {
  int cost, each, all;
  MOE_DEV int tiles(int u) const {  // that begin before unit u
    return (int)((uint32_t)(max(0, u - cost) + each - 1) / (uint32_t)each);
  }
};
MOE_DEV Units units_of(const Params& p, const Item& it) {
  const int wide = (it.ntok * p.a.group + 15) >> 4;  // query rows, by 16
  Units u;
  u.cost = kItemUnits + kItemRowUnits * wide;
  u.each = max(wide == 1 ? 4 : wide == 2 ? 5 : wide == 3 ? 7 : 8, 80 >> p.page_shift);
  u.all = it.hi > 0 ? u.cost + it.n * u.each : 0;    // (see clear_blind)
  return u;
}
// (A range of less than a tile would only add a part to be joined.)
MOE_DEV long long most_ranges(const Params&, long long total, int) { return total >> 3; }

// The CTA's part of an item, in shared memory: one warp walks the range, and the
// others read what they need of a part when they need it. (With a copy of the walk
// and of the part in registers of every warp, a tile took a third more
// instructions: what did not fit was worked out again at every tile.)
struct Part {
  int n;              // tiles; −1: there are no more parts
  int rows, wide;     // query rows, and those rounded up: 16, 32, 48 or 64
  int shift;          // log2 of the streams: 2, 1 or 0
  int whole, ends;    // all of the item; its last tile
  int once;           // no other item has its keys
  int b, h;           // request, key head
  int row0, ntok;     // packed rows of the item
  int pos0;           // position of its first token
  int hi, lo, sk;     // see Item
  int first, ns, gap; // tile j of the part is tile t = first + j, beyond ns of them t + gap
  // tiles that not all rows see whole: from edge_hi on, and [edge_sk, edge_lo)
  int edge_hi, edge_lo, edge_sk;
  MOE_DEV int tile(int j) const { return first + j + (first + j < ns ? 0 : gap); }
};
constexpr int kParts = 8;

// The next part of the walk with tiles in it; false when there is none.
MOE_DEV bool next_part(const Params& p, Walk& w, Request& r, Part* out) {
  const Attend8Args& a = p.a;
#pragma unroll 1
  while (w.left > 0) {
    const Item it = make_item(a, r, w.block, p.block);
    const Units units = units_of(p, it);
    const int u1 = min(w.u0 + w.left, units.all);
    const int t0 = units.tiles(w.u0), t1 = units.tiles(u1), n = t1 - t0;
    out->n = n;
    out->rows = it.ntok * a.group;
    out->wide = (out->rows + 15) & ~15;
    out->shift = out->wide == 16 ? 2 : out->wide == 32 ? 1 : 0;
    out->whole = n == it.n;
    out->ends = t1 == it.n;
    out->once = r.q <= p.block;
    out->b = w.b;
    out->h = w.h;
    out->row0 = it.row0;
    out->ntok = it.ntok;
    out->pos0 = it.pos0;
    out->hi = it.hi;
    out->lo = it.lo;
    out->sk = it.sk;
    out->first = t0;
    out->ns = it.ns;
    out->gap = it.lo_tile - it.ns;
    // key0 + 127 > pos0; key0 below the last row's window and not all of it sinks
    out->edge_hi = (it.pos0 + 1) >> 7;
    const int seen = a.window > 0 ? max(0, window_from(it.hi - 1, a.window)) : 0;
    out->edge_lo = (seen + kTile - 1) / kTile;
    out->edge_sk = it.sk / kTile;
    w.left -= u1 - w.u0;
    w.u0 = 0;
    if (w.left > 0 && ++w.block * p.block >= r.q) {
      if (++w.h == a.cache.n_kv_heads) {
        w.h = 0;
        bool bad;
        do {
          if (++w.b >= a.n_requests) return false;
          r = request(a, p.page_shift, w.b, &bad);
        } while (r.q == 0 || r.len == 0);
      }
      w.block = max(0, r.q - r.len) / p.block;   // (those before it see nothing)
    }
    if (n > 0) return true;
  }
  return false;
}

// A place in a ring (a tile's number in the CTA's range), counted modulo twice its
// stages: the stage, and the parity of its filling.
template <int kStages>
struct Place {
  int at;
  MOE_DEV explicit Place(unsigned from) : at((int)(from % (2u * kStages))) {}
  MOE_DEV int stage() const { return at >= kStages ? at - kStages : at; }
  MOE_DEV uint32_t parity() const { return at >= kStages; }
  MOE_DEV void next() { at = at + 1 == 2 * kStages ? 0 : at + 1; }
};

// How many tiles each of the four streams has had, modulo 256, a byte each: all
// roles count alike, and a barrier's parity follows from its stream's count.
MOE_DEV uint32_t count_of(uint32_t counts, int s) { return counts >> (8 * s) & 255u; }
MOE_DEV uint32_t add_counts(uint32_t counts, int n, int shift) {
  uint32_t r = 0;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int more = s >> shift == 0 && n > s ? ((n - 1 - s) >> shift) + 1 : 0;
    r |= (count_of(counts, s) + (uint32_t)more & 255u) << (8 * s);
  }
  return r;
}

// Barriers and words behind the ring.
template <int kStages>
struct Misc {
  uint64_t full[kStages], empty[kStages];        // keys' stages, then values'
  uint64_t part_full[kParts], part_empty[kParts];
  uint64_t raw_full, raw_empty;  // queries as they come
  uint64_t q_full;               // and as numbers
  uint64_t pg_full[kSlots], sc_full[kSlots], tile_done[kSlots];  // of a tile's slot
  uint64_t s_full[4], s_empty[4], p_full[4], p_done[4];  // of a stream
  uint64_t drain[2];
  Start start;
  long long part[8];
  uint32_t tmem;
  int lost;
  // NaN has been noted in the CTA's `spoiled` for the present item
  int spoils;
};
// A tile's slot: ks, log2 vs + kBase and pages of its 16-key blocks; key0, edge
struct Slot {
  float ks[kScaleBlocks], lv[kScaleBlocks];
  int page[kScaleBlocks];
  int key0, edge;
};
constexpr int kOffRef = 1152;                      // [4 groups][rows] −m of a column
constexpr int kOffQScale = kOffRef + 512;          // [2][64] a row's factor
constexpr int kOffStat = kOffQScale + 512;         // [4 groups][4 warps][rows]
constexpr int kOffSlots = kOffStat + 2048;
constexpr int kOffParts = kOffSlots + kSlots * (int)sizeof(Slot);
static_assert(kOffParts + kParts * (int)sizeof(Part) <= 6656, "misc words");

// ln 2's reciprocal: scores are kept in powers of two.
constexpr float kLog2e = 1.4426950408889634f;

// Row `row`, byte `at` of a tile of kRow-byte rows, swizzled at that width.
template <int kRow>
MOE_DEV uint32_t swizzled(uint32_t row, uint32_t at) {
  const uint32_t o = row * kRow + at;
  return o ^ (o >> 3 & (kRow == 128 ? 0x70u : 0x30u));
}

// Barriers and words by their address in shared memory.
MOE_DEV bool try_at(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
MOE_DEV bool try_at_longer(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity), "r"(kTryNs)
      : "memory");
  return done != 0;
}
MOE_DEV int ld_shared(uint32_t at) {
  int v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
MOE_DEV void ld_shared2(uint32_t at, uint64_t* a, uint64_t* b) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(*a), "=l"(*b) : "r"(at) : "memory");
}
MOE_DEV void st_shared4(uint32_t at, const uint32_t* v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}

// A wait that does not end at once (see wait_or_abort).
MOE_DEV bool wait_longer(uint32_t bar, uint32_t parity, volatile int* lost, int site) {
  bool done = false;
#pragma unroll 1
  for (int i = 0; !done && i < kTries && *lost == 0; ++i)
    done = __all_sync(0xffffffffu, try_at_longer(bar, parity));
  if (!done && *lost == 0) *lost = site;
  return __all_sync(0xffffffffu, done);
}

// Four values' e4m3 numbers: each is 16 times what the ones before it left. (In
// fp16: the differences of numbers and their multiples by 16 are exact.)
template <int kNum>
MOE_DEV void numbers_of(float a, float b, float c, float d, uint32_t (&out)[kNum]) {
  __half2 lo = __floats2half2_rn(a, b), hi = __floats2half2_rn(c, d);
#pragma unroll
  for (int i = 0; i < kNum; ++i) {
    out[i] = e4m3_of(lo, hi);
    if (i + 1 < kNum) {
      __half2 x, y;
      halves_of(out[i], &x, &y);
      lo = __hfma2(x, __float2half2_rn(-16.f), __hmul2(lo, __float2half2_rn(16.f)));
      hi = __hfma2(y, __float2half2_rn(-16.f), __hmul2(hi, __float2half2_rn(16.f)));
    }
  }
}
// What a number counts.
MOE_DEV constexpr float number_unit(int i) { return i == 0 ? 1.f : i == 1 ? 0x1p-4f : 0x1p-8f; }

// Four weights' e5m2 numbers, from their roundings to fp16: an e5m2 number is the
// upper byte of an fp16 number, and half a step of it added to the lower byte rounds
// to nearest. Each is 8 times what the ones before it left, which is exact, rounded. Of
// 11 bits the first leaves multiples of 2^-10 up to 2^-3, the second up to 2^-7, and that
// the third holds, so fp16's results see their weights' roundings to fp16 alone. For bf16
// the first is cut, an instruction less for two weights (prompt chunks 549 us
// otherwise): it leaves up to 2^-2, the second up to 2^-6, and the third is off by 2^-10
// at most. Weights below 2^-12 are off by half a step of the third, 2^-23; its ties go up
// for every second key and down for the others.
template <bool kF16>
MOE_DEV void weight_numbers(float a, float b, float c, float d, uint32_t ties,
                            uint32_t (&out)[kWeightNum]) {
  __half2 w[2] = {__floats2half2_rn(a, b), __floats2half2_rn(c, d)};
#pragma unroll
  for (int i = 0; i < kWeightNum; ++i) {
    uint32_t x[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      x[k] = *reinterpret_cast<const uint32_t*>(&w[k]);
      if (i == 2) x[k] += ties;
      else if (i == 1 || kF16) x[k] += 0x00800080u;
      if (i + 1 < kWeightNum) {
        const uint32_t upper = x[k] & 0xff00ff00u;
        w[k] = __hmul2(__hsub2(w[k], *reinterpret_cast<const __half2*>(&upper)),
                       __float2half2_rn(8.f));
      }
    }
    out[i] = __byte_perm(x[0], x[1], 0x7531);
  }
}
MOE_DEV constexpr float weight_unit(int i) {
  return i == 0 ? 1.f : i == 1 ? 0x1p-3f : 0x1p-6f;
}

// The largest of the warp's values; NaN are passed over.
MOE_DEV float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Bytes of w that are NaN, 0x80 each.
MOE_DEV uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// Query rows [n0, n1) of the part are those that see `key`.
MOE_DEV void visible(const Attend8Args& a, const Part& pt, int key, int* n0, int* n1) {
  const long long back = (long long)key - pt.pos0;     // of the first token that sees it
  *n0 = (int)min(max(back, 0ll), (long long)pt.ntok) * a.group;
  *n1 = pt.rows;
  if (a.window > 0 && key >= a.sinks)
    *n1 = (int)min(max(back + a.window, 0ll), (long long)pt.ntok) * a.group;
}

// In a tile of V that not all rows see whole: rows that no row of the item sees
// become zeros; NaN in rows that some see and others do not is taken out, and
// noted in `spoiled`. A thread takes the row of its key, the `per` groups of a
// stream every per-th piece of it.
template <int kDim>
MOE_DEV void clean_values(const Attend8Args& a, const Part& pt, unsigned char* tile, int key0,
                          int gl, int per, unsigned long long* spoiled, int* spoils) {
  const int kt = threadIdx.x & 127, key = key0 + kt;
  const bool none = key >= pt.hi || (key < pt.lo && key >= pt.sk);
  if (!none && !some_see(a, pt.pos0, pt.hi, key)) return;
  int n0, n1;
  visible(a, pt, key, &n0, &n1);
#pragma unroll 1
  for (int c = gl; c < kDim / 16; c += per) {
    uint4* at = reinterpret_cast<uint4*>(tile + kt * kDim + c * 16);
    if (none) {
      *at = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint4 x = *at;
    if (!(nan_bytes(x.x) | nan_bytes(x.y) | nan_bytes(x.z) | nan_bytes(x.w))) continue;
    const int d0 = (int)(swizzled<kDim>(kt, c * 16) - kt * kDim);  // its first column
    const unsigned long long rows =
        (n1 >= 64 ? ~0ull : (1ull << n1) - 1) & ~(n0 >= 64 ? ~0ull : (1ull << n0) - 1);
    unsigned char* bytes = reinterpret_cast<unsigned char*>(at);
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
      if ((bytes[i] & 0x7f) != 0x7f) continue;
      bytes[i] = 0;
      atomicOr(spoiled + d0 + i, rows);
      *static_cast<volatile int*>(spoils) = 1;
    }
  }
}

template <int kDim>
MOE_DEV const float* part_of(const Params& p, int cta, bool ends) {
  return p.part + (size_t)(2 * cta + (ends ? 0 : 1)) * slot_floats(kDim);
}

// Tokens that see nothing, at positions below 0 (a refused request's, whose cache
// length is 0, or those of a cache shorter than the pass), have no part in the work
// that is cut: the softmax threads of all CTAs share their rows, and clear them.
template <int kDim>
__device__ __noinline__ void clear_blind(const Attend8Args& a, int page_shift) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int b0 = 0; b0 < a.n_requests; b0 += 32) {
    Request mine = {0, 0, 0};
    bool bad;
    if (b0 + lane < a.n_requests) mine = request(a, page_shift, b0 + lane, &bad);
#pragma unroll 1
    for (uint32_t todo = __ballot_sync(0xffffffffu, mine.q > mine.len); todo; todo &= todo - 1) {
      const int from = __ffs(todo) - 1, q = __shfl_sync(0xffffffffu, mine.q, from);
      const int len = __shfl_sync(0xffffffffu, mine.len, from);
      const int first = __shfl_sync(0xffffffffu, mine.first, from);
      const int64_t n = (int64_t)(q - len) * a.n_heads * (kDim / 8);
      for (int64_t i = (int64_t)blockIdx.x * 512 + threadIdx.x - 128; i < n; i += gridDim.x * 512) {
        const int64_t row = i / (kDim / 8), t = row / a.n_heads;
        uint16_t* to = static_cast<uint16_t*>(a.out) + (first + t) * a.out_token_stride +
                       (row - t * a.n_heads) * a.out_head_stride;
        reinterpret_cast<uint4*>(to)[i % (kDim / 8)] = make_uint4(0, 0, 0, 0);
      }
      __syncwarp();
    }
  }
}

// The parts of an item joined in key order, those of CTAs `first` to this one: a
// thread has 4 columns of a row and loads 8 parts at once. (Barriers and flags as
// in attend.cu.)
template <int kDim, bool kF16>
MOE_DEV void join_parts(const Params& p, const Start& st, volatile int* lost) {
  const Attend8Args& a = p.a;
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
        *lost = 0xB70;
        if (exchange(word, given_up(p.call)) == p.call) break;
        word = nullptr;
        break;
      }
    }
    if (word) *word = 0ull;
  }
  asm volatile("bar.sync 2, 512;" ::: "memory");
  const int rows = st.ntok * a.group;
#pragma unroll 1
  for (int i = tid; i < rows * (kDim / 4); i += 512) {
    const int row = i / (kDim / 4), c4 = i % (kDim / 4);
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
          mc[j] = __ldcg(part + kRows * kDim + row);
          sc[j] = __ldcg(part + kRows * kDim + kRows + row);
          oc[j] = __ldcg(reinterpret_cast<const float4*>(part + row * kDim) + c4);
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
    const int t = row / a.group, g = row - t * a.group;
    uint16_t* out = static_cast<uint16_t*>(a.out) + (int64_t)(st.row0 + t) * a.out_token_stride +
                    (int64_t)(st.head0 + g) * a.out_head_stride;
    *reinterpret_cast<uint2*>(out + c4 * 4) =
        make_uint2(round16<kF16>(o.x * inv, o.y * inv), round16<kF16>(o.z * inv, o.w * inv));
  }
}

template <int kDim, int kNum>
__global__ void __launch_bounds__(kThreads, 1) attend8_kernel(const __grid_constant__ Params p) {
  using Z = Sizes<kDim, kNum>;
  constexpr bool kF16 = kNum == 3;
  constexpr int kStages = Z::kStages, kKeyStages = Z::kKeyStages;
  constexpr float kBase = moe::kBase<kF16>, kGrow = moe::kGrow<kF16>;
  using KeyPlace = Place<kKeyStages>;
  using ValuePlace = Place<Z::kValueStages>;
  using M = Misc<kStages>;
  static_assert(sizeof(M) <= kOffRef, "misc words");
  const Attend8Args& a = p.a;
  extern __shared__ __align__(1024) unsigned char smem[];
  if (smem_addr(smem) & 1023u) {               // the tiles' swizzle needs it
    if (threadIdx.x == 0) report_error(a.err, ERR_CHECK, 0xB23);
    return;
  }
  unsigned char* misc = smem + Z::kOffMisc;
  M& m = *reinterpret_cast<M*>(misc);
  float* refs = reinterpret_cast<float*>(misc + kOffRef);
  float* qscale = reinterpret_cast<float*>(misc + kOffQScale);
  float* stat = reinterpret_cast<float*>(misc + kOffStat);
  Slot* slots = reinterpret_cast<Slot*>(misc + kOffSlots);
  Part* parts = reinterpret_cast<Part*>(misc + kOffParts);
  // the same value in every lane, and known to be
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0) - 4;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&m.full[i], 1);
      mbar_init(&m.empty[i], 1);
    }
    for (int i = 0; i < kParts; ++i) {
      mbar_init(&m.part_full[i], 1);
      mbar_init(&m.part_empty[i], 19);         // the loader, both MMA warps, 16 of the softmax
    }
    mbar_init(&m.raw_full, 32);                // the lanes that copy, with their copies
    mbar_init(&m.raw_empty, 16);
    mbar_init(&m.q_full, 16);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&m.pg_full[i], 1);
      mbar_init(&m.sc_full[i], 1);
      mbar_init(&m.tile_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&m.s_full[i], 1);
      mbar_init(&m.s_empty[i], 16);            // a warp counts 1, 2 or 4 (see below)
      mbar_init(&m.p_full[i], 16);
      mbar_init(&m.p_done[i], 1);
    }
    mbar_init(&m.drain[0], 1);
    mbar_init(&m.drain[1], 1);
    fence_mbar_init();
    m.lost = m.spoils = 0;
    m.start.joins = 0;
  }
  if (warp == -3) umma::tmem_alloc(&m.tmem, Z::kCols);
  if (threadIdx.x == 0) {
    prefetch_tmap(&p.kmap);
    prefetch_tmap(&p.vmap);
  }
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < 128) p.spoiled[blockIdx.x * 128 + threadIdx.x] = 0;
  // (the ring holds the plan's counts until the first tiles are on their way)
  int blind = 0;                               // some tokens see nothing
  if (threadIdx.x < kPlanThreads) {
    find_start(p, reinterpret_cast<long long*>(smem + Z::kOffRing), m.part, &m.start);
  } else {
    for (int b = threadIdx.x - kPlanThreads; b < a.n_requests; b += kThreads - kPlanThreads) {
      bool bad;
      const Request r = request(a, p.page_shift, b, &bad);
      blind |= r.q > r.len;
    }
  }
  fence_proxy_async_smem();
  umma::fence_before_sync();
  blind = __syncthreads_or(blind);
  umma::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, m.tmem, 0);

  volatile int* lost = &m.lost;
  bool ok = true;  // no wait of this role has been lost
  auto wait_at = [&](uint32_t bar, uint32_t parity, int site) {
    if (!__all_sync(0xffffffffu, try_at(bar, parity)))
      ok = wait_longer(bar, parity, lost, site) && ok;
  };
  auto wait = [&](uint64_t* bar, uint32_t parity, int site) {
    wait_at(smem_addr(bar), parity, site);
  };
  auto wait_both = [&](uint64_t* a, uint32_t a_parity, uint64_t* b, uint32_t b_parity, int site) {
    const bool first = try_at(smem_addr(a), a_parity), second = try_at(smem_addr(b), b_parity);
    if (!__all_sync(0xffffffffu, first && second)) {
      wait(a, a_parity, site);
      wait(b, b_parity, site + 0x80);
    }
  };
  // a barrier of each stream, from that of stream 0 on: phase counts − 1 has ended
  auto wait_four = [&](uint64_t* bars, uint32_t counts, int site) {
    bool done = true;
#pragma unroll
    for (int s = 0; s < 4; ++s)
      done = try_at(smem_addr(bars + s), count_of(counts, s) & 1u ^ 1u) && done;
    if (!__all_sync(0xffffffffu, done)) {
#pragma unroll 1
      for (int s = 0; s < 4; ++s) wait(bars + s, count_of(counts, s) & 1u ^ 1u, site);
    }
  };
  // The parts, one after the other. A lost wait ends a role's walk: what a part
  // says may then be another's.
  int part_no = 0;
  auto next = [&]() -> const Part* {
    const int slot = part_no & (kParts - 1);
    wait(&m.part_full[slot], part_no >> 3 & 1u, 0xB32);
    return ok && parts[slot].n >= 0 ? parts + slot : nullptr;
  };
  auto done_with_part = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&m.part_empty[part_no & (kParts - 1)]);
    ++part_no;
  };
  uint32_t counts = 0;

  if (warp < 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == -4) {
    // ------------------------------------------------------------- loader --
    const int page = 1 << p.page_shift;
    const int rows = min(page, kTile);          // rows of a box
    // keys and values that one item reads alone are not kept in L2: the rows of
    // the other heads beside them are (single tokens 258 us otherwise, 243)
    const uint64_t stay = l2_evict_normal_policy(), go = l2_evict_first_policy();
    // Lanes 0-15 load K_{j + streams}, a box each, lanes 16-31 V_j: with one after the
    // other the loader was what a tile of 16 rows took. (A box takes its 80 cycles to
    // issue: a lane each, or one lane of the warp for all, which took longer.)
    const int half = lane >> 4, piece = lane & 15;
    const CUtensorMap* map = half ? &p.vmap : &p.kmap;
    const uint32_t to = smem_addr(smem) + Z::kOffRing + piece * rows * kDim;
    const int block = min(piece * rows / 16, kScaleBlocks - 1);  // first of the lane's box
    int tile_no = 0;
    KeyPlace k_at(0);                           // the next places in the rings
    ValuePlace v_at(0);
    for (const Part* pt; (pt = next()); done_with_part()) {
      const int n = pt->n, streams = 1 << pt->shift, head = pt->h;
      const uint64_t policy = pt->once ? go : stay;
#pragma unroll 1
      for (int j = -streams; ok && j < n; ++j) {
        const bool keys = j + streams < n, values = j >= 0;
        const bool has = half ? values : keys;
        const int no = tile_no + (half ? j : j + streams), slot = no & (kSlots - 1);
        const int k_stage = k_at.stage(), v_stage = kKeyStages + v_at.stage();
        const int stage = half ? v_stage : k_stage;
        // (a tile's pages are there for V when they were for K)
        const uint32_t empty = smem_addr(&m.empty[stage]), pages = smem_addr(&m.pg_full[slot]);
        const bool there = !has || (try_at(empty, (half ? v_at.parity() : k_at.parity()) ^ 1u) &&
                                    (half || try_at(pages, no / kSlots & 1u)));
        if (!__all_sync(0xffffffffu, there)) {
          if (keys) {
            const int first = tile_no + j + streams;
            wait(&m.pg_full[first & (kSlots - 1)], first / kSlots & 1u, 0xB30);
            wait(&m.empty[k_stage], k_at.parity() ^ 1u, 0xB31);
          }
          if (values) wait(&m.empty[v_stage], v_at.parity() ^ 1u, 0xB31);
        }
        if (ok) {
          const int pg = has && piece * rows < kTile ? slots[slot].page[block] : -1;
          const int row = page > kTile && has ? slots[slot].key0 & (page - 1) : 0;
          const uint32_t wanted = __ballot_sync(0xffffffffu, pg >= 0);
          if (piece == 0 && has)
            mbar_arrive_expect_tx(&m.full[stage],
                                  __popc(wanted >> (16 * half) & 0xffffu) * rows * kDim);
          __syncwarp();
          if (pg >= 0)
            tma_load_4d_at(to + stage * Z::kTileBytes, map, 0, head, row, pg, &m.full[stage],
                           policy);
          __syncwarp();
        }
        if (keys) k_at.next();
        if (values) v_at.next();
      }
      tile_no += n;
    }
    // After a lost wait the tiles still in flight must land before the CTA
    // ends; without one, every tile has been waited for by the MMA warp.
    if (!ok) {
#pragma unroll 1
      for (int i = 0; i < 2 * 500 * kStages; ++i) try_longer(&m.full[i / 1000], i & 1);
    }
  } else if (warp == -3 || warp == -2) {
    // ---------------------------------------------------------------- MMA --
    const bool scores = warp == -3;
    constexpr int kSteps = kDim / 32;
    constexpr uint32_t kRowHi = umma::kDescHi8<kDim>, kPHi = umma::kDescHi8<128>;
    constexpr uint32_t kOne = 1u << 16;                // (a K-major tile has no other distance)
    const uint32_t ring_at = (smem_addr(smem) + Z::kOffRing) >> 4;
    const uint32_t q_at = smem_addr(smem) >> 4;
    const uint32_t p_at = (smem_addr(smem) + Z::kOffP) >> 4;
    constexpr uint32_t kNextP = (kTile * 128u >> 4) << 16;  // the next 128 columns of P
    int tile_no = 0;
    auto commit = [&](uint64_t* bar) {                 // arrives when the MMAs so far are done
      if (ok) umma::commit_elect(bar);
    };
    for (const Part* pt; (pt = next()); done_with_part()) {
      const int n = pt->n, shift = pt->shift, streams = 1 << shift;
      if (scores) {                                    // S = K · Qᵀ
        const int cols = pt->wide * kNum;
        const int pitch = Z::kScoreColumns >> shift;   // columns between streams
        const uint32_t id = umma::idesc_f8(kTile, cols, false, false);
        // S may be laid out anew once the last scores of every stream are read
        wait_four(m.s_empty, counts, 0xB41);
        wait(&m.q_full, part_no & 1u, 0xB42);
#pragma unroll 1
        for (int j = 0; ok && j < n; ++j) {
          const int s = j & (streams - 1);
          const uint32_t k = count_of(counts, s) + (uint32_t)(j >> shift);
          const KeyPlace at(tile_no + j);
          // (who waits for the scores then has the scales too)
          wait_both(&m.full[at.stage()], at.parity(), &m.sc_full[(tile_no + j) & (kSlots - 1)],
                    (tile_no + j) / kSlots & 1u, 0xB43);
          wait(&m.s_empty[s], k & 1u ^ 1u, 0xB44);
          umma::fence_after_sync();
          if (ok)
            umma::mma_f8<kSteps, kRowHi, kRowHi, 2, 2>(
                tmem + s * pitch, (ring_at + at.stage() * (Z::kTileBytes >> 4)) & 0x3fffu | kOne,
                q_at & 0x3fffu | kOne, id, 0u);
          commit(&m.s_full[s]);
          commit(&m.empty[at.stage()]);
        }
      } else {                                         // Oᵀ (+)= Vᵀ · Pᵀ
        const int cols = pt->wide * kWeightNum;
        const int pitch = Z::kColumns >> shift;
        const uint32_t id = umma::idesc_f8(kDim, cols, true, true);
#pragma unroll 1
        for (int j = 0; ok && j < n; ++j) {
          const int s = j & (streams - 1);
          const uint32_t k = count_of(counts, s) + (uint32_t)(j >> shift);
          const ValuePlace at(tile_no + j);
          const int stage = kKeyStages + at.stage();
          const uint32_t first = s * pitch;            // column of P
          wait_both(&m.p_full[s], k & 1u, &m.full[stage], at.parity(), 0xB45);
          umma::fence_after_sync();
          if (ok)
            umma::mma_f8<4, kRowHi, kPHi, (32 * kDim >> 4), (32 * 128 >> 4)>(
                tmem + Z::kColO + s * pitch,
                (ring_at + stage * (Z::kTileBytes >> 4)) & 0x3fffu | kOne,
                (p_at + (first >> 7) * (kTile * 128 >> 4) + ((first & 127u) >> 4)) & 0x3fffu |
                    kNextP,
                id, j >= streams ? 1u : 0u);
          commit(&m.p_done[s]);
          commit(&m.empty[stage]);
          commit(&m.tile_done[(tile_no + j) & (kSlots - 1)]);
        }
      }
      tile_no += n;
      counts = add_counts(counts, n, shift);
    }
    // Every MMA, and every arrival that hangs on one, is done before tensor
    // memory is released.
    umma::commit_elect(&m.drain[scores]);
#pragma unroll 1
    for (int i = 0; i < kTries && !try_longer(&m.drain[scores], 0); ++i) {
    }
    __syncwarp();
  } else if (warp == -1) {
    // ------------------------------------------------------------- ahead --
    // Three things, each as soon as there is room for it: the parts; the pages and
    // scales of four tiles at a time, 8 lanes a tile, a lane its 16 keys (the pages
    // of the next four are asked for while the scales of these are on their way);
    // a part's queries, 16 bytes a lane.
    constexpr int kPieces = kDim / 8;                  // of a query row
    Walk w = m.start.w;
    Request r = m.start.r;
    bool more = true;                                  // parts to come
    int published = 0, queries = 0;                    // parts
    // tiles written; the next one's part, and place in it
    int tiles = 0, t_part = 0, t_next = 0;
    bool q_done = false;
    const int q = lane >> 3, block = lane & 7;
    const int page_mask = (1 << p.page_shift) - 1, block_shift = p.page_shift - p.blocks_shift;
    const int box = min(page_mask + 1, kTile) / 16;    // blocks of a box
    // the next four tiles: how many there are, and this lane's (tile < 0: none)
    int count = 0, tile = -1, edge = 0, page = -1, head = 0;
    bool wants = false;
    auto ask = [&]() {
      // the 8 lanes of a tile look for it from the part of the first of the four on
      int at = t_part, j = t_next + q;
      tile = page = -1;
      wants = false;
      while (at < published) {
        const int n = parts[at & (kParts - 1)].n;
        if (n < 0) at = published;
        if (j < n || n < 0) break;
        j -= n;
        ++at;
      }
      if (at < published) {
        const Part& pt = parts[at & (kParts - 1)];
        tile = pt.tile(j);
        head = pt.h;
        edge = tile >= pt.edge_hi || (tile < pt.edge_lo && tile >= pt.edge_sk);
        const int key = tile * kTile + block * 16;
        wants = key < pt.hi && (key + 16 > pt.lo || key < pt.sk);  // some row sees of the block
        if (wants) page = a.block_table[(size_t)pt.b * a.max_blocks + (key >> p.page_shift)];
      }
      __syncwarp();
      count = __popc(__ballot_sync(0xffffffffu, tile >= 0)) >> 3;
      t_next += count;
      while (t_part < published) {
        const int n = parts[t_part & (kParts - 1)].n;
        if (n < 0 || t_next < n) break;
        t_next -= n;
        ++t_part;
      }
    };
    int idle = 0;
    while (ok && (more || !q_done || count || t_part < published - 1)) {
      bool did = false;
      // parts
      if (more && published < min(queries, t_part) + kParts - 1) {
        const int slot = published & (kParts - 1);
        if (__all_sync(0xffffffffu, try_now(&m.part_empty[slot], published >> 3 & 1u ^ 1u))) {
          Part next_one;
          more = next_part(p, w, r, &next_one);
          if (!more) next_one.n = -1;
          if (lane == 0) {
            parts[slot] = next_one;
            mbar_arrive(&m.part_full[slot]);
          }
          __syncwarp();
          ++published;
          did = true;
        }
      }
      if (count == 0 && t_part < published) ask();
      // queries
      if (!q_done && queries < published &&
          __all_sync(0xffffffffu, try_now(&m.raw_empty, queries & 1u ^ 1u))) {
        const Part& pt = parts[queries & (kParts - 1)];
        const int rows = pt.n >= 0 ? pt.rows : 0;
        q_done = pt.n < 0;
        const uint32_t to = smem_addr(smem) + Z::kOffRaw;
        const uint16_t* from = static_cast<const uint16_t*>(a.q) +
                               (int64_t)pt.row0 * a.q_token_stride +
                               (int64_t)pt.h * a.group * a.q_head_stride;
#pragma unroll 1
        for (int i = lane; i < rows * kPieces; i += 32) {
          const int row = i / kPieces, t = row / a.group;
          const uint16_t* at = from + t * a.q_token_stride + (row - t * a.group) * a.q_head_stride +
                               i % kPieces * 8;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * 16), "l"(at)
                       : "memory");
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                         smem_addr(&m.raw_full))
                     : "memory");
        ++queries;
        did = true;
      }
      // tiles
      if (count > 0) {
        const int last = tiles + count - 1;            // (slots are given back in order)
        if (__all_sync(0xffffffffu, try_now(&m.tile_done[last & (kSlots - 1)],
                                            last / kSlots & 1u ^ 1u))) {
          const int now = count, first = tiles, mine = tile, is_edge = edge;
          int pg = page;
          const bool there = wants && pg >= 0 && pg < a.cache.n_pages;
          if (wants && !there) {
            report_error(a.err, ERR_CHECK, 0xB21);
            pg = (int)a.cache.n_pages;                 // out of the map: the box reads zeros
          }
          float ks = 1.f, vs = 1.f;
          if (there) {
            const int64_t at =
                ((((int64_t)pg * a.cache.n_kv_heads) + head) << p.blocks_shift) +
                ((mine * kTile + block * 16 & page_mask) >> block_shift);
            ks = __ldg(a.cache.k_scale + at);
            vs = __ldg(a.cache.v_scale + at);
          }
          // a box's page: that of any of its blocks that is wanted
#pragma unroll
          for (int o = 1; o < kScaleBlocks; o <<= 1) {
            const int other = __shfl_xor_sync(0xffffffffu, pg, o);
            if (o < box) pg = max(pg, other);
          }
          Slot& slot = slots[(first + q) & (kSlots - 1)];
          if (mine >= 0) {
            slot.page[block] = pg;
            if (block == 0) {
              slot.key0 = mine * kTile;
              slot.edge = is_edge;
            }
          }
          __syncwarp();
          if (lane < now) mbar_arrive(&m.pg_full[(first + lane) & (kSlots - 1)]);
          tiles += now;
          ask();
          const float least = pow2(MOE_KV8_MIN_EXP), most = pow2(MOE_KV8_MAX_EXP);
          if (!(ks >= least && ks <= most && vs >= least && vs <= most)) {
            report_error(a.err, ERR_CHECK, 0xB33);
            ks = ks > most ? most : ks >= least ? ks : least;
            vs = vs > most ? most : vs >= least ? vs : least;
          }
          const uint32_t bits = __float_as_uint(vs);   // (a power of two's is exact)
          const float l = bits & 0x7fffffu ? log2f(vs) : (float)((int)(bits >> 23) - 127);
          if (mine >= 0) {
            slot.ks[block] = ks;
            slot.lv[block] = l + kBase;
          }
          __syncwarp();
          if (lane < now) mbar_arrive(&m.sc_full[(first + lane) & (kSlots - 1)]);
          did = true;
        }
      }
      if (did) {
        idle = 0;
      } else {
        // (a limit of about half a second; see wait_or_abort)
        __nanosleep(100);
        if ((++idle & 255) == 255 && (*lost || idle > (1 << 22))) {
          if (*lost == 0) *lost = 0xB60;
          ok = false;
        }
        ok = __all_sync(0xffffffffu, ok);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ------------------------------------------------------------ softmax --
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    if (a.clear) clear_rows<kDim>(a);                  // while the first tiles are on their way
    if (blind) clear_blind<kDim>(a, p.page_shift);
    const int g = warp >> 2, quarter = warp & 3;       // group, and the warp's quarter of a tile
    const int kt = threadIdx.x & 127;                  // key of the tile, TMEM lane
    const uint32_t lanes = tmem + ((uint32_t)quarter << 21);  // 32 · quarter in the upper half
    float* ref = refs + g * 16;                // −m of the group's columns
    float* group_stat = stat + g * 4 * 16;     // [4 warps][rows]
    auto group_sync = [&]() {
      asm volatile("bar.sync %0, 128;" ::"r"(3 + g) : "memory");
    };
    auto all_sync = [&]() { asm volatile("bar.sync 2, 512;" ::: "memory"); };
    int tile_no = 0;                                   // of the part's first tile
    bool open = false;                                 // the last part does not end its item
    const Part* pt = nullptr;                          // the present part
    int gone = 0;                                      // some warp has lost a wait: all of them stop
#pragma unroll 1
    for (;;) {
      // The next part's queries into numbers: a warp takes every 16th row, divides
      // it by the power of two that makes its largest size 224 to 448, and leaves
      // that power with the scale as the row's factor. (For all but the first, the
      // products with the present part's are done, and the tensor cores begin with
      // the next one's while the present one's results go out.)
      const int no = pt ? part_no + 1 : part_no;
      const Part* then = parts + (no & (kParts - 1));
      wait(&m.part_full[no & (kParts - 1)], no >> 3 & 1u, 0xB32);
      wait(&m.raw_full, no & 1u, 0xB58);
      if (!ok || then->n < 0) then = nullptr;
      if (then) {
        constexpr int kMine = kDim / 32;               // columns of a lane
        const int rows = then->rows, wide = then->wide;
        const float to_log2 = a.scale * kLog2e;
        // (the chains of its four rows side by side)
        uint32_t x[4][kMine / 2];
        float top[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = min(warp + 16 * i, rows - 1);
          const unsigned char* at = smem + Z::kOffRaw + r * (kDim * 2) + lane * (kMine * 2);
          if constexpr (kMine == 4) {
            const uint2 w = *reinterpret_cast<const uint2*>(at);
            x[i][0] = w.x;
            x[i][1] = w.y;
          } else {
            x[i][0] = *reinterpret_cast<const uint32_t*>(at);
          }
        }
        auto element = [&](int i, int c) {
          const uint32_t w = x[i][c / 2] >> (16 * (c & 1));
          return kF16 ? __half2float(__ushort_as_half((unsigned short)(w & 0xffffu)))
                      : __uint_as_float(w << 16);
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          top[i] = 0.f;
#pragma unroll
          for (int c = 0; c < kMine; ++c) {
            const float v = element(i, c);
            top[i] = fmaxf(top[i], fabsf(v));
            if (v != v) top[i] = INFINITY;
          }
          top[i] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top[i])));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = warp + 16 * i;
          if (r >= rows) break;
          const uint32_t bits = __float_as_uint(top[i]);
          int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
          e = min(max(e, -120), 120);
          const float inv = pow2(-e);
          float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < kMine; ++c) v[c] = element(i, c);
          uint32_t num[kNum];
          numbers_of<kNum>(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv, num);
#pragma unroll
          for (int k = 0; k < kNum; ++k) {
            unsigned char* to = smem + swizzled<kDim>(k * wide + r, lane * kMine);
            if constexpr (kMine == 4)
              *reinterpret_cast<uint32_t*>(to) = num[k];
            else
              *reinterpret_cast<uint16_t*>(to) = (uint16_t)num[k];
          }
          // (a row with NaN or an infinity has NaN for its factor)
          if (lane == 0)
            qscale[(no & 1) * kRows + r] = top[i] <= 3.402823466e38f ? to_log2 * pow2(e) : NAN;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&m.raw_empty);
          mbar_arrive(&m.q_full);
        }
      }
      // the last products of every stream
      wait_four(m.p_done, counts, 0xB57);
      gone = !ok;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\t"
          "setp.ne.s32 p, %0, 0;\n\t"
          "bar.red.or.pred q, 2, 512, p;\n\t"
          "selp.s32 %0, 1, 0, q;\n\t}"
          : "+r"(gone)::"memory");
      if (gone) break;
      if (pt) {
        // ---- the present part's results out
        const int n = pt->n, shift = pt->shift, streams = 1 << shift;
        umma::fence_after_sync();
        const bool spoils = *static_cast<volatile int*>(&m.spoils);
        float* slot = p.part + (size_t)(2 * blockIdx.x + (pt->ends ? 0 : 1)) * slot_floats(kDim);
        // What each column of each stream counts: its sums join those of the row's
        // other streams, and are divided by Σ where the item is whole. The factors
        // take the references' place; column i is that of row i % width of its
        // stream.
        const int width = kRows >> shift;
        if (warp < kRows / 32) {
          const int i = threadIdx.x - 128, row = i & (width - 1);
          float top = -INFINITY, sum = 0.f;
#pragma unroll 1
          for (int z = row; z < kRows; z += width) top = fmaxf(top, -refs[z]);
#pragma unroll 1
          for (int z = row; z < kRows; z += width) {
            const float* l = stat + z / 16 * (4 * 16) + z % 16;
            // (a stream that saw none of the row's keys has zeros, or sums of NaN)
            sum = fmaf(l[0] + l[16] + (l[2 * 16] + l[3 * 16]),
                       top == -INFINITY ? 1.f : exp2_approx(-refs[z] - top), sum);
          }
          float by = top == -INFINITY ? 1.f : exp2_approx(-refs[i] - top);
          if (pt->whole) {
            by *= inverse(sum);
          } else if (i < pt->rows) {
            slot[kRows * kDim + i] = top;
            slot[kRows * kDim + kRows + i] = sum;
          }
          asm volatile("bar.sync 7, %0;" ::"n"(kRows) : "memory");
          refs[i] = by;
        }
        all_sync();
        // A thread has column d of V, and its group a quarter of the rows.
        const int d = kDim == 128 ? kt : quarter * 16 + (lane & 15);
        const bool valid = kDim == 128 || lane < 16;
        const int rows = pt->rows, wide = pt->wide, take = wide / 4, from = g * take;
        const uint32_t o_from = lanes + Z::kColO + from;
        const unsigned long long spoilt =
            spoils ? __ldcg(p.spoiled + blockIdx.x * 128 + d) : 0ull;
        uint16_t* through = reinterpret_cast<uint16_t*>(smem + Z::kOffP);
        const bool whole = pt->whole;
#pragma unroll 1
        for (int i = 0; i < take && from + i < rows; i += 4) {  // (take: a multiple of 4)
          float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
          for (int z = 0; z < streams && z < n; ++z) {
            uint32_t w[kWeightNum][4];
#pragma unroll
            for (int e = 0; e < kWeightNum; ++e)
              umma::ld_x4(o_from + z * (Z::kColumns >> shift) + e * wide + i, w[e]);
            const float4 by = *reinterpret_cast<const float4*>(refs + z * width + from + i);
            const float f[4] = {by.x, by.y, by.z, by.w};
            umma::wait_ld();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              float v = __uint_as_float(w[0][c]);
#pragma unroll
              for (int e = 1; e < kWeightNum; ++e)
                v = fmaf(__uint_as_float(w[e][c]), weight_unit(e), v);
              o[c] = fmaf(v, f[c], o[c]);
            }
          }
          if (spoilt >> (from + i) & 15ull) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (spoilt >> (from + i + c) & 1ull) o[c] = NAN;
          }
          if (whole) {
            const uint32_t w0 = round16<kF16>(o[0], o[1]), w1 = round16<kF16>(o[2], o[3]);
            uint16_t* to = through + (from + i) * kDim + d;
            if (valid) {
              to[0] = (uint16_t)w0;
              to[kDim] = (uint16_t)(w0 >> 16);
              to[2 * kDim] = (uint16_t)w1;
              to[3 * kDim] = (uint16_t)(w1 >> 16);
            }
          } else if (valid) {
#pragma unroll
            for (int c = 0; c < 4; ++c) slot[(from + i + c) * kDim + d] = o[c];
          }
        }
        open = !pt->ends;
        umma::fence_before_sync();
        // O and the factors have been read before any stream goes on
        all_sync();
        if (pt->whole) {
          // rows of results pass through P, 16 bytes a thread
          constexpr int kPieces = kDim / 8;
          uint16_t* out = static_cast<uint16_t*>(a.out) + (int64_t)pt->row0 * a.out_token_stride +
                          (int64_t)pt->h * a.group * a.out_head_stride;
#pragma unroll 1
          for (int i = threadIdx.x - 128; i < rows * kPieces; i += 512) {
            const int r = i / kPieces, t = r / a.group;
            *reinterpret_cast<uint4*>(out + t * a.out_token_stride +
                                      (r - t * a.group) * a.out_head_stride + i % kPieces * 8) =
                *reinterpret_cast<const uint4*>(through + i * 8);
          }
        }
        if (spoils) {
          if (threadIdx.x < 256) p.spoiled[blockIdx.x * 128 + threadIdx.x - 128] = 0;
          if (threadIdx.x == 128) m.spoils = 0;
        }
        done_with_part();
      }
      pt = then;
      if (!pt) break;

      // ---- a part's tiles
      const int n = pt->n, shift = pt->shift, streams = 1 << shift, wide = pt->wide;
      const int s = g >> (2 - shift), gl = g & (3 >> shift);  // stream, and group of it
      const int c0 = 16 * gl;                  // the group's first query row
      const bool active = c0 < wide;
      const uint32_t column = s * (Z::kColumns >> shift) + c0;  // of O and P
      const uint32_t s_addr = lanes + s * (Z::kScoreColumns >> shift) + c0;
      const uint32_t o_addr = lanes + Z::kColO + column;
      // a stream's barriers count 16: each of its 16 / streams warps arrives for as many
      auto arrive = [&](uint32_t bar) {
        __syncwarp();
        asm volatile(
            "{\n\t.reg .pred e;\n\t"
            "elect.sync _|e, 0xffffffff;\n\t"
            "@e mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
            "r"(streams)
            : "memory");
      };
      // rows that do not exist stay out of every vote; the others' references are 0
      // until they have seen a key
      if (quarter == 0 && lane < 16)
        ref[lane] = c0 + lane < pt->rows ? 0.f : -INFINITY;
      uint32_t fresh = low_bits(min(pt->rows - c0, 16));
      all_sync();
      const float* factor = qscale + (part_no & 1) * kRows + c0;
      uint64_t sums[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) sums[c] = 0;
      uint32_t k = count_of(counts, s);
      // what a tile needs, as shared-memory addresses
      const uint32_t bars = smem_addr(&m.s_full[s]);
      const uint32_t factors = smem_addr(factor), refs_at = smem_addr(ref);
      constexpr uint32_t kEmpty = 32, kPFull = 64, kPDone = 96;  // of the stream's, behind s_full
      const uint32_t first_slot = smem_addr(slots) + (kt >> 4) * 4;
      const uint32_t ties = kt & 1 ? 0x00800080u : 0x007f007fu;  // see weight_numbers
      uint32_t p_at[kWeightNum];                       // of the thread's weights
#pragma unroll
      for (int i = 0; i < kWeightNum; ++i) {
        const uint32_t at = column + i * wide;
        p_at[i] = smem_addr(smem) + Z::kOffP + (at >> 7) * (kTile * 128) +
                  swizzled<128>(kt, at & 127u);
      }
#pragma unroll 1
      for (int j = s; j < n; j += streams, ++k) {
        wait_at(bars, k & 1u, 0xB51);
        // (a lost wait leaves the sums wrong, and the barriers in step)
        const uint32_t slot = first_slot + (uint32_t)((tile_no + j) & (kSlots - 1)) * sizeof(Slot);
        const int edge = ld_shared(slot + offsetof(Slot, edge) - (kt >> 4) * 4);
        if (active) {
          umma::fence_after_sync();
          uint32_t x[16], y[kNum - 1][16];
          umma::ld_x16(s_addr, x);
#pragma unroll
          for (int i = 1; i < kNum; ++i) umma::ld_x16(s_addr + i * wide, y[i - 1]);
          const float ks = __int_as_float(ld_shared(slot)),
                      lv = __int_as_float(ld_shared(slot + offsetof(Slot, lv)));
          const float iv = exp2_approx(kBase - lv);    // 1 / vs
          umma::wait_ld();
          umma::fence_before_sync();
          arrive(bars + kEmpty);
          // q · K
#pragma unroll
          for (int i = 1; i < kNum; ++i) {
            const uint64_t unit = pair_f(number_unit(i), number_unit(i));
#pragma unroll
            for (int c = 0; c < 16; c += 2) {
              float lo, hi;
              split(fma2(pair(y[i - 1][c], y[i - 1][c + 1]), unit, pair(x[c], x[c + 1])), &lo, &hi);
              x[c] = __float_as_uint(lo);
              x[c + 1] = __float_as_uint(hi);
            }
          }
          const uint64_t ks2 = pair_f(ks, ks), lv2 = pair_f(lv, lv), iv2 = pair_f(iv, iv);
          // t = q·K·factor·ks + log2 vs + kBase − m, −inf for what a row does not see
          float t[16];
#pragma unroll
          for (int c = 0; c < 16; c += 4) {
            uint64_t f0, f1, r0, r1;
            ld_shared2(factors + c * 4, &f0, &f1);
            ld_shared2(refs_at + c * 4, &r0, &r1);
            split(fma2(mul2(pair(x[c], x[c + 1]), f0), ks2, add2(lv2, r0)), &t[c], &t[c + 1]);
            split(fma2(mul2(pair(x[c + 2], x[c + 3]), f1), ks2, add2(lv2, r1)), &t[c + 2],
                  &t[c + 3]);
          }
          if (edge) {
            int n0, n1;
            visible(a, *pt, slots[(tile_no + j) & (kSlots - 1)].key0 + kt, &n0, &n1);
            const uint32_t seen = low_bits(n1 - c0) & ~low_bits(n0 - c0);
            asm volatile("" ::: "memory");             // (a branch, not selections at every tile)
#pragma unroll
            for (int c = 0; c < 16; ++c) t[c] = seen >> c & 1u ? t[c] : -INFINITY;
          }
          float top = fmaxf(t[0], t[1]);
#pragma unroll
          for (int c = 2; c < 16; c += 2) top = max3(top, t[c], t[c + 1]);
          int grown = top > kBase + kGrow || fresh;
          asm volatile(
              "{\n\t.reg .pred p, q;\n\t"
              "setp.ne.s32 p, %0, 0;\n\t"
              "bar.red.or.pred q, %1, 128, p;\n\t"
              "selp.s32 %0, 1, 0, q;\n\t}"
              : "+r"(grown)
              : "r"(3 + g)
              : "memory");
          uint32_t cols = 0;                           // columns whose reference moves,
          float keep = 1.f;                            // and by how much (lane c: column c)
          if (grown) {
            // the tile's largest t of every column: a reference that it passes follows
            // it, and with it what has been summed up so far
            const int col = lane & 15;
            const float ref_was = ref[col];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float v = warp_max(t[c]);
              if (lane == c) group_stat[quarter * 16 + c] = v;
            }
            group_sync();
            float best = group_stat[col];
#pragma unroll
            for (int w = 1; w < 4; ++w) best = fmaxf(best, group_stat[w * 16 + col]);
            const bool first = fresh >> col & 1u;
            const bool follows = best > (first ? -INFINITY : kBase + kGrow);
            const float by = follows ? best - kBase : 0.f;
            if (quarter == 0 && lane < 16 && follows) ref[col] = ref_was - by;
            if (!first) keep = exp2_approx(-by);
            cols = __ballot_sync(0xffffffffu, follows) & 0xffffu;
            fresh &= ~cols;
#pragma unroll
            for (int c = 0; c < 16; c += 2) {
              if (!(cols >> c & 3u)) continue;
              t[c] -= __shfl_sync(0xffffffffu, by, c);
              t[c + 1] -= __shfl_sync(0xffffffffu, by, c + 1);
              sums[c / 2] = mul2(sums[c / 2], pair_f(__shfl_sync(0xffffffffu, keep, c),
                                                     __shfl_sync(0xffffffffu, keep, c + 1)));
            }
            group_sync();
          }
          // weights, their sum, and their numbers
          uint32_t num[kWeightNum][4];
#pragma unroll
          for (int c = 0; c < 16; c += 4) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = exp2_approx(t[c + e]);
            sums[c / 2] = fma2(pair_f(w[0], w[1]), iv2, sums[c / 2]);
            sums[c / 2 + 1] = fma2(pair_f(w[2], w[3]), iv2, sums[c / 2 + 1]);
            uint32_t v[kWeightNum];
            weight_numbers<kF16>(w[0], w[1], w[2], w[3], ties, v);
#pragma unroll
            for (int i = 0; i < kWeightNum; ++i) num[i][c / 4] = v[i];
          }
          // the product with the weights before them has read those, and added to O
          wait_at(bars + kPDone, k & 1u ^ 1u, 0xB55);
          if (cols && j >= streams) {
            umma::fence_after_sync();
#pragma unroll 1
            for (uint32_t todo = cols; todo; todo &= todo - 1) {
              const int c = __ffs(todo) - 1;
              const float by = __shfl_sync(0xffffffffu, keep, c);
              uint32_t o[kWeightNum];
#pragma unroll
              for (int i = 0; i < kWeightNum; ++i) o[i] = umma::ld_x1(o_addr + i * wide + c);
              umma::wait_ld();
#pragma unroll
              for (int i = 0; i < kWeightNum; ++i)
                umma::st_x1(o_addr + i * wide + c, __float_as_uint(__uint_as_float(o[i]) * by));
            }
            umma::wait_st();
            umma::fence_before_sync();
          }
#pragma unroll
          for (int i = 0; i < kWeightNum; ++i) st_shared4(p_at[i], num[i]);
        } else {
          arrive(bars + kEmpty);
          wait_at(bars + kPDone, k & 1u ^ 1u, 0xB52);
        }
        if (edge) {
          // (the stage's last tile has landed: the products up to the stream's tile
          // before this one are done, and that is less than the ring behind)
          const ValuePlace at(tile_no + j);
          const int stage = kKeyStages + at.stage();
          wait(&m.full[stage], at.parity(), 0xB56);
          if (ok)
            clean_values<kDim>(a, *pt, smem + Z::kOffRing + stage * Z::kTileBytes,
                               slots[(tile_no + j) & (kSlots - 1)].key0, gl, 4 >> shift,
                               p.spoiled + blockIdx.x * 128, &m.spoils);
        }
        fence_proxy_async_smem();
        arrive(bars + kPFull);
      }
      // the sums over keys: 16 columns of 32 lanes, by halves
      {
        float v[16];
#pragma unroll
        for (int c = 0; c < 8; ++c) split(sums[c], &v[2 * c], &v[2 * c + 1]);
#pragma unroll
        for (int half = 8; half > 0; half >>= 1) {
          const bool up = lane & (2 * half);
#pragma unroll
          for (int i = 0; i < half; ++i) {
            const float give = up ? v[i] : v[i + half], stays = up ? v[i + half] : v[i];
            v[i] = stays + __shfl_xor_sync(0xffffffffu, give, 2 * half);
          }
        }
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
        if (!(lane & 1)) group_stat[quarter * 16 + (lane >> 1)] = v[0];
      }
      // (a column that saw no key has no reference)
      if (quarter == 0 && lane < 16 && (fresh >> lane & 1u)) ref[lane] = INFINITY;
      counts = add_counts(counts, n, shift);
      tile_no += n;
      // all scores with these queries are there
      wait_four(m.s_full, counts, 0xB59);
    }
    // The last part is left to the CTA that ends its item, and an item that began
    // in earlier ranges joined, when all of the range's results are there.
    if (!gone && (open || m.start.joins)) {
      all_sync();
      unsigned long long before = 0;                   // (used at the end: it takes a while)
      if (open && threadIdx.x == 128) before = exchange(p.left + blockIdx.x, p.call);
      if (m.start.joins) join_parts<kDim, kF16>(p, m.start, lost);
      if (before == given_up(p.call)) p.left[blockIdx.x] = 0ull;
    }
  }
  umma::fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && m.lost) report_error(a.err, ERR_TIMEOUT, m.lost);
  if (warp == -3) umma::tmem_dealloc(tmem, Z::kCols);
}

template <int kDim, int kNum>
cudaError_t launch_t(Params& p, int ctas, cudaStream_t stream) {
  using Z = Sizes<kDim, kNum>;
  auto* kernel = attend8_kernel<kDim, kNum>;
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
constexpr size_t kSpoiledBytes = kMaxCtas * 128 * sizeof(unsigned long long);

}  // namespace

size_t attend8_workspace_bytes(int head_dim) {
  return kLeftBytes + kSpoiledBytes + 2 * kMaxCtas * slot_floats(head_dim) * sizeof(float);
}

cudaError_t launch_attend8(const Attend8Args& a, int num_sms, cudaStream_t stream) {
  Params p;
  memset(&p, 0, sizeof p);
  p.a = a;
  const moe_kv8_cache& c = a.cache;
  p.page_shift = 31 - __builtin_clz(c.page_size);
  p.blocks_shift = 31 - __builtin_clz(c.page_size / c.block);
  p.tpt = p.block = kRows / a.group;
  char* ws = static_cast<char*>(a.workspace);
  p.left = reinterpret_cast<unsigned long long*>(ws);
  p.spoiled = reinterpret_cast<unsigned long long*>(ws + kLeftBytes);
  p.part = reinterpret_cast<float*>(ws + kLeftBytes + kSpoiledBytes);
  p.call = call_number();
  // [page][row][head][dim]: a box is a head's rows of a page, or 128 of them
  const cuuint64_t dims[4] = {(uint64_t)c.head_dim, (uint64_t)c.n_kv_heads, (uint64_t)c.page_size,
                            (uint64_t)c.n_pages};
  const cuuint64_t strides[3] = {(uint64_t)c.head_stride, (uint64_t)c.token_stride,
                               (uint64_t)c.page_stride};
  const uint32_t box[4] = {(uint32_t)c.head_dim, 1,
                           (uint32_t)(c.page_size < kTile ? c.page_size : kTile), 1};
  const uint32_t steps[4] = {1, 1, 1, 1};
  const EncodeFn encode = encode_fn();
  if (!encode) return cudaErrorNotSupported;
  auto encode_maps = [&] {
    auto map = [&](CUtensorMap* to, const void* at) {
      return encode(to, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(at), dims, strides, box,
                    steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    c.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                    CU_TENSOR_MAP_L2_PROMOTION_NONE,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    return map(&p.kmap, c.k) && map(&p.vmap, c.v);
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
  if (c.head_dim == 128)
    return a.f16 ? launch_t<128, 3>(p, ctas, stream) : launch_t<128, 2>(p, ctas, stream);
  return a.f16 ? launch_t<64, 3>(p, ctas, stream) : launch_t<64, 2>(p, ctas, stream);
}

}  // namespace moe
