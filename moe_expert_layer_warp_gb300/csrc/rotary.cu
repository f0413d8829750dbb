// rotary.cu — rotary positions of a step's queries and keys: pair (a, b) of a
// token at position p becomes amplitude · (a cos θ − b sin θ, a sin θ + b cos θ)
// with θ = p · f_i.
//
// The angle. In turns, θ is the fraction of p · f_i / 2π: frequencies are
// given as multiples of 2^-64 turns, so the 64-bit product with the position
// drops whole turns by itself and is exact, however far the position is. Its
// nearest quarter turn is taken off, which leaves at most an eighth, and that
// in fp32 goes to sincospif: an angle is off by 2^-28 turns at most. (In fp32, a
// position of 900000 at one radian a position would leave 2^-5 radians.)
//
// Bound by memory: every element is read and written once. The sines and cosines of
// a CTA's tokens are worked out once for all their heads, into shared memory; then
// every thread takes 16 bytes of one half of a head's pairs and the matching 16 of
// the other (or 16 bytes of interleaved pairs, or of columns that are copied), 64
// bytes in flight at a time: with 16 of interleaved pairs, and a CTA's tokens one
// after the other, the call below took 115 us and more. 12345 tokens of 64 heads of
// 128 bf16 columns, 64 of them turned (405 MB): 71 us, 5.7 TB/s, 86 % of a copy's
// rate. 36 tokens of 40 heads: 2 us beyond an empty launch.
#include <type_traits>

#include "batch_launch.h"
#include "common.cuh"
#include "kv8_launch.h"
#include "round16.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 512;   // of a head
constexpr int kMaxTokens = 16;   // of a CTA

enum { kF32 = 0, kBf16 = 1, kFp16 = 2 };

template <int kType>
struct Chunk {                   // 16 bytes of a row
  static constexpr int kN = kType == kF32 ? 4 : 8;
  using T = std::conditional_t<kType == kF32, float, uint16_t>;
  uint4 w;
  MOE_DEV void load(const void* base, int64_t at) {
    w = *reinterpret_cast<const uint4*>(static_cast<const T*>(base) + at);
  }
  MOE_DEV void store(void* base, int64_t at) const {
    *reinterpret_cast<uint4*>(static_cast<T*>(base) + at) = w;
  }
  MOE_DEV void get(float (&v)[kN]) const {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kType == kF32) {
        v[i] = __uint_as_float(x[i]);
      } else if constexpr (kType == kBf16) {
        v[2 * i] = bf16lo(x[i]);
        v[2 * i + 1] = bf16hi(x[i]);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
  MOE_DEV void set(const float (&v)[kN]) {
    if constexpr (kType == kF32) {
      w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                     __float_as_uint(v[3]));
    } else {
      constexpr bool f16 = kType == kFp16;
      w = make_uint4(round16<f16>(v[0], v[1]), round16<f16>(v[2], v[3]), round16<f16>(v[4], v[5]),
                     round16<f16>(v[6], v[7]));
    }
  }
};

// amplitude · (cos, sin) of position · turn.
MOE_DEV float2 turn_of(int position, uint64_t turn, float amplitude) {
  const uint64_t x = (uint64_t)position * turn;
  const uint64_t quarter = (x + (1ull << 61)) >> 62;
  const int64_t rest = (int64_t)(x - (quarter << 62));          // within ±2^61
  float s, c;
  sincospif((float)(rest >> 29) * 0x1p-34f, &s, &c);            // half turns
  s *= amplitude;
  c *= amplitude;
  switch (quarter & 3) {
    case 0: return make_float2(c, s);
    case 1: return make_float2(-s, c);
    case 2: return make_float2(-c, -s);
    default: return make_float2(s, -c);
  }
}

// What a CTA turns: its tokens, and for queries and keys how their pieces are
// counted. by_…: what quotient() takes for the divisor per_….
struct Pieces {
  int per_head, per_token;
  uint32_t by_head, by_token;
};
struct Split {
  int tokens;
  Pieces of[2];
};

// a / d with by = ceil(2^32 / d), 0 for d = 1, exact while a · d < 2^32.
MOE_DEV int quotient(int a, uint32_t by) { return by ? __umulhi(a, by) : a; }

template <int kType, bool kInterleaved>
__global__ void __launch_bounds__(kThreads)
    rotary_kernel(const __grid_constant__ RotaryArgs a, const __grid_constant__ Split split) {
  constexpr int kN = Chunk<kType>::kN;
  constexpr int kAhead = kInterleaved ? 4 : 2;   // pieces that a thread has in flight
  __shared__ float2 table[kMaxPairs];            // [tokens][pairs]
  __shared__ int position[kMaxTokens];
  const moe_rotary_desc& d = a.desc;
  const int pairs = d.n_rotated / 2;
  pdl_wait();
  pdl_trigger();
  const int t0 = blockIdx.x * split.tokens, tokens = min(split.tokens, a.n_tokens - t0);
  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int t = i / pairs, p = a.positions[t0 + t], pair = i - t * pairs;
    if (pair == 0) position[t] = p;
    table[i] = turn_of(max(p, 0), d.turns[pair], d.amplitude);
  }
  __syncthreads();
  // a head's rotated pieces come first, then the columns that are copied
  const int turned = kInterleaved ? d.n_rotated / kN : pairs / kN;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const moe_rotary_rows& r = a.rows[which];
    const Pieces& n = split.of[which];
    const bool moves = r.in != r.out;
    const int total = tokens * n.per_token;
    for (int i0 = threadIdx.x; i0 < total; i0 += kAhead * kThreads) {
      Chunk<kType> x[kAhead], y[kAhead];
      int64_t to[kAhead];
      const float2* cs[kAhead];                  // null: a copy
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kThreads;
        if (i >= total) break;
        const int t = quotient(i, n.by_token), k = i - t * n.per_token;
        const int h = quotient(k, n.by_head), j = k - h * n.per_head;
        const int64_t from = (t0 + t) * r.in_token_stride + h * r.in_head_stride;
        int at = d.first + j * kN;
        if (j >= turned) {
          at = (j - turned) * kN;
          at += at < d.first ? 0 : d.n_rotated;
        }
        const bool turns = j < turned && position[t] >= 0;
        cs[u] = turns ? table + t * pairs + j * (kInterleaved ? kN / 2 : kN) : nullptr;
        to[u] = (t0 + t) * r.out_token_stride + h * r.out_head_stride + at;
        x[u].load(r.in, from + at);
        if (!kInterleaved && j < turned) y[u].load(r.in, from + at + pairs);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kThreads;
        if (i >= total) break;
        if (cs[u] == nullptr) {
          if (!moves) continue;
          x[u].store(r.out, to[u]);
          if constexpr (!kInterleaved) {         // a row without a position
            const int k = i - quotient(i, n.by_token) * n.per_token;
            if (k - quotient(k, n.by_head) * n.per_head < turned) y[u].store(r.out, to[u] + pairs);
          }
          continue;
        }
        float v[kN];
        x[u].get(v);
        if constexpr (kInterleaved) {
#pragma unroll
          for (int e = 0; e < kN; e += 2) {
            const float2 w = cs[u][e / 2];
            const float b = v[e];
            v[e] = b * w.x - v[e + 1] * w.y;
            v[e + 1] = b * w.y + v[e + 1] * w.x;
          }
        } else {
          float z[kN];
          y[u].get(z);
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            const float2 w = cs[u][e];
            const float b = v[e];
            v[e] = b * w.x - z[e] * w.y;
            z[e] = b * w.y + z[e] * w.x;
          }
          y[u].set(z);
          y[u].store(r.out, to[u] + pairs);
        }
        x[u].set(v);
        x[u].store(r.out, to[u]);
      }
    }
  }
}

uint32_t divisor(int d) { return (uint32_t)(((1ull << 32) + d - 1) / d); }

template <int kType>
auto kernel_of(bool interleaved) {
  return interleaved ? rotary_kernel<kType, true> : rotary_kernel<kType, false>;
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int dtype, int num_sms, cudaStream_t stream) {
  const moe_rotary_desc& d = a.desc;
  const int n = dtype == MOE_F32 ? 4 : 8;
  Split s = {};
  int64_t most = 1;                  // pieces of a token
  for (int w = 0; w < 2; ++w) {
    const moe_rotary_rows& r = a.rows[w];
    Pieces& p = s.of[w];
    p.per_head = (d.interleaved ? d.n_rotated : d.n_rotated / 2) / n +
                 (r.in != r.out ? (d.head_dim - d.n_rotated) / n : 0);
    p.per_token = r.n_heads * p.per_head;
    p.by_head = divisor(p.per_head);
    if (p.per_token > most) most = p.per_token;
  }
  // An angle for every thread, while that leaves every SM two CTAs. (Of a call with
  // the replay that measures it, 7 us: one token a CTA takes 73 us for 12345 tokens
  // of 40 heads and 44 for 17 short ones, this 54 and 20; 36 tokens take 9.3 us one
  // to a CTA, 11.4 four. Two thousand tokens: 18.5 with four CTAs to an SM, 15.5
  // with two.)
  int per = 2 * kThreads / d.n_rotated;
  if (per > kMaxTokens) per = kMaxTokens;
  if (per > a.n_tokens / (num_sms * 2)) per = a.n_tokens / (num_sms * 2);
  if (per < 1 || per * most * most >> 32) per = 1;
  s.tokens = per;
  for (Pieces& p : s.of)             // (1: the quotient is 0, as one token's index is)
    p.by_token = per > 1 && p.per_token > 0 ? divisor(p.per_token) : 1;
  const dim3 grid((a.n_tokens - 1) / per + 1);
  auto* kernel = dtype == MOE_F32    ? kernel_of<kF32>(d.interleaved)
                 : dtype == MOE_BF16 ? kernel_of<kBf16>(d.interleaved)
                                     : kernel_of<kFp16>(d.interleaved);
  return launch_pdl(kernel, grid, dim3(kThreads), 0, stream, a, s);
}

}  // namespace moe
