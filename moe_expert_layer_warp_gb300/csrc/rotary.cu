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
// Bound by memory: every element is read and written once. A token's sines and
// cosines, n_rotated / 2 pairs, are worked out once for all its heads, into
// shared memory; then every thread takes 16 bytes of one half of a head's pairs
// and the matching 16 of the other (or 16 bytes of interleaved pairs).
#include "batch_launch.h"
#include "common.cuh"
#include "kv8_launch.h"
#include "round16.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 512;   // of a head

enum { kF32 = 0, kBf16 = 1, kFp16 = 2 };

template <int kType>
struct Chunk {                   // 16 bytes of a row, in fp32
  static constexpr int kN = kType == kF32 ? 4 : 8;
  float v[kN];
  MOE_DEV void load(const void* base, int64_t at) {
    if constexpr (kType == kF32) {
      const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
      const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (kType == kBf16) {
          v[2 * i] = bf16lo(w[i]);
          v[2 * i + 1] = bf16hi(w[i]);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
          v[2 * i] = f.x;
          v[2 * i + 1] = f.y;
        }
      }
    }
  }
  MOE_DEV void store(void* base, int64_t at) const {
    if constexpr (kType == kF32) {
      *reinterpret_cast<float4*>(static_cast<float*>(base) + at) =
          make_float4(v[0], v[1], v[2], v[3]);
    } else {
      constexpr bool f16 = kType == kFp16;
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) =
          make_uint4(round16<f16>(v[0], v[1]), round16<f16>(v[2], v[3]), round16<f16>(v[4], v[5]),
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

template <int kType>
__global__ void __launch_bounds__(kThreads)
    rotary_kernel(const __grid_constant__ RotaryArgs a, int tokens_per_cta) {
  constexpr int kN = Chunk<kType>::kN;
  __shared__ float2 table[kMaxPairs];
  const moe_rotary_desc& d = a.desc;
  const int pairs = d.n_rotated / 2;
  pdl_wait();
  pdl_trigger();
  const int t0 = blockIdx.x * tokens_per_cta, t1 = min(t0 + tokens_per_cta, a.n_tokens);
  // a head's pieces: of its rotated columns, and of the others
  const int turned = d.interleaved ? d.n_rotated / kN : pairs / kN;
  const int rest = (d.head_dim - d.n_rotated) / kN;
  for (int t = t0; t < t1; ++t) {
    const int p = a.positions[t];
    if (p >= 0) {
      for (int i = threadIdx.x; i < pairs; i += kThreads)
        table[i] = turn_of(p, d.turns[i], d.amplitude);
    }
    __syncthreads();
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const moe_rotary_rows& r = a.rows[which];
      const bool moves = r.in != r.out;
      const int per_head = turned + (moves ? rest : 0);
      const int n = p < 0 && !moves ? 0 : r.n_heads * per_head;
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const int h = i / per_head, j = i - h * per_head;
        const int64_t from = t * r.in_token_stride + h * r.in_head_stride;
        const int64_t to = t * r.out_token_stride + h * r.out_head_stride;
        Chunk<kType> x, y;
        if (j >= turned) {                                      // a copy
          const int c = (j - turned) * kN, at = c < d.first ? c : c + d.n_rotated;
          x.load(r.in, from + at);
          x.store(r.out, to + at);
        } else if (d.interleaved) {
          const int at = d.first + j * kN;
          x.load(r.in, from + at);
          if (p >= 0) {
#pragma unroll
            for (int e = 0; e < kN; e += 2) {
              const float2 cs = table[(j * kN + e) / 2];
              y.v[e] = x.v[e] * cs.x - x.v[e + 1] * cs.y;
              y.v[e + 1] = x.v[e] * cs.y + x.v[e + 1] * cs.x;
            }
            x = y;
          }
          x.store(r.out, to + at);
        } else {
          const int at = d.first + j * kN;
          x.load(r.in, from + at);
          y.load(r.in, from + at + pairs);
          if (p >= 0) {
#pragma unroll
            for (int e = 0; e < kN; ++e) {
              const float2 cs = table[j * kN + e];
              const float u = x.v[e];
              x.v[e] = u * cs.x - y.v[e] * cs.y;
              y.v[e] = u * cs.y + y.v[e] * cs.x;
            }
          }
          x.store(r.out, to + at);
          y.store(r.out, to + at + pairs);
        }
      }
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int dtype, int num_sms, cudaStream_t stream) {
  // tokens one after the other while that leaves every SM eight CTAs
  int per = a.n_tokens / (num_sms * 8);
  if (per < 1) per = 1;
  const dim3 grid((a.n_tokens - 1) / per + 1);
  auto* kernel = dtype == MOE_F32    ? rotary_kernel<kF32>
                 : dtype == MOE_BF16 ? rotary_kernel<kBf16>
                                     : rotary_kernel<kFp16>;
  return launch_pdl(kernel, grid, dim3(kThreads), 0, stream, a, per);
}

}  // namespace moe
