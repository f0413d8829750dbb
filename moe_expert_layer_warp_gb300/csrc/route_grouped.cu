// route_grouped.cu — experts from router logits: softmax or sigmoid scores, a
// balance bias, groups, top-k, renormalised weights.
//
// Sources: "Deep Dive into Mixture of Experts: From 1991 to DeepSeek-V3", §5
// (DeepSeek-style routing sketch: scores, a bias that only selects, top-k).
//
// With s_e the score and c_e = s_e + bias_e, the result is a selection by
// comparisons of c (and of sums of two c), and what is asked for is the
// selection of exact arithmetic. fp32 decides almost every comparison: a
// value computed here is off by at most a bound that is known, so a
// difference larger than the two bounds has the right sign. Closer ones (a
// few tokens in ten thousand, with trained routers' spreads) are decided in
// fp64, whose rate is 1/64 of fp32's: by the choices of the few experts in
// question, one in a lane, and only where that does not settle it by all of
// the token's. (Everything in fp64 took 848 us for 20011 tokens of 256
// experts; close tokens whole in fp64, 81 us.) Without a bias, c is monotone
// in the logit, and experts are compared by their logits, exactly.
//
// 20011 tokens of 256 experts in 8 groups (sigmoid, bias, bf16) take 18.8 us;
// the logits alone would take 1.7. What bounds it is issuing a token's
// 790 instructions and waiting for one lane's after another's: scores 5 us,
// groups 4, the (k + 1)-th best 1, candidates and ranks 4, weights 4. A group's
// experts lie in its own lanes, so its sum takes log2(lanes) steps and no
// shared memory (groups across lanes: 28 us). Warps that stay and load the
// next token ahead were slower (22.9 us): the tokens that take fp64 then hold
// up others. 64 tokens take 3.4 us, 9 take 2.6: a launch and one token's chain.
#include <cuda_fp16.h>
#include <limits.h>
#include <math.h>

#include "batch_launch.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
// Blocks of an SM: 64 registers a thread, and what is rare spills. (With 6
// blocks of 80 registers, 20011 tokens took 21.3 us for 19.4.)
constexpr int kPerSm = 8;
constexpr uint32_t kAll = 0xffffffffu;

template <typename T>
MOE_DEV float widen(T v);
template <>
MOE_DEV float widen<float>(float v) { return v; }
template <>
MOE_DEV float widen<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
MOE_DEV float widen<__half>(__half v) { return __half2float(v); }

template <typename T>
MOE_DEV constexpr float lowest();
template <>
MOE_DEV constexpr float lowest<float>() { return -3.402823466e+38f; }
template <>
MOE_DEV constexpr float lowest<__nv_bfloat16>() { return -3.389531389e+38f; }
template <>
MOE_DEV constexpr float lowest<__half>() { return -65504.f; }

// The logit, −inf for a masked expert.
template <typename T>
MOE_DEV float load_logit(const T* p) {
  const float v = widen<T>(*p);
  return v <= lowest<T>() ? -INFINITY : v;
}

// What experts are compared by: kMasked for a masked expert, kAbsent for one
// that is not there or not among the groups kept; every other is above both.
constexpr float kAbsent = -INFINITY;
constexpr float kMasked = -3.402823466e+38f;

MOE_DEV float warp_most(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
MOE_DEV float warp_least(float v) {
  float r;
  asm("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

MOE_DEV double warp_max(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

MOE_DEV double warp_add(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// One token by one warp, everything in fp64: the chosen expert j and its
// weight in lane j. Expert e is in lane e % 32, register e / 32.
struct Chosen {
  int e;
  float w;
};
template <typename T>
__device__ __noinline__ Chosen route_exact(const moe_router_desc& r, const T* row,
                                           const float* bias) {
  constexpr int kPerLane = MOE_MAX_EXPERTS / 32;
  const int lane = threadIdx.x & 31;
  const int E = r.n_experts, size = E / r.n_groups;
  double s[kPerLane], c[kPerLane];
  uint32_t left = 0;  // experts of this lane still to choose from
  float l[kPerLane];
  double top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = lane + 32 * i;
    l[i] = e < E ? load_logit(row + e) : -INFINITY;
    if (e < E) left |= 1u << i;
    top = fmax(top, (double)l[i]);
  }
  if (r.score == MOE_SCORE_SOFTMAX) {
    top = warp_max(top);
    double sum = 0;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      s[i] = l[i] == -INFINITY ? 0.0 : exp((double)l[i] - top);
      sum += s[i];
    }
    sum = warp_add(sum);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) s[i] = sum > 0.0 ? s[i] / sum : 0.0;
  } else {
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      s[i] = l[i] == -INFINITY ? 0.0 : 1.0 / (1.0 + exp(-(double)l[i]));
  }
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = lane + 32 * i;
    c[i] = l[i] == -INFINITY ? -INFINITY : s[i] + (bias ? (double)bias[e] : 0.0);
  }
  // groups of one choice each, and experts, compare by logits if no bias is
  // there: scores may be too small even for fp64
  auto by_logit = [&] {
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) c[i] = l[i];
  };
  if (!bias && r.group_top != 2) by_logit();
  if (r.top_groups < r.n_groups) {
    // lane g ends with group g's score
    double mine = -INFINITY;
    for (int g = 0; g < r.n_groups; ++g) {
      double a = -INFINITY, b = -INFINITY;  // best and second best
#pragma unroll
      for (int i = 0; i < kPerLane; ++i) {
        const int e = lane + 32 * i;
        if (e / size == g && e < E) {
          b = fmax(b, fmin(a, c[i]));
          a = fmax(a, c[i]);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const double a2 = __shfl_xor_sync(kAll, a, o);
        const double b2 = __shfl_xor_sync(kAll, b, o);
        b = fmax(fmax(b, b2), fmin(a, a2));
        a = fmax(a, a2);
      }
      const double score = r.group_top == 2 ? a + b : a;
      if (lane == g) mine = score;
    }
    // a group is kept if fewer than top_groups come before it
    int before = 0;
    for (int g = 0; g < r.n_groups; ++g) {
      const double other = __shfl_sync(kAll, mine, g);
      if (other > mine || (other == mine && g < lane)) ++before;
    }
    const uint32_t kept = __ballot_sync(kAll, lane < r.n_groups && before < r.top_groups);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int e = lane + 32 * i;
      if (e < E && !((kept >> (e / size)) & 1u)) left &= ~(1u << i);
    }
  }
  if (!bias) by_logit();
  int my_e = 0;
  double my_s = 0;
  for (int j = 0; j < r.top_k; ++j) {
    double best = -INFINITY, bs = 0;
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int e = lane + 32 * i;
      if (((left >> i) & 1u) && (be == 0x7fffffff || c[i] > best)) {
        best = c[i];
        be = e;
        bs = s[i];
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double c2 = __shfl_xor_sync(kAll, best, o);
      const double s2 = __shfl_xor_sync(kAll, bs, o);
      const int e2 = __shfl_xor_sync(kAll, be, o);
      const bool swap = e2 != 0x7fffffff &&
                        (be == 0x7fffffff || c2 > best || (c2 == best && e2 < be));
      if (swap) {
        best = c2;
        bs = s2;
        be = e2;
      }
    }
    if (be < E && (be & 31) == lane) left &= ~(1u << (be >> 5));
    if (lane == j) {
      my_e = be < E ? be : 0;
      my_s = bs;
    }
  }
  double w = lane < r.top_k ? my_s : 0.0;
  if (r.renorm) {
    const double sum = warp_add(w);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  return Chosen{my_e, (float)(w * r.scale)};
}

// Order-preserving integer key of a double.
MOE_DEV unsigned long long order_key64(double f) {
  const long long u = __double_as_longlong(f == 0.0 ? 0.0 : f);
  return u < 0 ? ~(unsigned long long)u : (unsigned long long)u | 0x8000000000000000ull;
}

// What fp64 needs of a row for a softmax: its maximum and sum.
struct RowSum {
  double top, sum;
};
template <typename T>
__device__ __noinline__ RowSum row_sum64(const T* row, int E) {
  const int lane = threadIdx.x & 31;
  RowSum q{-INFINITY, 0.0};
  for (int e = lane; e < E; e += 32) q.top = fmax(q.top, (double)load_logit(row + e));
  q.top = warp_max(q.top);
  for (int e = lane; e < E; e += 32) {
    const double l = load_logit(row + e);
    if (l != -INFINITY) q.sum += exp(l - q.top);
  }
  q.sum = warp_add(q.sum);
  return q;
}

// The choice of one expert in fp64 (−inf for a masked one).
__device__ __noinline__ double choice64(float x, float bias, bool sigmoid, RowSum q) {
  if (x == -INFINITY) return -INFINITY;
  return (sigmoid ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - q.top) / q.sum) + (double)bias;
}

// exp of a non-positive or moderate argument by the hardware's base-2
// exponential: x·log2(e) is rounded (|x|·2^-24·1.45 of an exponent step at
// most) and the exponential itself is good to 2^-22, so the result is off by
// at most (|x| + 4)·2^-23 relative to it.
MOE_DEV float exp_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}

MOE_DEV float reciprocal_fast(float x) {  // good to 2^-23
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The descriptor, and what follows from it. Every group (all experts, if none
// is left out) has the same number of lanes, a power of two, and they have its
// experts in order, `per` each; the last ones may have fewer.
struct Router {
  moe_router_desc d;
  int groups, size, per;
  int shift;      // log2 of the lanes of a group
  int whole;      // every lane has kPer experts
  int wide;       // a lane's logits are aligned 16-byte pieces, or it has none
  int wide_bias;  // and its bias is
};

// One warp per token; a lane has kPer experts or fewer, consecutive ones.
template <typename T, int kPer>
__global__ void __launch_bounds__(kWarps * 32, kPerSm)
    route_grouped_kernel(const __grid_constant__ Router p, const T* __restrict__ logits,
                         int64_t row_stride, const float* __restrict__ bias, int n,
                         int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  // what the experts of the warp's token are compared by
  __shared__ alignas(16) float choice[kWarps][32][kPer];
  // the experts that may be among the k; then by rank
  __shared__ alignas(16) float cand_c[kWarps][32];
  __shared__ int cand_e[kWarps][32];
  pdl_wait();
  pdl_trigger();
  const moe_router_desc& r = p.d;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kWarps + warp;
  if (t >= n) return;
  const int E = r.n_experts, k = r.top_k;
  const T* row = logits + t * row_stride;
  const bool sigmoid = r.score == MOE_SCORE_SIGMOID;
  const bool by_logit = bias == nullptr;   // experts compare by their logits
  const bool grouped = p.groups > 1;
  const int share = 1 << p.shift;
  const int g = lane >> p.shift, sub = lane & (share - 1);
  const int first = g * p.size + sub * p.per;
  const int have = g < p.groups ? max(0, min(p.per, p.size - sub * p.per)) : 0;

  float l[kPer];
  if (p.wide) {
    constexpr int kVec = 16 / sizeof(T) < kPer ? 16 / sizeof(T) : kPer;
#pragma unroll
    for (int v = 0; v < kPer; v += kVec) {
      alignas(16) T piece[kVec];
      if constexpr (kVec * sizeof(T) == 16) {
        if (have)
          *reinterpret_cast<uint4*>(piece) = __ldg(reinterpret_cast<const uint4*>(row + first + v));
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) l[v + i] = have ? widen<T>(piece[i]) : -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) l[i] = i < have ? widen<T>(row[first + i]) : -INFINITY;
  }

  // softmax: the row's maximum and sum, for the choices and the weights
  float top = 0.f, inv = 1.f;
  if (!sigmoid) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) m = fmaxf(m, l[i]);
    top = warp_most(m);
    if (top <= lowest<T>()) top = 0.f;     // every expert masked: scores 0
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += l[i] <= lowest<T>() ? 0.f : expf(l[i] - top);
    sum = warp_sum(sum);
    inv = sum > 0.f ? 1.f / sum : 0.f;
  }

  // what experts, and groups, are compared by
  const bool sums = grouped && r.group_top == 2;
  float c[kPer];
  auto store_choices = [&] {
#pragma unroll
    for (int i = 0; i < kPer; i += kPer < 4 ? 2 : 4) {
      if constexpr (kPer < 4)
        *reinterpret_cast<float2*>(&choice[warp][lane][i]) = make_float2(c[i], c[i + 1]);
      else
        *reinterpret_cast<float4*>(&choice[warp][lane][i]) =
            make_float4(c[i], c[i + 1], c[i + 2], c[i + 3]);
    }
  };
  auto take_logits = [&] {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      c[i] = i >= have ? kAbsent : l[i] <= lowest<T>() ? kMasked : l[i];
  };
  if (!by_logit || sums) {
    if (sigmoid) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) c[i] = reciprocal_fast(1.f + exp_fast(-l[i]));
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) c[i] = exp_fast(l[i] - top) * inv;
    }
    if (!by_logit) {
      float b[kPer];
      if (p.wide_bias) {
        if constexpr (kPer >= 4) {
#pragma unroll
          for (int i = 0; i < kPer; i += 4) {
            const float4 f = have ? __ldg(reinterpret_cast<const float4*>(bias + first + i))
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            b[i] = f.x;
            b[i + 1] = f.y;
            b[i + 2] = f.z;
            b[i + 3] = f.w;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) b[i] = i < have ? __ldg(bias + first + i) : 0.f;
      }
      // (a finite bias may be as low as kMasked)
#pragma unroll
      for (int i = 0; i < kPer; ++i) c[i] = fmaxf(c[i] + b[i], -0x1.fffffcp127f);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) c[i] = l[i] <= lowest<T>() ? kMasked : c[i];
    if (!p.whole) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) c[i] = i < have ? c[i] : kAbsent;
    }
  } else {
    take_logits();
  }
  store_choices();

  bool unsure = false;
  if (grouped) {
    const int G = p.groups;
    float a = c[0], b = kAbsent;           // best and second best
#pragma unroll
    for (int i = 1; i < kPer; ++i) {
      b = fmaxf(b, fminf(a, c[i]));
      a = fmaxf(a, c[i]);
    }
    for (int o = 1; o < share; o <<= 1) {
      const float a2 = __shfl_xor_sync(kAll, a, o), b2 = __shfl_xor_sync(kAll, b, o);
      b = fmaxf(fmaxf(b, b2), fminf(a, a2));
      a = fmaxf(a, a2);
    }
    a = a > kMasked ? a : -INFINITY;
    b = b > kMasked ? b : -INFINITY;
    const float mine = r.group_top == 2 ? a + b : a;
    // how many groups come before this one: its lanes share the others
    int before = 0;
    for (int o = sub; o - sub < G; o += share) {
      const float other = __shfl_sync(kAll, mine, o << p.shift);
      before += o < G && (other > mine || (other == mine && o < g));
    }
    for (int o = 1; o < share; o <<= 1) before += __shfl_xor_sync(kAll, before, o);
    bool keep = g < G && before < r.top_groups;
    // Group sums compare only by a margin. A score is off by less than
    // 2^-19.4: s·|x| ≤ 0.37 for a softmax's x = l − top, s·(1 − s)·|x| ≤ 0.28
    // for a sigmoid, and the rest is relative to s ≤ 1; four scores make
    // 2^-17.4, and one group's two 2^-18.4. Roundings of c and of the sums go
    // by |a| + |b|.
    if (!by_logit || r.group_top == 2) {
      const float size_ab = (a == -INFINITY ? 0.f : fabsf(a)) + (b == -INFINITY ? 0.f : fabsf(b));
      const float margin = 0x1p-18f + size_ab * 0x1p-22f;
      const float worst_kept = warp_least(keep ? mine - margin : INFINITY);
      const float best_left = warp_most(g < G && !keep ? mine + margin : -INFINITY);
      if (worst_kept != -INFINITY && !(worst_kept > best_left)) {
        // the groups' sums in fp64, a group in a lane: its two best choices,
        // if they are its two best for certain
        float c1 = kMasked, c2 = kMasked, c3 = kMasked;
        int e1 = 0, e2 = 0;
        __syncwarp();
        if (lane < G) {
          for (int i = 0, from = lane * share, at = 0; i < p.size; ++i, ++at) {
            if (at == p.per) {
              ++from;
              at = 0;
            }
            const float o = choice[warp][from][at];
            const int e = lane * p.size + i;
            if (o > c1) {
              c3 = c2;
              c2 = c1;
              e2 = e1;
              c1 = o;
              e1 = e;
            } else if (o > c2) {
              c3 = c2;
              c2 = o;
              e2 = e;
            } else {
              c3 = fmaxf(c3, o);
            }
          }
        }
        const float next = r.group_top == 2 ? c3 : c2, last = r.group_top == 2 ? c2 : c1;
        const float apart = 0x1p-17f + warp_most(size_ab) * 0x1p-21f;
        unsure |= __any_sync(kAll, next != kMasked && !(last - next > apart));
        const RowSum q = sigmoid ? RowSum{0.0, 0.0} : row_sum64(row, E);
        double sum = -INFINITY;
        if (c1 != kMasked) {
          sum = choice64(load_logit(row + e1), bias ? bias[e1] : 0.f, sigmoid, q);
          if (r.group_top == 2)
            sum = c2 == kMasked ? -INFINITY
                                : sum + choice64(load_logit(row + e2), bias ? bias[e2] : 0.f,
                                                 sigmoid, q);
        }
        const unsigned long long mine64 = order_key64(sum);
        int rank = 0;
        for (int o = 0; o < G; ++o) {
          const unsigned long long other = __shfl_sync(kAll, mine64, o);
          if (other > mine64 || (other == mine64 && o < lane)) ++rank;
        }
        const uint32_t kept64 = __ballot_sync(kAll, lane < G && rank < r.top_groups);
        keep = g < G && ((kept64 >> g) & 1u);
      }
    }
    if (by_logit && sums) {                // the groups' by their scores: now the experts'
      take_logits();
      __syncwarp();
      store_choices();
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) c[i] = keep ? c[i] : kAbsent;
  }

  // At least k + 1 experts are no worse than the (k + 1)-th best of the lanes'
  // best ones, and few more: they go one to a lane and are ranked against
  // each other. Beside a bias, those that lie below it by no more than the
  // choices may be off come along.
  auto best_of_lane = [&] {
    float m = c[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) m = fmaxf(m, c[i]);
    return m;
  };
  float best = best_of_lane(), least = kAbsent;
  if (__popc(__ballot_sync(kAll, best != kAbsent)) > k) {
    for (int j = 0; j <= k; ++j) {
      least = warp_most(best);
      if (best == least) best = kAbsent;
    }
  } else {  // experts left in k lanes or fewer: a lane's next best takes its turn
    for (int j = 0; j <= k; ++j) {
      least = warp_most(best);
      if (best == least) {
        best = kAbsent;
#pragma unroll
        for (int i = 0; i < kPer; ++i) best = fmaxf(best, c[i] < least ? c[i] : kAbsent);
      }
    }
  }
  // what a choice near `least` may be off by: see bound() below
  if (!by_logit && least > kMasked)
    least -= 2.f * ((sigmoid ? 0x1p-20f : 0x1p-18f) + fabsf(least) * 0x1p-22f);
  least = fmaxf(least, kMasked);
  uint32_t in = 0;                         // this lane's, a bit each
#pragma unroll
  for (int i = 0; i < kPer; ++i) in |= c[i] >= least ? 1u << i : 0u;
  cand_c[warp][lane] = kAbsent;
  __syncwarp();
  int count = 0;
  for (uint32_t who; (who = __ballot_sync(kAll, in != 0)) != 0;) {
    const int at = count + __popc(who & ((1u << lane) - 1u));
    if (in) {
      const int i = __ffs(in) - 1;
      if (at < 32) {
        cand_c[warp][at] = choice[warp][lane][i];
        cand_e[warp][at] = first + i;
      }
      in &= in - 1;
    }
    count += __popc(who);
  }
  const bool crowd = count > 32;
  // what the bounds of two choices (see bound() below) never exceed together
  auto bounds_most = [&](float c1, float c2) {
    return (sigmoid ? 0x1p-19f : 0x1p-17f) + (fabsf(c1) + fabsf(c2)) * 0x1p-23f;
  };
  __syncwarp();
  float my_c = kAbsent;
  int my_e = 0;
  if (!crowd) {
    if (lane < count) {
      my_c = cand_c[warp][lane];
      my_e = cand_e[warp][lane];
    }
    int rank = 0;
    for (int o = 0; o < count; o += 4) {   // (none is below those past `count`)
      const float4 other = *reinterpret_cast<const float4*>(&cand_c[warp][o]);
      rank += (other.x > my_c) + (other.y > my_c) + (other.z > my_c) + (other.w > my_c);
    }
    if (__popc(__reduce_or_sync(kAll, lane < count ? 1u << rank : 0u)) != count) {
      // equal ones: the lower expert's first
      for (int o = 0; o < count; ++o)
        rank += cand_c[warp][o] == my_c && cand_e[warp][o] < my_e;
    }
    __syncwarp();
    if (lane < count) {
      cand_c[warp][rank] = my_c;
      cand_e[warp][rank] = my_e;
    }
  } else {
    // many equal ones: the largest left k + 1 times, of equal ones the lowest
    // expert's, which is in the lowest lane
    count = k + 1;
    for (int j = 0; j <= k; ++j) {
      const float mine = best_of_lane(), most = warp_most(mine);
      const int from = __ffs(__ballot_sync(kAll, mine == most)) - 1;
      if (lane == from) {
        int at = 0;
#pragma unroll
        for (int i = kPer - 1; i >= 0; --i)
          if (c[i] == most) at = i;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (i == at) c[i] = kAbsent;
        cand_c[warp][j] = most;
        cand_e[warp][j] = first + at;
      }
    }
    if (!by_logit) {
      // those left must lie below the k-th by what no bound exceeds, or equal
      // it in logit and bias (and come after it)
      __syncwarp();
      const float c_k = cand_c[warp][k - 1];
      const float x_k = load_logit(row + cand_e[warp][k - 1]);
      const float b_k = __ldg(bias + cand_e[warp][k - 1]);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (c[i] > kMasked && !(c_k - c[i] > bounds_most(c_k, c[i])) &&
            !(load_logit(row + first + i) == x_k && __ldg(bias + first + i) == b_k))
          unsure = true;
    }
  }
  __syncwarp();
  // rank j's expert in lane j
  my_c = lane < count ? cand_c[warp][lane] : kAbsent;
  my_e = lane < count ? cand_e[warp][lane] : 0;

  // the chosen experts' scores, accurately
  auto score_of = [&](float x) {
    return x == -INFINITY ? 0.f
           : sigmoid      ? reciprocal_fast(1.f + expf(-x))
                          : expf(x - top) * inv;
  };
  float x = lane < count ? load_logit(row + my_e) : -INFINITY;
  float s = score_of(x);
  if (!by_logit) {
    // Neighbours in the order of the k must differ by more than their bounds — for
    // a sigmoid s·((1 − s)·(|x|·2^-23.4 + 2^-22) + 2^-22), (1 − s)·|x| ≤ 0.28
    // for x > 0; for a softmax s·(|x|·2^-23.4 + 2^-19.4) — or be equal in
    // logit and bias: then the index decides, here as exactly. So must the last
    // of the k and every other candidate, not the next one alone: a large score
    // beside a negative bias has a larger bound than those before it. Most
    // tokens' do by what no bound exceeds.
    const float c2 = __shfl_down_sync(kAll, my_c, 1);
    const bool next = lane < k && lane + 1 < count && c2 > kMasked;
    if (__any_sync(kAll, next && !(my_c - c2 > bounds_most(my_c, c2)))) {
      auto bound = [&](float v_s, float v_x, float v_c) {
        return (sigmoid ? v_s * 0x1.6ap-21f + fmaxf(-v_x, 0.f) * v_s * 0x1p-23f
                        : v_s * (fabsf(v_x - top) * 0x1p-23f + 0x1p-19f)) +
               fabsf(v_c) * 0x1p-23f;
      };
      const float b = lane < count ? __ldg(bias + my_e) : 0.f;
      const float off = lane < count && x != -INFINITY ? bound(s, x, my_c) : 0.f;
      // the one before: of a candidate behind the k, the last of the k
      const int ahead = lane < k ? max(lane - 1, 0) : k - 1;
      const float c1 = __shfl_sync(kAll, my_c, ahead), off1 = __shfl_sync(kAll, off, ahead);
      const float x1 = __shfl_sync(kAll, x, ahead), b1 = __shfl_sync(kAll, b, ahead);
      const bool close = lane > 0 && lane < count && my_c > kMasked &&
                         !(c1 - my_c > off1 + off) && !(x1 == x && b1 == b);
      if (!__any_sync(kAll, close)) {
      } else if (crowd) {
        unsure = true;                     // others may be as close
      } else {                             // all candidates by fp64
        const RowSum q = sigmoid ? RowSum{0.0, 0.0} : row_sum64(row, E);
        const unsigned long long mine64 =
            lane < count ? order_key64(choice64(x, b, sigmoid, q)) : 0ull;
        int rank = 0;
        for (int o = 0; o < count; ++o) {
          const unsigned long long other = __shfl_sync(kAll, mine64, o);
          const int e_o = __shfl_sync(kAll, my_e, o);
          rank += other > mine64 || (other == mine64 && e_o < my_e);
        }
        __syncwarp();
        if (lane < count) cand_e[warp][rank] = my_e;
        __syncwarp();
        my_e = cand_e[warp][lane < count ? lane : 0];
        x = lane < count ? load_logit(row + my_e) : -INFINITY;
        s = score_of(x);
      }
    }
  }
  // scores that fp32 cannot hold, of which quotients are wanted
  if (r.renorm && lane < k && x != -INFINITY && s < 0x1p-100f) unsure = true;
  float w;
  if (__any_sync(kAll, unsure)) {
    const Chosen exact = route_exact<T>(r, row, bias);
    my_e = exact.e;
    w = exact.w;
  } else {
    w = lane < k ? s : 0.f;
    if (r.renorm) {
      const float sum = warp_sum(w);
      w = sum > 0.f ? __fdividef(w, sum) : 0.f;  // 2^-100 < sum ≤ 16: good to two steps
    }
    w *= r.scale;
  }
  if (lane < k) {
    topk_idx[(size_t)t * k + lane] = my_e;
    topk_w[(size_t)t * k + lane] = w;
  }
}

template <typename T, int kPer>
cudaError_t launch_t(Router p, const T* logits, int64_t row_stride, const float* bias, int n,
                     int32_t* topk_idx, float* topk_w, cudaStream_t stream) {
  const bool pieces = p.per == kPer && p.size % kPer == 0;  // a lane has kPer experts or none
  p.whole = pieces && p.groups * p.size == 32 * kPer;
  p.wide = pieces && kPer * sizeof(T) % 16 == 0 && row_stride * sizeof(T) % 16 == 0 &&
           (reinterpret_cast<uintptr_t>(logits) & 15u) == 0;
  p.wide_bias = pieces && kPer >= 4 && (reinterpret_cast<uintptr_t>(bias) & 15u) == 0;
  return launch_pdl(route_grouped_kernel<T, kPer>, dim3((n - 1) / kWarps + 1), dim3(kWarps * 32), 0,
                    stream, p, logits, row_stride, bias, n, topk_idx, topk_w);
}

template <typename T>
cudaError_t launch_e(const moe_router_desc& r, const void* logits, int64_t row_stride,
                     const float* bias, int n, int32_t* topk_idx, float* topk_w,
                     cudaStream_t stream) {
  const T* l = static_cast<const T*>(logits);
  Router p;
  p.d = r;
  p.groups = r.top_groups < r.n_groups ? r.n_groups : 1;
  p.size = r.n_experts / p.groups;
  p.shift = 0;
  while ((2 << p.shift) * p.groups <= 32) ++p.shift;
  p.per = ((p.size - 1) >> p.shift) + 1;   // 16 at most: more than 16 / groups lanes a group
  if (p.per <= 2) return launch_t<T, 2>(p, l, row_stride, bias, n, topk_idx, topk_w, stream);
  if (p.per <= 4) return launch_t<T, 4>(p, l, row_stride, bias, n, topk_idx, topk_w, stream);
  if (p.per <= 8) return launch_t<T, 8>(p, l, row_stride, bias, n, topk_idx, topk_w, stream);
  return launch_t<T, 16>(p, l, row_stride, bias, n, topk_idx, topk_w, stream);
}

}  // namespace

cudaError_t launch_route_grouped(const moe_router_desc& r, const void* logits, int dtype,
                                 int64_t row_stride, const float* bias, int n, int32_t* topk_idx,
                                 float* topk_w, cudaStream_t stream) {
  switch (dtype) {
    case MOE_F32:
      return launch_e<float>(r, logits, row_stride, bias, n, topk_idx, topk_w, stream);
    case MOE_BF16:
      return launch_e<__nv_bfloat16>(r, logits, row_stride, bias, n, topk_idx, topk_w, stream);
    default:
      return launch_e<__half>(r, logits, row_stride, bias, n, topk_idx, topk_w, stream);
  }
}

}  // namespace moe
