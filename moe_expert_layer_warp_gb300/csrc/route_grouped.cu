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
#include <limits.h>
#include <math.h>

#include "batch_launch.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
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

// Order-preserving integer keys of floats (−0 and +0 have one key); kNone is
// below every float's key.
constexpr int kNone = INT_MIN;
MOE_DEV int order_key(float f) {
  const int u = __float_as_int(f + 0.f);
  return u ^ ((u >> 31) & 0x7fffffff);
}
MOE_DEV float key_value(int key) { return __int_as_float(key ^ ((key >> 31) & 0x7fffffff)); }

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
template <typename T>
__device__ __noinline__ void route_exact(const moe_router_desc& r, const T* row,
                                         const float* bias, int* expert, float* weight) {
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
  *expert = my_e;
  *weight = (float)(w * r.scale);
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

// The descriptor, and what follows from it.
struct Router {
  moe_router_desc d;
  int size;         // experts of a group
  int to_group;     // e / size = e·to_group >> 16, for e < 256
  int share_shift;  // log2 of the lanes that look through one group
  int wide;         // rows are whole, aligned 16-byte pieces
};

// One warp per token; lane holds kPer consecutive experts.
template <typename T, int kPer>
__global__ void __launch_bounds__(kWarps * 32)
    route_grouped_kernel(const __grid_constant__ Router p, const T* __restrict__ logits,
                         int64_t row_stride, const float* __restrict__ bias, int n,
                         int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  // choices of the warp's token, one float of padding after every 32
  __shared__ float choice[kWarps][32 * kPer + kPer];
  // the experts that may be among the k, with their keys; then by rank
  __shared__ int2 cand[kWarps][32];
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
  const bool grouped = r.top_groups < r.n_groups;

  float l[kPer];
  if (p.wide) {
    constexpr int kVec = 16 / sizeof(T) < kPer ? 16 / sizeof(T) : kPer;
#pragma unroll
    for (int v = 0; v < kPer; v += kVec) {
      alignas(16) T piece[kVec];
      if (lane * kPer + v < E) {
        if constexpr (kVec * sizeof(T) == 16) {
          *reinterpret_cast<uint4*>(piece) =
              __ldg(reinterpret_cast<const uint4*>(row + lane * kPer + v));
        } else {
#pragma unroll
          for (int i = 0; i < kVec; ++i) piece[i] = row[lane * kPer + v + i];
        }
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const float x = lane * kPer + v < E ? widen<T>(piece[i]) : -INFINITY;
        l[v + i] = x <= lowest<T>() ? -INFINITY : x;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      l[i] = lane * kPer + i < E ? load_logit(row + lane * kPer + i) : -INFINITY;
  }

  // softmax: the row's maximum and sum, for the choices and the weights
  float top = 0.f, inv = 1.f;
  if (!sigmoid) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) m = fmaxf(m, l[i]);
    top = key_value(__reduce_max_sync(kAll, order_key(m)));
    if (top == -INFINITY) top = 0.f;       // every expert masked: scores 0
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += expf(l[i] - top);
    sum = warp_sum(sum);
    inv = sum > 0.f ? 1.f / sum : 0.f;
  }

  // what experts are compared by, as keys
  int key[kPer];
  bool unsure = false;
  if (by_logit) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = lane * kPer + i < E ? order_key(l[i]) : kNone;
  }
  if (!by_logit || (grouped && r.group_top == 2)) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane * kPer + i;
      const float s =
          sigmoid ? reciprocal_fast(1.f + exp_fast(-l[i])) : exp_fast(l[i] - top) * inv;
      float c = -INFINITY;
      if (e < E && l[i] != -INFINITY) c = by_logit ? s : s + __ldg(bias + e);
      if (!by_logit) key[i] = e < E ? order_key(c) : kNone;
      if (grouped) choice[warp][e + (e >> 5)] = c;
    }
  } else if (grouped) {                    // groups by their largest logit
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane * kPer + i;
      choice[warp][e + (e >> 5)] = l[i];
    }
  }

  if (grouped) {
    __syncwarp();
    const int G = r.n_groups, size = p.size, share = 1 << p.share_shift;
    const int g = lane >> p.share_shift, sub = lane & (share - 1);
    float a = -INFINITY, b = -INFINITY;    // best and second best
    if (g < G) {
      for (int i = sub; i < size; i += share) {
        const int e = g * size + i;
        const float c = choice[warp][e + (e >> 5)];
        b = fmaxf(b, fminf(a, c));
        a = fmaxf(a, c);
      }
    }
    for (int o = 1; o < share; o <<= 1) {
      const float a2 = __shfl_xor_sync(kAll, a, o), b2 = __shfl_xor_sync(kAll, b, o);
      b = fmaxf(fmaxf(b, b2), fminf(a, a2));
      a = fmaxf(a, a2);
    }
    const float mine = g < G ? (r.group_top == 2 ? a + b : a) : -INFINITY;
    int before = 0;
    for (int o = 0; o < G; ++o) {
      const float other = __shfl_sync(kAll, mine, o << p.share_shift);
      before += other > mine || (other == mine && o < g);
    }
    bool keep = g < G && before < r.top_groups;
    // Group sums compare only by a margin. A score is off by less than
    // 2^-19.4: s·|x| ≤ 0.37 for a softmax's x = l − top, s·(1 − s)·|x| ≤ 0.28
    // for a sigmoid, and the rest is relative to s ≤ 1; four scores make
    // 2^-17.4. Roundings of c and of the sums go by the largest |a| + |b|.
    if (!by_logit || r.group_top == 2) {
      const float size_ab = (a == -INFINITY ? 0.f : fabsf(a)) + (b == -INFINITY ? 0.f : fabsf(b));
      const float largest =
          __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(g < G ? size_ab : 0.f)));
      const float worst_kept =
          key_value(__reduce_min_sync(kAll, keep ? order_key(mine) : order_key(INFINITY)));
      const float best_left =
          key_value(__reduce_max_sync(kAll, order_key(g < G && !keep ? mine : -INFINITY)));
      const float margin = 0x1p-17f + largest * 0x1p-21f;
      if (worst_kept != -INFINITY && !(worst_kept - best_left > margin)) {
        // the groups' sums in fp64, a group in a lane: its two best choices,
        // if they are its two best for certain
        float c1 = -INFINITY, c2 = -INFINITY, c3 = -INFINITY;
        int e1 = 0, e2 = 0;
        if (lane < G) {
          for (int i = 0; i < size; ++i) {
            const int e = lane * size + i;
            const float c = choice[warp][e + (e >> 5)];
            if (c > c1) {
              c3 = c2;
              c2 = c1;
              e2 = e1;
              c1 = c;
              e1 = e;
            } else if (c > c2) {
              c3 = c2;
              c2 = c;
              e2 = e;
            } else {
              c3 = fmaxf(c3, c);
            }
          }
        }
        const float next = r.group_top == 2 ? c3 : c2, last = r.group_top == 2 ? c2 : c1;
        unsure |= __any_sync(kAll, next != -INFINITY && !(last - next > margin));
        const RowSum q = sigmoid ? RowSum{0.0, 0.0} : row_sum64(row, E);
        double sum = -INFINITY;
        if (c1 != -INFINITY) {
          sum = choice64(load_logit(row + e1), bias ? bias[e1] : 0.f, sigmoid, q);
          if (r.group_top == 2)
            sum = c2 == -INFINITY ? -INFINITY
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
    const uint32_t kept = __ballot_sync(kAll, keep && sub == 0);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane * kPer + i;
      if (!((kept >> ((e * p.to_group >> 16) << p.share_shift)) & 1u)) key[i] = kNone;
    }
  }

  // At least k + 1 experts are no worse than the (k + 1)-th best of the lanes'
  // best ones, and few more: they go one to a lane and are ranked against
  // each other. Beside a bias, those that lie below it by no more than the
  // choices may be off come along.
  auto best_below = [&](int limit) {       // this lane's largest key under `limit`
    int m = kNone;
#pragma unroll
    for (int i = 0; i < kPer; ++i) m = max(m, key[i] < limit ? key[i] : kNone);
    return m;
  };
  int best = best_below(INT_MAX);
  // (with experts left in k lanes or fewer, a lane's next best takes its turn)
  const bool few = __popc(__ballot_sync(kAll, best != kNone)) <= k;
  int least = kNone;
  for (int j = 0; j <= k; ++j) {
    least = __reduce_max_sync(kAll, best);
    if (best == least) best = few ? best_below(least) : kNone;
  }
  // what a choice near `least` may be off by: see bound() below
  const float off_max = (sigmoid ? 0x1p-20f : 0x1p-18f) + fabsf(key_value(least)) * 0x1p-22f;
  if (!by_logit && least > order_key(-INFINITY)) least = order_key(key_value(least) - 2.f * off_max);
  int count = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const bool in = key[i] != kNone && key[i] >= least;
    const uint32_t who = __ballot_sync(kAll, in);
    const int at = count + __popc(who & ((1u << lane) - 1u));
    if (in && at < 32) cand[warp][at] = make_int2(key[i], lane * kPer + i);
    count += __popc(who);
  }
  const bool crowd = count > 32;
  __syncwarp();
  if (!crowd) {
    const int2 my = lane < count ? cand[warp][lane] : make_int2(kNone, 0);
    int rank = 0;
    for (int o = 0; o < count; ++o) {
      const int2 other = cand[warp][o];
      rank += other.x > my.x || (other.x == my.x && other.y < my.y);
    }
    __syncwarp();
    if (lane < count) cand[warp][rank] = my;
  } else {
    // many equal ones: the largest key left k + 1 times, of equal ones the
    // lowest expert's, which is in the lowest lane
    count = k + 1;
    for (int j = 0; j <= k; ++j) {
      const int mine = best_below(INT_MAX), most = __reduce_max_sync(kAll, mine);
      const int from = __ffs(__ballot_sync(kAll, mine == most)) - 1;
      if (lane == from) {
        int at = 0;
#pragma unroll
        for (int i = kPer - 1; i >= 0; --i)
          if (key[i] == most) at = i;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (i == at) key[i] = kNone;
        cand[warp][j] = make_int2(most, lane * kPer + at);
      }
    }
  }
  __syncwarp();
  const int2 my = lane < count ? cand[warp][lane] : make_int2(kNone, 0);
  int my_e = my.y;                         // rank j's expert in lane j

  // the chosen experts' scores, accurately
  auto score_of = [&](float x) {
    return x == -INFINITY ? 0.f : sigmoid ? 1.f / (1.f + expf(-x)) : expf(x - top) * inv;
  };
  float x = lane < count ? load_logit(row + my_e) : -INFINITY;
  float s = score_of(x);
  if (!by_logit) {
    // Neighbours in the order must differ by more than their bounds — for a
    // sigmoid s·((1 − s)·(|x|·2^-23.4 + 2^-22) + 2^-22), (1 − s)·|x| ≤ 0.28
    // for x > 0; for a softmax s·(|x|·2^-23.4 + 2^-19.4) — or be equal in
    // logit and bias: then the index decides, here as exactly.
    auto bound = [&](float v_s, float v_x, float v_c) {
      return (sigmoid ? v_s * 0x1.6ap-21f + fmaxf(-v_x, 0.f) * v_s * 0x1p-23f
                      : v_s * (fabsf(v_x - top) * 0x1p-23f + 0x1p-19f)) +
             fabsf(v_c) * 0x1p-23f;
    };
    const float b = lane < count ? __ldg(bias + my_e) : 0.f;
    const float c = key_value(my.x);
    const float off = lane < count && x != -INFINITY ? bound(s, x, c) : 0.f;
    const float x2 = __shfl_down_sync(kAll, x, 1), b2 = __shfl_down_sync(kAll, b, 1);
    const float c2 = __shfl_down_sync(kAll, c, 1), off2 = __shfl_down_sync(kAll, off, 1);
    const bool close = lane < k && lane + 1 < count && x2 != -INFINITY && !(c - c2 > off + off2) &&
                       !(x == x2 && b == b2);
    if (!__any_sync(kAll, close)) {
    } else if (crowd) {
      unsure = true;                       // others may be as close
    } else {                               // all candidates by fp64
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
      if (lane < count) cand[warp][rank].y = my_e;
      __syncwarp();
      my_e = cand[warp][lane < count ? lane : 0].y;
      x = lane < count ? load_logit(row + my_e) : -INFINITY;
      s = score_of(x);
    }
  }
  // sigmoids that fp32 cannot hold, of which quotients are wanted
  if (sigmoid && r.renorm && lane < k && x != -INFINITY && s < 0x1p-100f) unsure = true;
  float w;
  if (__any_sync(kAll, unsure)) {
    route_exact<T>(r, row, bias, &my_e, &w);
  } else {
    w = lane < k ? s : 0.f;
    if (r.renorm) {
      const float sum = warp_sum(w);
      w = sum > 0.f ? w / sum : 0.f;
    }
    w *= r.scale;
  }
  if (lane < k) {
    topk_idx[(size_t)t * k + lane] = my_e;
    topk_w[(size_t)t * k + lane] = w;
  }
}

template <typename T, int kPer>
cudaError_t launch_t(const moe_router_desc& r, const T* logits, int64_t row_stride,
                     const float* bias, int n, int32_t* topk_idx, float* topk_w,
                     cudaStream_t stream) {
  Router p;
  p.d = r;
  p.size = r.n_experts / r.n_groups;
  p.to_group = (65536 + p.size - 1) / p.size;
  p.share_shift = 0;
  while ((2 << p.share_shift) * r.n_groups <= 32) ++p.share_shift;
  // rows in whole pieces: every lane's experts exist or none does
  p.wide = r.n_experts % kPer == 0 && (reinterpret_cast<uintptr_t>(logits) & 15u) == 0 &&
           row_stride * sizeof(T) % 16 == 0 && kPer * sizeof(T) % 16 == 0;
  return launch_pdl(route_grouped_kernel<T, kPer>, dim3((n - 1) / kWarps + 1), dim3(kWarps * 32), 0,
                    stream, p, logits, row_stride, bias, n, topk_idx, topk_w);
}

template <typename T>
cudaError_t launch_e(const moe_router_desc& r, const void* logits, int64_t row_stride,
                     const float* bias, int n, int32_t* topk_idx, float* topk_w,
                     cudaStream_t stream) {
  const T* l = static_cast<const T*>(logits);
  if (r.n_experts <= 64) return launch_t<T, 2>(r, l, row_stride, bias, n, topk_idx, topk_w, stream);
  if (r.n_experts <= 128)
    return launch_t<T, 4>(r, l, row_stride, bias, n, topk_idx, topk_w, stream);
  return launch_t<T, 8>(r, l, row_stride, bias, n, topk_idx, topk_w, stream);
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
