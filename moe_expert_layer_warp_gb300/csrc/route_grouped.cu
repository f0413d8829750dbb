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
// difference larger than the two bounds has the right sign. Only a token
// with a closer one is done again in fp64 (a few in ten thousand, with
// trained routers' spreads); doing all of them there took 848 us for 20011
// tokens of 256 experts, fp64 being 1/64 of fp32's rate. Without a bias, c is
// monotone in the logit, and experts are compared by their logits, exactly.
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

// Order-preserving integer keys of floats (−0 and +0 have one key; 0 is below
// every float's key).
MOE_DEV uint32_t order_key(float f) {
  uint32_t u = __float_as_uint(f);
  if ((u << 1) == 0u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
MOE_DEV float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
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

// exp of a non-positive or moderate argument by the hardware's base-2
// exponential: x·log2(e) is rounded (|x|·2^-24·1.45 of an exponent step at
// most) and the exponential itself is good to 2^-22, so the result is off by
// at most (|x| + 4)·2^-23 relative to it.
MOE_DEV float exp_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}

// One warp per token; lane holds kPer consecutive experts, so that a lower
// lane is a lower expert.
template <typename T, int kPer>
__global__ void __launch_bounds__(kWarps * 32)
    route_grouped_kernel(const __grid_constant__ moe_router_desc r, const T* __restrict__ logits,
                         int64_t row_stride, const float* __restrict__ bias, int n, int wide,
                         int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  // choices of the warp's token, one float of padding after every 32
  __shared__ float choice[kWarps][32 * kPer + kPer];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kWarps + warp;
  if (t >= n) return;
  const int E = r.n_experts, k = r.top_k;
  const T* row = logits + t * row_stride;
  const bool sigmoid = r.score == MOE_SCORE_SIGMOID;
  const bool by_logit = bias == nullptr;   // experts compare by their logits
  const bool grouped = r.top_groups < r.n_groups;

  float l[kPer];
  if (wide) {                              // rows of whole, aligned 16-byte pieces
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

  // what experts are compared by, as keys; 0: not to be chosen
  uint32_t key[kPer];
  bool unsure = false;
  if (by_logit) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = lane * kPer + i < E ? order_key(l[i]) : 0u;
  }
  if (!by_logit || (grouped && r.group_top == 2)) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane * kPer + i;
      // off by at most s·(|x| + 16)·2^-22, x = l or l − top (for a softmax the
      // sum adds its own errors, 13 roundings and 2^-22 of each term)
      const float s = sigmoid ? __frcp_rn(1.f + exp_fast(-l[i])) : exp_fast(l[i] - top) * inv;
      float c = -INFINITY;
      if (e < E && l[i] != -INFINITY) c = by_logit ? s : s + __ldg(bias + e);
      if (!by_logit) key[i] = e < E ? order_key(c) : 0u;
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
    // `share` lanes per group, a power of two
    const int G = r.n_groups, size = E / G;
    const int share = 1 << (31 - __clz(32 / G));
    const int g = lane / share, sub = lane & (share - 1);
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
      const float other = __shfl_sync(kAll, mine, o * share);
      if (other > mine || (other == mine && o < g)) ++before;
    }
    const bool keep = g < G && before < r.top_groups;
    // Group sums compare only by a margin. A score is off by less than
    // 2^-19.4: s·|x| ≤ 0.37 for a softmax's x = l − top, s·(1 − s)·|x| ≤ 0.23
    // for a sigmoid, and the rest is relative to s ≤ 1; four scores make
    // 2^-17.4. Roundings of c and of the sums go by the largest |a| + |b|.
    if (!by_logit || r.group_top == 2) {
      const float size_ab = (a == -INFINITY ? 0.f : fabsf(a)) + (b == -INFINITY ? 0.f : fabsf(b));
      const float largest =
          __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(g < G ? size_ab : 0.f)));
      const float worst_kept = key_value(__reduce_min_sync(kAll, keep ? order_key(mine) : 0xff800000u));
      const float best_left =
          key_value(__reduce_max_sync(kAll, g < G && !keep ? order_key(mine) : 0x007fffffu));
      const float margin = 0x1p-17f + largest * 0x1p-21f;
      if (worst_kept != -INFINITY && !(worst_kept - best_left > margin)) unsure = true;
    }
    const uint32_t kept = __ballot_sync(kAll, keep && sub == 0);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane * kPer + i;
      if (e < E && !((kept >> (e / size * share)) & 1u)) key[i] = 0u;
    }
  }

  // k + 1 rounds: the largest key left, of equal ones the lowest expert's;
  // round j's expert ends in lane j (the last is only for the comparison)
  uint32_t my_key = 0u;
  int my_e = 0;
  for (int j = 0; j <= k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) best = max(best, key[i]);
    const uint32_t most = __reduce_max_sync(kAll, best);
    const int from = __ffs(__ballot_sync(kAll, best == most)) - 1;
    int at = 0;
#pragma unroll
    for (int i = kPer - 1; i >= 0; --i)
      if (key[i] == most) at = i;
    if (lane == from) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i == at) key[i] = 0u;
    }
    const int e = __shfl_sync(kAll, lane * kPer + at, from);
    if (lane == j) {
      my_key = most;
      my_e = most ? e : 0;
    }
  }
  // the chosen experts' scores, accurately
  const bool mine = lane <= k && my_key != 0u;
  const float x = mine ? load_logit(row + my_e) : -INFINITY;
  const float s = x == -INFINITY ? 0.f : sigmoid ? 1.f / (1.f + expf(-x)) : expf(x - top) * inv;
  if (!by_logit) {
    // neighbours in the order must differ by more than their bounds, or be
    // equal in logit and bias: then the index decides, here as exactly
    const float b = mine ? __ldg(bias + my_e) : 0.f;
    const float c = key_value(my_key);
    const float off =
        s * (fabsf(sigmoid ? x : x - top) + 16.f) * 0x1p-22f + fabsf(c) * 0x1p-23f;
    const float x2 = __shfl_down_sync(kAll, x, 1), b2 = __shfl_down_sync(kAll, b, 1);
    const float c2 = __shfl_down_sync(kAll, c, 1), off2 = __shfl_down_sync(kAll, off, 1);
    const uint32_t key2 = __shfl_down_sync(kAll, my_key, 1);
    const bool close = lane < k && key2 != 0u && x2 != -INFINITY && !(c - c2 > off + off2) &&
                       !(x == x2 && b == b2);
    unsure |= __any_sync(kAll, close);
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
  // rows in whole pieces: every lane's experts exist or none does
  const int wide = r.n_experts % kPer == 0 && (reinterpret_cast<uintptr_t>(logits) & 15u) == 0 &&
                   row_stride * sizeof(T) % 16 == 0 && kPer * sizeof(T) % 16 == 0;
  return launch_pdl(route_grouped_kernel<T, kPer>, dim3((n - 1) / kWarps + 1), dim3(kWarps * 32), 0,
                    stream, r, logits, row_stride, bias, n, wide, topk_idx, topk_w);
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
