// route_grouped.cu — experts from router logits: softmax or sigmoid scores, a
// balance bias, groups, top-k, renormalised weights.
//
// Sources: "Deep Dive into Mixture of Experts: From 1991 to DeepSeek-V3", §5
// (DeepSeek-style routing sketch: scores, a bias that only selects, top-k).
#include <math.h>

#include "batch_launch.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr int kPerLane = MOE_MAX_EXPERTS / 32;

template <typename T>
MOE_DEV float load_logit(const T* p);
template <>
MOE_DEV float load_logit<float>(const float* p) { return *p; }
template <>
MOE_DEV float load_logit<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }
template <>
MOE_DEV float load_logit<__half>(const __half* p) { return __half2float(*p); }

template <typename T>
MOE_DEV constexpr float lowest();
template <>
MOE_DEV constexpr float lowest<float>() { return -3.402823466e+38f; }
template <>
MOE_DEV constexpr float lowest<__nv_bfloat16>() { return -3.389531389e+38f; }
template <>
MOE_DEV constexpr float lowest<__half>() { return -65504.f; }

MOE_DEV double warp_max(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

MOE_DEV double warp_add(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One warp per token, everything in fp64; expert e is in lane e % 32,
// register e / 32.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
    route_grouped_kernel(const __grid_constant__ moe_router_desc r, const T* __restrict__ logits,
                         int64_t row_stride, const float* __restrict__ bias, int n,
                         int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= n) return;
  const int E = r.n_experts, size = E / r.n_groups;
  const T* row = logits + t * row_stride;
  double s[kPerLane], c[kPerLane];
  uint32_t left = 0;  // experts of this lane still to choose from
  float l[kPerLane];
  double top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = lane + 32 * i;
    l[i] = e < E ? load_logit(row + e) : -INFINITY;
    if (l[i] <= lowest<T>()) l[i] = -INFINITY;
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
    for (int i = 0; i < kPerLane; ++i) s[i] = l[i] == -INFINITY ? 0.0 : 1.0 / (1.0 + exp(-(double)l[i]));
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
        const double a2 = __shfl_xor_sync(0xffffffffu, a, o);
        const double b2 = __shfl_xor_sync(0xffffffffu, b, o);
        b = fmax(fmax(b, b2), fmin(a, a2));
        a = fmax(a, a2);
      }
      const double score = r.group_top == 2 ? a + b : a;
      if (lane == g) mine = score;
    }
    // a group is kept if fewer than top_groups come before it
    int before = 0;
    for (int g = 0; g < r.n_groups; ++g) {
      const double other = __shfl_sync(0xffffffffu, mine, g);
      if (other > mine || (other == mine && g < lane)) ++before;
    }
    const uint32_t kept =
        __ballot_sync(0xffffffffu, lane < r.n_groups && before < r.top_groups);
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
      const double c2 = __shfl_xor_sync(0xffffffffu, best, o);
      const double s2 = __shfl_xor_sync(0xffffffffu, bs, o);
      const int e2 = __shfl_xor_sync(0xffffffffu, be, o);
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
      my_e = be;
      my_s = bs;
    }
  }
  double w = lane < r.top_k ? my_s : 0.0;
  if (r.renorm) {
    const double sum = warp_add(w);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  if (lane < r.top_k) {
    topk_idx[(size_t)t * r.top_k + lane] = my_e < E ? my_e : 0;
    topk_w[(size_t)t * r.top_k + lane] = (float)(w * r.scale);
  }
}

template <typename T>
cudaError_t launch_t(const moe_router_desc& r, const void* logits, int64_t row_stride,
                     const float* bias, int n, int32_t* topk_idx, float* topk_w,
                     cudaStream_t stream) {
  return launch_pdl(route_grouped_kernel<T>, dim3((n - 1) / kWarps + 1), dim3(kWarps * 32), 0,
                    stream, r, static_cast<const T*>(logits), row_stride, bias, n, topk_idx,
                    topk_w);
}

}  // namespace

cudaError_t launch_route_grouped(const moe_router_desc& r, const void* logits, int dtype,
                                 int64_t row_stride, const float* bias, int n, int32_t* topk_idx,
                                 float* topk_w, cudaStream_t stream) {
  switch (dtype) {
    case MOE_F32:
      return launch_t<float>(r, logits, row_stride, bias, n, topk_idx, topk_w, stream);
    case MOE_BF16:
      return launch_t<__nv_bfloat16>(r, logits, row_stride, bias, n, topk_idx, topk_w, stream);
    default:
      return launch_t<__half>(r, logits, row_stride, bias, n, topk_idx, topk_w, stream);
  }
}

}  // namespace moe
