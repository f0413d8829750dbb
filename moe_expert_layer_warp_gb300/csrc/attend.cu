// attend.cu — attention of every request's new tokens over its paged cache:
// causal, optionally within a sliding window beside a few first keys that
// stay visible.
//
// For a query row q at position p, with s_j = scale·(q·k_j) over the keys it
// sees, out = Σ_j e^(s_j − m) v_j / Σ_j e^(s_j − m), m = max_j s_j. The
// maximum and the two sums are carried along in one pass over the keys: when
// the maximum grows from m to m', what has been summed so far is multiplied
// by e^(m − m').
#include <math.h>

#include "batch_launch.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;

template <bool kF16>
MOE_DEV float2 widen(uint32_t w) {
  if constexpr (kF16) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  } else {
    return make_float2(bf16lo(w), bf16hi(w));
  }
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

// One warp per (token, query head), keys one after the other; a lane holds
// kDim/32 elements of the row.
template <int kDim, bool kF16>
__global__ void __launch_bounds__(kWarps * 32) attend_kernel(const __grid_constant__ AttendArgs a,
                                                             int page_shift) {
  pdl_wait();
  pdl_trigger();
  constexpr int kWords = kDim / 64;
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x, head = blockIdx.y * kWarps + (threadIdx.x >> 5);
  if (head >= a.n_heads) return;
  if (t == 0 && head == 0) {
    // row ranges out of order or past the rows are reported, and not followed
    bool bad = false;
    for (int r = lane; r < a.n_requests; r += 32)
      bad |= a.q_start[r] < 0 || a.q_start[r] > a.q_start[r + 1] || a.q_start[r + 1] > a.n_tokens;
    if (bad) report_error(a.err, ERR_CHECK, 0xA22);
  }
  // the last request that starts at or before t
  int b = 0;
  for (int r = 1; r < a.n_requests; ++r)
    if (a.q_start[r] <= t) b = r;
  const int first = a.q_start[b], last = a.q_start[b + 1];
  if (t < first || t >= last) return;
  int len = a.kv_len[b];
  if (len < 0 || len > ((int64_t)a.max_blocks << page_shift)) {
    if (lane == 0) report_error(a.err, ERR_CHECK, 0xA20);
    len = 0;
  }
  const int pos = len - (last - t);
  const uint32_t* q = reinterpret_cast<const uint32_t*>(
      static_cast<const uint16_t*>(a.q) + t * a.q_token_stride + head * a.q_head_stride);
  float2 x[kWords], acc[kWords];
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    x[w] = widen<kF16>(q[lane + 32 * w]);
    acc[w] = make_float2(0.f, 0.f);
  }
  float m = -INFINITY, sum = 0.f;
  const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  for (int j = min(a.sinks, lo) > 0 ? 0 : lo; j <= pos; ++j) {
    if (j < lo && j >= a.sinks) j = lo;
    const int page = a.block_table[(size_t)b * a.max_blocks + (j >> page_shift)];
    uint32_t kw[kWords], vw[kWords];
    if (page < 0 || page >= a.cache.n_pages) {
      if (lane == 0) report_error(a.err, ERR_CHECK, 0xA21);
#pragma unroll
      for (int w = 0; w < kWords; ++w) kw[w] = vw[w] = 0u;
    } else {
      const int64_t at = page * a.cache.page_stride +
                         (j & ((1 << page_shift) - 1)) * a.cache.token_stride +
                         (head / a.group) * a.cache.head_stride;
      const uint32_t* kp =
          reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.cache.k) + at);
      const uint32_t* vp =
          reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.cache.v) + at);
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        kw[w] = kp[lane + 32 * w];
        vw[w] = vp[lane + 32 * w];
      }
    }
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      const float2 kv = widen<kF16>(kw[w]);
      s += x[w].x * kv.x + x[w].y * kv.y;
    }
    s = warp_sum(s) * a.scale;
    const float grown = fmaxf(m, s);
    const float keep = expf(m - grown), p = expf(s - grown);
    m = grown;
    sum = sum * keep + p;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      const float2 vv = widen<kF16>(vw[w]);
      acc[w].x = acc[w].x * keep + p * vv.x;
      acc[w].y = acc[w].y * keep + p * vv.y;
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) +
                                              t * a.out_token_stride + head * a.out_head_stride);
#pragma unroll
  for (int w = 0; w < kWords; ++w) out[lane + 32 * w] = narrow<kF16>(acc[w].x * inv, acc[w].y * inv);
}

}  // namespace

size_t attend_workspace_bytes(int head_dim) {
  (void)head_dim;
  return 256;
}

cudaError_t launch_attend(const AttendArgs& a, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const bool f16 = a.cache.dtype == MOE_F16;
  auto* kernel = a.cache.head_dim == 128
                     ? (f16 ? attend_kernel<128, true> : attend_kernel<128, false>)
                     : (f16 ? attend_kernel<64, true> : attend_kernel<64, false>);
  const int page_shift = 31 - __builtin_clz(a.cache.page_size);
  return launch_pdl(kernel, dim3(a.n_tokens, (a.n_heads + kWarps - 1) / kWarps), dim3(kWarps * 32),
                    0, stream, a, page_shift);
}

}  // namespace moe
