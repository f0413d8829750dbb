// attend8.cu — attention of every request's new tokens over its paged cache of
// e4m3 codes: causal, optionally within a sliding window beside a few first
// keys that stay visible.
//
// For a query row q at position p, with s_j = scale·ks_j·(q·k_j) over the keys
// it sees, out = Σ_j e^(s_j − m) vs_j·v_j / Σ_j e^(s_j − m). A warp per row
// walks its keys one after the other with the running maximum and sums.
#include <math.h>

#include "batch_launch.h"
#include "common.cuh"
#include "fp8.cuh"
#include "kv8_launch.h"
#include "round16.cuh"

namespace moe {
namespace {

template <int kDim, bool kF16>
__global__ void __launch_bounds__(256) attend8_kernel(const __grid_constant__ Attend8Args a,
                                                      int page_shift, int block_shift) {
  constexpr int kN = kDim / 32;                  // columns of a lane
  pdl_wait();
  pdl_trigger();
  const moe_kv8_cache& c = a.cache;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t t = row / a.n_heads;
  const int h = (int)(row - t * a.n_heads), kh = h / a.group;
  if (t >= a.n_tokens) return;
  // the token's request: the last that begins at or before it
  int b = -1, first = 0, len = 0, q = 0;
  for (int i = 0; i < a.n_requests; ++i) {
    const int f = a.q_start[i], l = a.q_start[i + 1];
    if (f < 0 || l < f || l > a.n_tokens) report_error(a.err, ERR_CHECK, 0xB30);
    if (f <= t && t < l) {
      b = i;
      first = f;
      q = min(l, a.n_tokens) - f;
    }
  }
  uint16_t* out = static_cast<uint16_t*>(a.out) + t * a.out_token_stride + h * a.out_head_stride +
                  lane * kN;
  if (b < 0) {
    if (a.clear)
      for (int i = 0; i < kN; ++i) out[i] = 0;
    return;
  }
  len = a.kv_len[b];
  if (len < 0 || len > MOE_MAX_CACHE_LEN || len > ((int64_t)a.max_blocks << page_shift)) {
    report_error(a.err, ERR_CHECK, 0xB31);
    len = 0;
  }
  const int pos = len - q + (int)(t - first);
  float x[kN], o[kN];
  for (int i = 0; i < kN; ++i) {
    const uint16_t w = (static_cast<const uint16_t*>(a.q) + t * a.q_token_stride +
                        h * a.q_head_stride)[lane * kN + i];
    x[i] = (kF16 ? __half2float(__ushort_as_half(w)) : __uint_as_float((uint32_t)w << 16)) *
           a.scale;
    o[i] = 0.f;
  }
  float m = -INFINITY, sum = 0.f;
  const int lo = a.window > 0 ? max(0, max(pos, 0) - a.window + 1) : 0;
  const int blocks = c.page_size >> block_shift;
  for (int j = 0; j <= pos && j < len; ++j) {
    if (j < lo && j >= a.sinks) {
      j = lo - 1;
      continue;
    }
    const int page = a.block_table[(size_t)b * a.max_blocks + (j >> page_shift)];
    float ks = 1.f, vs = 1.f;
    uint32_t kw = 0, vw = 0;
    if (page < 0 || page >= c.n_pages) {
      report_error(a.err, ERR_CHECK, 0xB32);
    } else {
      const int r = j & (c.page_size - 1);
      const int64_t at = page * c.page_stride + r * c.token_stride + kh * c.head_stride + lane * kN;
      if (kN == 4) {
        kw = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(c.k) + at);
        vw = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(c.v) + at);
      } else {
        kw = *reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(c.k) + at);
        vw = *reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(c.v) + at);
      }
      const int64_t s = ((int64_t)page * c.n_kv_heads + kh) * blocks + (r >> block_shift);
      ks = c.k_scale[s];
      vs = c.v_scale[s];
      const float least = pow2(MOE_KV8_MIN_EXP), most = pow2(MOE_KV8_MAX_EXP);
      if (!(ks >= least && ks <= most && vs >= least && vs <= most)) {
        report_error(a.err, ERR_CHECK, 0xB33);
        ks = fminf(fmaxf(ks, least), most);
        vs = fminf(fmaxf(vs, least), most);
      }
    }
    const float4 k4 = floats_of(kw), v4 = floats_of(vw);
    const float kf[4] = {k4.x, k4.y, k4.z, k4.w}, vf[4] = {v4.x, v4.y, v4.z, v4.w};
    float s = 0.f;
    for (int i = 0; i < kN; ++i) s = fmaf(x[i], kf[i], s);
    s = warp_sum(s) * ks;
    const float top = fmaxf(m, s);
    const float keep = m == -INFINITY ? 0.f : expf(m - top), p = expf(s - top);
    m = top;
    sum = sum * keep + p;
    for (int i = 0; i < kN; ++i) o[i] = fmaf(p * vs, vf[i], o[i] * keep);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  for (int i = 0; i < kN; i += 2)
    *reinterpret_cast<uint32_t*>(out + i) = round16<kF16>(o[i] * inv, o[i + 1] * inv);
}

}  // namespace

size_t attend8_workspace_bytes(int) { return 256; }

cudaError_t launch_attend8(const Attend8Args& a, int, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.n_tokens * a.n_heads;
  const dim3 grid((unsigned)((rows + 7) / 8));
  const int ps = 31 - __builtin_clz(a.cache.page_size), bs = 31 - __builtin_clz(a.cache.block);
  auto* kernel = a.cache.head_dim == 128
                     ? (a.f16 ? attend8_kernel<128, true> : attend8_kernel<128, false>)
                     : (a.f16 ? attend8_kernel<64, true> : attend8_kernel<64, false>);
  return launch_pdl(kernel, grid, dim3(256), 0, stream, a, ps, bs);
}

}  // namespace moe
