// kv8_cache.cu — new keys and values into a paged cache of e4m3 codes with a
// scale for each block of tokens and head, and rows of it back.
//
// With A the largest finite size among a block's new elements of one head,
// e(A) is the smallest exponent with A ≤ 448 · 2^e, and the block's scale 2^e
// the larger of that and the one it has (or that alone, when the block starts
// anew). Powers of two divide exactly, so a code is the one rounding of its
// element; where the scale grows, the other codes are divided by the growth,
// which rounds only those that fall below 2^-6.
//
// Both are bound by memory, or by a launch and a chain of loads for a few tokens.
#include "batch_launch.h"
#include "common.cuh"
#include "fp8.cuh"
#include "kv8_launch.h"
#include "round16.cuh"

namespace moe {
namespace {

enum { kF32 = 0, kBf16 = 1, kFp16 = 2 };

struct Eight {
  float v[8];
};
template <int kType>
MOE_DEV Eight load8(const void* base, int64_t at) {
  Eight r;
  if constexpr (kType == kF32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    r.v[0] = a.x, r.v[1] = a.y, r.v[2] = a.z, r.v[3] = a.w;
    r.v[4] = b.x, r.v[5] = b.y, r.v[6] = b.z, r.v[7] = b.w;
  } else {
    const uint4 x =
        __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kType == kBf16) {
        r.v[2 * i] = bf16lo(w[i]);
        r.v[2 * i + 1] = bf16hi(w[i]);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        r.v[2 * i] = f.x;
        r.v[2 * i + 1] = f.y;
      }
    }
  }
  return r;
}

// The smallest e in [MOE_KV8_MIN_EXP, MOE_KV8_MAX_EXP] with a ≤ 448 · 2^e, where
// that range has one. (448 = 1.75 · 2^8.)
MOE_DEV int exponent_for(float a) {
  const uint32_t bits = __float_as_uint(a);
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, MOE_KV8_MIN_EXP), MOE_KV8_MAX_EXP);
}

constexpr int kAppendThreads = 128;
constexpr int kHold = 4;  // pieces of 8 elements that a thread keeps from the first pass

// A CTA takes the blocks whose first token in the call is one of `per` tokens,
// for one head, of keys or of values: a pass over the block's new rows for their
// largest size, then one that writes codes.
template <int kType>
__global__ void __launch_bounds__(kAppendThreads)
    kv8_append_kernel(const __grid_constant__ Append8Args a, int page_shift, int block_shift,
                      int row_shift, int per) {
  __shared__ uint32_t written[8];      // rows of the block that the call writes
  __shared__ float warp_max[kAppendThreads / 32];
  pdl_wait();
  pdl_trigger();
  const moe_kv8_cache& c = a.cache;
  const int tid = threadIdx.x, lane = tid & 31, h = blockIdx.y;
  const int64_t n_slots = c.n_pages << page_shift;
  const int blocks = c.page_size >> block_shift;   // of a page
  const int block = 1 << block_shift;
  const void* src = blockIdx.z ? a.v : a.k;
  uint8_t* codes = static_cast<uint8_t*>(blockIdx.z ? c.v : c.k) + h * c.head_stride;
  float* scales = blockIdx.z ? c.v_scale : c.k_scale;
  const int pieces = 1 << row_shift;               // of a row, 8 elements each
  auto block_of = [&](int t) -> int64_t {          // -1: none
    const int64_t s = a.slots[t];
    return s >= 0 && s < n_slots ? s >> block_shift : -1;
  };
  const int t_end = min((int)(blockIdx.x + 1) * per, a.n_tokens);
  for (int t0 = blockIdx.x * per; t0 < t_end; ++t0) {
    const int64_t slot0 = a.slots[t0];
    if (slot0 < 0 || slot0 >= n_slots) {
      if (slot0 != -1 && tid == 0) report_error(a.err, ERR_CHECK, 0xB10);
      continue;
    }
    const int64_t b = slot0 >> block_shift;
    if (t0 > 0 && block_of(t0 - 1) == b) continue;  // an earlier token's
    int n = 0;                                      // tokens of the block
    for (bool more = true; more;) {
      const int t = t0 + n + lane;
      const uint32_t same = __ballot_sync(0xffffffffu, t < a.n_tokens && block_of(t) == b);
      n += same == 0xffffffffu ? 32 : __ffs(~same) - 1;
      more = same == 0xffffffffu;
    }
    // the new rows' largest finite size, and which rows they are
    __syncthreads();
    if (tid < 8) written[tid] = 0;
    __syncthreads();
    const int all = n << row_shift;
    Eight held[kHold];
    float top = 0.f;
    auto piece = [&](int i) {
      return load8<kType>(src, (int64_t)(t0 + (i >> row_shift)) * a.token_stride +
                                   h * a.head_stride + (i & (pieces - 1)) * 8);
    };
    auto size_of = [&](const Eight& x) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float s = fabsf(x.v[e]);
        top = fmaxf(top, s <= 3.402823466e38f ? s : 0.f);
      }
    };
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
      const int i = tid + k * kAppendThreads;
      if (i < all) {
        held[k] = piece(i);
        size_of(held[k]);
      }
    }
    for (int i = tid + kHold * kAppendThreads; i < all; i += kAppendThreads) size_of(piece(i));
    for (int i = tid; i < n; i += kAppendThreads) {
      const int row = (int)(a.slots[t0 + i] & (block - 1));
      atomicOr(&written[row >> 5], 1u << (row & 31));
    }
    // (sizes are not negative: their bits order as they do)
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    if (lane == 0) warp_max[tid >> 5] = top;
    const int64_t page = b / blocks;
    float* scale = scales + (page * c.n_kv_heads + h) * blocks + (b - page * blocks);
    // (a scale that this library did not write counts by its exponent)
    const int was = min(max((int)(__float_as_uint(*scale) >> 23 & 0xffu) - 127, MOE_KV8_MIN_EXP),
                        MOE_KV8_MAX_EXP);
    __syncthreads();
    for (int w = 0; w < kAppendThreads / 32; ++w) top = fmaxf(top, warp_max[w]);
    const bool anew = written[0] & 1u;
    const int needs = exponent_for(top), e = anew ? needs : max(was, needs);
    if (tid == 0) *scale = pow2(e);
    uint8_t* page_codes = codes + page * c.page_stride;
    const int first = (int)(b - page * blocks) << block_shift;   // its first row in the page
    if (!anew && e > was) {
      const float by = pow2(was - e);
      for (int i = tid; i < block << row_shift; i += kAppendThreads) {
        const int row = i >> row_shift;
        if (written[row >> 5] >> (row & 31) & 1u) continue;
        uint2* at = reinterpret_cast<uint2*>(page_codes + (first + row) * c.token_stride +
                                             (i & (pieces - 1)) * 8);
        const uint2 x = *at;
        const float4 lo = floats_of(x.x), hi = floats_of(x.y);
        *at = make_uint2(e4m3_of(lo.x * by, lo.y * by) |
                             (uint32_t)e4m3_of(lo.z * by, lo.w * by) << 16,
                         e4m3_of(hi.x * by, hi.y * by) |
                             (uint32_t)e4m3_of(hi.z * by, hi.w * by) << 16);
      }
    }
    const float inv = pow2(-e);
    auto write = [&](const Eight& x, int i) {
      const int row = (int)(a.slots[t0 + (i >> row_shift)] & (c.page_size - 1));
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // x · 0 makes NaN of an infinity, and adds nothing to the others
        const float lo = fmaf(x.v[2 * k], inv, x.v[2 * k] * 0.f);
        const float hi = fmaf(x.v[2 * k + 1], inv, x.v[2 * k + 1] * 0.f);
        w[k] = e4m3_of(lo, hi);
      }
      *reinterpret_cast<uint2*>(page_codes + row * c.token_stride + (i & (pieces - 1)) * 8) =
          make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    };
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
      const int i = tid + k * kAppendThreads;
      if (i < all) write(held[k], i);
    }
    for (int i = tid + kHold * kAppendThreads; i < all; i += kAppendThreads) write(piece(i), i);
  }
}

constexpr int kReadThreads = 256;

// A thread takes 8 codes.
template <int kType>
__global__ void __launch_bounds__(kReadThreads)
    kv8_read_kernel(const __grid_constant__ Read8Args a, int page_shift, int block_shift,
                    int row_shift) {
  pdl_wait();
  pdl_trigger();
  const moe_kv8_cache& c = a.cache;
  const int64_t n_slots = c.n_pages << page_shift;
  const int blocks = c.page_size >> block_shift;
  const int per_row = c.n_kv_heads << row_shift;
  const int64_t n = (int64_t)a.n * per_row;
  const uint8_t* codes = static_cast<const uint8_t*>(blockIdx.y ? c.v : c.k);
  const float* scales = blockIdx.y ? c.v_scale : c.k_scale;
  void* out = blockIdx.y ? a.v : a.k;
  for (int64_t i = (int64_t)blockIdx.x * kReadThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kReadThreads) {
    const int t = (int)(i / per_row);
    const int j = (int)(i - (int64_t)t * per_row);
    const int h = j >> row_shift, e = (j & ((1 << row_shift) - 1)) * 8;
    const int64_t slot = a.slots[t];
    float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
    if (slot >= 0 && slot < n_slots) {
      const int64_t page = slot >> page_shift;
      const int row = (int)(slot & (c.page_size - 1));
      const float s = __ldg(scales + (page * c.n_kv_heads + h) * blocks + (row >> block_shift));
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(
          codes + page * c.page_stride + row * c.token_stride + h * c.head_stride + e));
      lo = floats_of(x.x);
      hi = floats_of(x.y);
      lo = make_float4(lo.x * s, lo.y * s, lo.z * s, lo.w * s);
      hi = make_float4(hi.x * s, hi.y * s, hi.z * s, hi.w * s);
    } else if (slot != -1) {
      report_error(a.err, ERR_CHECK, 0xB20);
    }
    const int64_t to = t * a.token_stride + h * a.head_stride + e;
    if constexpr (kType == kF32) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + to);
      p[0] = lo;
      p[1] = hi;
    } else {
      constexpr bool f16 = kType == kFp16;
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + to) =
          make_uint4(round16<f16>(lo.x, lo.y), round16<f16>(lo.z, lo.w), round16<f16>(hi.x, hi.y),
                     round16<f16>(hi.z, hi.w));
    }
  }
}

int log2i(int v) { return 31 - __builtin_clz(v); }

}  // namespace

cudaError_t launch_kv8_append(const Append8Args& a, int src_dtype, int num_sms,
                              cudaStream_t stream) {
  const moe_kv8_cache& c = a.cache;
  // tokens whose blocks a CTA takes: one, while the GPU has room for a CTA each
  int per = 1;
  while (per < 16 && (int64_t)a.n_tokens * c.n_kv_heads * 2 > (int64_t)per * num_sms * 16) per *= 2;
  const dim3 grid((a.n_tokens - 1) / per + 1, c.n_kv_heads, 2);
  auto* kernel = src_dtype == MOE_F32    ? kv8_append_kernel<kF32>
                 : src_dtype == MOE_BF16 ? kv8_append_kernel<kBf16>
                                         : kv8_append_kernel<kFp16>;
  return launch_pdl(kernel, grid, dim3(kAppendThreads), 0, stream, a, log2i(c.page_size),
                    log2i(c.block), log2i(c.head_dim / 8), per);
}

cudaError_t launch_kv8_read(const Read8Args& a, int dtype, int num_sms, cudaStream_t stream) {
  const moe_kv8_cache& c = a.cache;
  const int row_shift = log2i(c.head_dim / 8);
  const int64_t n = ((int64_t)a.n * c.n_kv_heads) << row_shift;
  const int64_t ctas = (n + kReadThreads - 1) / kReadThreads, most = (int64_t)num_sms * 32;
  const dim3 grid((unsigned)(ctas < most ? ctas : most), 2);
  auto* kernel = dtype == MOE_F32    ? kv8_read_kernel<kF32>
                 : dtype == MOE_BF16 ? kv8_read_kernel<kBf16>
                                     : kv8_read_kernel<kFp16>;
  return launch_pdl(kernel, grid, dim3(kReadThreads), 0, stream, a, log2i(c.page_size),
                    log2i(c.block), row_shift);
}

}  // namespace moe
