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
// Bound by memory, or by a launch and a chain of loads for a few tokens. 4747 rows
// of 8 heads of 128 fp32 columns, keys and values, in blocks of 32 (49 MB): 13 us
// beyond an empty launch, 3.7 TB/s: the chain from slots to rows to a block's
// largest size to its codes, which is what 36 rows' 2 us are too. Read back, 32001
// rows of 8 heads of 128 columns in bf16 (196 MB, 131 of them written): 44 us, 4.5
// TB/s; filling those 131 MB alone takes 35. (More rows a thread, their loads ahead,
// were slower: 2 rows 51 us, 8 rows 65, against 49 on the same card.)
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

// A CTA takes the blocks whose first token in the call is one of `per` tokens (16 at
// most), for one head, of keys or of values: a pass over the block's new rows for
// their largest size, then one that writes codes. What both need of the slots is
// loaded once, a token a lane.
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
  const int c0 = blockIdx.x * per, c1 = min(c0 + per, a.n_tokens);
  // lane l: the slot of token c0 − 1 + l (-1: none), and its block
  auto slot_of = [&](int t) -> int64_t { return t >= 0 && t < a.n_tokens ? a.slots[t] : -1; };
  auto block_of = [&](int64_t s) -> int64_t {
    return s >= 0 && s < n_slots ? s >> block_shift : -1;
  };
  const int64_t slot_l = slot_of(c0 - 1 + lane), block_l = block_of(slot_l);
  if (tid < 32 && lane > 0 && c0 - 1 + lane < c1 && block_l < 0 && slot_l != -1)
    report_error(a.err, ERR_CHECK, 0xB10);
  // tokens that are the first of their block in the call
  const int64_t before = __shfl_up_sync(0xffffffffu, block_l, 1);
  uint32_t leaders = __ballot_sync(0xffffffffu, lane > 0 && c0 - 1 + lane < c1 && block_l >= 0 &&
                                                    block_l != before);
  for (; leaders; leaders &= leaders - 1) {
    const int l0 = __ffs(leaders) - 1, t0 = c0 - 1 + l0;
    const int64_t b = __shfl_sync(0xffffffffu, block_l, l0);
    // its tokens: those that follow with the same block
    uint32_t other = __ballot_sync(0xffffffffu, block_l != b) & (0xffffffffu << l0);
    int n = (other ? __ffs(other) - 1 : 32) - l0;
    for (bool more = other == 0; more;) {
      other = __ballot_sync(0xffffffffu, block_of(slot_of(t0 + n + lane)) != b);
      n += other ? __ffs(other) - 1 : 32;
      more = other == 0;
    }
    // the scale that the block has (one that this library did not write counts by
    // its exponent)
    const int64_t page = b / blocks;
    float* scale = scales + (page * c.n_kv_heads + h) * blocks + (b - page * blocks);
    const uint32_t was_bits = __float_as_uint(*scale);
    // the new rows' largest finite size, and which rows they are
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
    for (int k = 0; k < kHold; ++k)
      if (tid + k * kAppendThreads < all) held[k] = piece(tid + k * kAppendThreads);
    __syncthreads();                               // (the block before is done with these)
    if (tid < 8) written[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kAppendThreads) {
      const int row = (int)(a.slots[t0 + i] & (block - 1));
      atomicOr(&written[row >> 5], 1u << (row & 31));
    }
#pragma unroll
    for (int k = 0; k < kHold; ++k)
      if (tid + k * kAppendThreads < all) size_of(held[k]);
    for (int i = tid + kHold * kAppendThreads; i < all; i += kAppendThreads) size_of(piece(i));
    // (sizes are not negative: their bits order as they do)
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    if (lane == 0) warp_max[tid >> 5] = top;
    __syncthreads();
    for (int w = 0; w < kAppendThreads / 32; ++w) top = fmaxf(top, warp_max[w]);
    const int was =
        min(max((int)(was_bits >> 23 & 0xffu) - 127, MOE_KV8_MIN_EXP), MOE_KV8_MAX_EXP);
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
    for (int k = 0; k < kHold; ++k)
      if (tid + k * kAppendThreads < all) write(held[k], tid + k * kAppendThreads);
    for (int i = tid + kHold * kAppendThreads; i < all; i += kAppendThreads) write(piece(i), i);
  }
}

constexpr int kReadThreads = 256;

// A thread takes 8 codes of a row's keys and the same 8 of its values.
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
  // a row takes `of` threads, and a CTA that many rows
  const int of = min(per_row, kReadThreads), rows = kReadThreads / of;
  const int group = threadIdx.x / of;
  const int64_t t = (int64_t)blockIdx.x * rows + group;
  if (group >= rows || t >= a.n) return;
  const int64_t slot = a.slots[t];
  const bool there = slot >= 0 && slot < n_slots;
  if (!there && slot != -1) report_error(a.err, ERR_CHECK, 0xB20);
  const int64_t page = slot >> page_shift;
  const int row = (int)slot & (c.page_size - 1);
  for (int j = threadIdx.x - group * of; j < per_row; j += of) {
    const int h = j >> row_shift, e = (j & ((1 << row_shift) - 1)) * 8;
    const int64_t to = t * a.token_stride + h * a.head_stride + e;
    uint2 x[2] = {make_uint2(0, 0), make_uint2(0, 0)};
    float s[2] = {0.f, 0.f};
    if (there) {
      const int64_t at = (page * c.n_kv_heads + h) * blocks + (row >> block_shift);
      const int64_t from = page * c.page_stride + row * c.token_stride + h * c.head_stride + e;
      x[0] = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.k) + from));
      x[1] = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.v) + from));
      s[0] = __ldg(c.k_scale + at);
      s[1] = __ldg(c.v_scale + at);
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      void* out = which ? a.v : a.k;
      const float by = s[which];
      float4 lo = floats_of(x[which].x), hi = floats_of(x[which].y);
      lo = make_float4(lo.x * by, lo.y * by, lo.z * by, lo.w * by);
      hi = make_float4(hi.x * by, hi.y * by, hi.z * by, hi.w * by);
      if constexpr (kType == kF32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + to);
        p[0] = lo;
        p[1] = hi;
      } else {
        constexpr bool f16 = kType == kFp16;
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + to) =
            make_uint4(round16<f16>(lo.x, lo.y), round16<f16>(lo.z, lo.w),
                       round16<f16>(hi.x, hi.y), round16<f16>(hi.z, hi.w));
      }
    }
  }
}

int log2i(int v) { return 31 - __builtin_clz(v); }

}  // namespace

cudaError_t launch_kv8_append(const Append8Args& a, int src_dtype, int num_sms,
                              cudaStream_t stream) {
  const moe_kv8_cache& c = a.cache;
  // Tokens whose blocks a CTA takes: one, while the GPU has room for a CTA each.
  // (With the replay that measures it, 7 us: 36 tokens of 8 heads take 9.3 us one to
  // a CTA and 11.4 sixteen, 4747 tokens 83 us one, 46 two, 28 four, 21 sixteen.)
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
  const int row_shift = log2i(c.head_dim / 8), per_row = c.n_kv_heads << row_shift;
  const int rows = per_row < kReadThreads ? kReadThreads / per_row : 1;
  const dim3 grid((unsigned)((a.n - 1) / rows + 1));
  auto* kernel = dtype == MOE_F32    ? kv8_read_kernel<kF32>
                 : dtype == MOE_BF16 ? kv8_read_kernel<kBf16>
                                     : kv8_read_kernel<kFp16>;
  return launch_pdl(kernel, grid, dim3(kReadThreads), 0, stream, a, log2i(c.page_size),
                    log2i(c.block), row_shift);
}

}  // namespace moe
