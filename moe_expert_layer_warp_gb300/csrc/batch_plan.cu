// batch_plan.cu — the batch plan (pages, slots and positions of every new
// token, from request lengths) and the append of keys and values to their
// slots.
//
// Plan. With q_b new tokens, c_b cached ones and h_b pages held, request b
// needs n_b = max(0, ceil((c_b + q_b) / page) − h_b) pages, and takes them
// from the free list at head + Σ_{a<b} n_a: everything follows from two
// prefix sums over at most 1024 requests. The work is a few hundred
// kilobytes at most, so a call is bound by its launch and one chain of
// dependent loads. Every CTA therefore redoes the prefix sums for itself,
// which costs less than handing them over through a second launch, and then
// maps its own tokens and fills its own share of the table rows. No CTA reads
// what another writes: a token's page is read from the table only below h_b,
// from the free list otherwise. One request takes 2.6 us of GPU time, 1000
// requests (20 of them prompts in chunks of up to 2048 tokens) 4.1 us; a launch
// alone takes 1.6.
//
// Append. A thread moves 8 elements of one head's row, 16 bytes of the cache:
// with heads of 64 or 128 columns a row is 8 or 16 such pieces, so a warp
// writes whole lines whatever the order of the slots. 12345 tokens of 8 heads
// of 128 columns (fp32 rounded to fp16, 149 MB) take 23.6 us, 6.3 TB/s, 93 % of a
// copy's rate; 36 tokens 1.6 us, the launch.
#include "batch_launch.h"
#include "common.cuh"
#include "round16.cuh"

namespace moe {
namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPerThread = MOE_MAX_REQUESTS / kPlanThreads;

// What a CTA keeps of each request after the prefix sums.
struct PlanRow {
  int cached, held;
  int take;   // index in free_pages of its first new page
  int given;  // pages it gets; −1: refused
};

__global__ void __launch_bounds__(kPlanThreads)
    plan_batch_kernel(moe_batch b, int page_shift, int n_tokens, int64_t* __restrict__ slots,
                      int32_t* __restrict__ positions, unsigned int* err) {
  __shared__ PlanRow row[MOE_MAX_REQUESTS];
  __shared__ int start[MOE_MAX_REQUESTS];
  __shared__ long long part_q[kPlanWarps], part_need[kPlanWarps];
  __shared__ int part_given[kPlanWarps];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = b.n_requests, page = 1 << page_shift;
  // requests tid·kPerThread + i of this thread; the loads go out together
  int q[kPerThread], cached[kPerThread], held[kPerThread];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int r = tid * kPerThread + i;
    q[i] = r < B ? b.q_len[r] : 0;
    cached[i] = r < B ? b.cached[r] : 0;
    held[i] = r < B ? b.held[r] : 0;
  }
  long long head = b.free_range[0], end = b.free_range[1];
  bool bad = head < 0 || end > b.free_capacity;
  head = max(head, 0ll);
  end = min(end, (long long)b.free_capacity);
  int need[kPerThread];
  bool fits[kPerThread];
  long long sq = 0, sn = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    if ((q[i] | cached[i] | held[i]) < 0) {
      bad = true;
      q[i] = max(q[i], 0);
      cached[i] = max(cached[i], 0);
      held[i] = max(held[i], 0);
    }
    const long long total = (long long)cached[i] + q[i];
    const long long blocks = (total + page - 1) >> page_shift;
    fits[i] = blocks <= b.max_blocks && total <= 0x7fffffff;
    need[i] = fits[i] ? max(0, (int)blocks - held[i]) : 0;
    sq += q[i];
    sn += need[i];
  }
  // exclusive prefix sums of tokens and needed pages: in the warp, then over
  // the warps
  long long iq = sq, in = sn;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long tq = __shfl_up_sync(0xffffffffu, iq, o);
    const long long tn = __shfl_up_sync(0xffffffffu, in, o);
    if (lane >= o) {
      iq += tq;
      in += tn;
    }
  }
  if (lane == 31) {
    part_q[warp] = iq;
    part_need[warp] = in;
  }
  __syncthreads();
  long long q0 = iq - sq, n0 = in - sn, total_q = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) {
    if (w < warp) {
      q0 += part_q[w];
      n0 += part_need[w];
    }
    total_q += part_q[w];
  }
  const bool writer = blockIdx.x == 0;
  int given_sum = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int r = tid * kPerThread + i;
    const bool ok = fits[i] && (need[i] == 0 || head + n0 + need[i] <= end);
    const int given = ok ? need[i] : -1;
    const int first = (int)min(q0, 0x7fffffffll);
    if (r < B) {
      row[r] = PlanRow{cached[i], held[i], ok ? (int)(head + n0) : 0, given};
      start[r] = first;
      if (writer) {
        b.q_start[r] = first;
        b.kv_len[r] = ok ? cached[i] + q[i] : 0;
        b.held_out[r] = held[i] + (ok ? need[i] : 0);
      }
    } else {
      start[r] = 0x7fffffff;  // past every token
    }
    given_sum += ok ? need[i] : 0;
    q0 += q[i];
    n0 += need[i];
  }
  if (writer) {
    given_sum = __reduce_add_sync(0xffffffffu, given_sum);
    if (lane == 0) part_given[warp] = given_sum;
    if (total_q > n_tokens) bad = true;
    if (bad) report_error(err, ERR_CHECK, 0xA00);
  }
  __syncthreads();
  const int total = (int)min(total_q, 0x7fffffffll);
  if (writer && tid == 0) {
    int g = 0;
    for (int w = 0; w < kPlanWarps; ++w) g += part_given[w];
    *b.free_head = (int)head + g;
    b.q_start[B] = total;
  }
  // new table entries, a warp per request
  for (int r = blockIdx.x * kPlanWarps + warp; r < B; r += gridDim.x * kPlanWarps) {
    const PlanRow p = row[r];
    int32_t* dst = b.block_table + (size_t)r * b.max_blocks + p.held;
    for (int i = lane; i < p.given; i += 32) dst[i] = b.free_pages[p.take + i];
  }
  // slots and positions, a thread per token (64 bits: a step of the grid from a t
  // near 2^31 passes 32)
  for (int64_t at0 = blockIdx.x * kPlanThreads + tid; at0 < n_tokens;
       at0 += gridDim.x * kPlanThreads) {
    const int t = (int)at0;
    int64_t slot = -1;
    int pos = -1;
    if (t < total) {
      int r = 0;  // the last request that starts at or before t
#pragma unroll
      for (int step = MOE_MAX_REQUESTS / 2; step > 0; step >>= 1)
        if (start[r + step] <= t) r += step;
      const PlanRow p = row[r];
      const int at = t - start[r];
      // a refused request's positions may pass 32 bits; they are not used
      pos = (int)min((long long)p.cached + at, 0x7fffffffll);
      if (p.given >= 0) {
        const int block = pos >> page_shift;
        const int pg = block < p.held ? b.block_table[(size_t)r * b.max_blocks + block]
                                      : b.free_pages[p.take + block - p.held];
        if (pg >= 0) {
          slot = ((int64_t)pg << page_shift) + (pos & (page - 1));
        } else {
          report_error(err, ERR_CHECK, 0xA01);
        }
      }
    }
    slots[t] = slot;
    positions[t] = pos;
  }
}

// ---------------------------------------------------------------- append --
// A copy bound by memory: one thread per 8 elements (16 bytes of the cache),
// keys and values in one launch.
constexpr int kAppendThreads = 256;

template <bool kSrcF32, bool kF16>
__global__ void __launch_bounds__(kAppendThreads)
    kv_append_kernel(const __grid_constant__ AppendArgs a, int page_shift, int chunk_shift) {
  pdl_wait();
  pdl_trigger();
  const moe_kv_cache& c = a.cache;
  const int per_head = 1 << chunk_shift;  // chunks of one head's row
  const int per_row = c.n_kv_heads << chunk_shift;
  const int64_t n = (int64_t)a.n_tokens * per_row;
  const int64_t n_slots = c.n_pages << page_shift;
  const void* src = blockIdx.y ? a.v : a.k;
  void* dst = blockIdx.y ? c.v : c.k;
  for (int64_t i = (int64_t)blockIdx.x * kAppendThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kAppendThreads) {
    const int t = (int)(i / per_row);
    const int j = (int)(i - (int64_t)t * per_row);
    const int h = j >> chunk_shift, e = (j & (per_head - 1)) * 8;
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= n_slots) {
      if (slot != -1) report_error(a.err, ERR_CHECK, 0xA10);
      continue;
    }
    const int64_t from = t * a.token_stride + h * a.head_stride + e;
    const int64_t to = (slot >> page_shift) * c.page_stride +
                       (slot & ((1 << page_shift) - 1)) * c.token_stride + h * c.head_stride + e;
    uint4 v;
    if constexpr (kSrcF32) {
      const float4 lo = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(src) + from));
      const float4 hi =
          __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(src) + from) + 1);
      v = make_uint4(round16<kF16>(lo.x, lo.y), round16<kF16>(lo.z, lo.w),
                     round16<kF16>(hi.x, hi.y), round16<kF16>(hi.z, hi.w));
    } else {
      v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + from));
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + to) = v;
  }
}

int log2i(int v) { return 31 - __builtin_clz(v); }

}  // namespace

cudaError_t launch_plan_batch(const moe_batch& b, int n_tokens, int64_t* slots, int32_t* positions,
                              unsigned int* err, cudaStream_t stream) {
  // a CTA per 256 tokens; the grid of a long batch stops at two CTAs per SM
  const int ctas = n_tokens > 0 ? (n_tokens - 1) / kPlanThreads + 1 : 1;
  return launch_pdl(plan_batch_kernel, dim3(ctas < 304 ? ctas : 304), dim3(kPlanThreads), 0, stream,
                    b, log2i(b.page_size), n_tokens, slots, positions, err);
}

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream) {
  const int chunk_shift = log2i(a.cache.head_dim / 8);
  const int64_t n = ((int64_t)a.n_tokens * a.cache.n_kv_heads) << chunk_shift;
  const int64_t ctas = (n + kAppendThreads - 1) / kAppendThreads;
  const dim3 grid((unsigned)(ctas < 152 * 32 ? ctas : 152 * 32), 2);
  const int page_shift = log2i(a.cache.page_size);
  const bool f16 = a.cache.dtype == MOE_F16;
  auto* kernel = a.src_f32 ? (f16 ? kv_append_kernel<true, true> : kv_append_kernel<true, false>)
                           : kv_append_kernel<false, false>;  // a copy: no type matters
  return launch_pdl(kernel, grid, dim3(kAppendThreads), 0, stream, a, page_shift, chunk_shift);
}

}  // namespace moe
