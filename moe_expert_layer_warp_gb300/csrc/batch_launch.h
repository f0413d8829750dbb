// batch_launch.h — host-side launchers of the kernels behind moe_batch.h, and
// what its entry points share with api.cu. Internal to libmoewarp.so:
// batch_api.cu validates arguments, then calls these.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"
#include "moe_batch.h"

namespace moe {

// Defined in api.cu: the current device's SM count and error word, and the
// text behind moe_last_cuda_error_string().
moe_status call_device(int* num_sms, unsigned int** err);
moe_status fail_cuda(cudaError_t e, const char* where);
moe_status refuse(moe_status st, const char* where, const char* why);

cudaError_t launch_plan_batch(const moe_batch& b, int n_tokens, int64_t* slots, int32_t* positions,
                              unsigned int* err, cudaStream_t stream);

struct AppendArgs {
  moe_kv_cache cache;
  const void* k;
  const void* v;
  int64_t token_stride, head_stride;
  int n_tokens;
  int src_f32;  // source fp32, else the cache's type
  const int64_t* slots;
  unsigned int* err;
};
cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream);

struct AttendArgs {
  moe_kv_cache cache;
  int n_heads, group;  // query heads, query heads per key head
  int window, sinks;   // window 0: none
  float scale;
  const void* q;
  int64_t q_token_stride, q_head_stride;
  int n_tokens, n_requests, max_blocks;
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* block_table;
  void* out;
  int64_t out_token_stride, out_head_stride;
  int clear;           // rows of no request become zeros
  void* workspace;
  unsigned int* err;
};
size_t attend_workspace_bytes(int head_dim);
cudaError_t launch_attend(const AttendArgs& a, int num_sms, cudaStream_t stream);

cudaError_t launch_route_grouped(const moe_router_desc& r, const void* logits, int dtype,
                                 int64_t row_stride, const float* bias, int n, int32_t* topk_idx,
                                 float* topk_w, cudaStream_t stream);

}  // namespace moe
