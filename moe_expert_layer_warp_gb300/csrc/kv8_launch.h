// kv8_launch.h — host-side launchers of the kernels behind moe_kv8.h. Internal
// to libmoewarp.so: kv8_api.cu validates arguments, then calls these.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "batch_launch.h"
#include "moe_kv8.h"

namespace moe {

struct RotaryArgs {
  moe_rotary_desc desc;
  moe_rotary_rows rows[2];  // queries and keys; no heads: none
  const int32_t* positions;
  int n_tokens;
};
cudaError_t launch_rotary(const RotaryArgs& a, int dtype, int num_sms, cudaStream_t stream);

struct Append8Args {
  moe_kv8_cache cache;
  const void* k;
  const void* v;
  int64_t token_stride, head_stride;
  int n_tokens;
  const int64_t* slots;
  unsigned int* err;
};
cudaError_t launch_kv8_append(const Append8Args& a, int src_dtype, int num_sms,
                              cudaStream_t stream);

struct Read8Args {
  moe_kv8_cache cache;
  const int64_t* slots;
  int n;
  void* k;
  void* v;
  int64_t token_stride, head_stride;
  unsigned int* err;
};
cudaError_t launch_kv8_read(const Read8Args& a, int dtype, int num_sms, cudaStream_t stream);

struct Attend8Args {
  moe_kv8_cache cache;
  int f16;             // q and out: fp16, else bf16
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
size_t attend8_workspace_bytes(int head_dim);
cudaError_t launch_attend8(const Attend8Args& a, int num_sms, cudaStream_t stream);

}  // namespace moe
