// batch_api.cu — the extern "C" entry points declared in
// include/moe_batch.h: argument checks, then one launcher each. Nothing here
// allocates device memory. Every refusal leaves its reason for
// moe_last_cuda_error_string().
#include <math.h>
#include <stdint.h>

#include "batch_launch.h"

namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A tensor map's strides are below 2^40 bytes; no GPU holds an array near it.
constexpr int64_t kMaxStride = int64_t(1) << 38;

bool page_size_ok(int32_t p) { return p == 16 || p == 32 || p == 64 || p == 128 || p == 256; }

// The cache descriptor's reason for a refusal, or null.
const char* cache_fault(const moe_kv_cache* c, moe_status* st) {
  *st = MOE_EINVAL;
  if (!c) return "null cache descriptor";
  if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16))
    return "cache pages null or not 16-byte aligned";
  if (c->n_pages < 1 || c->n_pages > 0x7fffffff) return "n_pages out of range";
  if (c->n_kv_heads < 1 || c->head_dim < 1 || c->page_size < 1) return "cache sizes out of range";
  if (c->dtype != MOE_F32 && c->dtype != MOE_BF16 && c->dtype != MOE_F16)
    return "unknown cache type";
  if (c->page_stride < 1 || c->token_stride < 1 || c->head_stride < 1 || c->page_stride % 8 != 0 ||
      c->token_stride % 8 != 0 || c->head_stride % 8 != 0)
    return "cache strides must be positive multiples of 8 elements";
  if (c->page_stride >= kMaxStride || c->token_stride >= kMaxStride ||
      c->head_stride >= kMaxStride)
    return "cache stride out of range";
  *st = MOE_EUNSUPPORTED;
  if (c->dtype == MOE_F32) return "the cache holds bf16 or fp16";
  if (!page_size_ok(c->page_size)) return "page_size must be 16, 32, 64, 128 or 256";
  if (c->head_dim != 64 && c->head_dim != 128) return "head_dim must be 64 or 128";
  *st = MOE_OK;
  return nullptr;
}

const char* attn_fault(const moe_kv_cache* c, const moe_attn_desc* a, moe_status* st) {
  if (const char* why = cache_fault(c, st)) return why;
  *st = MOE_EINVAL;
  if (!a) return "null attention descriptor";
  if (a->n_heads < 1 || a->n_heads % c->n_kv_heads != 0)
    return "n_heads must be a multiple of n_kv_heads";
  if (a->window < 0 || a->sinks < 0) return "window and sinks must not be negative";
  if (!(a->scale > 0.f) || !isfinite(a->scale)) return "scale must be finite and positive";
  if (a->n_heads / c->n_kv_heads > MOE_MAX_HEAD_GROUP) {
    *st = MOE_EUNSUPPORTED;
    return "more than 128 query heads per key head";
  }
  *st = MOE_OK;
  return nullptr;
}

// moe_attend and moe_attend_padded.
moe_status attend(const moe_kv_cache* cache, const moe_attn_desc* attn, const void* q,
                  int64_t q_token_stride, int64_t q_head_stride, int32_t n_tokens,
                  const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table,
                  int32_t max_blocks, int32_t n_requests, void* workspace, size_t workspace_bytes,
                  void* out, int64_t out_token_stride, int64_t out_head_stride, void* stream,
                  const char* fn, bool padded) {
  moe_status st;
  if (const char* why = attn_fault(cache, attn, &st)) return moe::refuse(st, fn, why);
  auto bad = [&](const char* why) { return moe::refuse(MOE_EINVAL, fn, why); };
  if (n_requests < 1 || n_requests > MOE_MAX_REQUESTS) return bad("n_requests out of range");
  if (n_tokens < 0 || max_blocks < 1) return bad("n_tokens or max_blocks out of range");
  if (q_token_stride < 1 || q_head_stride < 1 || q_token_stride % 8 != 0 ||
      q_head_stride % 8 != 0 || q_token_stride >= kMaxStride || q_head_stride >= kMaxStride)
    return bad("q strides must be positive multiples of 8 elements");
  // rows of out must not overlap: a token's heads before the next token, or a
  // head's tokens before the next head, whatever lies between
  const int64_t D = cache->head_dim, H = attn->n_heads;
  auto holds = [D](int64_t outer, int64_t inner, int64_t n) {  // n rows `inner` apart
    return outer >= D && (outer - D) / inner >= n - 1;
  };
  const bool heads_in = out_head_stride >= D &&
                        (n_tokens < 2 || holds(out_token_stride, out_head_stride, H));
  const bool tokens_in = out_token_stride >= D &&
                         (H < 2 || holds(out_head_stride, out_token_stride, n_tokens));
  if (out_token_stride % 8 != 0 || out_head_stride % 8 != 0 || !(heads_in || tokens_in))
    return bad("out strides must be multiples of 8 elements and rows must not overlap");
  if (n_tokens == 0) return MOE_OK;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16))
    return bad("q or out null or not 16-byte aligned");
  if (!q_start || !kv_len || !block_table || !aligned(q_start, 4) || !aligned(kv_len, 4) ||
      !aligned(block_table, 4))
    return bad("q_start, kv_len or block_table null or misaligned");
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < moe::attend_workspace_bytes(cache->head_dim))
    return bad("workspace null, not 256-byte aligned or too small");
  // a window beyond the longest cache is one of its length
  const int window = attn->window < MOE_MAX_CACHE_LEN ? attn->window : MOE_MAX_CACHE_LEN;
  int sms;
  moe::AttendArgs a = {*cache, attn->n_heads, attn->n_heads / cache->n_kv_heads, window,
                       attn->window > 0 ? attn->sinks : 0, attn->scale, q, q_token_stride,
                       q_head_stride, n_tokens, n_requests, max_blocks, q_start, kv_len,
                       block_table, out, out_token_stride, out_head_stride, padded ? 1 : 0, workspace,
                       nullptr};
  st = moe::call_device(&sms, &a.err);
  if (st != MOE_OK) return st;
  const cudaError_t e = moe::launch_attend(a, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : moe::fail_cuda(e, fn);
}

}  // namespace

extern "C" {

moe_status moe_plan_batch(const moe_batch* b, int32_t n_tokens, int64_t* slots,
                          int32_t* positions, void* stream) {
  const char* fn = "moe_plan_batch";
  auto bad = [&](const char* why) { return moe::refuse(MOE_EINVAL, fn, why); };
  if (!b) return bad("null batch");
  if (b->n_requests < 1 || b->n_requests > MOE_MAX_REQUESTS) return bad("n_requests out of range");
  if (b->max_blocks < 1 || b->free_capacity < 0 || n_tokens < 0)
    return bad("max_blocks, free_capacity or n_tokens out of range");
  if (!b->q_len || !b->cached || !b->held || !b->free_range || !b->block_table || !b->q_start ||
      !b->kv_len || !b->held_out || !b->free_head)
    return bad("null array");
  if (b->free_capacity > 0 && !b->free_pages) return bad("null free_pages");
  if (n_tokens > 0 && (!slots || !positions)) return bad("null slots or positions");
  for (const void* p : {(const void*)b->q_len, (const void*)b->cached, (const void*)b->held,
                        (const void*)b->free_pages, (const void*)b->free_range,
                        (const void*)b->block_table, (const void*)b->q_start,
                        (const void*)b->kv_len, (const void*)b->held_out,
                        (const void*)b->free_head, (const void*)positions})
    if (!aligned(p, 4)) return bad("misaligned array");
  if (!aligned(slots, 8)) return bad("misaligned slots");
  if (b->held_out == b->held || b->kv_len == b->cached || b->free_head == b->free_range ||
      b->free_head == b->free_range + 1)
    return bad("an output is one of the inputs");
  if (!page_size_ok(b->page_size))
    return moe::refuse(MOE_EUNSUPPORTED, fn, "page_size must be 16, 32, 64, 128 or 256");
  int sms;
  unsigned int* err;
  const moe_status st = moe::call_device(&sms, &err);
  if (st != MOE_OK) return st;
  const cudaError_t e = moe::launch_plan_batch(*b, n_tokens, slots, positions, err,
                                               static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : moe::fail_cuda(e, "moe_plan_batch launch");
}

moe_status moe_kv_append(const moe_kv_cache* cache, const void* k, const void* v,
                         int32_t src_dtype, int64_t token_stride, int64_t head_stride,
                         int32_t n_tokens, const int64_t* slots, void* stream) {
  const char* fn = "moe_kv_append";
  moe_status st;
  if (const char* why = cache_fault(cache, &st)) return moe::refuse(st, fn, why);
  auto bad = [&](const char* why) { return moe::refuse(MOE_EINVAL, fn, why); };
  if (n_tokens < 0) return bad("n_tokens out of range");
  if (src_dtype != MOE_F32 && src_dtype != cache->dtype)
    return bad("src_dtype must be the cache's type or MOE_F32");
  const int width = src_dtype == MOE_F32 ? 4 : 2;
  if (token_stride < 0 || head_stride < 0 || token_stride * width % 16 != 0 ||
      head_stride * width % 16 != 0)
    return bad("source strides must be multiples of 16 bytes");
  if (n_tokens == 0) return MOE_OK;
  if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8))
    return bad("k, v or slots null or misaligned");
  int sms;
  moe::AppendArgs a = {*cache, k, v, token_stride, head_stride, n_tokens,
                       src_dtype == MOE_F32 ? 1 : 0, slots, nullptr};
  st = moe::call_device(&sms, &a.err);
  if (st != MOE_OK) return st;
  const cudaError_t e = moe::launch_kv_append(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : moe::fail_cuda(e, "moe_kv_append launch");
}

size_t moe_attend_workspace_bytes(const moe_kv_cache* cache, const moe_attn_desc* attn) {
  moe_status st;
  if (attn_fault(cache, attn, &st)) return 0;
  return moe::attend_workspace_bytes(cache->head_dim);
}

moe_status moe_attend(const moe_kv_cache* cache, const moe_attn_desc* attn, const void* q,
                      int64_t q_token_stride, int64_t q_head_stride, int32_t n_tokens,
                      const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table,
                      int32_t max_blocks, int32_t n_requests, void* workspace,
                      size_t workspace_bytes, void* out, int64_t out_token_stride,
                      int64_t out_head_stride, void* stream) {
  return attend(cache, attn, q, q_token_stride, q_head_stride, n_tokens, q_start, kv_len,
                block_table, max_blocks, n_requests, workspace, workspace_bytes, out,
                out_token_stride, out_head_stride, stream, "moe_attend", false);
}

moe_status moe_attend_padded(const moe_kv_cache* cache, const moe_attn_desc* attn, const void* q,
                             int64_t q_token_stride, int64_t q_head_stride, int32_t n_tokens,
                             const int32_t* q_start, const int32_t* kv_len,
                             const int32_t* block_table, int32_t max_blocks, int32_t n_requests,
                             void* workspace, size_t workspace_bytes, void* out,
                             int64_t out_token_stride, int64_t out_head_stride, void* stream) {
  return attend(cache, attn, q, q_token_stride, q_head_stride, n_tokens, q_start, kv_len,
                block_table, max_blocks, n_requests, workspace, workspace_bytes, out,
                out_token_stride, out_head_stride, stream, "moe_attend_padded", true);
}

moe_status moe_route_grouped(const moe_router_desc* r, const void* logits, int32_t dtype,
                             int64_t row_stride, const float* bias, int32_t n, int32_t* topk_idx,
                             float* topk_w, void* stream) {
  const char* fn = "moe_route_grouped";
  auto bad = [&](const char* why) { return moe::refuse(MOE_EINVAL, fn, why); };
  if (!r) return bad("null router descriptor");
  if (r->n_experts < 1 || r->n_experts > MOE_MAX_EXPERTS) return bad("n_experts out of range");
  if (r->n_groups < 1 || r->n_groups > MOE_MAX_GROUPS || r->n_experts % r->n_groups != 0)
    return bad("n_groups must divide n_experts and be at most 32");
  const int size = r->n_experts / r->n_groups;
  if (r->top_groups < 1 || r->top_groups > r->n_groups) return bad("top_groups out of range");
  if (r->group_top < 1 || r->group_top > 2 || r->group_top > size)
    return bad("group_top must be 1 or 2 and at most a group's experts");
  if (r->top_k < 1 || r->top_k > MOE_MAX_TOPK || r->top_k > r->top_groups * size)
    return bad("top_k out of range");
  if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) return bad("unknown score");
  if (r->renorm != 0 && r->renorm != 1) return bad("renorm must be 0 or 1");
  if (!isfinite(r->scale)) return bad("scale must be finite");
  if (dtype != MOE_F32 && dtype != MOE_BF16 && dtype != MOE_F16) return bad("unknown logits type");
  if (n < 0 || row_stride < r->n_experts) return bad("n or row_stride out of range");
  if (n == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w || !aligned(logits, dtype == MOE_F32 ? 4 : 2) ||
      !aligned(bias, 4) || !aligned(topk_idx, 4) || !aligned(topk_w, 4))
    return bad("null or misaligned array");
  int sms;
  unsigned int* err;
  const moe_status st = moe::call_device(&sms, &err);
  if (st != MOE_OK) return st;
  const cudaError_t e = moe::launch_route_grouped(*r, logits, dtype, row_stride, bias, n, topk_idx,
                                                  topk_w, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : moe::fail_cuda(e, "moe_route_grouped launch");
}

}  // extern "C"
