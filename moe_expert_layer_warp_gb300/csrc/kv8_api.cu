// kv8_api.cu — the extern "C" entry points declared in include/moe_kv8.h:
// argument checks, then one launcher each. Nothing here allocates device
// memory. Every refusal leaves its reason for moe_last_cuda_error_string().
#include <math.h>
#include <stdint.h>

#include "kv8_launch.h"

namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A tensor map's strides are below 2^40 bytes; no GPU holds an array near it.
constexpr int64_t kMaxStride = int64_t(1) << 38;

bool power_of_two(int32_t v) { return v > 0 && (v & (v - 1)) == 0; }

int width(int32_t dtype) { return dtype == MOE_F32 ? 4 : 2; }
bool known(int32_t dtype) { return dtype == MOE_F32 || dtype == MOE_BF16 || dtype == MOE_F16; }

// Whether rows of D elements, tokens and heads with the given strides, do not
// overlap: a token's heads before the next token, or a head's tokens before the
// next head, whatever lies between.
bool rows_apart(int64_t D, int64_t tokens, int64_t heads, int64_t token_stride,
                int64_t head_stride) {
  auto holds = [D](int64_t outer, int64_t inner, int64_t n) {  // n rows `inner` apart
    return outer >= D && (outer - D) / inner >= n - 1;
  };
  return (head_stride >= D && (tokens < 2 || holds(token_stride, head_stride, heads))) ||
         (token_stride >= D && (heads < 2 || holds(head_stride, token_stride, tokens)));
}

// The cache descriptor's reason for a refusal, or null.
const char* cache_fault(const moe_kv8_cache* c, moe_status* st) {
  *st = MOE_EINVAL;
  if (!c) return "null cache descriptor";
  if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16))
    return "cache pages null or not 16-byte aligned";
  if (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return "cache scales null or misaligned";
  if (c->n_pages < 1 || c->n_pages > 0x7fffffff) return "n_pages out of range";
  if (c->n_kv_heads < 1 || c->n_kv_heads > 0x7fff || c->head_dim < 1 || c->page_size < 1)
    return "cache sizes out of range";
  if (c->page_stride < 1 || c->token_stride < 1 || c->head_stride < 1 ||
      c->page_stride % 16 != 0 || c->token_stride % 16 != 0 || c->head_stride % 16 != 0)
    return "cache strides must be positive multiples of 16";
  if (c->page_stride >= kMaxStride || c->token_stride >= kMaxStride ||
      c->head_stride >= kMaxStride)
    return "cache stride out of range";
  *st = MOE_EUNSUPPORTED;
  const int32_t p = c->page_size;
  if (!power_of_two(p) || p < 16 || p > 256) return "page_size must be 16, 32, 64, 128 or 256";
  if (!power_of_two(c->block) || c->block < 16 || c->block > p)
    return "block must be a power of two, 16 to page_size";
  if (c->head_dim != 64 && c->head_dim != 128) return "head_dim must be 64 or 128";
  *st = MOE_OK;
  return nullptr;
}

const char* attn_fault(const moe_kv8_cache* c, const moe_attn_desc* a, moe_status* st) {
  if (const char* why = cache_fault(c, st)) return why;
  *st = MOE_EINVAL;
  if (!a) return "null attention descriptor";
  if (a->n_heads < 1 || a->n_heads % c->n_kv_heads != 0)
    return "n_heads must be a multiple of n_kv_heads";
  if (a->window < 0 || a->sinks < 0) return "window and sinks must not be negative";
  if (!(a->scale > 0.f) || !isfinite(a->scale)) return "scale must be finite and positive";
  if (a->n_heads / c->n_kv_heads > 64) {
    *st = MOE_EUNSUPPORTED;
    return "more than 64 query heads per key head";
  }
  *st = MOE_OK;
  return nullptr;
}

// One of moe_rotary's rows: its reason for a refusal, or null.
const char* rows_fault(const moe_rotary_rows* r, int32_t D, int32_t dtype, int32_t n_tokens) {
  if (r->n_heads < 0) return "n_heads out of range";
  if (r->n_heads == 0) return nullptr;
  const int w = width(dtype);
  for (int64_t s : {r->in_token_stride, r->in_head_stride, r->out_token_stride, r->out_head_stride})
    if (s < 0 || s >= kMaxStride || s * w % 16 != 0)
      return "strides must be multiples of 16 bytes";
  if (!rows_apart(D, n_tokens, r->n_heads, r->out_token_stride, r->out_head_stride))
    return "rows of out must not overlap";
  if (r->in == r->out && (r->in_token_stride != r->out_token_stride ||
                          r->in_head_stride != r->out_head_stride))
    return "rows rotated in place need equal strides";
  if (n_tokens > 0 && (!r->in || !r->out || !aligned(r->in, 16) || !aligned(r->out, 16)))
    return "rows null or not 16-byte aligned";
  return nullptr;
}

// moe_attend8 and moe_attend8_padded.
moe_status attend8(const moe_kv8_cache* cache, const moe_attn_desc* attn, int32_t dtype,
                   const void* q, int64_t q_token_stride, int64_t q_head_stride, int32_t n_tokens,
                   const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table,
                   int32_t max_blocks, int32_t n_requests, void* workspace, size_t workspace_bytes,
                   void* out, int64_t out_token_stride, int64_t out_head_stride, void* stream,
                   const char* fn, bool padded) {
  moe_status st;
  if (const char* why = attn_fault(cache, attn, &st)) return moe::refuse(st, fn, why);
  auto bad = [&](const char* why) { return moe::refuse(MOE_EINVAL, fn, why); };
  if (dtype != MOE_BF16 && dtype != MOE_F16) return bad("q and out must be bf16 or fp16");
  if (n_requests < 1 || n_requests > MOE_MAX_REQUESTS) return bad("n_requests out of range");
  if (n_tokens < 0 || max_blocks < 1) return bad("n_tokens or max_blocks out of range");
  if (q_token_stride < 1 || q_head_stride < 1 || q_token_stride % 8 != 0 ||
      q_head_stride % 8 != 0 || q_token_stride >= kMaxStride || q_head_stride >= kMaxStride)
    return bad("q strides must be positive multiples of 8 elements");
  if (out_token_stride % 8 != 0 || out_head_stride % 8 != 0 ||
      !rows_apart(cache->head_dim, n_tokens, attn->n_heads, out_token_stride, out_head_stride))
    return bad("out strides must be multiples of 8 elements and rows must not overlap");
  if (n_tokens == 0) return MOE_OK;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16))
    return bad("q or out null or not 16-byte aligned");
  if (!q_start || !kv_len || !block_table || !aligned(q_start, 4) || !aligned(kv_len, 4) ||
      !aligned(block_table, 4))
    return bad("q_start, kv_len or block_table null or misaligned");
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < moe::attend8_workspace_bytes(cache->head_dim))
    return bad("workspace null, not 256-byte aligned or too small");
  // a window beyond the longest cache is one of its length
  const int window = attn->window < MOE_MAX_CACHE_LEN ? attn->window : MOE_MAX_CACHE_LEN;
  int sms;
  moe::Attend8Args a = {*cache, dtype == MOE_F16 ? 1 : 0, attn->n_heads,
                        attn->n_heads / cache->n_kv_heads, window,
                        attn->window > 0 ? attn->sinks : 0, attn->scale, q, q_token_stride,
                        q_head_stride, n_tokens, n_requests, max_blocks, q_start, kv_len,
                        block_table, out, out_token_stride, out_head_stride, padded ? 1 : 0,
                        workspace, nullptr};
  st = moe::call_device(&sms, &a.err);
  if (st != MOE_OK) return st;
  const cudaError_t e = moe::launch_attend8(a, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : moe::fail_cuda(e, fn);
}

}  // namespace

extern "C" {

moe_status moe_rotary_turns(const double* radians, int32_t n, uint64_t* turns) {
  const char* fn = "moe_rotary_turns";
  if (n < 0 || (n > 0 && (!radians || !turns)))
    return moe::refuse(MOE_EINVAL, fn, "n out of range or null array");
  // 1/2π in two doubles, and the product with it in two
  const double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  for (int32_t i = 0; i < n; ++i) {
    const double f = fabs(radians[i]);
    if (!(f <= 0x1p40))
      return moe::refuse(MOE_EINVAL, fn, "angles must be finite, at most 2^40 in size");
    const double p = f * hi, e = fma(f, hi, -p) + f * lo;
    // the fraction of a turn: p's own exactly, as two 32-bit halves (the rest's
    // share is rounded), then e
    const double frac = p - floor(p), top = floor(frac * 0x1p32);
    const double rest = (frac * 0x1p32 - top) * 0x1p32;
    const uint64_t v = ((uint64_t)top << 32) + (uint64_t)(int64_t)llround(rest) +
                       (uint64_t)(int64_t)llround(e * 0x1p64);
    turns[i] = radians[i] < 0 ? 0 - v : v;
  }
  return MOE_OK;
}

moe_status moe_rotary(const moe_rotary_desc* d, int32_t dtype, const moe_rotary_rows* q,
                      const moe_rotary_rows* k, const int32_t* positions, int32_t n_tokens,
                      void* stream) {
  const char* fn = "moe_rotary";
  auto bad = [&](const char* why) { return moe::refuse(MOE_EINVAL, fn, why); };
  if (!d) return bad("null rotary descriptor");
  if (d->head_dim < 16 || d->n_rotated < 16 || d->first < 0 ||
      d->first > d->head_dim - d->n_rotated)
    return bad("the rotated columns must lie within a head");
  if (d->interleaved != 0 && d->interleaved != 1) return bad("interleaved must be 0 or 1");
  if (!isfinite(d->amplitude)) return bad("amplitude must be finite");
  if (!d->turns || !aligned(d->turns, 8)) return bad("turns null or misaligned");
  if (!known(dtype)) return bad("unknown type");
  if (n_tokens < 0) return bad("n_tokens out of range");
  if (d->head_dim % 16 != 0 || d->head_dim > 1024 || d->n_rotated % 16 != 0 || d->first % 8 != 0)
    return moe::refuse(MOE_EUNSUPPORTED, fn,
                       "head_dim and n_rotated must be multiples of 16, at most 1024, first one "
                       "of 8");
  moe::RotaryArgs a = {*d, {{}, {}}, positions, n_tokens};
  const moe_rotary_rows* rows[2] = {q, k};
  int64_t heads = 0;
  for (int i = 0; i < 2; ++i) {
    if (!rows[i]) continue;
    if (const char* why = rows_fault(rows[i], d->head_dim, dtype, n_tokens)) return bad(why);
    a.rows[i] = *rows[i];
    heads += rows[i]->n_heads;
  }
  if (heads > 0x7fff) return bad("n_heads out of range");
  if (n_tokens == 0 || heads == 0) return MOE_OK;
  if (!positions || !aligned(positions, 4)) return bad("positions null or misaligned");
  const moe_rotary_rows &x = a.rows[0], &y = a.rows[1];
  if (x.n_heads > 0 && y.n_heads > 0 &&
      (x.out == y.out || (x.out == y.in && x.out != x.in) || (y.out == x.in && y.out != y.in)))
    return bad("rows of q and k must not share memory that is written");
  int sms;
  unsigned int* err;
  const moe_status st = moe::call_device(&sms, &err);
  if (st != MOE_OK) return st;
  const cudaError_t e = moe::launch_rotary(a, dtype, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : moe::fail_cuda(e, "moe_rotary launch");
}

moe_status moe_kv8_append(const moe_kv8_cache* cache, const void* k, const void* v,
                          int32_t src_dtype, int64_t token_stride, int64_t head_stride,
                          int32_t n_tokens, const int64_t* slots, void* stream) {
  const char* fn = "moe_kv8_append";
  moe_status st;
  if (const char* why = cache_fault(cache, &st)) return moe::refuse(st, fn, why);
  auto bad = [&](const char* why) { return moe::refuse(MOE_EINVAL, fn, why); };
  if (n_tokens < 0) return bad("n_tokens out of range");
  if (!known(src_dtype)) return bad("unknown source type");
  const int w = width(src_dtype);
  if (token_stride < 0 || head_stride < 0 || token_stride >= kMaxStride ||
      head_stride >= kMaxStride || token_stride * w % 16 != 0 || head_stride * w % 16 != 0)
    return bad("source strides must be multiples of 16 bytes");
  if (n_tokens == 0) return MOE_OK;
  if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8))
    return bad("k, v or slots null or misaligned");
  if (cache->k == cache->v || cache->k_scale == cache->v_scale)
    return bad("the cache's keys and values share memory");
  int sms;
  moe::Append8Args a = {*cache, k, v, token_stride, head_stride, n_tokens, slots, nullptr};
  st = moe::call_device(&sms, &a.err);
  if (st != MOE_OK) return st;
  const cudaError_t e =
      moe::launch_kv8_append(a, src_dtype, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : moe::fail_cuda(e, "moe_kv8_append launch");
}

moe_status moe_kv8_read(const moe_kv8_cache* cache, const int64_t* slots, int32_t n,
                        int32_t dtype, void* k, void* v, int64_t token_stride, int64_t head_stride,
                        void* stream) {
  const char* fn = "moe_kv8_read";
  moe_status st;
  if (const char* why = cache_fault(cache, &st)) return moe::refuse(st, fn, why);
  auto bad = [&](const char* why) { return moe::refuse(MOE_EINVAL, fn, why); };
  if (n < 0) return bad("n out of range");
  if (!known(dtype)) return bad("unknown type");
  const int w = width(dtype);
  if (token_stride < 0 || head_stride < 0 || token_stride >= kMaxStride ||
      head_stride >= kMaxStride || token_stride * w % 16 != 0 || head_stride * w % 16 != 0 ||
      !rows_apart(cache->head_dim, n, cache->n_kv_heads, token_stride, head_stride))
    return bad("strides must be multiples of 16 bytes and rows must not overlap");
  if (n == 0) return MOE_OK;
  if (!k || !v || k == v || !slots || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8))
    return bad("k, v or slots null, the same or misaligned");
  int sms;
  moe::Read8Args a = {*cache, slots, n, k, v, token_stride, head_stride, nullptr};
  st = moe::call_device(&sms, &a.err);
  if (st != MOE_OK) return st;
  const cudaError_t e = moe::launch_kv8_read(a, dtype, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : moe::fail_cuda(e, "moe_kv8_read launch");
}

size_t moe_attend8_workspace_bytes(const moe_kv8_cache* cache, const moe_attn_desc* attn) {
  moe_status st;
  if (attn_fault(cache, attn, &st)) return 0;
  return moe::attend8_workspace_bytes(cache->head_dim);
}

moe_status moe_attend8(const moe_kv8_cache* cache, const moe_attn_desc* attn, int32_t dtype,
                       const void* q, int64_t q_token_stride, int64_t q_head_stride,
                       int32_t n_tokens, const int32_t* q_start, const int32_t* kv_len,
                       const int32_t* block_table, int32_t max_blocks, int32_t n_requests,
                       void* workspace, size_t workspace_bytes, void* out,
                       int64_t out_token_stride, int64_t out_head_stride, void* stream) {
  return attend8(cache, attn, dtype, q, q_token_stride, q_head_stride, n_tokens, q_start, kv_len,
                 block_table, max_blocks, n_requests, workspace, workspace_bytes, out,
                 out_token_stride, out_head_stride, stream, "moe_attend8", false);
}

moe_status moe_attend8_padded(const moe_kv8_cache* cache, const moe_attn_desc* attn, int32_t dtype,
                              const void* q, int64_t q_token_stride, int64_t q_head_stride,
                              int32_t n_tokens, const int32_t* q_start, const int32_t* kv_len,
                              const int32_t* block_table, int32_t max_blocks, int32_t n_requests,
                              void* workspace, size_t workspace_bytes, void* out,
                              int64_t out_token_stride, int64_t out_head_stride, void* stream) {
  return attend8(cache, attn, dtype, q, q_token_stride, q_head_stride, n_tokens, q_start, kv_len,
                 block_table, max_blocks, n_requests, workspace, workspace_bytes, out,
                 out_token_stride, out_head_stride, stream, "moe_attend8_padded", true);
}

}  // extern "C"
