/*
 * moe_batch.h — C ABI of libmoewarp.so, second part: what surrounds the MoE
 * layer when one step verifies the passes of several requests at once, on
 * one GB300 (sm_103a). In the order a decoder block calls them:
 *   moe_plan_batch     block tables, slots and positions from request lengths
 *   moe_kv_append      the pass's keys and values into a paged cache
 *   moe_attend         every new token's attention over that cache
 *                      (moe_attend_padded: and zeros for rows of no request)
 *   moe_route_grouped  experts from router logits: softmax or sigmoid scores,
 *                      balance bias, groups, top-k, renormalised weights
 * and then moe_build_union, an expert engine and moe_combine of moe_warp.h. One
 * expert pass takes MOE_MAX_TOKENS tokens and MOE_MAX_PAIRS (token, expert)
 * pairs at most (128 and 512: 64 tokens at top 8), far fewer than one call
 * here may hold. A larger step goes through the experts in several passes over
 * slices of moe_route_grouped's rows, which the caller cuts.
 *
 * A verification pass of a request is its n = γ+1 newest tokens; a prompt
 * that enters in chunks is, for these calls, a longer pass of the same kind.
 * The new tokens of all requests are packed one request after the other:
 * request b owns rows q_start[b] .. q_start[b+1]-1 of every [n_tokens] array.
 *
 * Conventions
 *   - The descriptors are host structs, read during the call only; every
 *     other pointer is a DEVICE pointer. The caller owns all memory, and the
 *     library allocates none.
 *   - Every call is asynchronous on `stream` (a cudaStream_t), captures into
 *     a CUDA graph, and never synchronises. Request lengths are read on the
 *     device only.
 *   - Arguments are checked on the host before any launch: MOE_EINVAL for a
 *     bad one, MOE_EUNSUPPORTED for a valid shape that no kernel covers,
 *     MOE_ECUDA for a failed launch; moe_last_cuda_error_string() says what
 *     was wrong. Values that only the device sees (lengths, pages, slots) are
 *     checked there: a bad one is reported through moe_last_device_error
 *     (MOE_EDEVICE), and nothing is read or written out of range for it.
 *   - Outputs must not overlap inputs unless the argument says so.
 *   - Strides count elements. Rows of head_dim elements are contiguous.
 *   - These calls have no gradients: the library serves.
 */
#ifndef MOE_BATCH_H
#define MOE_BATCH_H

#include "moe_warp.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_MAX_REQUESTS 1024   /* requests per call */
#define MOE_MAX_GROUPS 32       /* expert groups */
#define MOE_MAX_HEAD_GROUP 128  /* query heads per key head */
#define MOE_MAX_CACHE_LEN 2147483391 /* kv_len of moe_attend: 2^31 − 257, so that tile ends fit */

/* Element types of the calls below (the first two are moe_wdtype's values). */
typedef enum { MOE_F32 = 0, MOE_BF16 = 1, MOE_F16 = 2 } moe_dtype;

/* ------------------------------------------------------------------ plan --
 * The requests of one step and the pages they hold. A request's cache
 * position p lives in page block_table[b][p / page_size], row p % page_size. */
typedef struct {
  int32_t n_requests;        /* B, 1 .. MOE_MAX_REQUESTS */
  int32_t max_blocks;        /* columns of block_table */
  int32_t page_size;         /* tokens per page: 16, 32, 64, 128 or 256 */
  int32_t free_capacity;     /* entries of free_pages */
  const int32_t* q_len;      /* [B] new tokens of each request (0 allowed) */
  const int32_t* cached;     /* [B] tokens already in its cache */
  const int32_t* held;       /* [B] pages it holds: the valid entries of its table row */
  const int32_t* free_pages; /* [free_capacity] page ids */
  const int32_t* free_range; /* [2] {head, end}: free_pages[head .. end-1] may be taken */
  int32_t* block_table;      /* [B][max_blocks] in/out: entries from held[b] on are written */
  int32_t* q_start;          /* [B+1] out: first packed row of each request; [B] the total */
  int32_t* kv_len;           /* [B] out: cached + q_len, or 0 for a refused request */
  int32_t* held_out;         /* [B] out: pages held now (must not be `held`) */
  int32_t* free_head;        /* [1] out: head + pages taken (must not be in free_range) */
} moe_batch;

/* Gives every request the pages its new tokens need and maps every token:
 *   need_b = max(0, ceil((cached_b + q_b) / page_size) − held_b),
 * taken from the free list in request order: request b's first new page is
 * free_pages[head + Σ_{a<b} need_a]. Pages held for drafted tokens that a
 * verifier turned down are used again. A request is refused when the pages
 * up to and including its own run past `end`, or when it does not fit
 * max_blocks (it then counts no need); one that needs no new page is never
 * refused for want of pages. A refused request takes no pages, its kv_len is
 * 0, its tokens' slots are −1.
 *   n_tokens  rows of slots and positions, ≥ Σ q_len (more is padding; with
 *             fewer, the tokens beyond are dropped and reported).
 *   slots     [n_tokens] int64 out: page · page_size + row, −1 for tokens of
 *             refused requests and for padding.
 *   positions [n_tokens] int32 out: cached_b + i of each new token, −1 for
 *             padding.
 * The call does not change its inputs except table entries from held[b] on,
 * so calling it again gives the same result. Deterministic.               */
moe_status moe_plan_batch(const moe_batch* batch, int32_t n_tokens, int64_t* slots,
                          int32_t* positions, void* stream);

/* ----------------------------------------------------------------- cache --
 * A pool of pages of keys and one of values with the same layout: element
 * (page, row, head, i) is at page·page_stride + row·token_stride +
 * head·head_stride + i. Strides are multiples of 8 elements, base pointers
 * 16-byte aligned; both [page][row][head] and [page][head][row] orders fit.  */
typedef struct {
  void* k;
  void* v;
  int64_t n_pages;
  int32_t page_size;         /* 16, 32, 64, 128 or 256 */
  int32_t n_kv_heads;
  int32_t head_dim;          /* 64 or 128 */
  int32_t dtype;             /* MOE_BF16 or MOE_F16 */
  int64_t page_stride, token_stride, head_stride;
} moe_kv_cache;

/* Writes n_tokens new keys and values to their slots, rounding to the cache's
 * type once (to nearest even).
 *   k, v      [n_tokens][n_kv_heads][head_dim] with the given token and head
 *             strides (shared by both; multiples of 16 bytes), of type
 *             src_dtype: the cache's own or MOE_F32.
 *   slots     [n_tokens] int64, as moe_plan_batch writes them; −1 skips a
 *             token. Two tokens must not share a slot.                      */
moe_status moe_kv_append(const moe_kv_cache* cache, const void* k, const void* v,
                         int32_t src_dtype, int64_t token_stride, int64_t head_stride,
                         int32_t n_tokens, const int64_t* slots, void* stream);

/* ------------------------------------------------------------- attention --*/
typedef struct {
  int32_t n_heads; /* query heads, a multiple of n_kv_heads: head h reads key head
                      h / (n_heads / n_kv_heads) */
  int32_t window;  /* 0: all earlier keys; W > 0: the W newest, the token's own included
                      (any W up to 2^31 − 1) */
  int32_t sinks;   /* with a window: this many first keys of the request stay visible */
  float scale;     /* of the products q·k; finite, > 0 */
} moe_attn_desc;

/* Bytes of scratch moe_attend needs (0 on invalid arguments). It depends on
 * the descriptors alone; 256-byte aligned, not initialised, reusable by
 * consecutive calls on one stream, not shared by calls that overlap.        */
size_t moe_attend_workspace_bytes(const moe_kv_cache* cache, const moe_attn_desc* attn);

/* out_i = Σ_j softmax_j(scale · q_i·k_j) · v_j over the keys token i sees:
 * token i of request b is at position p = kv_len[b] − q_len_b + i, q_len_b =
 * q_start[b+1] − q_start[b], and sees keys j ≤ p, with a window only those
 * with p − j < window or j < sinks. A token that sees no key (kv_len 0, or
 * shorter than the pass) gets zeros, one with NaN among its scores NaN. The
 * keys and values of the new tokens themselves are read from the cache: append
 * them first.
 *   q         [n_tokens][n_heads][head_dim] of the cache's type, strides
 *             positive multiples of 8, 16-byte aligned.
 *   q_start   [n_requests+1], kv_len [n_requests] (each ≤ MOE_MAX_CACHE_LEN),
 *             block_table [n_requests][max_blocks]: as moe_plan_batch writes
 *             them.
 *   out       same shape and type, with its own strides (multiples of 8,
 *             16-byte aligned). Rows of no request are not written.
 * Table entries of pages that hold no key any new token of the request sees
 * are not read, and what lies in the cache at a position that a token does not
 * see (beyond kv_len, a later token's, behind the window) has no effect on it,
 * NaN and infinities included.
 * Scores, softmax statistics and sums are fp32; softmax weights are rounded
 * to the cache's type before the product with v. Deterministic for the batch:
 * the same inputs give the same bits. Keys are cut among the SMs by all
 * requests' lengths, so a request's last bits may change with its neighbours'.
 */
moe_status moe_attend(const moe_kv_cache* cache, const moe_attn_desc* attn, const void* q,
                      int64_t q_token_stride, int64_t q_head_stride, int32_t n_tokens,
                      const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table,
                      int32_t max_blocks, int32_t n_requests, void* workspace,
                      size_t workspace_bytes, void* out, int64_t out_token_stride,
                      int64_t out_head_stride, void* stream);

/* moe_attend for batches padded to a fixed number of tokens: rows of `out` that
 * belong to no request (those from q_start[n_requests] on) are written zeros. */
moe_status moe_attend_padded(const moe_kv_cache* cache, const moe_attn_desc* attn, const void* q,
                             int64_t q_token_stride, int64_t q_head_stride, int32_t n_tokens,
                             const int32_t* q_start, const int32_t* kv_len,
                             const int32_t* block_table, int32_t max_blocks, int32_t n_requests,
                             void* workspace, size_t workspace_bytes, void* out,
                             int64_t out_token_stride, int64_t out_head_stride, void* stream);

/* --------------------------------------------------------------- routing --*/
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;

typedef struct {
  int32_t n_experts;  /* E ≤ MOE_MAX_EXPERTS */
  int32_t top_k;      /* k ≤ MOE_MAX_TOPK, ≤ top_groups · (E / n_groups) */
  int32_t n_groups;   /* ≤ MOE_MAX_GROUPS, divides E; experts of a group are consecutive */
  int32_t top_groups; /* groups kept per token, 1 .. n_groups */
  int32_t group_top;  /* 1 or 2: a group's score is the sum of its best 1 or 2 choice scores */
  int32_t score;      /* moe_score */
  int32_t renorm;     /* 1: a token's weights are divided by their sum */
  float scale;        /* multiplies the weights; finite */
} moe_router_desc;

/* Per token, from router logits l_e ("Deep Dive into Mixture of Experts", §5,
 * DeepSeek-style routing sketch, with scores and groups as parameters):
 *   score   s_e = 1/(1+e^−l_e), or the softmax of l over all E experts;
 *   choice  c_e = s_e + bias_e (bias NULL: s_e);
 *   groups  the top_groups groups with the largest sums of their group_top
 *           best choices; then the top_k experts of those groups by choice.
 *           Equal values go to the lower index, in both steps;
 *   weight  s_e (without the bias), divided by the sum over the k kept when
 *           renorm, times scale.
 * A logit of −inf or of its type's lowest finite value masks an expert:
 * score 0, choice −inf; it is kept, with weight 0, only when a token has
 * fewer than k others in its groups. If every kept score is 0 the weights
 * are 0. +inf and NaN logits are not supported (the indices stay in range).
 * The selection is that of exact arithmetic: without a bias experts compare
 * by their logits, and where two choices or group sums lie closer than fp32
 * resolves, they are compared in fp64.
 *   logits    [n][E] of `dtype` (MOE_F32, MOE_BF16, MOE_F16), rows row_stride
 *             apart (row_stride ≥ E), aligned to their type.
 *   bias      [E] fp32 finite, or NULL.
 *   topk_idx  [n][k] out, in descending order of choice (moe_build_union
 *             reads it); topk_w [n][k] fp32 out. n may be 0.                */
moe_status moe_route_grouped(const moe_router_desc* router, const void* logits, int32_t dtype,
                             int64_t row_stride, const float* bias, int32_t n, int32_t* topk_idx,
                             float* topk_w, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BATCH_H */
