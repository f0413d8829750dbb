/*
 * moe_kv8.h — C ABI of libmoewarp.so, third part: a step's keys and queries
 * between projection and attention when the paged cache is held in 8 bits.
 * In the order a decoder block calls them, with moe_plan_batch before and
 * the expert layer behind them:
 *   moe_rotary      rotary positions of the new tokens' queries and keys
 *                   (moe_rotary_turns: its table of frequencies)
 *   moe_kv8_append  their keys and values into a paged cache of 8-bit codes
 *                   with a scale for each block of tokens and head
 *   moe_attend8     every new token's attention over that cache
 *                   (moe_attend8_padded: and zeros for rows of no request)
 *   moe_kv8_read    rows of the cache as the values they stand for
 *
 * The conventions are those of moe_batch.h: host structs are read during the
 * call only, every other pointer is a DEVICE pointer unless the argument says
 * otherwise, calls are asynchronous, capture into a CUDA graph, allocate
 * nothing and never synchronise; arguments are checked on the host, and values
 * that only the device sees there (moe_last_device_error). No gradients.
 */
#ifndef MOE_KV8_H
#define MOE_KV8_H

#include "moe_batch.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- rotary --*/
typedef struct {
  int32_t head_dim;      /* D, a multiple of 16, at most 1024 */
  int32_t n_rotated;     /* r ≤ D columns of every head are rotated, a multiple of 16 */
  int32_t first;         /* the first of them, a multiple of 8, first + r ≤ D */
  int32_t interleaved;   /* 0: columns i and i + r/2 of them are a pair; 1: 2i and 2i + 1 */
  float amplitude;       /* multiplies rotated columns (long contexts' scaling; else 1); finite */
  const uint64_t* turns; /* [r/2] angle per position of pair i, in 2^-64 turns (moe_rotary_turns) */
} moe_rotary_desc;

/* Rows [n_tokens][n_heads][head_dim] of queries or keys. in and out: 16-byte
 * aligned, strides (in elements) multiples of 16 bytes; out may be in, with the
 * same strides, and must not overlap it otherwise. Rows of out must not overlap,
 * nor the other call argument's rows. */
typedef struct {
  const void* in;
  void* out;
  int32_t n_heads;
  int64_t in_token_stride, in_head_stride;
  int64_t out_token_stride, out_head_stride;
} moe_rotary_rows;

/* Host to host: turns[i] = radians[i] / 2π as a fraction of 2^64 (rounded to
 * nearest; whole turns drop out), for n finite angles per position. The product
 * with a position is then exact modulo one turn, however far it is.          */
moe_status moe_rotary_turns(const double* radians, int32_t n, uint64_t* turns);

/* Rotates pair (a, b) of a token at position p by θ = p · radians[i]:
 *   (a, b) -> amplitude · (a cos θ − b sin θ, a sin θ + b cos θ)
 * in fp32, rounded once to the rows' type. Columns that are not rotated, and
 * every column of a token whose position is negative (padding), are copied (or
 * left, where out is in).
 *   dtype      of both rows: MOE_F32, MOE_BF16 or MOE_F16.
 *   q, k       either may be NULL, or have no heads.
 *   positions  [n_tokens] int32, as moe_plan_batch writes them.              */
moe_status moe_rotary(const moe_rotary_desc* rotary, int32_t dtype, const moe_rotary_rows* q,
                      const moe_rotary_rows* k, const int32_t* positions, int32_t n_tokens,
                      void* stream);

/* ------------------------------------------------------- cache in 8 bits --
 * Pages of codes (e4m3: sign, 4 bits of exponent, 3 of mantissa, at most ±448,
 * NaN, no infinities) in the layouts of moe_kv_cache, and one fp32 scale for
 * each block of `block` consecutive rows of a page and each head, for keys and
 * for values: an element stands for code · scale. Strides count codes (bytes)
 * and are multiples of 16.                                                  */
typedef struct {
  void* k;
  void* v;
  float* k_scale;        /* [n_pages][n_kv_heads][page_size / block] */
  float* v_scale;
  int64_t n_pages;
  int32_t page_size;     /* 16, 32, 64, 128 or 256 */
  int32_t n_kv_heads;
  int32_t head_dim;      /* 64 or 128 */
  int32_t block;         /* rows of a scale: a power of two, 16 .. page_size */
  int64_t page_stride, token_stride, head_stride;
} moe_kv8_cache;

/* Exponents of the scales that moe_kv8_append writes, and the range in which
 * moe_attend8 takes scales from elsewhere. */
#define MOE_KV8_MIN_EXP (-50)
#define MOE_KV8_MAX_EXP 50

/* Writes n_tokens new keys and values to their slots. For every block that they
 * touch and every head, keys and values apart: with A the largest finite size
 * among the block's new elements and e(A) the smallest exponent with
 * A ≤ 448 · 2^e, kept within [−50, 50], the block's scale becomes
 *   2^e(A)           if a new token stands in the block's first row: the block
 *                    starts anew, what its other rows held is given up;
 *   max(old, 2^e(A)) otherwise; where it grows, the codes of the block's other
 *                    rows are divided by the growth and rounded again.
 * Codes are the quotients by the scale, rounded to nearest even; beyond
 * 448 · 2^50 they are held at ±448. Infinities and NaN become NaN. (A power of
 * two costs nothing: e4m3 has the same relative step at every size, and a scale
 * that grows then changes only codes below 2^-6.)
 *   k, v       as for moe_kv_append, of type src_dtype: MOE_F32, MOE_BF16 or
 *              MOE_F16.
 *   slots      [n_tokens] int64, −1 skips a token. The tokens of one block are
 *              consecutive rows of the call with none between them, skipped ones
 *              neither, as moe_plan_batch orders them (else what the block holds
 *              is not defined), and no two share a slot (where one does, codes
 *              of either may stay).
 *              Rows of a block are first written from its first row on. Keys and
 *              values of the cache do not share memory.                      */
moe_status moe_kv8_append(const moe_kv8_cache* cache, const void* k, const void* v,
                          int32_t src_dtype, int64_t token_stride, int64_t head_stride,
                          int32_t n_tokens, const int64_t* slots, void* stream);

/* Rows of the cache as the values they stand for, rounded to `dtype` (MOE_F32
 * and MOE_BF16 hold them exactly for scales of moe_kv8_append; MOE_F16 may
 * round, or overflow to infinity).
 *   slots      [n] int64; −1 gives zeros. The same slot may stand twice.
 *   k, v       [n][n_kv_heads][head_dim] out, 16-byte aligned, with the given
 *              token and head strides (shared, multiples of 16 bytes, rows do
 *              not overlap).                                                 */
moe_status moe_kv8_read(const moe_kv8_cache* cache, const int64_t* slots, int32_t n,
                        int32_t dtype, void* k, void* v, int64_t token_stride, int64_t head_stride,
                        void* stream);

/* Bytes of scratch moe_attend8 needs (0 on invalid arguments); see
 * moe_attend_workspace_bytes. */
size_t moe_attend8_workspace_bytes(const moe_kv8_cache* cache, const moe_attn_desc* attn);

/* moe_attend over a cache in 8 bits: out_i = Σ_j softmax_j(scale · q_i·k_j) · v_j
 * with k_j and v_j the values that the codes stand for, and with the masks,
 * arguments and promises of moe_attend, but
 *   dtype      MOE_BF16 or MOE_F16: the type of q and out;
 *   n_heads    at most 64 for each key head.
 * Scales of blocks with a visible key lie within [2^-50, 2^50]: others are
 * reported, and read as the nearer end.
 * The codes go to the tensor cores as they are; queries go as sums of two e4m3
 * numbers (bf16) or three (fp16), which hold all bits of a bf16 or fp16 query whose
 * size is within 2^-14 of its row's largest. The products of a softmax weight p_j
 * and its block's value scale vs_j are rounded, to either side alike: off by 2^-9
 * (bf16) or 2^-11 (fp16) of themselves, or by 2^-26 or 2^-32 of the row's largest
 * product where that is more. Sums and statistics are fp32; over n keys the tensor
 * cores' sums are cut by n/32 · 2^-23 of their terms' sizes, as moe_attend's are
 * by n/16. A result is then off by
 *   (2^-9 + n · 2^-28) Σ p_j |v_j| + 2^-26 max_j(p_j vs_j) Σ |code_j|    (bf16)
 *   (2^-11 + n · 2^-28) Σ p_j |v_j| + 2^-32 max_j(p_j vs_j) Σ |code_j|   (fp16)
 * at most, the codes those of the keys that the row sees, beside its scores' errors
 * in fp32 and its own rounding. What the sum's last term says: a block whose scale is
 * far above the others' takes their bits, though its codes be zeros. A query row
 * with NaN or an infinity gives NaN (or zeros, where it sees nothing).         */
moe_status moe_attend8(const moe_kv8_cache* cache, const moe_attn_desc* attn, int32_t dtype,
                       const void* q, int64_t q_token_stride, int64_t q_head_stride,
                       int32_t n_tokens, const int32_t* q_start, const int32_t* kv_len,
                       const int32_t* block_table, int32_t max_blocks, int32_t n_requests,
                       void* workspace, size_t workspace_bytes, void* out,
                       int64_t out_token_stride, int64_t out_head_stride, void* stream);

/* moe_attend8 with zeros written to rows of `out` that belong to no request. */
moe_status moe_attend8_padded(const moe_kv8_cache* cache, const moe_attn_desc* attn, int32_t dtype,
                              const void* q, int64_t q_token_stride, int64_t q_head_stride,
                              int32_t n_tokens, const int32_t* q_start, const int32_t* kv_len,
                              const int32_t* block_table, int32_t max_blocks, int32_t n_requests,
                              void* workspace, size_t workspace_bytes, void* out,
                              int64_t out_token_stride, int64_t out_head_stride, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_KV8_H */
