/*
 * spear_serve.h -- C ABI of the serving operators that run beside the W4
 * linear layer of spear_w4ec.h on MI355X (gfx950):
 *
 *   - a paged key/value cache in fp16 or 8 bits: writing new tokens
 *     (quantising them on the way) and reading sequences back;
 *   - attention of new tokens over that cache: one token a sequence (decode),
 *     a few drafted ones, or a prompt's chunk, in one ragged batch;
 *   - verification of drafted tokens against the target's probabilities from
 *     random numbers that the caller gives.
 *
 * The conventions of spear_w4ec.h hold: tensors are device pointers owned by
 * the caller and borrowed until the work enqueued on `stream` (a hipStream_t,
 * NULL = the null stream) completes; nothing is allocated, freed or
 * synchronized; argument checks come before anything is enqueued and return a
 * spear_status_t; no C++ exception crosses this interface; functions are
 * reentrant.  All of them can be captured into a HIP graph.
 *
 * The cache.  Pages [num_pages][kv_heads][page_size][head_dim] for the keys
 * and the same for the values, contiguous, 16-byte aligned: one head's tokens
 * of a page are one run of memory.  Token i of a sequence lies in page
 * block_table[b][i / page_size], place i % page_size; its slot is
 * page * page_size + place.  dtype SPEAR_KV_FP16 holds fp16.  SPEAR_KV_INT8
 * holds int8 codes with one fp32 scale per token and head in
 * [num_pages][kv_heads][page_size]:
 *     s = max|x| / 127 over the head's head_dim values, code = rint(x / s)
 * (float32 divisions, ties to even; 0 where s = 0), standing for code * s.  A
 * row that holds an infinity or NaN gets the scale infinity or NaN and reads
 * back without a finite value.
 *
 * Memory safety against device data the host cannot check: lengths and offsets
 * are clamped to the tensors' bounds, page numbers outside [0, num_pages) are
 * read as the last page, slots outside the cache are not written.  With offsets
 * that do not rise, a row that comes before its sequence's first is read back as
 * zeros, and an attention call so large that the rows they repeat could pass its
 * 32-bit counts computes nothing.
 */
#ifndef SPEAR_SERVE_H
#define SPEAR_SERVE_H

#include "spear_w4ec.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum spear_kv_dtype {
  SPEAR_KV_FP16 = 0,
  SPEAR_KV_INT8 = 1
} spear_kv_dtype_t;

/* Shape of a paged cache. */
typedef struct spear_kv_desc {
  int32_t dtype;      /* spear_kv_dtype_t */
  int32_t num_pages;  /* >= 1 */
  int32_t kv_heads;   /* >= 1 */
  int32_t head_dim;   /* 64 or 128 */
  int32_t page_size;  /* a power of two, 16 to 1024 */
} spear_kv_desc_t;

/*
 * spear_kv_append -- write new tokens' keys and values into the cache.
 *   k, v     fp16 [tokens][kv_heads][head_dim], 16-byte aligned, the last
 *            dimension contiguous; strides of the first two in elements
 *            (multiples of 8), so they may be parts of a joint projection's
 *            output.
 *   slots    int64 [tokens]; a slot outside [0, num_pages * page_size) writes
 *            nothing (-1 for padding).  Two tokens with the same slot race.
 *   k_scale, v_scale  fp32, written beside the codes (SPEAR_KV_INT8; may be
 *            NULL for SPEAR_KV_FP16).
 * tokens = 0 does nothing; tokens * kv_heads may be up to 2^27.
 * Errors: NULL_POINTER, INVALID_SHAPE (sizes, strides not multiples of 8),
 *         UNSUPPORTED (head_dim, page_size, size), INVALID_ARGUMENT (dtype),
 *         MISALIGNED, HIP.
 */
spear_status_t spear_kv_append(const spear_kv_desc_t* kv, int32_t tokens, const void* k, int64_t k_token_stride,
                               int64_t k_head_stride, const void* v, int64_t v_token_stride,
                               int64_t v_head_stride, const int64_t* slots, void* k_cache, void* v_cache,
                               float* k_scale, float* v_scale, void* stream);

/*
 * spear_kv_gather -- read whole sequences back in fp16.
 *   block_table  int32 [batch][table_stride], entries of a sequence's pages in
 *            order; entries past its last page are not read (batch 0: may be NULL).
 *   cu_kv    int32 [batch + 1], rising from 0: sequence b fills rows
 *            cu_kv[b] .. cu_kv[b + 1] - 1 of the outputs with its first tokens.
 *   k_out, v_out  fp16 [rows][kv_heads][head_dim], contiguous, 16-byte
 *            aligned; rows at and past cu_kv[batch] are set to zero.  An 8-bit
 *            cache gives fp16(code * s).  rows * kv_heads may be up to 2^28.
 * Errors: as spear_kv_append.
 */
spear_status_t spear_kv_gather(const spear_kv_desc_t* kv, int32_t batch, int32_t rows, const int32_t* block_table,
                               int64_t table_stride, const int32_t* cu_kv, const void* k_cache, const void* v_cache,
                               const float* k_scale, const float* v_scale, void* k_out, void* v_out, void* stream);

/* One attention call. */
typedef struct spear_attention_desc {
  spear_kv_desc_t kv;
  int32_t batch;      /* sequences; >= 0 */
  int32_t total_q;    /* rows of q and out; 0 is a no-op */
  int32_t max_q;      /* the longest sequence's new tokens (>= 1; a smaller value is slower, not wrong) */
  int32_t max_pages;  /* entries of a block table row; >= 1 */
  int32_t q_heads;    /* a multiple of kv_heads */
  float scale;        /* factor of the scores, |scale| <= 1e30; usually 1 / sqrt(head_dim) */
  int32_t device_cus; /* 0: query the current device; > 0: plan for that many CUs, no device access */
} spear_attention_desc_t;

/*
 * spear_attention_workspace_bytes -- device workspace of a call (host only).
 * The workspace is one of spear_w4ec_linear's kind: zero-filled before its first
 * use, its 1 MiB header's counters returned to zero by the call, the rest
 * scratch; calls that run concurrently must not share it.
 * Errors: NULL_POINTER, INVALID_SHAPE, INVALID_ARGUMENT, UNSUPPORTED, HIP.
 */
spear_status_t spear_attention_workspace_bytes(const spear_attention_desc_t* desc, size_t* bytes);

/*
 * spear_paged_attention -- attention of each sequence's new tokens over its
 * cached ones (the new ones already among them).  With L = kv_lens[b] cached
 * tokens and n = cu_q[b + 1] - cu_q[b] new ones, new token i stands at
 * position L - n + i and sees the keys j <= L - n + i:
 *     out = softmax_j(scale q . k_j) v
 * per head; query head h reads kv head h / (q_heads / kv_heads).  A token
 * that sees no key (L - n + i < 0) gives zeros, as does one whose visible
 * scores are all -infinity.  What the cache holds past a token's position (or
 * past kv_lens) never reaches its output, be it infinite or NaN.
 *   q        fp16 [total_q][q_heads][head_dim], 16-byte aligned, last dimension
 *            contiguous, strides of the first two in elements (multiples of 8).
 *   cu_q     int32 [batch + 1], rising from 0: rows of sequence b.
 *   kv_lens  int32 [batch], 0 to max_pages * page_size.
 *   block_table  int32 [batch][table_stride], as for spear_kv_gather.
 *   out      fp16 [total_q][q_heads][head_dim], contiguous, 16-byte aligned;
 *            rows of no sequence are left as they are.
 * Softmax statistics and sums are held in fp32; the weights of the values are
 * rounded to fp16 for the matrix cores; codes of an 8-bit cache enter them
 * exactly.  The result does not depend on scheduling.
 * Errors: NULL_POINTER, INVALID_SHAPE, INVALID_ARGUMENT, UNSUPPORTED,
 *         MISALIGNED, WORKSPACE_TOO_SMALL, HIP.
 */
spear_status_t spear_paged_attention(const spear_attention_desc_t* desc, const void* q, int64_t q_token_stride,
                                     int64_t q_head_stride, const int32_t* cu_q, const int32_t* kv_lens,
                                     const int32_t* block_table, int64_t table_stride, const void* k_cache,
                                     const void* v_cache, const float* k_scale, const float* v_scale, void* out,
                                     void* workspace, size_t workspace_bytes, void* stream);

/* One verification call. */
typedef struct spear_verify_desc {
  int32_t batch;       /* sequences; 0 is a no-op; below 2^24 */
  int32_t max_drafts;  /* K >= 0 drafted tokens at most per sequence; up to 2^20 */
  int32_t vocab;       /* V >= 1; up to 2^30 */
  int32_t device_cus;  /* as in spear_attention_desc_t */
} spear_verify_desc_t;

/*
 * spear_verify_workspace_bytes -- device workspace of a call (host only): one
 * of spear_w4ec_linear's kind, zero-filled before its first use; the call
 * returns the counters of its header to zero.
 * Errors: NULL_POINTER, INVALID_SHAPE, INVALID_ARGUMENT (device_cus),
 *         UNSUPPORTED (sizes), HIP.
 */
spear_status_t spear_verify_workspace_bytes(const spear_verify_desc_t* desc, size_t* bytes);

/*
 * spear_verify_draft -- keep the drafted tokens that the target's
 * probabilities allow and draw the next token, so that the tokens are
 * distributed as if drawn from the target (speculative sampling by
 * acceptance and residual).  For sequence b with n drafted tokens x_0 .. :
 *   - x_i is kept while u[b][i] * q_i(x_i) < p_i(x_i) (fp32 product); a is the
 *     number kept before the first that is not (or n);
 *   - the next token is drawn with weights w = max(p_a - q_a, 0) if a < n, or
 *     w = p_a if a = n or that is zero everywhere, as the winner of an
 *     exponential race: the largest w(j) / noise[b][j] over w(j) > 0 (fp32, ties
 *     to the lowest j); -1 if there is no such j.
 *   target   fp32 [batch][K + 1][V], draft fp32 [batch][K][V] (NULL: each
 *            drafted token had probability 1, as copied drafts have); the last
 *            dimension contiguous, strides of the first two in elements.
 *   drafted  int32 [batch][K], u fp32 [batch][K] in [0, 1), noise fp32
 *            [batch][V] drawn from Exp(1); contiguous.  A drafted token outside
 *            [0, V) is not kept.
 *   num_drafts  int32 [batch], 0 to K each (clamped); NULL: K for all.
 *   accepted output int32 [batch]: a.  tokens output int32 [batch][K + 1]: the
 *            kept tokens, the drawn one, then -1.
 * Errors: NULL_POINTER, INVALID_SHAPE, INVALID_ARGUMENT, UNSUPPORTED,
 *         MISALIGNED, WORKSPACE_TOO_SMALL, HIP.
 */
spear_status_t spear_verify_draft(const spear_verify_desc_t* desc, const float* target, int64_t target_batch_stride,
                                  int64_t target_row_stride, const float* draft, int64_t draft_batch_stride,
                                  int64_t draft_row_stride, const int32_t* drafted, const float* u,
                                  const float* noise, const int32_t* num_drafts, int32_t* accepted,
                                  int32_t* tokens, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEAR_SERVE_H */
