/*
 * awq_attn.h - C ABI of attention over a cache of 4-bit keys and values (same library, libawq_mi355x.so).
 *
 * What a layer does between its exported QKV product (awq_w4a16_gemm) and its exported output product:
 *   awq_rope            rotary positions of queries and keys, over one or several axes; and its gradient
 *   awq_kv4_write       new keys and values quantized into their slots of a paged cache
 *   awq_kv4_attention   attention of new tokens over the cache: single tokens, drafts, prompts
 *   awq_kv4_read        cached keys and values back as numbers
 *
 * The cache. A page holds page_size consecutive tokens of one sequence, of all n_kv heads, keys and values:
 *   codes   uint8 [n_pages, 2, n_kv, page_size, head_dim / 2]: for keys (0) and values (1), two codes a byte, the even
 *           channel in the low nibble;
 *   params  float16 [n_pages, 2, n_kv, n_groups, page_size, 2]: (step, offset) of each group of AWQ_GROUP_SIZE consecutive
 *           channels of a head (the last group is shorter where head_dim is no multiple of it; n_groups =
 *           ceil(head_dim / 128)).
 * A code c stands for offset + c * step, c = 0 .. 15. A group whose step or offset is not finite stands for NaNs.
 * Pages are contiguous; from page to page there are page_codes bytes and page_params (step, offset) pairs, so that the
 * layers of a model may share a page. head_dim is a multiple of 32 up to AWQ_KV4_MAX_HEAD_DIM, page_size a power of two
 * from AWQ_KV4_MIN_PAGE to AWQ_KV4_MAX_PAGE. Token i of a sequence with page table `table` lies in slot
 * table[i / page_size] * page_size + i % page_size. codes are 16-byte aligned, page_codes a multiple of 16; params
 * 16-byte aligned, page_params a multiple of 4.
 *
 * Conventions are those of awq.h and awq_moe.h: device pointers owned by the caller, no allocation, work enqueued on
 * `stream` without synchronising, argument errors found on the host before anything is enqueued. In addition:
 *   - A [n_tokens, n_heads, head_dim] argument has a pitch from token to token and one from head to head, in elements
 *     (either may be the larger one; channels are consecutive; elements do not overlap). Its pointer needs only the
 *     alignment of an element.
 *   - Slots, page numbers, lengths and offsets are checked on the device: an entry outside its range is skipped or
 *     clamped, never followed out of a buffer.
 *   - No tokens at all is AWQ_ERR_NO_TOKENS; a sequence may have none.
 *   - Outputs must not overlap inputs unless stated otherwise. Two calls may run at the same time unless they share a
 *     workspace or an output, or one writes slots that the other reads or writes.
 */
#ifndef AWQ_ATTN_MI355X_H
#define AWQ_ATTN_MI355X_H

#include "awq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define AWQ_KV4_MAX_HEAD_DIM 256
#define AWQ_KV4_MIN_PAGE 16
#define AWQ_KV4_MAX_PAGE 1024
#define AWQ_MAX_ROPE_DIM 512
#define AWQ_MAX_ROPE_AXES 8
#define AWQ_MAX_HEADS 1024
#define AWQ_MAX_ATTN_TOKENS ((int64_t)1 << 23) /* tokens of one call */
#define AWQ_MAX_ATTN_SEQS (1 << 20)

/* ------------------------------------------------------------------ rotary positions */

typedef enum {
  AWQ_ROPE_HALF = 0,  /* pair i is channels (i, i + rot_dim / 2) */
  AWQ_ROPE_PAIRS = 1  /* pair i is channels (2 i, 2 i + 1) */
} awq_rope_style;

/* For every token t, head and pair i < rot_dim / 2 of channels (a, b), with
 * angle = positions[axis[i], t] * inv_freq[i]:
 *   out_a = scale * (x_a cos(angle) - x_b sin(angle)),  out_b = scale * (x_b cos(angle) + x_a sin(angle)).
 * Channels from rot_dim on are copied. The angle is formed and reduced in float64.
 *   x, out     [n_tokens, n_heads, head_dim] of dtype (AWQ_DTYPE_F32, BF16 or F16). out may be x with the same pitches.
 *              The query and key heads of a fused QKV row are one x.
 *   positions  [n_axes, ld_positions] int32 or int64 (position_bytes 4 or 8), magnitudes below 2^31.
 *   inv_freq   float32 [rot_dim / 2].
 *   axis       int32 [rot_dim / 2], which axis a pair turns with (NULL: axis 0; an entry outside [0, n_axes): angle 0).
 * rot_dim is even, 2 .. head_dim; head_dim up to AWQ_MAX_ROPE_DIM. */
AWQ_API int awq_rope(const void* x, int64_t ld_x, int64_t ld_x_head, int dtype, int64_t n_tokens, int64_t n_heads,
                     int64_t head_dim, const void* positions, int64_t ld_positions, int position_bytes, int n_axes,
                     const float* inv_freq, const int32_t* axis, int64_t rot_dim, int style, float scale, void* out,
                     int64_t ld_out, int64_t ld_out_head, void* stream);

/* The gradient of awq_rope with respect to x: every pair turned back, times scale. d_x may be d_out. */
AWQ_API int awq_rope_backward(const void* d_out, int64_t ld_d_out, int64_t ld_d_out_head, int dtype, int64_t n_tokens,
                              int64_t n_heads, int64_t head_dim, const void* positions, int64_t ld_positions,
                              int position_bytes, int n_axes, const float* inv_freq, const int32_t* axis, int64_t rot_dim,
                              int style, float scale, void* d_x, int64_t ld_d_x, int64_t ld_d_x_head, void* stream);

/* ------------------------------------------------------------------ the cache */

/* Quantizes the keys and values of n_tokens tokens into their slots. For each token, head and group, with x clamped to
 * +-AWQ_KV4_LARGEST:
 *   step   = float16((max x - min x) / 15), offset = float16(min x), each rounded once (the quotient as in float64);
 *   code   = min(max(round_to_even((x - offset) / step), 0), 15), the quotient before its rounding as in float64
 *            (0 where step is 0).
 * A group that holds a NaN or an infinity gets NaN for step and offset.
 *   k, v   [n_tokens, n_kv, head_dim] of dtype (AWQ_DTYPE_F32, BF16 or F16).
 *   slots  [n_tokens] int32 or int64 (slot_bytes 4 or 8); a token whose slot is outside [0, n_pages * page_size) is not
 *          written (padding). Of two tokens with the same slot each byte is one's or the other's.
 * Other slots are left as they were. */
#define AWQ_KV4_LARGEST 65024.0f
AWQ_API int awq_kv4_write(const void* k, int64_t ld_k, int64_t ld_k_head, const void* v, int64_t ld_v, int64_t ld_v_head,
                          int dtype, int64_t n_tokens, int64_t n_kv, int64_t head_dim, const void* slots, int slot_bytes,
                          uint8_t* codes, int64_t page_codes, void* params, int64_t page_params, int64_t n_pages,
                          int page_size, void* stream);

/* The cached keys and values of slots, rounded once to dtype: k[i], v[i] = slot slots[i]. Rows of slots outside the cache
 * are left as they were. k or v may be NULL (not wanted). Arguments as awq_kv4_write. */
AWQ_API int awq_kv4_read(const uint8_t* codes, int64_t page_codes, const void* params, int64_t page_params, int64_t n_pages,
                         int page_size, int64_t n_kv, int64_t head_dim, const void* slots, int slot_bytes, int64_t n_tokens,
                         int dtype, void* k, int64_t ld_k, int64_t ld_k_head, void* v, int64_t ld_v, int64_t ld_v_head,
                         void* stream);

/* ------------------------------------------------------------------ attention over the cache */

/* Workspace bytes of awq_kv4_attention (0 on invalid sizes, and where none is needed). max_kv as there; 0: enough for any table. */
AWQ_API size_t awq_kv4_attention_workspace_bytes(int64_t n_tokens, int64_t n_seqs, int ragged, int64_t n_heads,
                                                 int64_t n_kv, int64_t head_dim, int causal, int64_t window, int64_t max_kv);

/* Sequence s has the new tokens q_offsets[s] .. q_offsets[s + 1] - 1 (q_len of them), and kv_len[s] cached tokens, the
 * last q_len of which are usually the new ones. Its new token i stands at p = kv_len - q_len + i and sees the cached
 * tokens j < kv_len with j <= p (causal) and j > p - window (window > 0). For each head h (keys and values of head
 * h / (n_heads / n_kv)):
 *   out = sum over seen j of softmax_j(scale * q . k_j) v_j,  lse = log sum over seen j of exp(scale * q . k_j)
 * out = 0 and lse = -infinity where nothing is seen (an lse past float32's range is an infinity, too). Tokens on a page outside [0, n_pages) are not seen.
 *   q          [n_tokens, n_heads, head_dim] of q_dtype (AWQ_DTYPE_BF16 or AWQ_DTYPE_F16).
 *   table      int32 [n_seqs, ld_table], table_width pages of each sequence used at most; kv_len is clamped to
 *              [0, table_width * page_size].
 *   kv_len     int32 [n_seqs].
 *   q_offsets  int32 [n_seqs + 1], ascending, or NULL: n_tokens / n_seqs new tokens for each (n_tokens is a multiple of
 *              n_seqs then). Rows of out and lse that belong to no sequence are left as they were.
 * n_tokens * n_heads is at most 2^27, table_width * page_size at most 2^30.
 * One kernel, for few rows or for many, takes all sequences of a call; which one goes by the mean of n_tokens / n_seqs *
 * n_heads / n_kv. A call that mixes single tokens and a long prompt is right, but two calls are faster.
 *   max_kv     the largest kv_len, as far as the caller knows: how the work is split goes by it, what is computed does not
 *              (up to the order of sums). 0: table_width * page_size.
 *   out        [n_tokens, n_heads, head_dim] of out_dtype (q_dtype or AWQ_DTYPE_F32). May be q, of the same type and pitches.
 *   lse        float32 [n_tokens, n_heads], contiguous, or NULL.
 * Products and sums are held in float32. Queries, the cache's numbers (keys only where a key head has many rows) and the
 * softmax's numerators (of float16 queries only there, too) are rounded to float16 for the matrix units (queries by way of a
 * power of two of each row, float16 ones only where a key head has few rows). A seen number of the cache past float16's
 * largest counts there as +-65504 (awq_kv4_write writes none); what a row does not see has no influence on it, whatever the
 * memory holds. */
AWQ_API int awq_kv4_attention(const void* q, int64_t ld_q, int64_t ld_q_head, int q_dtype, int64_t n_tokens, int64_t n_heads,
                              int64_t n_kv, int64_t head_dim, const uint8_t* codes, int64_t page_codes, const void* params,
                              int64_t page_params, int64_t n_pages, int page_size, const int32_t* table, int64_t ld_table,
                              int64_t table_width, const int32_t* kv_len, const int32_t* q_offsets, int64_t n_seqs,
                              float scale, int causal, int64_t window, int64_t max_kv, void* out, int64_t ld_out,
                              int64_t ld_out_head, int out_dtype, float* lse, void* workspace, size_t workspace_bytes,
                              void* stream);

#ifdef __cplusplus
}
#endif
#endif /* AWQ_ATTN_MI355X_H */
