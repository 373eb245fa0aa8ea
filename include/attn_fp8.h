/*
 * attn_fp8.h -- C ABI of the 8-bit KV cache: quantising it as it is written,
 * decoding over it, and reading it back into bf16 pages.
 *
 * Half the bytes of the bf16 cache of attn_decode.h: twice the context in the
 * same memory, and a decode, which is bound by reading the cache, in about
 * half the time.  The layer shapes, pages, block tables, lengths, streams,
 * workspaces, errors and status bits are attn_decode.h's; this header states
 * what differs.
 *
 * Format.  A cache is four arrays:
 *   k_pool, v_pool    e4m3 [num_pages, 16, Hkv, D]: sign, 4 exponent bits
 *                     (bias 7), 3 mantissa bits; largest 448, no infinity
 *   k_scale, v_scale  E8M0 [num_pages, Hkv, 16]: one byte s per position and
 *                     KV head, standing for 2^(s - 127); 255 is NaN, and 0
 *                     (which no append writes: a cleared page) reads as zero
 * Position l of sequence b, KV head c, page P = block_table[b][l / 16], row
 * r = l % 16 holds  k[i] = e4m3(k_pool[P][r][c][i]) * 2^(k_scale[P][c][r] - 127),
 * and v alike.
 *
 * The appends round each head's row y once: 2^(s - 127) is the smallest power
 * of two with max|y| <= 448 * 2^(s - 127) (s clamped to [1, 254]), the values
 * are y * 2^(127 - s) rounded to e4m3, to nearest even.  So a value is off by
 * at most 2^-4 of itself, or 2^-10 * 2^(s - 127) where it is below
 * 2^-6 * 2^(s - 127) (less than 2^-13.8 of the row's largest).  A row that
 * holds a NaN or an infinity is stored with s = 255 and reads as NaN.
 */
#ifndef ATTN_FP8_H
#define ATTN_FP8_H

#include "attn_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * attn_kv_append_sliding_fp8 / attn_kv_append_global_fp8 -- norms, RoPE and
 * append of a chunk of tokens per sequence (one token each in a decode step)
 * into an 8-bit cache: attn_kv_append_*_chunk with keys and values quantised
 * from their fp32 results.  q_out stays bf16.
 *
 * k_pool, v_pool, k_scale, v_scale: all required (no values-only form), 16
 * bytes aligned; written at the tokens' positions only.  Every other argument
 * is attn_kv_append_*_chunk's.
 */
int32_t attn_kv_append_sliding_fp8(const void* qkv, const void* w_q, const void* w_k, const int32_t* block_table,
                                   const int32_t* seq_lens, const int32_t* cu_q, void* q_out, void* k_pool,
                                   void* v_pool, uint8_t* k_scale, uint8_t* v_scale, int32_t batch, int32_t total_q,
                                   int32_t max_blocks, int64_t num_pages, int32_t* status, void* stream);
int32_t attn_kv_append_global_fp8(const void* qkv, const void* w_q, const void* w_k, const int32_t* block_table,
                                  const int32_t* seq_lens, const int32_t* cu_q, void* q_out, void* k_pool,
                                  void* v_pool, uint8_t* k_scale, uint8_t* v_scale, int32_t batch, int32_t total_q,
                                  int32_t max_blocks, int64_t num_pages, int32_t* status, void* stream);

/*
 * attn_kv_read_sliding_fp8 / attn_kv_read_global_fp8 -- cached positions read
 * back into bf16 pages, for the calls that take a bf16 cache
 * (attn_prefill_*).
 *
 * For every sequence the last min(L, span) positions (span <= 0: all L) go
 * from page block_table[b][l / 16] to page out_table[b][l / 16], row l % 16,
 * of k_out and v_out.  Exact wherever the value lies in bf16's normal range
 * (an append's values do, but for rows whose largest is below 2^-100);
 * rounded to nearest even otherwise.
 *
 * k_out, v_out  bf16 [out_pages, 16, Hkv, D], 16 bytes aligned; rows of other
 *               positions are not written
 * out_table     int32 [batch, max_blocks], entries of read positions in
 *               [0, out_pages); may be block_table (the same page ids)
 * max_seq_len   host bound on seq_lens (sizes the launch only)
 * status        a page id outside its pool raises ATTN_DEV_BAD_PAGE and that
 *               page is left out; a bad length as in the decode calls
 * A chunk of n queries on a sliding layer sees span = window + n - 1.
 */
int32_t attn_kv_read_sliding_fp8(const void* k_pool, const void* v_pool, const uint8_t* k_scale,
                                 const uint8_t* v_scale, const int32_t* block_table, const int32_t* seq_lens,
                                 void* k_out, void* v_out, const int32_t* out_table, int32_t batch,
                                 int32_t max_blocks, int64_t num_pages, int64_t out_pages, int32_t max_seq_len,
                                 int32_t span, int32_t* status, void* stream);
int32_t attn_kv_read_global_fp8(const void* k_pool, const void* v_pool, const uint8_t* k_scale, const uint8_t* v_scale,
                                const int32_t* block_table, const int32_t* seq_lens, void* k_out, void* v_out,
                                const int32_t* out_table, int32_t batch, int32_t max_blocks, int64_t num_pages,
                                int64_t out_pages, int32_t max_seq_len, int32_t span, int32_t* status, void* stream);

/*
 * attn_decode_sliding_fp8 / attn_decode_global_fp8 -- attn_decode_sliding and
 * attn_decode_global over an 8-bit cache: the same softmax over the keys and
 * values as they read back.  num_splits as there; the automatic plan and the
 * workspace are attn_decode_fp8_plan's.
 *
 * q is bf16.  Products run in f16 on e4m3 values (exact), scales are applied
 * in fp32, sums are fp32; the weights are rounded to f16 (2^-11 relative at
 * most) before they meet the values.  A page id outside [0, num_pages) on a visible
 * position raises ATTN_DEV_BAD_PAGE and reads as zeros.  A visible NaN (a
 * scale of 255, or the e4m3 NaN) gives NaN outputs; what lies outside the
 * visible positions is never used.  Every array 16 bytes aligned.
 */
int32_t attn_decode_sliding_fp8(const void* q, const void* k_pool, const void* v_pool, const uint8_t* k_scale,
                                const uint8_t* v_scale, const int32_t* block_table, const int32_t* seq_lens, void* o,
                                int32_t batch, int32_t max_blocks, int64_t num_pages, int32_t max_seq_len,
                                int32_t window, int32_t out_dtype, int32_t num_splits, void* workspace,
                                size_t workspace_bytes, int32_t* status, void* stream);
int32_t attn_decode_global_fp8(const void* q, const void* k_pool, const void* v_pool, const uint8_t* k_scale,
                               const uint8_t* v_scale, const int32_t* block_table, const int32_t* seq_lens, void* o,
                               int32_t batch, int32_t max_blocks, int64_t num_pages, int32_t max_seq_len,
                               int32_t window, int32_t out_dtype, int32_t num_splits, void* workspace,
                               size_t workspace_bytes, int32_t* status, void* stream);

/*
 * attn_decode_fp8_plan -- the launch plan of the calls above, as pure host
 * arithmetic: thread blocks per KV head, kernels launched (1 or 2) and workspace
 * bytes (any of the three may be NULL) on a device of num_sms multiprocessors.
 * Arguments and errors as attn_decode_plan.  attn_decode_fp8_workspace_size --
 * the workspace for the current CUDA device (0, with attn_last_error, on bad
 * arguments or when no device can be queried).
 */
int32_t attn_decode_fp8_plan(int32_t kind, int32_t batch, int32_t max_seq_len, int32_t window, int32_t num_splits,
                             int32_t num_sms, int32_t* out_num_splits, int32_t* out_launches,
                             size_t* out_workspace_bytes);
size_t attn_decode_fp8_workspace_size(int32_t kind, int32_t batch, int32_t max_seq_len, int32_t window,
                                      int32_t num_splits);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_FP8_H */
