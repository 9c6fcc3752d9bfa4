/*
 * kvq_fp4.h -- C ABI of libkvq's microscaled 4-bit cache (NVFP4: E2M1 codes,
 * an E4M3 scale for every 16 consecutive dims of a row) for NVIDIA GB300.
 *
 * The "nvfp4" cache dtype of the "vLLM FP8 quantized KV cache guide" (the
 * kv_cache_dtype list), beside the FP8 caches of kvq.h:
 *
 *   kvq_fp4_write         quantize bf16 K/V and scatter them into the pages
 *   kvq_fp4_read          gather tokens back to bf16, by block table
 *   kvq_fp4_decode_attn   attention of one query token per sequence
 *   kvq_fp4_prefill_attn  attention of a chunk of query tokens per sequence
 *
 * Conventions (streams, status codes, dev_status bits, ownership) are those
 * of kvq.h.  A value of the cache is
 *   x^ = e2m1(code) * e4m3(block scale) * s
 * with s a binary32 scale per tensor or per KV head.  code * block scale has
 * at most six significand bits and lies in 2^-10 .. 2688, so it is exact in
 * binary16 and in bfloat16; only s rounds.
 *
 * Cache layout, per layer and per tensor (K and V separately), uint8:
 *   [num_blocks][num_kv_heads][9 * head_dim]
 * a page of one KV head being 16 token rows of head_dim / 2 code bytes (dim
 * 2i in the low four bits of byte i, dim 2i + 1 in the high four), then 16
 * token rows of head_dim / 16 E4M3 scale bytes.  4.5 bits a value against
 * the FP8 cache's 8.  One page is one run of 1152 (576) bytes, so a kernel
 * fetches codes and scales with a single copy.
 *
 * Code e2m1: sign, two exponent bits, one significand bit: 0, 0.5, 1, 1.5, 2,
 * 3, 4, 6 and their negatives.  It has neither infinities nor NaN.
 *
 * Supported shapes: head_dim 64 or 128; block_size == 16; for the attentions
 * num_q_heads % num_kv_heads == 0 with a quotient of at most 8 (any of
 * 1 .. 8).  Device pointers are 16-byte aligned; index arrays and scales
 * 4-byte, slot_mapping 8-byte, workspaces 256-byte aligned.  Caches of any
 * size: offsets are 64-bit.
 */
#ifndef KVQ_FP4_H_
#define KVQ_FP4_H_

#include "kvq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of one KV head's page of one tensor. */
#define KVQ_FP4_PAGE_BYTES(head_dim) (9 * (head_dim))

/*
 * kvq_fp4_write -- quantize and scatter K and V into the paged 4-bit cache.
 *
 * For every token t with slot = slot_mapping[t] >= 0, every KV head h and
 * every 16 consecutive dims x_0 .. x_15 of k[t][h] (and likewise of v):
 *   a  = max_i |x_i|, an infinity counting as the largest finite bf16
 *   sb = e4m3(a / (6 s_h))          both quotients and 6 s_h, sb s_h are
 *   c_i = e2m1(x_i / (sb s_h))      binary32, round to nearest even
 * with e4m3 and e2m1 rounding to nearest even and saturating (448, 6).  The
 * codes keep the sign of x_i.  A block whose sb or sb s_h is 0 has codes of
 * 0; one that holds a NaN has the scale code 0x7F (NaN) and codes of 0, so
 * that its 16 values read as NaN.  With s_h = amax / 2688 (amax the head's
 * largest magnitude: the E4M3 scale of kvq_calibrate_scales over 6) the
 * largest block scale is 448.
 *
 *   k, v, token_stride, slot_mapping   as for kvq_write (slots distinct)
 *   k_cache, v_cache   uint8, layout above, num_blocks blocks
 *   k_scale, v_scale   fp32 device arrays of 1 (KVQ_SCALE_PER_TENSOR) or
 *                      num_kv_heads (KVQ_SCALE_PER_HEAD) values, finite, > 0
 *   dev_status         optional; KVQ_DEV_BAD_SLOT
 * num_tokens == 0 is a no-op.
 */
KVQ_API int kvq_fp4_write(const void* k, const void* v, int64_t token_stride,
                          const int64_t* slot_mapping, int64_t num_tokens, int num_kv_heads,
                          int head_dim, void* k_cache, void* v_cache, int64_t num_blocks,
                          int block_size, const float* k_scale, int k_scale_len,
                          const float* v_scale, int v_scale_len, int scale_granularity,
                          uint32_t* dev_status, kvq_stream_t stream);

/*
 * kvq_fp4_read -- gather tokens of each sequence back to bf16.
 *
 * Row cu_lens[b] + j of k_out and v_out, 0 <= j < cu_lens[b+1] - cu_lens[b],
 * is token starts[b] + j of sequence b, at offset (starts[b] + j) % 16 of
 * block block_tables[b][(starts[b] + j) / 16]:
 *   bf16(fp32(code * block scale * s_h)), both roundings to nearest even.
 *
 *   block_tables   int32 [num_seqs][max_blocks_per_seq]
 *   starts         int32 [num_seqs], or NULL for zeros
 *   cu_lens        int32 [num_seqs + 1], 0 = cu_lens[0] <= ... <=
 *                  cu_lens[num_seqs] <= num_rows
 *   k_out, v_out   bf16 [num_rows][num_kv_heads][head_dim], consecutive rows
 *                  out_stride elements apart (>= num_kv_heads * head_dim, a
 *                  multiple of 8); rows from cu_lens[num_seqs] on are left
 *                  as they were
 *   dev_status     optional; KVQ_DEV_BAD_BLOCK (a block id outside
 *                  [0, num_blocks): its rows are zero), KVQ_DEV_BAD_SEQLEN (a
 *                  token position outside [0, max_blocks_per_seq *
 *                  block_size): its row is zero)
 * num_rows == 0 is a no-op.
 */
KVQ_API int kvq_fp4_read(const void* k_cache, const void* v_cache, int64_t num_blocks,
                         int block_size, int num_kv_heads, int head_dim,
                         const int32_t* block_tables, int max_blocks_per_seq,
                         const int32_t* starts, const int32_t* cu_lens, int num_seqs,
                         int64_t num_rows, const float* k_scale, int k_scale_len,
                         const float* v_scale, int v_scale_len, int scale_granularity,
                         void* k_out, void* v_out, int64_t out_stride, uint32_t* dev_status,
                         kvq_stream_t stream);

/*
 * kvq_fp4_workspace_size -- bytes of device workspace that
 * kvq_fp4_decode_attn (num_seqs sequences) and kvq_fp4_prefill_attn (any
 * number of sequences) need; one buffer serves both (61 MB at 152 SMs and
 * head_dim 128, half of that at 64, until decode batches need more).
 * num_sms <= 0 queries the current device.  Returns 0 for invalid sizes.
 */
KVQ_API size_t kvq_fp4_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads,
                                      int head_dim, int num_sms);

/*
 * kvq_fp4_decode_attn -- grouped-query attention of one new token per
 * sequence over the 4-bit cache, dequantization fused.
 *
 * Sequence b holds L_b = seq_lens[b] tokens, the new one (at L_b - 1)
 * included; its query attends to the tokens t < L_b with
 *   t >= L_b - sliding_window  (always, where sliding_window is 0)
 *   or t < num_sinks           (the first tokens, which stay visible)
 *   O = softmax(q K^^T / sqrt(head_dim)) V^
 * and a sequence of no tokens, or none whose page is good, gives a zero row.
 *
 *   q              bf16 [num_seqs][num_q_heads][head_dim]; query head h reads
 *                  KV head h / (num_q_heads / num_kv_heads)
 *   block_tables   int32 [num_seqs][max_blocks_per_seq]; only the entries of
 *                  pages that hold a visible token are read
 *   seq_lens       int32 [num_seqs]
 *   k_scale, v_scale, scale_granularity   as for kvq_fp4_write
 *   workspace      device scratch of kvq_fp4_workspace_size bytes, its first
 *                  KVQ_WS_COUNTER_BYTES zero before the first call and left
 *                  zero by every completed one, as for kvq_decode_attn; calls
 *                  that may run at the same time need a workspace each
 *   out            bf16 [num_seqs][num_q_heads][head_dim]
 *   dev_status     optional; KVQ_DEV_BAD_BLOCK (the page is masked out),
 *                  KVQ_DEV_BAD_SEQLEN (L_b < 0 or > max_blocks_per_seq *
 *                  block_size: a zero row), KVQ_DEV_WAIT_TIMEOUT
 * Statistics and sums are binary32.  The logits use q as f16 after a scaling by
 * a power of two: exact for values within 2^31 of the query head's largest, off
 * by 2^-39 of that at most for smaller ones, as in kvq_decode_attn.  Finite
 * queries of any magnitude are fine: logits past binary32's integers leave the
 * largest one's token.  Each probability reaches the product with V^ as one f16,
 * within 2^-11 of its value or 2^-32 of the row's largest.
 * Limits: num_seqs <= 4096; num_seqs * num_kv_heads <= 65536; num_seqs *
 * (max_blocks_per_seq + 8) * num_kv_heads < 2^31; num_kv_heads <= 256;
 * max_blocks_per_seq * block_size < 2^31.
 */
KVQ_API int kvq_fp4_decode_attn(const void* q, const void* k_cache, const void* v_cache,
                                const int32_t* block_tables, int max_blocks_per_seq,
                                const int32_t* seq_lens, int num_seqs, int num_q_heads,
                                int num_kv_heads, int head_dim, int64_t num_blocks,
                                int block_size, const float* k_scale, int k_scale_len,
                                const float* v_scale, int v_scale_len, int scale_granularity,
                                int sliding_window, int num_sinks, void* workspace,
                                size_t workspace_bytes, void* out, uint32_t* dev_status,
                                kvq_stream_t stream);

/*
 * kvq_fp4_prefill_attn -- attention of a chunk of new tokens per sequence
 * over the 4-bit cache (a prompt, a chunk of one over its cached prefix, a
 * few draft tokens), dequantization fused.
 *
 * Sequence b holds L_b = seq_lens[b] tokens in the cache, the chunk's own
 * included; its last n_b = cu_q_lens[b+1] - cu_q_lens[b] are the queries.
 * Query row cu_q_lens[b] + j is the token at pos = L_b - n_b + j and attends
 * to the tokens t <= pos with
 *   t > pos - sliding_window   (always, where sliding_window is 0)
 *   or t < num_sinks.
 *
 *   q              bf16 [num_q_tokens][num_q_heads][head_dim]
 *   cu_q_lens      int32 [num_seqs + 1], device: 0 = cu_q_lens[0] <= ... <=
 *                  cu_q_lens[num_seqs] <= num_q_tokens; rows of out from
 *                  cu_q_lens[num_seqs] on are left as they were
 *   max_q_len      host: an upper bound of every n_b; the rows of a longer
 *                  chunk past it, rounded up to whole tiles of 128 /
 *                  (num_q_heads / num_kv_heads) queries (0: all its rows), are
 *                  left as they were and KVQ_DEV_BAD_QLEN is raised
 *   workspace      as for kvq_fp4_decode_attn
 *   out            bf16 [num_q_tokens][num_q_heads][head_dim]
 *   dev_status     optional; KVQ_DEV_BAD_BLOCK, KVQ_DEV_BAD_SEQLEN (L_b < n_b
 *                  or L_b > max_blocks_per_seq * block_size: zero rows),
 *                  KVQ_DEV_BAD_QLEN (rows past max_q_len, or a chunk whose
 *                  cu_q_lens are negative, decrease or pass num_q_tokens: its
 *                  rows are left as they were), KVQ_DEV_WAIT_TIMEOUT
 * Precision as for kvq_fp4_decode_attn.  Limits: num_seqs <= 65535;
 * num_kv_heads <= 256; max_blocks_per_seq * block_size < 2^30; num_q_tokens
 * <= 2^30; num_seqs * num_kv_heads * (max_q_len / 16 + 1) < 2^31.
 * num_q_tokens == 0 is a no-op.
 */
KVQ_API int kvq_fp4_prefill_attn(const void* q, const int32_t* cu_q_lens, int64_t num_q_tokens,
                                 int max_q_len, const void* k_cache, const void* v_cache,
                                 const int32_t* block_tables, int max_blocks_per_seq,
                                 const int32_t* seq_lens, int num_seqs, int num_q_heads,
                                 int num_kv_heads, int head_dim, int64_t num_blocks,
                                 int block_size, const float* k_scale, int k_scale_len,
                                 const float* v_scale, int v_scale_len, int scale_granularity,
                                 int sliding_window, int num_sinks, void* workspace,
                                 size_t workspace_bytes, void* out, uint32_t* dev_status,
                                 kvq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_FP4_H_ */
