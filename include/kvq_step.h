/*
 * kvq_step.h -- C ABI of libkvq's operators around a serving step over the
 * paged caches of kvq.h (and, where rows and pages move, of kvq_fp4.h), for
 * NVIDIA GB300:
 *
 *   kvq_rope_write    per-head norm and rotation of q and k, and the
 *                     quantize-and-scatter of k and v, in one pass
 *   kvq_tree_attn     attention of trees of drafted tokens over the cache
 *   kvq_tree_commit   move the accepted path's rows together, in every layer
 *   kvq_pages_init, kvq_pages_alloc, kvq_pages_free, kvq_pages_fork
 *                     a pool of pages that sequences take, give back and share
 *   kvq_copy_pages    copy pages in every layer's caches
 *
 * A step of speculative decoding writes the drafts behind each sequence's
 * tokens (kvq_rope_write), attends (kvq_tree_attn), keeps the accepted path
 * (kvq_tree_commit) and gives the pages behind it back (kvq_pages_free).  A
 * step of beam search, or samples of one prompt, forks the block tables
 * (kvq_pages_fork) and copies the pages that are not full (kvq_copy_pages).
 * "10.4 KV Cache quantization: INT8, KIVI 2-bit, FP8 KV" has the cache's
 * math (sections 10.4.2, 10.4.5); these operators are this library's own.
 *
 * Conventions (streams, status codes, dev_status bits, ownership, supported
 * shapes) are those of kvq.h.  Nothing is allocated and nothing is kept
 * between calls; every call can be captured into a graph.
 */
#ifndef KVQ_STEP_H_
#define KVQ_STEP_H_

#include "kvq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further bits OR-ed into *dev_status. */
#define KVQ_DEV_NO_PAGES 64u  /* the pool has too few free pages: nothing was taken      */
#define KVQ_DEV_BAD_TREE 128u /* a parent not before its node, or a path that is no path */

/*
 * kvq_rope_write -- norm, rotate, quantize and scatter.
 *
 * For every token t and every head row x of q[t] and k[t], in binary32:
 *   y = x / sqrt(mean_d x_d^2 + eps) * w_d     (w = q_weight or k_weight; no
 *                                               norm where it is NULL)
 *   z_a = y_a cos - y_b sin,  z_b = y_a sin + y_b cos
 * for each of the num_pairs pairs i of dims, (a, b) = (i, i + num_pairs) or,
 * where `interleaved`, (2i, 2i + 1); the dims past 2 num_pairs stay y.  The
 * angle of pair i is positions[axis[i]][t] * turns[i] / 2^64 turns, a turn
 * being 2 pi; the product is taken modulo 2^64, so it is exact at any
 * position and an angle is off by what its turns[i] is off, times the
 * position.  cos and sin are within 2^-20 absolute.  Then
 *   q_out[t] = bf16(z)
 *   the cache row of slot_mapping[t] gets cast_fp8(z / sK) and cast_fp8(v / sV)
 * as kvq_write forms them (bf16(z) and v's bits with KVQ_FMT_BF16), with z in
 * binary32: K is rounded once.  Finite rows of any magnitude are normed; a NaN
 * or an infinity in a row reaches that row only.  Codes and scales for KVQ_SCALE_PER_TOKEN_HEAD as kvq_write_token_head
 * forms them, amax / fmt_max over the finite values of z (and v).
 *
 *   q, k, v         bf16 [num_tokens][heads][head_dim]; a token's heads are
 *                   consecutive, consecutive tokens q_stride, k_stride and
 *                   v_stride elements apart (multiples of 8, at least the
 *                   token's heads * head_dim): slices of one projection's
 *                   output fit.
 *   positions       int32 [num_axes][num_tokens], any values; num_axes <= 16
 *   turns           int64 [num_pairs]: round(2^64 * f_i / (2 pi)) for a
 *                   frequency of f_i radians a position, taken modulo 2^64
 *   axis            uint8 [num_pairs], below num_axes (a larger one counts as
 *                   axis 0); NULL: all axis 0
 *   num_pairs       a multiple of 8, 0 .. head_dim / 2
 *   q_weight, k_weight   bf16 [head_dim] or NULL, each on its own
 *   slot_mapping    int64 [num_tokens]; a negative one's k and v are not
 *                   written (its q is); slots distinct
 *   k_cache .. fmt  as for kvq_write; with KVQ_SCALE_PER_TOKEN_HEAD (FP8 only)
 *                   k_scale and v_scale are the scale caches, outputs, of
 *                   num_blocks * num_kv_heads * 16 floats
 *   q_out           bf16 [num_tokens][num_q_heads][head_dim], tokens
 *                   q_out_stride elements apart; q itself is fine (in place,
 *                   same stride), any other overlap is not
 *   dev_status      optional; KVQ_DEV_BAD_SLOT
 * num_tokens == 0 is a no-op.  num_q_heads + num_kv_heads <= 65535.
 */
KVQ_API int kvq_rope_write(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                           const void* v, int64_t v_stride, int64_t num_tokens, int num_q_heads,
                           int num_kv_heads, int head_dim, const int32_t* positions, int num_axes,
                           const int64_t* turns, const uint8_t* axis, int num_pairs,
                           int interleaved, const void* q_weight, const void* k_weight, float eps,
                           const int64_t* slot_mapping, void* k_cache, void* v_cache,
                           int64_t num_blocks, int block_size, float* k_scale, int k_scale_len,
                           float* v_scale, int v_scale_len, int scale_granularity, int fmt,
                           void* q_out, int64_t q_out_stride, uint32_t* dev_status,
                           kvq_stream_t stream);

/* Most nodes of one sequence's tree. */
#define KVQ_TREE_MAX_NODES 256

/*
 * kvq_tree_workspace_size -- bytes of device workspace that kvq_tree_attn
 * needs for any batch of these heads; its contents before a call and after it
 * mean nothing.  num_sms <= 0 queries the current device.  Returns 0 for
 * invalid sizes.
 */
KVQ_API size_t kvq_tree_workspace_size(int num_q_heads, int num_kv_heads, int head_dim, int num_sms);

/*
 * kvq_tree_attn -- attention of trees of drafted tokens over the paged cache,
 * dequantization fused.
 *
 * Sequence b holds L_b = seq_lens[b] tokens in the cache, of which the last
 * n_b = cu_q_lens[b+1] - cu_q_lens[b] are the nodes of its tree (written
 * there before the call); P_b = L_b - n_b tokens precede the tree.  Query row
 * cu_q_lens[b] + j is node j.  Its parent is node parents[cu_q_lens[b] + j] <
 * j, or -1 where it follows the tokens before the tree directly; its depth is
 * the number of its ancestors and its position P_b + depth.  It attends to
 * the tokens t < P_b with t > position - sliding_window (all of them where
 * sliding_window is 0), and to itself and its ancestors (with a window the
 * nearest sliding_window of these):
 *   O = softmax(q K^T / sqrt(head_dim)) V^
 * A row that sees nothing whose page is good is zero.
 *
 *   q               bf16 [num_q_tokens][num_q_heads][head_dim]
 *   cu_q_lens       int32 [num_seqs + 1], device: 0 = cu_q_lens[0] <= ... <=
 *                   cu_q_lens[num_seqs] <= num_q_tokens; rows of out from
 *                   cu_q_lens[num_seqs] on are left as they were
 *   parents         int32 [num_q_tokens], or NULL: every node's parent is the
 *                   node before it (drafts in a row, causal)
 *   caches, block_tables, seq_lens, scales, scale_granularity, fmt, q_scale
 *                   as for kvq_prefill_attn, every granularity included
 *   flags           0 or KVQ_Q_FP8, as for kvq_prefill_attn
 *   workspace       device scratch of kvq_tree_workspace_size bytes, 256-byte
 *                   aligned; calls that may run at the same time (two graphs
 *                   among them) need one each
 *   out             bf16 [num_q_tokens][num_q_heads][head_dim]; no input
 *   dev_status      optional; KVQ_DEV_BAD_BLOCK (the page is masked out),
 *                   KVQ_DEV_BAD_SEQLEN (L_b < n_b or L_b > max_blocks_per_seq
 *                   * block_size: zero rows), KVQ_DEV_BAD_QLEN (n_b past
 *                   KVQ_TREE_MAX_NODES, or cu_q_lens that are negative,
 *                   decrease or pass num_q_tokens: the rows are left as they
 *                   were), KVQ_DEV_BAD_TREE (a parent that is not before its
 *                   node, or below -1, counts as -1), KVQ_DEV_WAIT_TIMEOUT
 * Statistics and sums are binary32, the output is rounded once.  Over FP8
 * caches the query row is scaled by a power of two that takes its largest
 * value to [2^7, 2^8) and enters the products as two E4M3 parts: exact for
 * values within 2^8 of the row's largest, off by 2^-17 of that at most
 * below; finite queries of any magnitude are fine.  A NaN or an infinity in a
 * query row makes that row NaN (with KVQ_Q_FP8 an infinity is cast_fp8's).  A weight enters the
 * product with V^ as its f16, in three E5M2 parts: within 2^-11 of its value
 * and 2^-24 of the row's largest.  Over a bf16 cache the query is taken as it is and a
 * weight as two bf16 parts, within 2^-17.  With KVQ_SCALE_PER_TOKEN_HEAD the
 * weight carries its value's scale relative to the largest that its row has
 * seen, and the 2^-24 is of the row's largest weight times that scale; scales
 * of tokens that a row does not see are nothing to it.  A NaN or an infinity in
 * a cache reaches the rows that see its token, and no others: one in V^ its own
 * dim, an infinity as an infinity or a NaN.  V of a bf16 cache may be finite
 * values up to 2^90.
 *
 * Without parents the call does what kvq_prefill_attn does, and with one node
 * a sequence what kvq_decode_attn does, as exactly (the decode's weights have
 * two f16 parts).  Which is faster (GB300, 32 heads of 128 over 8 KV heads):
 * one token a sequence, kvq_decode_attn (32 x 2049 tokens of FP8: 34 us, here
 * 56, kvq_prefill_attn 122); chunks over an FP8 cache, this call up to some 16
 * tokens, and while sequences are few and long (32 x 16 tokens over 2048: 62
 * us against 106; 1 x 64 over 32768: 60 against 497), kvq_prefill_attn from
 * some 64 tokens of many sequences on (32 x 64 over 2048: 133 against 103;
 * 8 x 256: 196 against 104); chunks over a bf16 cache, this call (32 x 64 over
 * 2048: 127 against 979).
 * Limits: num_seqs <= 4096; num_kv_heads <= 256; num_q_heads / num_kv_heads
 * <= 8; num_blocks * num_kv_heads * block_size < 2^31; max_blocks_per_seq *
 * block_size < 2^30; num_seqs * num_kv_heads * T * (max_blocks_per_seq / 4 +
 * 12) < 2^31 with T = 1 where num_q_tokens * num_q_heads / num_kv_heads <=
 * 128, else 16; beyond them KVQ_ERR_UNSUPPORTED.  num_q_tokens == 0 is a no-op.
 */
KVQ_API int kvq_tree_attn(const void* q, const int32_t* cu_q_lens, int64_t num_q_tokens,
                          const int32_t* parents, const void* k_cache, const void* v_cache,
                          const int32_t* block_tables, int max_blocks_per_seq,
                          const int32_t* seq_lens, int num_seqs, int num_q_heads,
                          int num_kv_heads, int head_dim, int64_t num_blocks, int block_size,
                          const float* q_scale, int q_scale_len, const float* k_scale,
                          int k_scale_len, const float* v_scale, int v_scale_len,
                          int scale_granularity, int fmt, int sliding_window, unsigned flags,
                          void* workspace, size_t workspace_bytes, void* out,
                          uint32_t* dev_status, kvq_stream_t stream);

/*
 * One cache tensor of one layer, for the calls that move rows or pages.  A
 * page of one KV head is 16 rows of row_bytes, then 16 rows of sub_bytes:
 *   FP8 cache             row_bytes = head_dim, sub_bytes = 0
 *   bf16 cache            row_bytes = 2 * head_dim, sub_bytes = 0
 *   scale cache           row_bytes = 4, sub_bytes = 0
 *   4-bit cache           row_bytes = head_dim / 2, sub_bytes = head_dim / 16
 * row_bytes and sub_bytes are multiples of 4 up to 512 (sub_bytes may be 0);
 * data is 16-byte aligned, [num_blocks][num_kv_heads] pages.
 */
typedef struct {
  void* data;
  int32_t row_bytes;
  int32_t sub_bytes;
} kvq_rows;

/*
 * kvq_tree_commit -- keep the accepted path of each sequence's tree.
 *
 * For sequence b, P_b = seq_lens[b] - (cu_q_lens[b+1] - cu_q_lens[b]), and
 * every i < num_accepted[b]: the row of token P_b + accepted[b][i] moves to
 * token P_b + i, in every cache and KV head, and
 *   new_lens[b] = P_b + num_accepted[b].
 * accepted[b] holds node numbers from the tree's first level down, so they
 * rise; rows are read before any of them is written over.
 *
 *   caches          host array of num_caches tensors (kinds mixed), all of
 *                   num_blocks blocks and num_kv_heads heads; at most 1024,
 *                   none twice (KVQ_ERR_ARG)
 *   accepted        int32 [num_seqs][max_path]
 *   num_accepted    int32 [num_seqs], 0 .. min(n_b, max_path)
 *   new_lens        int32 [num_seqs], out; no part of an input (KVQ_ERR_ARG)
 *   dev_status      optional; KVQ_DEV_BAD_TREE (a path that does not rise,
 *                   leaves [0, n_b), or a count outside its range: nothing of
 *                   the sequence moves, new_lens[b] = seq_lens[b]),
 *                   KVQ_DEV_BAD_SEQLEN (seq_lens[b] < n_b or past
 *                   max_blocks_per_seq * block_size: the same),
 *                   KVQ_DEV_BAD_QLEN (cu_q_lens below 0 or decreasing: the
 *                   same), KVQ_DEV_BAD_BLOCK (a row to or from such a page is
 *                   not moved)
 * num_seqs <= 65535, max_path <= 4096.  With no caches only new_lens is written.
 */
KVQ_API int kvq_tree_commit(const kvq_rows* caches, int num_caches, int64_t num_blocks,
                            int num_kv_heads, int block_size, const int32_t* cu_q_lens,
                            const int32_t* block_tables, int max_blocks_per_seq,
                            const int32_t* seq_lens, int num_seqs, const int32_t* accepted,
                            int max_path, const int32_t* num_accepted, int32_t* new_lens,
                            uint32_t* dev_status, kvq_stream_t stream);

/*
 * A pool of pages: KVQ_POOL_WORDS(num_blocks) int32 words on the device.
 *   [0], [2], [3]   0    [1]   how many pages are free
 *   [4 + i]                  how many table entries hold page i
 *   [4 + num_blocks + i / 32], bit i % 32    page i is free
 * The calls below take the lowest free pages first, so tables and pool
 * depend on the calls' arguments alone.  A pool's calls are ordered on one
 * stream (or by the caller).  num_blocks <= 2^24.
 */
#define KVQ_POOL_HEADER 4
#define KVQ_POOL_WORDS(num_blocks) (KVQ_POOL_HEADER + (num_blocks) + ((num_blocks) + 31) / 32)

/* kvq_pages_init -- every page free. */
KVQ_API int kvq_pages_init(int32_t* pool, int64_t num_blocks, kvq_stream_t stream);

/*
 * kvq_pages_alloc -- pages for tokens to come.  Sequence by sequence, entries
 * ceil(old_lens[b] / 16) .. ceil(new_lens[b] / 16) - 1 of block_tables[b] get
 * the lowest free pages, each held once; nothing where new_lens[b] is the
 * smaller.  If the pool has too few for all of them, nothing changes and
 * KVQ_DEV_NO_PAGES is raised.  A length below 0 or past max_blocks_per_seq *
 * 16: the sequence is passed over, KVQ_DEV_BAD_SEQLEN.  num_seqs <= 4096.
 */
KVQ_API int kvq_pages_alloc(int32_t* pool, int64_t num_blocks, int32_t* block_tables,
                            int max_blocks_per_seq, const int32_t* old_lens,
                            const int32_t* new_lens, int num_seqs, uint32_t* dev_status,
                            kvq_stream_t stream);

/*
 * kvq_pages_free -- give pages back.  Entries ceil(new_lens[b] / 16) ..
 * ceil(old_lens[b] / 16) - 1 of block_tables[b] become -1 and their pages lose
 * a holder each; a page without one is free.  Nothing where new_lens[b] is
 * the larger; lengths out of range as for kvq_pages_alloc.  An entry outside
 * [0, num_blocks), or of a page that nothing holds: KVQ_DEV_BAD_BLOCK, the
 * entry becomes -1 and the pool does not change for it.  num_seqs <= 4096.
 */
KVQ_API int kvq_pages_free(int32_t* pool, int64_t num_blocks, int32_t* block_tables,
                           int max_blocks_per_seq, const int32_t* old_lens,
                           const int32_t* new_lens, int num_seqs, uint32_t* dev_status,
                           kvq_stream_t stream);

/*
 * kvq_pages_fork -- tables of sequences that go on from others.
 *
 * Row b of out_tables is to go on from row s = parents[b] of tables, of
 * lens[s] tokens: its full pages are shared (held once more), a last page
 * that is not full is replaced by the lowest free one, and copies[b] = (that
 * page, the new one), (-1, -1) where there is none.  Entries past the last
 * page are -1; out_lens[b] = lens[s].  parents[b] < 0 gives an empty row; one
 * of num_src or more, or whose length is out of range, too, with
 * KVQ_DEV_BAD_SEQLEN.  A shared entry outside [0, num_blocks), or of a page
 * that nothing holds, is -1 in out_tables (KVQ_DEV_BAD_BLOCK); so is a last
 * page's, which then takes no page and is not copied.  If the pool has too
 * few pages nothing is written and KVQ_DEV_NO_PAGES is raised.
 *
 *   tables       int32 [num_src][max_blocks_per_seq], lens int32 [num_src]
 *   parents      int32 [num_out]
 *   out_tables   int32 [num_out][max_blocks_per_seq], out_lens int32
 *                [num_out], copies int32 [num_out][2]; apart from the inputs,
 *                the pool and each other (KVQ_ERR_ARG)
 * What out_tables held before is not given back: free it first.
 * num_src, num_out <= 4096.
 */
KVQ_API int kvq_pages_fork(int32_t* pool, int64_t num_blocks, const int32_t* tables,
                           const int32_t* lens, int num_src, int max_blocks_per_seq,
                           const int32_t* parents, int num_out, int32_t* out_tables,
                           int32_t* out_lens, int32_t* copies, uint32_t* dev_status,
                           kvq_stream_t stream);

/*
 * kvq_copy_pages -- page copies[i][0] onto page copies[i][1] of every cache,
 * all heads, for every i < num_copies with neither below 0.  Pages outside
 * [0, num_blocks): KVQ_DEV_BAD_BLOCK, not copied.  Targets are distinct and no
 * pair's source.  caches as for kvq_tree_commit, but of any number.  num_copies <= 2^20.
 */
KVQ_API int kvq_copy_pages(const kvq_rows* caches, int num_caches, int64_t num_blocks,
                           int num_kv_heads, int block_size, const int32_t* copies,
                           int num_copies, uint32_t* dev_status, kvq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_STEP_H_ */
