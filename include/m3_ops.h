/*
 * m3_ops.h -- C ABI of the serving operators: what a host needs around the
 * decode of m3.h to run requests of different lengths from one paged cache.
 *
 *   m3_kv_map       page tables and slot maps from the requests' lengths
 *   m3_kv_store     K/V rows of new tokens into the pages
 *   m3_attn_prompt  causal attention over packed prompts of different lengths
 *   m3_attn_prefix  one-token attention of a batch that shares a long prefix
 *   m3_logit_rules  penalties, biases and grammar masks on logits
 *
 * Conventions:
 *  - Stateless, as m3_quantize_int8: every pointer is device memory of the
 *    CURRENT device unless marked HOST, the work is asynchronous on
 *    `cuda_stream` (cudaStream_t, 0: the legacy default stream), nothing is
 *    allocated or kept, and a call can be captured into a CUDA graph.  Two
 *    calls may run at once as long as their outputs and workspaces differ.
 *  - Returns an m3_status; arguments are checked on the host before anything
 *    is launched (m3_last_error() has the message).  Lengths, page numbers,
 *    slots and token numbers live on the device, so the kernels check them:
 *    what lies outside is never read or written, as each call says.
 *  - dtype is M3_KV_BF16 or M3_KV_F16; strides are in elements.
 *  - The pool: [n_pages][2][Hkv][page][D], K heads then V heads of a page,
 *    contiguous, 16-byte aligned -- the page of m3_kv_alloc without its chunk
 *    swizzle.  page: a power of two, 16..1024.  Slot = number * page + offset.
 *  - Every device-side wait is bounded; m3_ops_sync_status reports one that
 *    gave up.
 */
#ifndef M3_OPS_H_
#define M3_OPS_H_

#include "m3.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { M3_LOGITS_F32 = 0, M3_LOGITS_BF16 = 1, M3_LOGITS_F16 = 2 };

/* Page tables and slot maps of n_req requests (1..8192), in one launch:
 * request r has cached[r] tokens in its pages and brings fresh[r] new ones
 * (negative counts as 0).  Its table row holds the pages of the cached
 * tokens in columns 0..ceil(cached / page) - 1; the columns its new tokens
 * need besides (none past max_pages) are filled from the free list, in
 * request order, starting at free_pages[*free_at].  Where the list has ended,
 * or holds a number outside 0..n_pages - 1, the column gets -1.  Other
 * columns stay as they are.
 *  cached, free_at: nullable (0).  table: [n_req][ld_table] in and out.
 *  start: added to every position (tokens ahead of the table: a shared prefix).
 *  cu [n_req + 1]: sums of fresh.  lens [n_req]: cached + fresh.
 *  taken [1]: pages the requests need from the list -- more than it holds
 *    means the -1 entries above.
 *  positions, seqs (int32) and slots (int64), [n_tokens] each: of token
 *    cu[r] + i the position start + cached[r] + i, the request r, and the slot
 *    (-1 where it has no page).  Tokens past cu[n_req], the padding of a
 *    captured graph, get -1 in all three; tokens past n_tokens are dropped.
 * Sums past 2^31 - 1 stop there.  positions, seqs and slots are 16-byte aligned.
 * The outputs are other memory than fresh, cached, free_pages and free_at. */
M3_API int m3_kv_map(int n_req, const int32_t* fresh, const int32_t* cached,
                     const int32_t* free_pages, int n_free, const int32_t* free_at, int32_t* table,
                     int max_pages, int64_t ld_table, int page, int n_pages, int start,
                     int n_tokens, int32_t* cu, int32_t* positions, int64_t* slots, int32_t* seqs,
                     int32_t* lens, int32_t* taken, void* cuda_stream);

/* K/V rows of n_tokens tokens into the pool: k, v [n_tokens][Hkv][D] with
 * strides between tokens and heads (the columns of a fused projection will
 * do), slots [n_tokens].  A slot outside the pool (-1) stores nothing.  The
 * slots are distinct: of two equal ones either token's values may stay.
 * D: a multiple of 8, up to 1024. */
M3_API int m3_kv_store(int dtype, int n_tokens, int Hkv, int D, const void* k, int64_t k_token,
                       int64_t k_head, const void* v, int64_t v_token, int64_t v_head,
                       const int64_t* slots, void* pool, int n_pages, int page, void* cuda_stream);

/* Causal attention of n_seq (up to 8192) packed sequences: queries q [n_q][Hq][D], of
 * sequence s the rows cu_q[s]..cu_q[s + 1] - 1, keys and values k, v
 * [n_k][Hkv][D], rows cu_k[s]..cu_k[s + 1] - 1 (cu_k null: cu_q; then n_k = n_q).
 * The last query sits on the last key: of Lq queries and Lk keys query i
 * attends to keys 0..i + Lk - Lq, so a sequence may continue cached keys.
 *   out = softmax(scale q k^T) v, lse = ln sum exp(scale q k) (nullable,
 *   [n_q][Hq] contiguous)
 * A query with no key gets out = 0 and lse = -inf.  Rows of q past
 * cu_q[n_seq] are not computed and their outputs stay as they are.  Lengths
 * that the arrays do not hold are cut to what they do.
 * Scores, sums and lse are fp32; the weights are rounded to dtype before
 * their product with v.  Keys and values that a query does not attend to never
 * reach it, infinities and NaN among them (those in values of a query's own
 * sequence, up to 127 keys behind it, make its row slow).
 * A row whose scores are all -inf counts as one without a key; out is other
 * memory than q, k and v.
 * D: 64 or 128; Hq a multiple of Hkv, Hq / Hkv <= 64; q, k, v, out 16-byte aligned with
 * strides that are multiples of 8; scale > 0. */
M3_API int m3_attn_prompt(int dtype, int n_seq, int n_q, int n_k, int Hq, int Hkv, int D,
                          const void* q, int64_t q_token, int64_t q_head, const void* k,
                          int64_t k_token, int64_t k_head, const void* v, int64_t v_token,
                          int64_t v_head, const int32_t* cu_q, const int32_t* cu_k, float scale,
                          void* out, int64_t o_token, int64_t o_head, float* lse,
                          void* cuda_stream);

/* Bytes of workspace that m3_attn_prefix needs for such a call (0 for a call
 * it refuses); prefix_pages and max_pages are the numbers of pages. */
M3_API int64_t m3_attn_prefix_workspace(int n_rows, int Hq, int Hkv, int D, int prefix_pages,
                                        int page, int max_pages);

/* One-token attention of n_rows rows that share a prefix: row b attends to
 * positions 0..prefix_len - 1 in the pages prefix_pages[], read once for the
 * whole batch (where it is short, by each row), and to its own lens[b] positions in the pages of its table
 * row.  q, out [n_rows][Hq][D] with strides, lse as in m3_attn_prompt.
 * lens[b] < 0 marks a row of padding: its out and lse stay as they are.  A row
 * with nothing to attend to gets out = 0 and lse = -inf.  lens[b] past
 * max_pages * page is cut to that.  Positions on a page whose number is
 * outside 0..n_pages - 1 are left out.  What lies in the pages past a length
 * does not matter.
 *  n_prefix_pages: entries of prefix_pages, ceil(prefix_len / page) at least.
 *  The work is split by n_prefix_pages and max_pages, not by the lengths: a
 *    table no wider than the rows need is faster where rows are few.
 *  workspace: of m3_attn_prefix_workspace's size for this n_prefix_pages,
 *    16-byte aligned, the call's own while it runs; calls (and captured
 *    graphs) that may run at once need one each.
 * Types, alignment and memory as m3_attn_prompt. */
M3_API int m3_attn_prefix(int dtype, int n_rows, int Hq, int Hkv, int D, const void* q,
                          int64_t q_row, int64_t q_head, const void* pool, int n_pages, int page,
                          const int32_t* prefix_pages, int n_prefix_pages, int prefix_len,
                          const int32_t* table, int max_pages, int64_t ld_table,
                          const int32_t* lens, float scale, void* out, int64_t o_row,
                          int64_t o_head, float* lse, void* workspace, int64_t workspace_bytes,
                          void* cuda_stream);

/* Rules on n_rows rows of `vocab` logits ahead of a draw, in this order, in
 * fp32 with one rounding to the logits' type (M3_LOGITS_*) at the end.  With c the
 * number of times token i stands in the row's history:
 *   c > 0:  x = x > 0 ? x / repetition : x * repetition
 *   x -= frequency * c + (c > 0 ? presence : 0)
 *   x += the row's biases of token i, added in their order
 *   x = -inf where the grammar does not allow token i
 *  history [n_rows][ld_history] int32, n_history (up to 2^24) per row, of
 *    which the first hist_len[r] count (nullable: all); numbers outside the vocabulary do not.
 *  repetition (> 0), frequency, presence: fp32 [n_rows], nullable (1, 0, 0).
 *  bias_ids int32, bias fp32: [n_rows][n_bias], up to 4096; ids outside the
 *    vocabulary are skipped.
 *  mask uint32 [n_masks][ceil(vocab / 32)]: bit i % 32 of word i / 32 set:
 *    allowed.  mask_row [n_rows]: the mask of each row, outside 0..n_masks - 1:
 *    none; nullable, then n_masks is 1 (for all rows) or n_rows.
 *  out: logits itself (same stride) or memory that does not overlap it. */
M3_API int m3_logit_rules(int dtype, int n_rows, int vocab, const void* logits, int64_t ld_logits,
                          void* out, int64_t ld_out, const int32_t* history, int n_history,
                          int64_t ld_history, const int32_t* hist_len, const float* repetition,
                          const float* frequency, const float* presence, const int32_t* bias_ids,
                          const float* bias, int n_bias, const uint32_t* mask, int n_masks,
                          const int32_t* mask_row, void* cuda_stream);

/* Synchronise `cuda_stream` and return the first error that a kernel of this
 * header recorded on the current device since the last call (M3_ETIMEOUT),
 * clearing it, or M3_OK.  One word serves all callers of the device: whoever asks
 * first gets the error, and what any of them computed since the last M3_OK is in
 * doubt.  Until it is cleared, waits that last over a millisecond (no sound one
 * does) give up early. */
M3_API int m3_ops_sync_status(void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* M3_OPS_H_ */
