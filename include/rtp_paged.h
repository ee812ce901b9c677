/*
 * rtp_paged.h -- operators over a caller-owned paged KV cache on NVIDIA B200 (sm_100a).
 *
 * These serve engines that keep keys and values in fixed-size pages of a shared pool instead of
 * one contiguous cache per layer (rtp.h).  They hold no state between calls: the caller owns the
 * pages, the block table, the lengths, the workspace and the streams.  (The page bounds of the
 * selection and the accumulated weights of the eviction are the caller's arrays as well.)
 *
 *   rtp_paged_append   norms of queries and keys per head, rotation by position, K and V rows
 *                      written to their pages, page bounds kept
 *   rtp_paged_bounds   page bounds recomputed from the stored keys
 *   rtp_paged_decode   attention of new tokens over their sequences' pages (all of them, a window
 *                      with sinks, or a list of pages), split over the length and joined
 *   rtp_paged_select   the pages a query attends to, by an upper bound of its scores in each page
 *   rtp_paged_evict    a cache brought back to a budget by the attention weight its slots drew
 *   rtp_paged_take_errors   what the kernels had to leave out since the last look
 *
 * Conventions shared by every entry point
 *   - Device pointers are plain addresses on the current device; every call is asynchronous and
 *     ordered on the stream it is given, allocates nothing and never waits, so it can be captured
 *     into a graph.  Lengths and tables are read on the device: a captured call follows them.
 *   - Argument errors are found on the host before any launch: RTP_EINVAL, no side effects,
 *     rtp_last_error(NULL) says what.  Errors that only the device can see (a page number outside
 *     the pool, a length outside the table, a sequence or row number outside the batch) never make a
 *     kernel read or write outside its arrays: what such an entry names is left out, and
 *     RTP_PAGED_ERANGE is set in the err word of rtp_paged_kv, if there is one.
 *   - Calls that share a workspace must not overlap on the GPU: one workspace per stream, and one
 *     per captured graph if graphs may run at the same time.  A workspace needs no initial value,
 *     and nothing in it outlives the call.
 *   - Results do not depend on timing: no sum is formed in an order that varies between runs.
 */
#ifndef RTP_PAGED_H_
#define RTP_PAGED_H_

#include <stddef.h>

#include "rtp.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { RTP_FP16 = 0, RTP_BF16 = 1, RTP_E4M3 = 2 } rtp_dtype;

/* Bits of rtp_paged_kv.err */
#define RTP_PAGED_ERANGE 2u   /* a page, length, sequence or row number out of range was left out */
#define RTP_PAGED_ETIMEOUT 4u /* a bounded in-kernel wait gave up; results of that call are invalid */

/* A paged cache of one layer.  Element (page, head, slot, d) of k lies at
 * k + page * k_stride[0] + head * k_stride[1] + slot * k_stride[2] + d (elements; v alike), so
 * pages may be laid out head by head or token by token, and K and V may share an allocation. */
typedef struct {
  void* k;                    /* DEVICE, 16-byte aligned */
  void* v;
  int64_t k_stride[3];        /* each a multiple of 16 bytes, and positive */
  int64_t v_stride[3];
  int64_t n_pages;            /* pages in the pool */
  int32_t page_size;          /* slots per page: 16, 32, 64 or 128 */
  int32_t n_kv_heads;         /* Hkv */
  int32_t head_dim;           /* D: 64 or 128 */
  int32_t dtype;              /* rtp_dtype of the pages */
  float k_scale, v_scale;     /* key = stored * k_scale, value = stored * v_scale (> 0) */
  const int32_t* block_table; /* DEVICE [n_seqs][table_stride]: page of slots i*page_size ... */
  int64_t table_stride;       /* >= max_pages */
  int32_t max_pages;          /* entries of a table row that may be used */
  int32_t n_seqs;
  void* bounds;               /* DEVICE [n_pages][Hkv][2][D] in the pages' dtype, contiguous and
                                 16-byte aligned: the least and the greatest stored key of each
                                 page in each dimension; NULL: not kept */
  uint32_t* err;              /* DEVICE error word, or NULL */
} rtp_paged_kv;

/* Move kv->err to *bits (DEVICE) and clear it, in one step: an error that another stream reports
 * meanwhile is in this answer or in the next.  Of kv only err is looked at. */
rtp_status rtp_paged_take_errors(const rtp_paged_kv* kv, uint32_t* bits, cudaStream_t stream);

/* Append new tokens.  Token t of sequence b is row cu_new[b] + i of q, k and v (cu_new DEVICE
 * [n_seqs + 1], ascending from 0; rows that no sequence names are left alone, RTP_PAGED_ERANGE tells
 * of offsets that descend, begin elsewhere or pass n_tokens; NULL: one token per sequence, row b,
 * n_tokens == n_seqs) and goes to slot seq_len[b] + i (seq_len: DEVICE, the lengths BEFORE the
 * call).  For each head row x of q and k, in fp32 and rounded once:
 *     y = x / sqrt(mean(x^2) + eps) * weight      (weight NULL: y = x)
 *     z = y rotated by its position: pair (c, c + D/2) by position * rope_base^(-2c/D)
 * q_out[t] = z of q; the page receives z of k divided by k_scale and v divided by v_scale (e4m3
 * saturates at 448).  positions: DEVICE [n_tokens], NULL: a token's slot (of a cache that evicts,
 * slots are not positions).  slot_pos: DEVICE [n_seqs][Hkv][slot_pos_stride] or NULL, receives
 * each new slot's position.  Of a token whose slot lies outside the table, and of all tokens of a
 * sequence of negative length, q alone is taken.  With kv->bounds, a page whose slot 0 is written
 * starts its bounds from this call's keys; other pages' bounds are widened by them.  (After dropping
 * tokens from a page, its bounds stay valid but wide until rtp_paged_bounds.)
 *
 * q, k, v: DEVICE fp16 or bf16 (dtype; that of the pages unless those are e4m3), heads
 * contiguous, rows q_stride, k_stride, v_stride elements apart (multiples of 8).  q_out: rows
 * q_out_stride apart; it may be q itself.  q and q_out may both be NULL (n_q_heads is then
 * ignored).  max_new: about the most tokens of one sequence (1 to n_tokens; sizes a launch).  A page
 * written to must belong to one sequence only. */
rtp_status rtp_paged_append(const rtp_paged_kv* kv, const void* q, const void* k, const void* v, int32_t dtype,
                            int64_t q_stride, int64_t k_stride, int64_t v_stride, int32_t n_tokens,
                            int32_t n_q_heads, const int32_t* cu_new, int32_t max_new, const int32_t* seq_len,
                            const int32_t* positions, const void* q_weight, const void* k_weight, float eps,
                            double rope_base, void* q_out, int64_t q_out_stride, int32_t* slot_pos,
                            int64_t slot_pos_stride, cudaStream_t stream);

/* Recompute kv->bounds of every page that holds one of the first seq_len[b] slots of a sequence,
 * from those slots' keys.  Sequences that share a page must use it to the same slot (as they do a
 * full page of a common prefix): each writes the bounds of what it uses. */
rtp_status rtp_paged_bounds(const rtp_paged_kv* kv, const int32_t* seq_len, cudaStream_t stream);

/* Attention of query rows over their sequences' pages:
 *     out[r][h] = softmax_j(sm_scale * q[r][h] . key_j) value_j,  h reads KV head h / (Hq / Hkv),
 * over slots j < row_len[r] of sequence row_seq[r] (NULL: row r reads sequence r).  A row with no
 * slot gives zeros and lse = -inf.
 *   window > 0: only slots j >= row_len - window or j < n_sink.  (Slots, not positions: after an
 *     eviction, which fills holes with later rows, they are not the last tokens.)
 *   sel != NULL: only the slots of the listed pages: sel DEVICE [n_rows][Hkv][sel_stride] page
 *     indexes of the sequence (not pool pages), sel_count DEVICE [n_rows][Hkv]; each page at most
 *     once (a repeated page counts twice); indexes outside the row's pages are skipped (-1 may pad
 *     a list).  window must be 0.
 *   scores != NULL: scores[r][g][j] += sum over KV head g's query heads of their weight on slot j,
 *     for the slots attended (DEVICE fp32 [n_rows][Hkv][scores_stride], scores_stride >=
 *     max_pages * page_size).  Row r must be sequence r (row_seq NULL); sel must be NULL.
 * q, out: DEVICE fp16 or bf16 (q_dtype; that of the pages unless those are e4m3), heads contiguous,
 * rows q_stride / out_stride elements apart (multiples of 8).  lse: DEVICE fp32 [n_rows][Hq]
 * natural logarithms of the softmax sums, or NULL.  sm_scale 0: 1/sqrt(D).  1 <= n_rows <= 65535,
 * Hq / Hkv <= 64.  Scores and the softmax are kept in fp32; the weights are rounded to 16 bits (to
 * fp16 for e4m3 pages) for the product with the values. */
rtp_status rtp_paged_decode(const rtp_paged_kv* kv, const void* q, int32_t q_dtype, int64_t q_stride,
                            int32_t n_rows, int32_t n_q_heads, const int32_t* row_seq, const int32_t* row_len,
                            int32_t window, int32_t n_sink, float sm_scale, const int32_t* sel,
                            const int32_t* sel_count, int64_t sel_stride, void* out, int64_t out_stride, float* lse,
                            float* scores, int64_t scores_stride, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream);

/* Bytes of workspace (16-byte aligned) that such a call needs; 0 on bad arguments. */
size_t rtp_paged_decode_workspace(const rtp_paged_kv* kv, int32_t n_rows, int32_t n_q_heads, int with_scores);

/* Pages each row attends to.  A page's score for KV head g is
 *     max over g's query heads of  sum_d max(q_d * lo_d, q_d * hi_d),
 * lo and hi its bounds: no key of the page scores higher.  It is summed in fp64, so that the choice
 * is the exact one.  Of the row's ceil(row_len / page_size) pages, the first n_first and the last
 * n_recent are always taken, then others in (score desc, page asc) order, min(top_pages, pages) in
 * all.  sel: DEVICE [n_rows][Hkv][sel_stride] receives their indexes ascending, then -1 up to
 * top_pages; sel_count: DEVICE [n_rows][Hkv].  Needs kv->bounds, n_first + n_recent <= top_pages
 * <= sel_stride.  A score that is not a number ranks last, and so does a page outside the pool, with
 * RTP_PAGED_ERANGE, where there is a choice; where a page is taken without one it is not looked at. */
rtp_status rtp_paged_select(const rtp_paged_kv* kv, const void* q, int32_t q_dtype, int64_t q_stride,
                            int32_t n_rows, int32_t n_q_heads, const int32_t* row_seq, const int32_t* row_len,
                            int32_t top_pages, int32_t n_first, int32_t n_recent, int32_t* sel, int64_t sel_stride,
                            int32_t* sel_count, void* workspace, size_t workspace_bytes, cudaStream_t stream);

size_t rtp_paged_select_workspace(const rtp_paged_kv* kv, int32_t n_rows, int32_t n_q_heads);

/* Bring every sequence of more than `budget` slots back to `budget`, for each KV head by itself.
 * positions: DEVICE int32 [n_seqs][Hkv][stride], the position of each slot's key; scores: DEVICE
 * fp32, alike, what the slots drew (rtp_paged_decode).  Of the first seq_len[b] slots these stay:
 * those with position < n_sink or > newest - n_recent (newest: the largest position), then others
 * in (score desc, position asc, slot asc) order, `budget` in all (n_sink + n_recent <= budget; a
 * score that is not a number ranks last).  Survivors in slots >= budget move into the freed slots
 * below it, in slot order: K and V rows, score, position; all other rows stay where they are, and
 * rows at and behind `budget` keep their bytes.  out_len[b] (DEVICE) = min(seq_len[b], budget);
 * out_scores and out_positions (may be scores and positions; no arrays share memory otherwise, so
 * out_len is not seq_len) receive slots 0 .. out_len - 1, then 0 and -1 up to stride.  budget and
 * stride are at most 2^24.  Pages moved into keep their bounds; call rtp_paged_bounds where those are
 * in use.  A page must belong to one sequence only. */
rtp_status rtp_paged_evict(const rtp_paged_kv* kv, const int32_t* seq_len, int32_t budget, int32_t n_recent,
                           int32_t n_sink, const float* scores, const int32_t* positions, int64_t stride,
                           float* out_scores, int32_t* out_positions, int32_t* out_len, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream);

size_t rtp_paged_evict_workspace(const rtp_paged_kv* kv, int64_t stride);

#ifdef __cplusplus
}
#endif

#endif /* RTP_PAGED_H_ */
