/*
 * specverify_cache.h -- the 4-bit paged KV cache of specverify.h beyond a verify's rows: the
 * attention of whole prompts over it, and a cache held to a budget of positions.
 *
 * A request starts with reserve -> per layer (append, prompt_attention, and
 * attention_weights of the prompt's last rows) -> evict; where requests are held to a budget a
 * step is reserve -> per layer (append_at, whose q_out is kept, attention) -> verify -> drain ->
 * per layer attention_weights of the rows that were committed -> release -> evict.
 *
 * Pages, tables, offsets, statuses and return values are those of specverify.h.  A workspace
 * that is NULL or not 16-byte aligned is SV_ERR_NULL.  Work is split by the bounds max_context and
 * total_context, not by the lengths on the device: loose ones cost time, not accuracy.
 */
#ifndef SPECVERIFY_CACHE_H
#define SPECVERIFY_CACHE_H

#include "specverify.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * spec_kv_append for sequences whose positions and cache slots differ, as after
 * spec_kv_evict: row cu[b] + j is stored at slot context_lens[b] + j and turned by the
 * angles of position context_lens[b] + position_offsets[b] + j, which max_position bounds
 * (a negative offset is SV_ROW_BAD_PARAM).
 *   position_offsets  int32 [batch], or NULL: all 0
 * Everything else: as spec_kv_append.
 */
int spec_kv_append_at(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                      int64_t ld_v, int dtype, const float* q_weight, const float* k_weight,
                      float eps, const float* cos_sin, int max_position, int rot_dim,
                      int interleaved, const int32_t* cu_seqlens, const int32_t* context_lens,
                      const int32_t* position_offsets, int batch, int total_rows, int heads,
                      int kv_heads, int head_dim, void* pages, int64_t num_pages, int page_size,
                      const int32_t* page_table, int64_t ld_table, void* q_out, int64_t ld_qout,
                      void* k_values, void* v_values, int32_t* status, void* stream);

/* Bytes of workspace spec_kv_prompt_attention needs with these sizes (0 on invalid sizes,
 * and on those past two more limits: total_rows * heads, each KV head's rounded up to blocks of
 * 128 or 256 with a block more per request, stays below 2^31, at head_dim 256 below 2^30; and
 * (total_context / 32 + batch) * kv_heads, with a window the tiles of 32 positions that rows see
 * at most, below 2^24).  Most of it is the requests' cache in bf16: 4 head_dim bytes per KV head
 * and position, total_context positions (with a window: those that rows see, at most). */
size_t spec_kv_prompt_workspace_bytes(int dtype, int batch, int total_rows, int heads,
                                      int kv_heads, int head_dim, int max_context,
                                      int64_t total_context, int window, int sinks);

/*
 * Attention of whole prompts over the cache: spec_kv_attention for any number of rows per
 * request.  Row j of request b, at position p = context_lens[b] + j, sees the positions
 * t <= p, and with window > 0 only t > p - window or t < sinks; its own and the earlier
 * rows' K and V are in the cache (spec_kv_append), and so is what lies before them
 * (context_lens[b] > 0: a prompt in parts, or after a prefix that spec_kv_fork shares).
 * Formula, precision and what never reaches a row: as spec_kv_attention.
 *   q, out         [total_rows][heads][head_dim] of dtype, rows ld_q / ld_out apart, without
 *                  an element in common (SV_ERR_SHAPE; columns of one wider array are fine);
 *                  total_rows * heads < 2^31 (and spec_kv_prompt_workspace_bytes's limits)
 *   max_context    bound of context_lens[b] + rows; requests past it are
 *                  SV_ROW_BAD_PARAM, like context_lens[b] < 0
 *   total_context  bound of the sum of context_lens[b] + rows over the requests, at most
 *                  2^30; requests with which the sum passes it are SV_ROW_BAD_PARAM
 *   scale, window, sinks, status: as spec_kv_attention
 *   workspace      spec_kv_prompt_workspace_bytes(), any contents; calls that may run at
 *                  once (two captured graphs among them) need their own
 * Rows of BAD_PARAM and BAD_PAGE requests are NaN; rows of BAD_K requests (none here for
 * too many rows) and of no request are left as they were.  Identical inputs give identical
 * bits, and a request's rows depend on the call's sizes but not on the other requests.
 */
int spec_kv_prompt_attention(const void* q, int64_t ld_q, int dtype, const int32_t* cu_seqlens,
                             const int32_t* context_lens, int batch, int total_rows, int heads,
                             int kv_heads, int head_dim, const void* pages, int64_t num_pages,
                             int page_size, const int32_t* page_table, int64_t ld_table,
                             int max_context, int64_t total_context, float scale, int window,
                             int sinks, void* out, int64_t ld_out, int32_t* status,
                             void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace spec_kv_attention_weights needs with these sizes (0 on invalid sizes,
 * and on those that would be 2^23 workgroups or more). */
size_t spec_kv_weights_workspace_bytes(int dtype, int batch, int max_k, int heads, int kv_heads,
                                       int head_dim, int max_context, int window, int sinks);

/*
 * The attention weight that cached positions get from the call's rows: per request b, KV
 * head h and position t < n = context_lens[b] + rows
 *   out[b][h][t] = (t < context_lens[b] ? in[b][h][t] : 0)
 *                + sum over rows j < row_counts[b] and query heads of h of softmax_t(scale q.k)
 * the softmax over what the row sees, as in spec_kv_attention.  After a verify, row_counts =
 * accepted + 1 counts the rows that were committed; positions that were given back start from
 * 0 again when they are next written, for a call's own positions take nothing from `in`.  The
 * call goes before spec_kv_release: the rows that do not count need their pages as well (a
 * request whose release gave one back is SV_ROW_BAD_PAGE).
 * With the last 64 rows of a prompt and in = NULL it makes a new request's weights.  Scores
 * and sums in fp32, weights not rounded.  A row that sees a K block stored as NaN, or whose
 * scores leave fp32's range (see spec_kv_attention), adds nothing.
 *   q              [total_rows][heads][head_dim] of dtype, rows ld_q apart (spec_kv_append's
 *                  q_out)
 *   row_counts     int32 [batch], or NULL: all rows; outside [0, rows] is SV_ROW_BAD_PARAM
 *   weights_in     float [batch][kv_heads][ld_weights], or NULL: zeros
 *   weights_out    the same layout; weights_in itself, or memory apart from it (SV_ERR_SHAPE
 *                  where they overlap).  Written for t < n only; requests whose status is
 *                  not SV_ROW_OK are left as they were
 *   ld_weights     at least max_context
 *   max_k, max_context, scale, window, sinks, status: as spec_kv_attention
 *   workspace      spec_kv_weights_workspace_bytes(), any contents; calls that may run at
 *                  once (two captured graphs among them) need their own
 * Identical inputs give identical bits, and a request's weights depend on the call's sizes
 * but not on the other requests.
 */
int spec_kv_attention_weights(const void* q, int64_t ld_q, int dtype, const int32_t* cu_seqlens,
                              const int32_t* context_lens, const int32_t* row_counts, int batch,
                              int total_rows, int max_k, int heads, int kv_heads, int head_dim,
                              const void* pages, int64_t num_pages, int page_size,
                              const int32_t* page_table, int64_t ld_table, int max_context,
                              float scale, int window, int sinks, const float* weights_in,
                              float* weights_out, int64_t ld_weights, int32_t* status,
                              void* workspace, size_t workspace_bytes, void* stream);

/*
 * Holds requests to a budget of positions.  Request b with n = seq_lens[b] > m = budgets[b] > 0
 * keeps, per layer and KV head, its first `sinks` positions, its last `recent`, and of the
 * others the m - sinks - recent of the largest weights (the lower position where weights are
 * equal; NaN counts as less than every number, -0 as 0).  What stays moves to slots 0 .. m-1
 * in its order, codes as they are, and its weights with it (0 at m .. n-1); seq_lens[b] = m,
 * the pages past it leave the table (-1) with their counts down by one, evicted[b] += n - m.
 * Other requests (budgets[b] <= 0, or n <= m) stay as they are, SV_ROW_OK.  Bytes of slots
 * from m on are left as they were.
 * From then on slots are not positions: pass `evicted` to spec_kv_append_at, and note that
 * the window and the first positions of an attention count slots.  No other call changes
 * `evicted` or `weights`: the caller sets evicted[b] = 0 when slot b takes a new sequence (its
 * first weights then come from weights_in = NULL), and after spec_kv_fork of all of an evicted
 * request copies evicted[src] to evicted[dst], and the weights of src, in every layer, to dst.
 * status: SV_ROW_BAD_PARAM for sinks + recent > m where n > m, or, whatever the budget, a length
 * that is negative or past ld_weights or the table row; SV_ROW_BAD_PAGE for a page id outside the pool, or one of the
 * ceil(m / page_size) pages that stay having a count other than 1 (evict before forking);
 * the request then stays as it is.
 *   budgets        int32 [batch]
 *   weights        float [layers][batch][kv_heads][ld_weights]
 *   pages          pool of layer 0, layer l at + l * layer_bytes (a multiple of 16)
 *   evicted        int32 [batch], or NULL
 * Returns SV_ERR_SHAPE for sizes outside the limits above, or layers * batch * kv_heads of
 * 2^22 and more.
 */
int spec_kv_evict(const int32_t* budgets, int batch, int sinks, int recent, float* weights,
                  int64_t ld_weights, int kv_heads, int head_dim, int page_size, int32_t* seq_lens,
                  int32_t* page_table, int64_t ld_table, int32_t* ref_counts, int64_t num_pages,
                  void* pages, int layers, int64_t layer_bytes, int32_t* evicted, int32_t* status,
                  void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_CACHE_H */
