/*
 * dcp_paged.h -- C ABI of libdcpcombine.so, second part: one rank's shard of a paged
 * key-value cache under decode context parallelism (DCP), on NVIDIA B200 (sm_100a).
 *
 * dcp_combine.h merges the partial attention results of N ranks.  The calls here produce a
 * rank's partial result and keep the cache it is computed from:
 *
 *   dcp_kv_append            rows of new tokens -> the pages of the rank that owns their positions
 *   dcp_paged_attention      attention of one new token per request over the rank's shard,
 *                            with its LSE (and, on request, its logits)
 *   dcp_paged_attention_pack the same, written straight into the packed send buffer of dcp_pack
 *   dcp_kv_weights           logits + LSE over all shards -> accumulated attention weights
 *   dcp_kv_evict             the positions of largest accumulated weight moved into new pages
 *
 * The cache.  A request's positions on this rank are numbered 0, 1, ... ("local positions").
 * Local position p of request b lies in slot p mod page_size of page
 * block_table[b][p / page_size]; each slot holds `heads` key rows and `heads` value rows of
 * head_dim elements.  Pages may be shared between requests (a common prefix) by every call
 * that only reads them.
 *
 * Which positions a rank holds (vllm-ascend, vllm_ascend/attention/context_parallel/sfa_cp.py,
 * _get_dcp_local_seq_lens): blocks of `interleave` consecutive positions of a request are dealt
 * round-robin to `num_shards` ranks.  With B = interleave * num_shards, rank `shard` holds
 *   (L / B) * interleave + min(max(L mod B - shard * interleave, 0), interleave)
 * of a request's L = seq_lens[b] positions.  num_shards = 1 takes seq_lens as the local lengths
 * themselves (a cache after dcp_kv_evict, or no DCP).  A negative length counts as 0, and a length
 * is cut to what the block table's max_pages pages can hold.
 *
 * A block-table entry that a length reaches but that is outside [0, num_pages) names no memory:
 * nothing is read or written there, and the positions in it count as not held (attention), or
 * are left out (append, evict).  Entries past a request's length are not read.
 *
 * The conventions of dcp_combine.h hold here too: device pointers on the current device, the
 * caller owns every buffer, asynchronous on `cuda_stream`, every argument checked on the host
 * before any launch, outputs must not overlap inputs (or one another) unless a call says so,
 * sizes and strides in elements, B == 0 a no-op, no host synchronisation, safe to capture into
 * a CUDA graph.
 */
#ifndef DCP_PAGED_H
#define DCP_PAGED_H

#include <stdint.h>

#include "dcp_combine.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest head_dim of the paged calls. */
#define DCP_MAX_PAGED_DIM 256
/* Largest number of key heads of a paged cache. */
#define DCP_MAX_PAGED_HEADS (1 << 20)

/*
 * A paged cache and the block table of the requests at hand.  Element d of key head h in slot
 * s of page p is at k + p*k_stride_page + s*k_stride_slot + h*k_stride_head + d (elements of
 * `dtype`), values alike, so [pages, slots, heads, D], [pages, heads, slots, D] and K/V
 * interleaved pools are all described.
 *
 * Requirements: dtype a dcp_dtype; head_dim in [1, DCP_MAX_PAGED_DIM] with rows a multiple of
 * 16 bytes; heads in [1, DCP_MAX_PAGED_HEADS]; page_size >= 1; num_pages >= 0; max_pages >= 0; max_pages * page_size
 * < 2^31 - 1024; k and v 16-byte aligned; strides >= 0 and multiples of 16 bytes; block_table 4-byte
 * aligned, entry (b, j) at b*table_stride + j.  In a cache that a call writes (append, evict's dst) the
 * rows must not overlap; strides (of dimensions of two or more entries) under which they do are refused.
 */
typedef struct {
    void *k;
    void *v;
    const int32_t *block_table; /* [requests, max_pages], device */
    int64_t num_pages;
    int64_t k_stride_page, k_stride_slot, k_stride_head;
    int64_t v_stride_page, v_stride_slot, v_stride_head;
    int64_t table_stride;
    int64_t max_pages;
    int32_t page_size;
    int32_t heads;
    int32_t head_dim;
    int32_t dtype;
} dcp_paged_kv;

/*
 * Bytes of workspace that dcp_paged_attention and dcp_paged_attention_pack need on the current
 * device for these sizes (0 for none, -1 for sizes they refuse).  It does not depend on B or on
 * any length.
 */
int64_t dcp_paged_attention_workspace(int64_t H, int32_t heads, int32_t head_dim, int32_t dtype);

/*
 * Attention of one new token per request over this rank's shard of the cache.  Query head h
 * reads key head h / (H / heads).  With n held positions of request b and
 * x_p = scale * (q[b,h] . k_p):
 *   m      = max_p x_p
 *   result = sum_p exp(x_p - m) v_p / sum_p exp(x_p - m)      (fp32 sums, one rounding)
 *   lse    = ln(sum_p exp(x_p - m)) + m                       (log2 in base 2)
 * A request without held positions gives 0 and -inf, which dcp_lse_combine then leaves out.
 * A position whose logit is -inf adds nothing (16-bit types), a row whose logits are all -inf counts as
 * empty.  A value that is not finite gives its column what IEEE products with the weights give: infinities
 * of one sign that infinity; a NaN, both signs, or an infinity whose weight is 0 (a logit of -inf, or
 * one some 90 or more below the row's largest) NaN.  A row that meets a non-finite fp32 key is NaN; fp32 keys
 * and values of magnitude 2^128 - 2^116 or more make NaN of their row, or of their column.
 * For 16-bit types exp(x_p - m) is carried into the product with v as two 16-bit parts; fp32
 * products are formed from two tf32 parts of each factor (2^-20 of the product).
 *
 * q           [B, H, head_dim] of kv->dtype; element (b, h, d) at b*q_stride_b + h*q_stride_h + d.
 * seq_lens    [B] int32, device.
 * Pages of a multiple of 8 slots are read with tensor copies, through maps the call encodes (as
 * dcp_pack does); a wait for them that runs out (never, while the copies work) is counted by
 * dcp_wait_timeouts.  Other page sizes, and pools whose maps the driver refuses, are read row by row.
 * Same result up to the order of sums.
 *
 * result      [B, H, head_dim] of kv->dtype, contiguous.
 * lse         [B, H] fp32, contiguous.
 * logits      NULL, or fp32: x_p of head h goes to b*logits_stride_b + h*logits_stride_h + p for
 *             the held positions p < logits_cap (the others are left as they were; a position
 *             in a page outside the pool gets -inf).  Its rows must not overlap: strides under which
 *             rows of logits_cap do are refused (B or H of 1: its stride does not matter).
 * workspace   at least dcp_paged_attention_workspace bytes, 16-byte aligned; its contents need no
 *             initialisation and mean nothing afterwards.  Calls that may run at the same time
 *             need one each.
 *
 * Requirements: those of dcp_paged_kv, and no row of a pool further than 2^32 units from its start,
 * a unit being the largest power of two up to 4096 bytes that divides all strides (64 GB for
 * strides of odd multiples of 16 bytes); H a multiple of heads (else DCP_ERR_SHAPE); q and result
 * 16-byte aligned, q strides multiples of 16 bytes and >= 0; B*H < 2^31; shard in
 * [0, num_shards), num_shards in [1, DCP_MAX_SHARDS], interleave >= 1; scale finite.
 */
int32_t dcp_paged_attention(const dcp_paged_kv *kv, const void *q, const int32_t *seq_lens, void *result, float *lse,
                            float *logits, int64_t B, int64_t H, int64_t q_stride_b, int64_t q_stride_h,
                            int64_t logits_stride_b, int64_t logits_stride_h, int64_t logits_cap, float scale,
                            int32_t shard, int32_t num_shards, int32_t interleave, int32_t is_lse_base_on_e,
                            void *workspace, int64_t workspace_bytes, void *cuda_stream);

/*
 * The same with the result written as dcp_pack would write it: send_buf [world_size, B,
 * H/world_size, head_dim + P] of kv->dtype, contiguous, row (r, b, h) = the result row of head
 * r*H/world_size + h followed by the 4 bytes of its LSE.  The same values as dcp_paged_attention,
 * then dcp_pack.
 * Requirements: as above; world_size in [1, DCP_MAX_SHARDS]; H % world_size == 0 (else
 * DCP_ERR_SHAPE); send_buf 16-byte aligned.
 */
int32_t dcp_paged_attention_pack(const dcp_paged_kv *kv, const void *q, const int32_t *seq_lens, void *send_buf,
                                 float *logits, int64_t B, int64_t H, int32_t world_size, int64_t q_stride_b,
                                 int64_t q_stride_h, int64_t logits_stride_b, int64_t logits_stride_h,
                                 int64_t logits_cap, float scale, int32_t shard, int32_t num_shards,
                                 int32_t interleave, int32_t is_lse_base_on_e, void *workspace,
                                 int64_t workspace_bytes, void *cuda_stream);

/*
 * Writes the key and value rows of new tokens into the cache.  The tokens of request r are
 * t = query_start_loc[r] .. query_start_loc[r+1]-1, the last ones of its seq_lens[r] positions:
 * token t has position seq_lens[r] - (query_start_loc[r+1] - t).  This rank writes those whose
 * position it holds (blocks of `interleave` positions dealt to num_shards ranks); the others, tokens
 * outside every request, with a negative position, past max_pages pages or in a page outside
 * the pool are skipped.  Bit-exact copies.  Where two tokens of one call land in the same slot (pages
 * shared between requests that both append), each element of its rows is one of the two tokens', without
 * an order: the key row may hold parts of both, and the value row another mixture.
 *
 * k_new, v_new  [T, heads, head_dim] of kv->dtype; element (t, h, d) at t*stride_t + h*stride_h + d.
 * seq_lens      [num_reqs] int32, device: lengths over all shards, the new tokens included (a length of 0
 *               leaves out the request's tokens, as after an eviction those that another rank owns).
 * query_start_loc [num_reqs + 1] int32, device, non-decreasing (other values give unspecified
 *               rows but no access outside the arrays).
 *
 * Requirements: those of dcp_paged_kv; T >= 0 (0 is a no-op), num_reqs >= 0; T * heads < 2^31;
 * k_new and v_new 16-byte aligned, strides multiples of 16 bytes and >= 0.
 */
int32_t dcp_kv_append(const dcp_paged_kv *kv, const void *k_new, const void *v_new, const int32_t *seq_lens,
                      const int32_t *query_start_loc, int64_t T, int32_t num_reqs, int64_t k_stride_t,
                      int64_t k_stride_h, int64_t v_stride_t, int64_t v_stride_h, int32_t shard, int32_t num_shards,
                      int32_t interleave, void *cuda_stream);

/*
 * Adds this step's attention weights to the accumulated ones:
 *   weights[b,j,p] += sum over the H/heads query heads h of key head j of
 *                     exp(logits[b,h,p] - global_lse[b,h])
 * for the held positions p of each request (p < cap).  global_lse is the LSE over ALL shards
 * (base e, or base 2 with is_lse_base_on_e = 0; logits are natural), so the weights of a
 * request's positions over all ranks sum to 1 per query head.  A head whose global LSE is NaN
 * or infinite adds nothing.  The heads are summed in order, in fp32, and added to the weight once.
 *
 * logits      fp32; element (b, h, p) at b*logits_stride_b + h*logits_stride_h + p.
 * global_lse  fp32; element (b, h) at b*lse_stride_b + h*lse_stride_h.
 * seq_lens    [B] int32, device.
 * weights     fp32, updated in place; element (b, j, p) at b*weights_stride_b + j*weights_stride_h + p.
 *
 * Requirements: B >= 0; heads >= 1; H a multiple of heads (else DCP_ERR_SHAPE); cap in [0, 2^31);
 * strides >= 0; the rows of weights must not overlap (strides under which they do are refused); all pointers 4-byte aligned; B*H < 2^31.
 */
int32_t dcp_kv_weights(const float *logits, const float *global_lse, const int32_t *seq_lens, float *weights,
                       int64_t B, int64_t H, int64_t heads, int64_t cap, int64_t logits_stride_b,
                       int64_t logits_stride_h, int64_t lse_stride_b, int64_t lse_stride_h, int64_t weights_stride_b,
                       int64_t weights_stride_h, int32_t shard, int32_t num_shards, int32_t interleave,
                       int32_t is_lse_base_on_e, void *cuda_stream);

/*
 * Eviction.  For each request b and key head j with n held positions:
 *   - n <= keep: every position is kept;
 *   - otherwise the last `recent` positions are kept, and of the n - recent before them the
 *     keep - recent of largest weights[b,j,p] (ties to the lowest position; +0 and -0 tie;
 *     NaN ranks below every number).
 * The kept positions, in increasing order, become local positions 0, 1, ... of the request in
 * dst: their key and value rows are copied to dst's pages and their weights to new_weights, whose
 * remaining entries become 0.  The selection is per key head, the new length
 * min(n, keep) the same for all of them.
 *
 * src         the cache read; `heads`, head_dim and dtype must equal dst's.
 * dst         the cache written (pools may be the same): its block table names the new pages,
 *             max_pages * page_size >= keep.  Pages written must not be pages that any request of
 *             the call reads, nor named twice, else the rows there are unspecified.  Rows whose source or
 *             destination page is outside its pool are not copied.
 * weights     fp32 [B, heads, cap], element (b, j, p) at b*weights_stride_b + j*weights_stride_h + p;
 *             lengths are cut to cap.
 * new_weights fp32 [B, heads, new_cap], strides alike; all new_cap entries are written; new_cap
 *             >= keep.  Must not overlap weights, nor its rows one another (strides under which they
 *             do are refused).
 * kept        [B, heads, keep] int32, contiguous: the kept positions, then -1.
 * new_lens    [B] int32: min(n, keep).
 *
 * Requirements: those of dcp_paged_kv for both; keep in [1, 2^31), recent in [0, keep];
 * B * heads < 2^31; weights, new_weights, kept, new_lens 4-byte aligned.
 */
int32_t dcp_kv_evict(const dcp_paged_kv *src, const dcp_paged_kv *dst, const int32_t *seq_lens, const float *weights,
                     float *new_weights, int32_t *kept, int32_t *new_lens, int64_t B, int64_t cap, int64_t new_cap,
                     int64_t weights_stride_b, int64_t weights_stride_h, int64_t new_weights_stride_b,
                     int64_t new_weights_stride_h, int64_t keep, int64_t recent, int32_t shard, int32_t num_shards,
                     int32_t interleave, void *cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* DCP_PAGED_H */
