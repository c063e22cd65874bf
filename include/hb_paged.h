/*
 * hb_paged.h -- C ABI (in libhb.so) of attention over a paged bf16 KV cache
 * whose sequences share long prefixes, and of eviction from such a cache by
 * accumulated attention weight.
 *
 * The calls stand beside hb_decode_attention_noalloc (hb.h), hb_kv4_decode and
 * the page table hb_pages_* (hb_cache.h): the same pools, 16-token blocks,
 * block tables, positions and grouped-query heads.  None needs an hb_ctx.
 * They are for a program with a model of its own: hb_forward takes a row's
 * position for its place in the cache, which an eviction ends.
 *
 *   "SARATHI ..." (paper-graph-ui summary), section 3.4 "Decode-Maximal
 *   Batching": what a decode costs is its KV read, which rows behind one
 *   prefix can share; "The Memory Constraint": the KV cache bounds the batch.
 *   "Sarathi-Serve Guide: Chunked-Prefills & LLM Serving" (aifetchly),
 *   production checklist: 16-token blocks, prefix reuse; "Deep Dive": a
 *   decode with ctx cached tokens attends keys 0..ctx.
 *
 * Conventions, as in hb_cache.h: return 0 (HB_OK) or a negative HB_E* code.
 * Arguments the host can see are checked before any launch; on an error code
 * other than HB_ECUDA nothing was enqueued.  Work is enqueued on cuda_stream
 * (a cudaStream_t, NULL = the legacy default stream) of the current device,
 * which must be the one the pointers belong to; no call waits, allocates or
 * keeps state, so every call may be captured into a CUDA graph.  Calls on
 * different streams, and graphs that can run at the same time, need
 * workspaces of their own.  "device" pointers are device memory, "host"
 * pointers are read during the call.
 */
#ifndef HB_PAGED_H
#define HB_PAGED_H

#include <stdint.h>

#include "hb.h"

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#pragma GCC visibility push(default)
#endif

/* K (post-RoPE) and V pools: device bf16 [num_blocks][n_kv_heads][16]
 * [head_dim], 16-byte aligned, head_dim 64 or 128, fewer than 2^27 blocks. */
typedef struct {
    void *k, *v;
    int num_blocks, n_kv_heads, head_dim;
} hb_paged_pool;

/* A pool of one fp32 number for each token and kv head: device fp32
 * [num_blocks][n_kv_heads][16], 16-byte aligned, found through block tables
 * of its own (which may be the cache's); fewer than 2^27 blocks. */
typedef struct {
    float *data;
    int num_blocks, n_kv_heads;
} hb_weight_pool;

/* ------------------------------------------------- shared prefixes
 *
 * Decode attention of rows in groups.  Row j at position ctx_lens[j] attends
 * keys 0..ctx_lens[j] of its own sequence, softmax(q k^T / sqrt(head_dim)) v,
 * head h reading kv head h / (n_heads / n_kv_heads), as in
 * hb_decode_attention_noalloc.  Rows are ordered by group: the first
 * group_rows[0] rows are group 0, and so on.  The first prefix_lens[g] tokens
 * of all rows of group g are the same (a fork's shared pages, and the same
 * tokens in each row's copy of a part-filled one); their keys are read once
 * for the whole group, whole blocks of them through the table of the group's
 * first row (also where that is a padding row).
 *   q, out:       device bf16, row j at q + j * q_stride elements, [n_heads]
 *                 [head_dim] dense inside a row; 16-byte aligned, strides
 *                 multiples of 8 and >= n_heads * head_dim (any stride for
 *                 one row).  out may not overlap q or the pools
 *   block_tables: device int32 [n_rows][bt_stride], bt_stride >=
 *                 max_ctx / 16 + 1: the whole table of each row, prefix
 *                 included
 *   ctx_lens:     device int32 [n_rows], each in [prefix_len - 1, max_ctx] (of
 *                 its group, and not below 0), or -1: a padding row, which
 *                 attends nothing and gets zeros
 *   group_rows:   host int32 [n_groups], each > 0, n_rows in all
 *   prefix_lens:  host int32 [n_groups], each in [0, max_ctx + 1]
 *   max_ctx:      what ctx_lens may be at most.  Prefixes are cut beside own keys
 *                 as long as it allows: one far above them is right, but leaves a
 *                 prefix of few kv heads to few SMs
 *   workspace:    device, 16-byte aligned, of at least
 *                 hb_decode_shared_workspace() bytes (which may be 0); its
 *                 contents mean nothing before and after the call
 * A row whose ctx_lens entry lies outside its range, or whose keys lie in a
 * block id outside the pool, gets NaN and reads nothing there; a bad block of
 * a prefix makes its group's rows NaN.  Bytes of slots past a row's context
 * never reach its result.  Sums and softmax statistics are fp32 (a q . k that
 * overflows it makes its row NaN), the weights keep 16 significant bits;
 * an infinity in V that a row sees is its result in that channel, beside the
 * opposite one NaN, and either where its weight is 0 in fp32;
 * results of differently shaped calls, or beside rows of other lengths, agree to
 * fp32 rounding, not bit for bit; one call repeated gives the same bits.
 * Errors: HB_EINVAL, HB_ERANGE (bt_stride or workspace too small, max_ctx of
 * 2^27 or more, more than 65535 rows, more work than one launch holds),
 * HB_ECUDA.  n_rows = n_groups = 0 does nothing. */
int hb_decode_shared(const hb_paged_pool *pool, const void *q, long long q_stride, const int32_t *block_tables,
                     int bt_stride, const int32_t *ctx_lens, int n_rows, int n_heads, int max_ctx,
                     const int32_t *group_rows, const int32_t *prefix_lens, int n_groups, void *out,
                     long long out_stride, void *workspace, long long workspace_bytes, void *cuda_stream);
long long hb_decode_shared_workspace(int n_rows, int n_heads, int n_kv_heads, int head_dim, int max_ctx,
                                     const int32_t *group_rows, const int32_t *prefix_lens, int n_groups);

/* ------------------------------------------------- weights
 *
 * Attention of n_queries rows a sequence (1: a decode; more: a window of a
 * prompt's last rows), which also adds up how much weight each key got.
 * Query i of sequence j is row j * n_queries + i, at position p = ctx_lens[j]
 * - (n_queries - 1) + i, and attends keys 0..p (none where p < 0: such a row
 * gets zeros).  With the weights p[i][h][t] of its softmax,
 *   w[t] = decay * w[t] + sum of p[i][h][t] over i and the heads h of a kv head
 * for every token t <= ctx_lens[j] and kv head.  A token of the call's own rows
 * (t > ctx_lens[j] - n_queries) starts from 0 whatever its slot held, and with
 * decay 0 every token does.
 *   q, out:        as for hb_decode_shared, n_seqs * n_queries rows
 *   block_tables:  device int32 [n_seqs][bt_stride], ctx_lens [n_seqs], each
 *                  in [0, max_ctx], or -1: a padding sequence, whose rows get
 *                  zeros and whose weights stay as they are
 *   weights, weight_tables: device int32 [n_seqs][wt_stride], wt_stride >=
 *                  max_ctx / 16 + 1.  No two sequences of a call may have a
 *                  weight block in common, nor has one sequence a block twice:
 *                  its slots would hold either's sums
 *   max_ctx:       as above: a window's common keys are cut by it
 *   decay:         finite, in [0, 1]
 *   workspace:     as above, hb_decode_weigh_workspace() bytes (4 for each row,
 *                  head and key of max_ctx, and partial results)
 * A sequence whose ctx_lens entry lies outside [-1, max_ctx] gets NaN and its
 * weights stay as they are.  A sequence with a block id outside the pool gets
 * NaN.  A row and head whose softmax is not a number, from a bad block or from
 * its keys, adds nothing to the weights.  A weight block outside its pool is
 * neither read nor written.  Weights that are 0 in fp32 are added as 0; sums
 * are fp32 and in a fixed order.
 * Errors: as for hb_decode_shared; n_queries in [1, 1024], n_seqs * n_queries
 * at most 65535.  n_seqs = 0 does nothing. */
int hb_decode_weigh(const hb_paged_pool *pool, const void *q, long long q_stride, const int32_t *block_tables,
                    int bt_stride, const int32_t *ctx_lens, int n_seqs, int n_queries, int n_heads, int max_ctx,
                    const hb_weight_pool *weights, const int32_t *weight_tables, int wt_stride, float decay, void *out,
                    long long out_stride, void *workspace, long long workspace_bytes, void *cuda_stream);
long long hb_decode_weigh_workspace(int n_seqs, int n_queries, int n_heads, int n_kv_heads, int head_dim, int max_ctx);

/* Test hook for the failure path of the two attention calls: in this thread's
 * next hb_decode_shared or hb_decode_weigh that attends keys for several rows
 * at once, the first CTA to do so leaves out one copy, so that its waits run
 * out (after 2 s, as they always would).  The rows and heads of that CTA become
 * NaN, after its copies and products under way have ended, and add nothing to
 * weights; the others, and the calls after it, are as ever. */
void hb_paged_test_lost_block(void);

/* ------------------------------------------------- eviction
 *
 * Choose the tokens that stay: for each sequence j and kv head, of its
 * lens[j] tokens the first n_first, the last n_recent, and of those between
 * the ones of the largest weight, keep in all (the lower position first where
 * weights are equal; a NaN, and a token whose weight block lies outside the
 * pool, below every number).  A sequence of at most keep tokens keeps all.
 *   weight_tables: device int32 [n_seqs][wt_stride], wt_stride >=
 *                  (max_len + 15) / 16
 *   lens:          device int32 [n_seqs], each in [0, max_len]; outside, none
 *                  is kept
 *   kept:          device int32 [n_seqs][n_kv_heads][keep]: the positions in
 *                  ascending order, then -1
 * keep > 0, n_first and n_recent >= 0, n_first + n_recent <= keep.
 * Errors: HB_EINVAL, HB_ERANGE (wt_stride too small, max_len above 2^27, more
 * work than one launch holds), HB_ECUDA.  n_seqs = 0 does nothing. */
int hb_evict_select(const hb_weight_pool *weights, const int32_t *weight_tables, int wt_stride, const int32_t *lens,
                    int n_seqs, int max_len, int keep, int n_first, int n_recent, int32_t *kept, void *cuda_stream);

/* Move the kept tokens: for each sequence, kv head and i < keep with
 * kept[i] >= 0, slot i of the new table gets K and V of slot kept[i] of the
 * old one (and, unless weights is NULL, slot i of new_weight_tables gets its
 * weight).  kept as hb_evict_select writes it: ascending, so kept[i] >= i,
 * then -1; other orders give wrong results where blocks are reused.
 *   block_tables, new_tables: device int32 [n_seqs][bt_stride] and
 *     [n_seqs][new_stride]; new_stride >= (keep + 15) / 16
 * A new block is either one that no sequence of the call reads, or the old
 * table's own at the same place (a cache compacted where it is: the two
 * tables may be the same memory), and no block is written twice.
 * The same holds for the weights' tables (strides wt_stride, new_wt_stride).
 * A position beyond the old table, or a block id outside the pool, old or new,
 * is skipped: the new slot stays as it was.
 * Errors: as for hb_evict_select; HB_ERANGE also where num_blocks * n_kv_heads
 * * 16 of either pool passes 2^32 - 2. */
int hb_evict_move(const hb_paged_pool *pool, const int32_t *block_tables, int bt_stride, const int32_t *new_tables,
                  int new_stride, const int32_t *kept, int n_seqs, int keep, const hb_weight_pool *weights,
                  const int32_t *weight_tables, int wt_stride, const int32_t *new_weight_tables, int new_wt_stride,
                  void *cuda_stream);

#if defined(__GNUC__)
#pragma GCC visibility pop
#endif

#ifdef __cplusplus
}
#endif

#endif /* HB_PAGED_H */
