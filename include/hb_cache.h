/*
 * hb_cache.h -- C ABI (in libhb.so) of a paged KV cache held in 4 bits, of
 * the attention that reads it, and of the operations on pages: copying them
 * on the device, and forking, compacting and freeing them on the host.
 *
 * The calls stand beside hb_append_kv, hb_read_kv and
 * hb_decode_attention_noalloc (hb.h): 16-token blocks found through block
 * tables, the same positions, slots and grouped-query heads.  None needs an
 * hb_ctx, except hb_copy_blocks, which works on a context's own pools.
 *
 *   "SARATHI ..." (paper-graph-ui summary), section 3.4 "The Memory
 *   Constraint": the KV cache bounds the batch size; "Decode-Maximal
 *   Batching": what a decode costs is its KV read.  A token in 4 bits takes
 *   144 bytes per head of 128 (K and V) instead of 512.
 *   "Sarathi-Serve Guide: Chunked-Prefills & LLM Serving" (aifetchly),
 *   production checklist, "Paged KV-Cache Page Sizing": 16-token blocks;
 *   "Deep Dive": chunk row i at position offset + i attends to keys
 *   0..offset + i, a decode with ctx cached tokens to keys 0..ctx.
 *
 * Conventions: return 0 (HB_OK) or a negative HB_E* code (hb.h).  Arguments
 * the host can see are checked before any launch; on an error code other
 * than HB_ECUDA and HB_ENOMEM (no host memory, from any call) nothing was
 * enqueued.  Work is enqueued on cuda_stream (a
 * cudaStream_t, NULL = the legacy default stream) of the current device,
 * which must be the one the pointers belong to; no call waits, allocates or
 * keeps state, so every call may be captured into a CUDA graph.  Calls on
 * different streams, and graphs that can run at the same time, need
 * workspaces of their own.  "device" pointers are device memory.
 */
#ifndef HB_CACHE_H
#define HB_CACHE_H

#include <stdint.h>

#include "hb.h"

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#pragma GCC visibility push(default)
#endif

/* ------------------------------------------------- the cache in 4 bits
 *
 * data: device bytes [num_blocks][n_kv_heads][18 head_dim], 16-byte aligned
 * (head_dim 64 or 128, NB = head_dim / 16).  Each (block, kv head) holds
 *   K codes   [token 16][t 4][NB][2]        byte b of (token, t, block i):
 *             channels 16 i + 4 t + 2 b (low 4 bits) and the next (high)
 *   V codes   [h 2][g 8][t 4][u 2][NB]      token 4 t + 2 h + u, channels
 *             16 i + 2 g (low 4 bits) and the next (high)
 *   K scales  [token 16][NB], V scales [NB][token 16]
 * A code is e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), a scale
 * e4m3; the value is code * scale * k_scale (or v_scale).
 *
 * Quantisation of 16 neighbouring channels x of a token's head: the scale is
 * max|x| / (6 k_scale) rounded to e4m3 (nearest, ties to even, at most 448),
 * each code x / (scale k_scale) rounded to e2m1 (nearest, ties to even, at
 * most 6), both quotients of fp32 numbers.  A scale that rounds to 0 stores
 * zeros.  An infinity stores the largest value, 6 * 448 * k_scale; a NaN
 * makes its 16 channels NaN.  k_scale, v_scale: finite, in [2^-60, 2^60]; 1
 * suits keys and values of ordinary size (below 2688). */
typedef struct {
    void *data;
    int num_blocks, n_kv_heads, head_dim;
    float k_scale, v_scale;
} hb_kv4_pool;

/* Bytes of a pool's data, or HB_EINVAL for dimensions it cannot have. */
long long hb_kv4_pool_bytes(int num_blocks, int n_kv_heads, int head_dim);

/* Quantise n_tokens rows of K (post-RoPE) and V and store row i at slots[i]
 * (block * 16 + offset, as hb_plan gives them).
 *   k, v:  device bf16, row i at k + i * k_stride elements, [n_kv_heads]
 *          [head_dim] dense inside a row; 16-byte aligned, strides multiples
 *          of 8 and >= n_kv_heads * head_dim (any stride for one row)
 *   slots: device int32 [n_tokens].  A slot outside [0, 16 num_blocks) (-1
 *          marks padding) stores nothing.  Two rows with one slot race: the
 *          slot then holds a mix of the two.
 * Errors: HB_EINVAL (bad argument), HB_ERANGE (more work than one
 * launch holds: n_tokens * n_kv_heads of the order of 10^10), HB_ECUDA.
 * n_tokens = 0 does nothing. */
int hb_kv4_append(const hb_kv4_pool *pool, const void *k, long long k_stride, const void *v, long long v_stride,
                  const int32_t *slots, int n_tokens, void *cuda_stream);

/* Read back the values at slots as bf16: code * (scale * k_scale) in fp32,
 * rounded to bf16.  Layout and conditions of hb_kv4_append.  A row whose slot
 * lies outside the pool is left as it was. */
int hb_kv4_read(const hb_kv4_pool *pool, const int32_t *slots, int n_tokens, void *k, long long k_stride, void *v,
                long long v_stride, void *cuda_stream);

/* Decode attention over the 4-bit cache, the counterpart of
 * hb_decode_attention_noalloc: query j at position ctx_lens[j] attends keys
 * 0..ctx_lens[j] of its own sequence, softmax(q k^T / sqrt(head_dim)) v, head
 * h reading kv head h / (n_heads / n_kv_heads).  The values are those that
 * hb_kv4_read gives, before their rounding to bf16; sums and softmax
 * statistics are fp32.  The weights lie in f16 (11 bits) about the row's
 * largest: a key may add nothing to the sum of V where its weight is below
 * 2^-36 of the largest, or, where one query (head_dim 128) or two (64) share a
 * kv head, where its weight times its V scale is below 2^-34 of the largest
 * weight times the largest V scale of the 16 channels.
 *   q, out:       device bf16, row j at q + j * q_stride elements, [n_heads]
 *                 [head_dim] dense inside a row; conditions as k above.
 *                 out may not overlap q or the pool
 *   block_tables: device int32 [n_decodes][bt_stride], bt_stride >=
 *                 max_ctx / 16 + 1
 *   ctx_lens:     device int32 [n_decodes], each in [0, max_ctx], or -1: a
 *                 padding row, which attends nothing and gets zeros
 *   workspace:    device, 16-byte aligned, of at least
 *                 hb_kv4_decode_workspace() bytes (which may be 0); its
 *                 contents mean nothing before and after the call
 * A row whose ctx_lens entry lies outside [-1, max_ctx], or whose table holds
 * a block id outside the pool among those it needs, gets NaN and reads
 * nothing there.  Bytes of slots past a row's context never reach its result.
 * The split of a row's keys depends on max_ctx, n_decodes and the heads, so
 * results of differently shaped calls agree to fp32 rounding, not bit for
 * bit; one call repeated gives the same bits.
 * Errors: HB_EINVAL, HB_ERANGE (bt_stride too small, workspace too small, more
 * than 65535 rows, or max_ctx of 2^27 or more), HB_ECUDA.  n_decodes = 0 does
 * nothing. */
int hb_kv4_decode(const hb_kv4_pool *pool, const void *q, long long q_stride, const int32_t *block_tables,
                  int bt_stride, const int32_t *ctx_lens, int n_decodes, int n_heads, int max_ctx, void *out,
                  long long out_stride, void *workspace, long long workspace_bytes, void *cuda_stream);
long long hb_kv4_decode_workspace(int n_decodes, int n_heads, int n_kv_heads, int head_dim, int max_ctx);

/* Attention of one prefill chunk over the 4-bit cache: row i at position
 * chunk_offset + i attends keys 0..chunk_offset + i, which the cache must
 * hold by then (hb_kv4_append before this call on the same stream).
 *   q, out:      as for hb_kv4_decode, chunk_len rows
 *   block_table: device int32 [n_blocks] covering positions
 *                0..chunk_offset + chunk_len - 1 (HB_ERANGE if n_blocks is
 *                too small).  A block id outside the pool makes the rows that
 *                attend to it NaN (and may make other rows of the chunk NaN)
 * Workspace and errors as for hb_kv4_decode, rounding as there or with V scales
 * of any size beside each other (2^-36 of the largest weight); chunk_offset +
 * chunk_len is at most 2^27, chunk_len times the heads of a kv head at most
 * 2^24 (HB_ERANGE, also for a chunk of more work than a launch can count, of
 * the order of 10^15 scores).  chunk_len = 0 does nothing. */
int hb_kv4_chunk(const hb_kv4_pool *pool, const void *q, long long q_stride, const int32_t *block_table, int n_blocks,
                 int chunk_offset, int chunk_len, int n_heads, void *out, long long out_stride, void *workspace,
                 long long workspace_bytes, void *cuda_stream);
long long hb_kv4_chunk_workspace(int chunk_offset, int chunk_len, int n_heads, int n_kv_heads, int head_dim);

/* Test hook for the failure path of the two attention calls: in this thread's
 * next hb_kv4_decode or hb_kv4_chunk that launches, the first CTA leaves out
 * the copy of its first page, so that its waits run out (after 2 s at most,
 * as they always would).  The rows and heads of that CTA become NaN, after
 * its copies and products under way have ended; the others, and the calls
 * after it, are as ever. */
void hb_kv4_test_lost_page(void);

/* ------------------------------------------------- pages on the device
 *
 * Copy page src[i] to page dst[i], i < n, in each of n_pools pools: pool p's
 * page b is the page_bytes bytes at data + p * pool_stride + b * page_bytes.
 * A pool is any array of pages (a bf16 K or V pool of a layer, an hb_kv4_pool),
 * device memory; data, pool_stride and page_bytes are multiples of 16, and no
 * pool reaches into the next.
 *   src, dst: host int32 [n], in [0, num_blocks); read during the call.  A
 *             page may be the source of several copies (forks), but a
 *             destination may be neither repeated nor a source of the same
 *             call, so the order of the copies does not matter.
 * Errors: HB_EINVAL (bad argument, or src and dst that break this rule),
 * HB_ERANGE (a page outside [0, num_blocks)), HB_ECUDA.  n = 0 does nothing. */
int hb_copy_pages(void *data, long long pool_stride, int n_pools, long long page_bytes, int num_blocks,
                  const int32_t *src, const int32_t *dst, int n, void *cuda_stream);

/* hb_copy_pages over the K and V pools of every layer of a context, on its
 * stream.  Errors as above, with their text in hb_last_error. */
int hb_copy_blocks(hb_ctx *ctx, const int32_t *src, const int32_t *dst, int n);

/* ------------------------------------------------- pages on the host
 *
 * A page table: which pages each sequence's tokens lie in, with a count of
 * the sequences that hold each page.  Host only; it says which pages to copy
 * (hb_copy_pages, hb_copy_blocks) and touches no device memory.  Free pages
 * are handed out lowest id first.  Not thread-safe.  Pointers to arrays are
 * host memory of the caller. */
typedef struct hb_pages hb_pages;

/* A table of num_blocks free pages of 16 tokens (at most 2^27 - 1, as many as
 * a pool of the 4-bit cache may have).  HB_EINVAL, HB_ENOMEM. */
int hb_pages_create(int num_blocks, hb_pages **out);
void hb_pages_destroy(hb_pages *p);

/* Grow sequence seq (any int; a new one starts empty) to n_tokens tokens.
 * The pages that the new tokens need are taken; and if their first lies in
 * a part-filled page that another sequence holds too, seq gets a page of its
 * own in its place: *copy_src and *copy_dst then name the pages to copy
 * before the new tokens are written (else both are -1).  A call that does
 * not grow the sequence changes nothing.  HB_EINVAL (NULL, n_tokens < the
 * sequence's length or < 0), HB_ENOMEM (not enough free pages; nothing
 * changed). */
int hb_pages_extend(hb_pages *p, int seq, int n_tokens, int32_t *copy_src, int32_t *copy_dst);

/* child, which must not exist, becomes a sequence that shares every page of
 * parent's first n_tokens tokens (0 <= n_tokens <= its length; -1: all of
 * them).  No page is taken or copied.  HB_EINVAL. */
int hb_pages_fork(hb_pages *p, int parent, int child, int n_tokens);

/* Forget a sequence; pages that no other sequence holds become free.
 * HB_EINVAL when there is none. */
int hb_pages_release(hb_pages *p, int seq);

/* Move held pages to the front: each of the highest held pages moves to the
 * lowest free one while that lowers its id, at most max_moves of them.  The
 * tables are changed at once; copy page src[i] to dst[i] (src and dst have
 * room for max_moves and meet the rule of hb_copy_pages) before the cache is
 * used again.  Returns the number of moves (0: compact already) or
 * HB_EINVAL. */
int hb_pages_compact(hb_pages *p, int32_t *src, int32_t *dst, int max_moves);

/* The pages of a sequence in order: up to max_blocks of them to table.
 * Returns how many it has (its length in tokens to *n_tokens unless NULL), or
 * HB_EINVAL when there is no such sequence. */
int hb_pages_table(hb_pages *p, int seq, int32_t *table, int max_blocks, int *n_tokens);

/* Free pages; sequences that hold page block (HB_ERANGE outside the table). */
int hb_pages_num_free(hb_pages *p);
int hb_pages_refcount(hb_pages *p, int block);

#if defined(__GNUC__)
#pragma GCC visibility pop
#endif

#ifdef __cplusplus
}
#endif

#endif /* HB_CACHE_H */
