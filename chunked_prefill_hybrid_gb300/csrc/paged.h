// paged.h -- what the calls of include/hb_paged.h share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "hb_paged.h"

namespace hb {
namespace paged {

constexpr int MAX_KEYS = 1 << 27;
constexpr int INLINE_GROUPS = 16;  // groups that fit the kernels' parameters

// Rows row0..row0 + rows - 1; prefix: tokens that they share, as the caller
// says; shared: those of them that are attended once for the group, in whole
// blocks, by the CTAs from cta0 on: `parts` runs of part_len sub-tiles of 64 keys.
struct Group {
    int row0, rows, prefix, shared;
    int cta0, parts, part_len;
};

// One attention over a paged cache: rows that attend their own keys from
// their group's shared ones on (hb_decode_shared), or all of them with
// nq queries a sequence (hb_decode_weigh).
struct Attn {
    const bf16 *k, *v;
    int num_blocks, n_kv, n_heads, group;  // group: query heads of a kv head
    const bf16 *q;
    long long q_stride;
    const int *tables;
    int bt_stride;
    const int *ctx_lens;
    int max_ctx, nq;
    float c2;                  // log2(e) / sqrt(d): weights are 2^((s - m) c2)
    int split_len, n_splits;   // of a row's own keys
    int col_tiles;             // CTAs of the queries of a kv head
    int first_slot, n_slots;   // partials of a row: its group's parts, then from first_slot on its own splits
    bool beside;               // the rows' own keys run beside the prefixes' kernel, launched before
    bf16 *out;
    long long out_stride;
    float2 *part_ml;           // [row][head][slot] (m, l)
    float *part_o;             // [row][head][slot][D]
    float *scores;             // [seq][head of the kv head's queries][score_stride], or null
    long long score_stride;
    int n_groups;              // 0: no groups
    const Group *groups;       // device, where they do not fit here
    Group few[INLINE_GROUPS];

    __device__ __forceinline__ Group at(int i) const { return groups ? groups[i] : few[i]; }
    // The group of a row.
    __device__ __forceinline__ Group of(int row) const
    {
        int lo = 0, hi = n_groups - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (at(mid).row0 <= row)
                lo = mid;
            else
                hi = mid - 1;
        }
        return at(lo);
    }
};

// The groups' shared keys, for all rows of a group at once (prefix_attention.cu).
int launch_prefix(const hb_paged_pool *pool, const Attn &p, int ctas, cudaStream_t s);

int check_pool(const hb_paged_pool *p);
int check_weight_pool(const hb_weight_pool *p);

}  // namespace paged
}  // namespace hb
