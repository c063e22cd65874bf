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
constexpr int SLOTS = 3 * 152;     // CTAs of the own keys' kernel that run at once
constexpr int SPLIT_MIN = 256;     // keys of a split at least
constexpr int BALANCE_SEQS = 256;

// Rows row0..row0 + rows - 1; prefix: tokens that they share, as the caller
// says; shared: those of them that are attended once for the group, in whole
// blocks, by the CTAs from cta0 on: `parts` runs of part_len sub-tiles of 64 keys.
struct Group {
    int row0, rows, prefix, shared;
    int cta0, parts, part_len;
};

// A pool of attention weights, and what an attention does with it.
struct Weigh {
    float *w;
    int num_blocks;
    const int *tables;
    int stride;
    float decay;
};

// One attention over a paged cache: of rows in groups that share prefixes
// (hb_decode_shared; every row has a table), or of nq rows a sequence
// (hb_decode_weigh; every sequence has a table).  Either way a part of the keys
// may be attended for a group or a sequence at once (prefix_attention.cu), and
// the others, its "own", row by row.
struct Attn {
    const bf16 *k, *v;
    int num_blocks, n_kv, n_heads, group;  // group: query heads of a kv head
    const bf16 *q;
    long long q_stride;
    const int *tables;
    int bt_stride;
    const int *ctx_lens;
    int max_ctx, n_seqs, nq;   // n_seqs: entries of ctx_lens
    float c2;                  // log2(e) / sqrt(d): weights are 2^((s - m) c2)
    int split_len, n_splits;   // of a row's own keys, unless
    bool balance;              // splits go by the lengths that the sequences have, BALANCE_SEQS of them at most
    int col_tiles;             // CTAs of the queries of a kv head
    int first_slot, n_slots;   // partials of a row: those of the common part, then from first_slot on its own splits
    bool direct;               // a row has one partial, which is its result
    bool beside;               // the own keys' kernel runs beside that of the common ones, launched before
    bf16 *out;
    long long out_stride;
    float2 *part_ml;           // [row][head][slot] (m, l)
    float *part_o;             // [row][head][slot][D]
    float *scores;             // [seq][kv head][query][score_stride]
    long long score_stride;
    float2 *final_ml;          // [row][head] (m, 1 / l, or 0 where that is not a number)
    bool fused;                // the attention's CTAs update the weights themselves
    bool lose;                 // the common keys' first CTA leaves out its first copy (hb_paged_test_lost_block)
    Weigh weigh;
    int seq_parts, seq_part_len;  // without groups: runs of the common keys of a sequence (0: none is common)
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
    // balance: keys of a split, by a whole warp.  As many CTAs as run at once for all
    // keys there are, or with up to twice as many keys each where the rows' last
    // splits, which are not full, would make more of them; n_splits hold the longest.
    __device__ __forceinline__ int balanced() const
    {
        constexpr int EACH = BALANCE_SEQS / 32;
        const int tiles = n_kv * col_tiles;
        int subs[EACH], sum = 0, most = 0;  // sub-tiles of 64 keys
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int j = i * 32 + (int)(threadIdx.x & 31);
            const int ctx = j < n_seqs ? ctx_lens[j] : -1;
            subs[i] = ctx < 0 || ctx > max_ctx ? 0 : (ctx + 64) >> 6;
            sum += subs[i];
            most = max(most, subs[i]);
        }
        sum = __reduce_add_sync(0xffffffffu, sum);
        most = __reduce_max_sync(0xffffffffu, most);
        const int least = max(SPLIT_MIN / 64, (most + n_splits - 1) / n_splits);
        int len = 0;
#pragma unroll 1
        for (int c = 8; c <= 16; ++c) {
            len = max(least, (int)(((long long)sum * tiles * c + 8 * SLOTS - 1) / (8 * SLOTS)));
            const float inv = __frcp_rn((float)len);
            int n = 0;
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                n += (int)ceilf(__fmul_rn(subs[i] - 0.5f, inv));
            if (__reduce_add_sync(0xffffffffu, n) * tiles <= SLOTS)
                break;
        }
        return len * 64;
    }
    // A sequence's rows as a group: common are the whole blocks that all of
    // them see.  Its context is in range.
    __device__ __forceinline__ Group sequence(int seq, int ctx) const
    {
        Group g = {seq * nq, nq, 0, 0, 0, 0, seq_part_len};
        const int all = ctx + 1 - (nq - 1);
        if (seq_parts > 0 && all >= 16) {
            g.shared = all & ~15;
            g.parts = ((g.shared + 63) / 64 + seq_part_len - 1) / seq_part_len;
        }
        return g;
    }
};

// The common keys, for all rows of a group or sequence at once.
int launch_prefix(const hb_paged_pool *pool, const Attn &p, int ctas, cudaStream_t s);

int check_pool(const hb_paged_pool *p);
int check_weight_pool(const hb_weight_pool *p);

}  // namespace paged
}  // namespace hb
