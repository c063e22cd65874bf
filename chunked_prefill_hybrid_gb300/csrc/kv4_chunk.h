// kv4_chunk.h -- host interface of the tcgen05 chunk attention over the 4-bit
// cache (kv4_chunk.cu).
#pragma once

#include "common.cuh"

namespace hb {

constexpr int KC_ROWS = 256;    // query columns (row x head of a kv head) of an item at most: two MMA tiles of 128
constexpr int KC_KEYS = 128;    // keys of a tile
constexpr int KC_CTAS = 152;    // CTAs at most: one per SM

// Where a CTA's work begins: key tile kt0 of item (kvh, qt), and how many
// units it has.
struct KcStart {
    int kvh, qt, kt0, units;
};

struct Kv4Chunk {
    const uint8_t *pool;
    int num_blocks, n_kv, group, n_heads;
    float ks, vs;
    const bf16 *q;
    long long q_stride;
    const int *table;
    int offset, cols;           // cols = chunk_len * group
    bf16 *out;
    long long out_stride;
    // work: units are (item, key tile); item = (kv head, `rows` columns), kv
    // head major; CTA c takes the units of start[c]
    int rows;                   // 256, or 128: both halves of a CTA on the same columns, on alternate key tiles
    int n_qt, ctas;             // items of a kv head; CTAs
    long long units;
    bool shared;                // some item is shared by several CTAs
    double us;                  // estimated time
    KcStart start[KC_CTAS];
    float *part_o;              // [2 ctas][D / 4][256][4]: CTA c's segment that starts with it, and its last
    float2 *part_ml;            // [2 ctas][256] (m in log2, l)
    bool lose;                  // the first CTA leaves out the copy of its first page (hb_kv4_test_lost_page)
};

// Plan the work of a chunk (host): everything but the pointers.  False when a
// CTA would have more units than it can count.
bool kv4_chunk_plan(Kv4Chunk &p, int chunk_len, int head_dim);
long long kv4_chunk_workspace_bytes(const Kv4Chunk &p, int head_dim);
cudaError_t launch_kv4_chunk(const Kv4Chunk &p, int head_dim, cudaStream_t s);

}  // namespace hb
