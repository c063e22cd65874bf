// evict.cu -- eviction from a paged cache by accumulated attention weight: the
// choice of the tokens that stay, and their move (include/hb_paged.h).
#include <cuda_runtime.h>

#include "paged.h"

namespace hb {
namespace {

using namespace paged;

constexpr int SEL_THREADS = 1024;
constexpr int SEL_KEYS = 4;  // neighbouring tokens of a thread
constexpr int MOVE_THREADS = 256;
constexpr int MOVE_DEPTH = 8;  // pieces that a thread has under way, twice

// Order-preserving integers: a NaN is 0, below the lowest number's; both zeros
// are equal; a token that stays in any case is above all.
constexpr uint32_t STAYS = 0xffffffffu;
__device__ __forceinline__ uint32_t rank_of(float w)
{
    uint32_t u = __float_as_uint(w);
    if ((u & 0x7fffffffu) > 0x7f800000u)
        return 0u;
    if (u == 0x80000000u)
        u = 0u;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct Select {
    const float *w;
    int num_blocks, n_kv;
    const int *tables;
    int stride;
    const int *lens;
    int max_len, keep, first, recent;
    int *kept;
};

// The ranks of tokens at .. at + 3 (at a multiple of 4) of a sequence of len.
__device__ __forceinline__ void ranks(const Select &p, const int *tab, int kvh, int at, int len, uint32_t (&r)[SEL_KEYS])
{
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    bool ok = false;
    if (at < len) {
        const int blk = __ldg(tab + (at >> 4));
        ok = blk >= 0 && blk < p.num_blocks;
        if (ok)
            v = *reinterpret_cast<const float4 *>(p.w + ((size_t)blk * p.n_kv + kvh) * 16 + (at & 15));
    }
    const float x[SEL_KEYS] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < SEL_KEYS; ++j)
        r[j] = at + j < p.first || at + j >= len - p.recent ? STAYS : ok ? rank_of(x[j]) : 0u;
}

// One CTA: a sequence's kv head.  The keep-th largest rank by its bytes from the
// top, a histogram each; then the tokens above it, and the first of those that
// equal it, in order.
__global__ void __launch_bounds__(SEL_THREADS) k_evict_select(const Select p)
{
    __shared__ int hist[256];
    __shared__ int s_byte, s_left;
    __shared__ int s_warp[32], s_total;
    const int kvh = blockIdx.x, seq = blockIdx.y;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    int len = p.lens[seq];
    if (len < 0 || len > p.max_len)
        len = 0;
    int *kept = p.kept + ((size_t)seq * p.n_kv + kvh) * p.keep;
    if (len <= p.keep) {
        for (int i = threadIdx.x; i < p.keep; i += SEL_THREADS)
            kept[i] = i < len ? i : -1;
        return;
    }
    const int *tab = p.tables + (size_t)seq * p.stride;
    uint32_t prefix = 0, mask = 0;
    int left = p.keep;  // to be taken of the ranks that have the prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (threadIdx.x < 256)
            hist[threadIdx.x] = 0;
        __syncthreads();
        for (int at = threadIdx.x * SEL_KEYS; at < len; at += SEL_THREADS * SEL_KEYS) {
            uint32_t r[SEL_KEYS];
            ranks(p, tab, kvh, at, len, r);
#pragma unroll
            for (int j = 0; j < SEL_KEYS; ++j)
                if (at + j < len && (r[j] & mask) == prefix)
                    atomicAdd(&hist[(r[j] >> shift) & 255], 1);
        }
        __syncthreads();
        if (warp == 0) {  // the byte in whose bin the left-th largest lies
            int mine[8], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                mine[j] = hist[255 - lane * 8 - j];
                sum += mine[j];
            }
            int upto = sum;
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, upto, x);
                if (lane >= x)
                    upto += y;
            }
            int before = upto - sum;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (before < left && before + mine[j] >= left) {
                    s_byte = 255 - lane * 8 - j;
                    s_left = left - before;
                }
                before += mine[j];
            }
        }
        __syncthreads();
        prefix |= (uint32_t)s_byte << shift;
        mask |= 0xffu << shift;
        left = s_left;
        __syncthreads();
    }
    // all above prefix, and the first `left` that equal it
    int done = 0, equal = 0;  // taken, and equals met, before this round
    for (int base = 0; base < len; base += SEL_THREADS * SEL_KEYS) {
        const int at = base + threadIdx.x * SEL_KEYS;
        uint32_t r[SEL_KEYS];
        ranks(p, tab, kvh, at, len, r);
        int count = 0;  // above in the low half, equal in the high
#pragma unroll
        for (int j = 0; j < SEL_KEYS; ++j)
            if (at + j < len)
                count += r[j] > prefix ? 1 : r[j] == prefix ? 1 << 16 : 0;
        int upto = count;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, x);
            if (lane >= x)
                upto += y;
        }
        if (lane == 31)
            s_warp[warp] = upto;
        __syncthreads();
        if (warp == 0) {
            const int v = s_warp[lane];
            int u = v;
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, u, x);
                if (lane >= x)
                    u += y;
            }
            s_warp[lane] = u - v;
            if (lane == 31)
                s_total = u;
        }
        __syncthreads();
        const int before = s_warp[warp] + upto - count, total = s_total;
        int above = before & 0xffff, same = equal + (before >> 16);
        const int met = min(equal, left);  // equals taken before this round
#pragma unroll
        for (int j = 0; j < SEL_KEYS; ++j)
            if (at + j < len) {
                const bool take = r[j] > prefix || (r[j] == prefix && same < left);
                if (take)
                    kept[done + above + (min(same, left) - met)] = at + j;
                above += r[j] > prefix;
                same += r[j] == prefix;
            }
        done += (total & 0xffff) + (min(equal + (total >> 16), left) - met);
        equal += total >> 16;
        __syncthreads();
    }
}

struct Move {
    uint8_t *pool[2];
    int num_blocks, n_kv;
    const int *from, *to;
    int from_stride, to_stride;
    const int *kept;
    int keep, slices;
    float *w;             // null: none
    int w_blocks;
    const int *w_from, *w_to;
    int w_from_stride, w_to_stride;
};

// Pieces of T of the tokens of one kv head, PER of them of each token (piece
// first.. of a row of `row` bytes): token i from slot kept[i].  A CTA goes
// through the tokens in order and stores a batch only when all its threads have
// loaded it: kept[i] >= i, so what a batch overwrites belongs to it or to the
// batches before, and the next one may be on its way already.
template <typename T>
__device__ __forceinline__ void move_rows(uint8_t *pool, int num_blocks, int n_kv, int kvh, int row, int first, int per,
                                          const int *from, int from_stride, const int *to, int to_stride,
                                          const int *kept, int keep)
{
    const int r = threadIdx.x / per, c = first + threadIdx.x % per;
    const int rows = MOVE_THREADS / per, batch = rows * MOVE_DEPTH;
    T v[2][MOVE_DEPTH];
    T *dst[2][MOVE_DEPTH];
    auto load = [&](int base, T (&x)[MOVE_DEPTH], T *(&d)[MOVE_DEPTH]) {
#pragma unroll
        for (int u = 0; u < MOVE_DEPTH; ++u) {
            const int i = base + u * rows + r;
            d[u] = nullptr;
            const int src = i < keep && r < rows ? __ldg(kept + i) : -1;
            if (src < 0 || (src >> 4) >= from_stride)
                continue;
            const int b0 = from[src >> 4], b1 = to[i >> 4];
            if (b0 < 0 || b0 >= num_blocks || b1 < 0 || b1 >= num_blocks || (b0 == b1 && src == i))
                continue;
            const uint8_t *s = pool + (((size_t)b0 * n_kv + kvh) * 16 + (src & 15)) * row;
            x[u] = reinterpret_cast<const T *>(s)[c];
            d[u] = reinterpret_cast<T *>(pool + (((size_t)b1 * n_kv + kvh) * 16 + (i & 15)) * row) + c;
        }
    };
    auto store = [&](const T (&x)[MOVE_DEPTH], T *const (&d)[MOVE_DEPTH]) {
#pragma unroll
        for (int u = 0; u < MOVE_DEPTH; ++u)
            if (d[u])
                *d[u] = x[u];
    };
    load(0, v[0], dst[0]);
    for (int base = 0; base < keep; base += 2 * batch) {
        load(base + batch, v[1], dst[1]);
        __syncthreads();
        store(v[0], dst[0]);
        load(base + 2 * batch, v[0], dst[0]);
        __syncthreads();
        store(v[1], dst[1]);
    }
}

template <int D>
__global__ void __launch_bounds__(MOVE_THREADS) k_evict_move(const Move p)
{
    pdl_wait();
    pdl_trigger();
    const int seq = blockIdx.y;
    const int each = 2 * p.slices + (p.w ? 1 : 0);
    const int kvh = blockIdx.x / each, part = blockIdx.x % each;
    const int *kept = p.kept + ((size_t)seq * p.n_kv + kvh) * p.keep;
    if (part < 2 * p.slices) {
        const int per = D / 8 / p.slices;
        move_rows<uint4>(p.pool[part & 1], p.num_blocks, p.n_kv, kvh, D * 2, (part >> 1) * per, per,
                         p.from + (size_t)seq * p.from_stride, p.from_stride, p.to + (size_t)seq * p.to_stride,
                         p.to_stride, kept, p.keep);
    } else {
        move_rows<float>((uint8_t *)p.w, p.w_blocks, p.n_kv, kvh, 4, 0, 1, p.w_from + (size_t)seq * p.w_from_stride,
                         p.w_from_stride, p.w_to + (size_t)seq * p.w_to_stride, p.w_to_stride, kept, p.keep);
    }
}

}  // namespace
}  // namespace hb

using namespace hb;
using namespace hb::paged;

extern "C" int hb_evict_select(const hb_weight_pool *weights, const int32_t *weight_tables, int wt_stride,
                               const int32_t *lens, int n_seqs, int max_len, int keep, int n_first, int n_recent,
                               int32_t *kept, void *cuda_stream)
try {
    const int rc = check_weight_pool(weights);
    if (rc)
        return rc;
    if (n_seqs < 0 || max_len < 0 || keep < 1 || n_first < 0 || n_recent < 0 || (long long)n_first + n_recent > keep)
        return HB_EINVAL;
    if (n_seqs == 0)
        return HB_OK;
    if (!weight_tables || !lens || !kept || (uintptr_t)weight_tables % 4 || (uintptr_t)lens % 4 || (uintptr_t)kept % 4)
        return HB_EINVAL;
    if (max_len > MAX_KEYS || keep > MAX_KEYS || wt_stride < (max_len + 15) / 16 || n_seqs > 65535)
        return HB_ERANGE;
    const Select p = {weights->data, weights->num_blocks, weights->n_kv_heads, weight_tables, wt_stride, lens,
                      max_len,       keep,                n_first,             n_recent,      kept};
    return launch_kernel(true, k_evict_select, dim3((unsigned)weights->n_kv_heads, (unsigned)n_seqs),
                         dim3(SEL_THREADS), 0, (cudaStream_t)cuda_stream, p) == cudaSuccess
               ? HB_OK
               : HB_ECUDA;
} catch (...) {
    return HB_ENOMEM;
}

extern "C" int hb_evict_move(const hb_paged_pool *pool, const int32_t *block_tables, int bt_stride,
                             const int32_t *new_tables, int new_stride, const int32_t *kept, int n_seqs, int keep,
                             const hb_weight_pool *weights, const int32_t *weight_tables, int wt_stride,
                             const int32_t *new_weight_tables, int new_wt_stride, void *cuda_stream)
try {
    int rc = check_pool(pool);
    if (rc || (weights && (rc = check_weight_pool(weights))))
        return rc;
    if (n_seqs < 0 || keep < 1 || (weights && weights->n_kv_heads != pool->n_kv_heads))
        return HB_EINVAL;
    if (n_seqs == 0)
        return HB_OK;
    if (!block_tables || !new_tables || !kept || (uintptr_t)block_tables % 4 || (uintptr_t)new_tables % 4 ||
        (uintptr_t)kept % 4 || bt_stride < 1)
        return HB_EINVAL;
    if (weights && (!weight_tables || !new_weight_tables || (uintptr_t)weight_tables % 4 ||
                    (uintptr_t)new_weight_tables % 4 || wt_stride < 1))
        return HB_EINVAL;
    if (keep > MAX_KEYS || new_stride < (keep + 15) / 16 || (weights && new_wt_stride < (keep + 15) / 16) ||
        n_seqs > 65535)
        return HB_ERANGE;
    Move p = {};
    p.pool[0] = (uint8_t *)pool->k;
    p.pool[1] = (uint8_t *)pool->v;
    p.num_blocks = pool->num_blocks;
    p.n_kv = pool->n_kv_heads;
    p.from = block_tables;
    p.from_stride = bt_stride;
    p.to = new_tables;
    p.to_stride = new_stride;
    p.kept = kept;
    p.keep = keep;
    p.slices = 1;
    if (weights) {
        p.w = weights->data;
        p.w_blocks = weights->num_blocks;
        p.w_from = weight_tables;
        p.w_from_stride = wt_stride;
        p.w_to = new_weight_tables;
        p.w_to_stride = new_wt_stride;
    }
    const long long gx = (long long)p.n_kv * (2 * p.slices + (weights ? 1 : 0));
    if (gx > 0x7fffffffll)
        return HB_ERANGE;
    return launch_kernel(true, pool->head_dim == 128 ? k_evict_move<128> : k_evict_move<64>,
                         dim3((unsigned)gx, (unsigned)n_seqs), dim3(MOVE_THREADS), 0, (cudaStream_t)cuda_stream,
                         p) == cudaSuccess
               ? HB_OK
               : HB_ECUDA;
} catch (...) {
    return HB_ENOMEM;
}
