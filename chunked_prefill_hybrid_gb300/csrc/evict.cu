// evict.cu -- eviction from a paged cache by accumulated attention weight: the
// choice of the tokens that stay, and their move (include/hb_paged.h).
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "kv4_host.h"
#include "paged.h"
#include "tc_ptx.cuh"

namespace hb {
namespace {

using namespace paged;

constexpr int MOVE_THREADS = 256;
constexpr int CLUSTER = 8;         // CTAs of a long sequence's kv head
constexpr int WIDE = 16;            // or, for very few of them, sixteen
constexpr int MOST_RANKS = 49152;  // of tokens that a CTA keeps in shared memory

// ------------------------------------------------------------------- choice

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
    int room;  // tokens of a CTA whose ranks fit its shared memory
};

// Weights of tokens at .. at + 3 (at a multiple of 4), through their block.
__device__ __forceinline__ float4 weights_at(const Select &p, int blk, int kvh, int at)
{
    if (blk < 0 || blk >= p.num_blocks)
        return make_float4(__int_as_float(0x7fc00000), __int_as_float(0x7fc00000), __int_as_float(0x7fc00000),
                           __int_as_float(0x7fc00000));
    return *reinterpret_cast<const float4 *>(p.w + ((size_t)blk * p.n_kv + kvh) * 16 + (at & 15));
}

// Their ranks in a sequence of len tokens.
__device__ __forceinline__ uint4 ranks(const Select &p, const float4 &v, int at, int len)
{
    const int late = len - p.recent;
    uint4 r;
    r.x = at < p.first || at >= late ? STAYS : rank_of(v.x);
    r.y = at + 1 < p.first || at + 1 >= late ? STAYS : rank_of(v.y);
    r.z = at + 2 < p.first || at + 2 >= late ? STAYS : rank_of(v.z);
    r.w = at + 3 < p.first || at + 3 >= late ? STAYS : rank_of(v.w);
    return r;
}

// A number in the shared memory of another CTA of the cluster.
__device__ __forceinline__ int remote(const int *at, uint32_t cta)
{
    int v;
    asm volatile("{\n.reg .b32 a;\nmapa.shared::cluster.u32 a, %1, %2;\nld.shared::cluster.s32 %0, [a];\n}\n"
                 : "=r"(v)
                 : "r"((uint32_t)__cvta_generic_to_shared(at)), "r"(cta)
                 : "memory");
    return v;
}

__device__ __forceinline__ void set_remote(const int *at, uint32_t cta, int v)
{
    asm volatile("{\n.reg .b32 a;\nmapa.shared::cluster.u32 a, %0, %1;\nst.shared::cluster.s32 [a], %2;\n}\n" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(at)),
                 "r"(cta), "r"(v)
                 : "memory");
}

// Sum over the lanes before this one and itself.
__device__ __forceinline__ int scan_warp(int v, int lane)
{
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, x);
        if (lane >= x)
            v += y;
    }
    return v;
}

// A CTA, or a cluster of them with a piece of the tokens each: one sequence's
// kv head.  The keep-th largest rank by its digits of BITS bits from the top, a
// histogram each (added up over the cluster in its shared memory), and no further
// than the tokens' ranks differ (18 x 40 of 1025: one pass of four less, 1.4 us);
// then the tokens above it, and the first of those that equal it, in order.  Latency
// bounds it, not memory: three or four passes of shared memory atomics and barriers.
template <int THREADS, int BITS, int CTAS>
__global__ void __launch_bounds__(THREADS) k_evict_select(const Select p)
{
    constexpr int PASSES = (32 + BITS - 1) / BITS, BINS = 1 << BITS, EACH = BINS / THREADS, WARPS = THREADS / 32;
    static_assert(EACH * THREADS == BINS);
    extern __shared__ __align__(16) uint32_t cache[];
    __shared__ int hist[PASSES][BINS], totals[CTAS > 1 ? BINS : 1];
    __shared__ int s_digit, s_left, s_all, s_count[2];
    __shared__ int s_warp[WARPS], s_total;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = blockIdx.x % CTAS, kvh = blockIdx.x / CTAS, seq = blockIdx.y;
    for (int i = threadIdx.x; i < PASSES * BINS; i += THREADS)
        hist[0][i] = 0;
    if (threadIdx.x < 2)
        s_count[threadIdx.x] = 0;
    pdl_wait();
    pdl_trigger();
    int len = p.lens[seq];
    if (len < 0 || len > p.max_len)
        len = 0;
    int *kept = p.kept + ((size_t)seq * p.n_kv + kvh) * p.keep;
    if (len <= p.keep) {  // the same for the whole cluster
        for (int i = part * THREADS + threadIdx.x; i < p.keep; i += CTAS * THREADS)
            kept[i] = i < len ? i : -1;
        return;
    }
    const int *tab = p.tables + (size_t)seq * p.stride;
    const int piece = ((len + CTAS - 1) / CTAS + 15) & ~15;
    const int t0 = min(len, part * piece), t1 = min(len, t0 + piece);
    const bool cached = piece <= p.room;
    auto fetch = [&](int at) {
        return cached ? *reinterpret_cast<const uint4 *>(cache + (at - t0))
                      : ranks(p, weights_at(p, __ldg(tab + (at >> 4)), kvh, at), at, len);
    };
    __syncthreads();  // the histograms are empty
    uint32_t prefix = 0, mask = 0;
    int left = p.keep;  // to be taken of the ranks that have the prefix
#pragma unroll 1
    for (int pass = 0; pass < PASSES; ++pass) {
        const int shift = max(0, 32 - BITS * (pass + 1));
        const uint32_t bins = pass == PASSES - 1 ? (1u << (32 - BITS * (PASSES - 1))) - 1 : BINS - 1;
        int *h = hist[pass];
        auto count = [&](const uint4 &r, int at) {
            if ((r.x & mask) == prefix)
                atomicAdd(&h[(r.x >> shift) & bins], 1);
            if (at + 1 < t1 && (r.y & mask) == prefix)
                atomicAdd(&h[(r.y >> shift) & bins], 1);
            if (at + 2 < t1 && (r.z & mask) == prefix)
                atomicAdd(&h[(r.z >> shift) & bins], 1);
            if (at + 3 < t1 && (r.w & mask) == prefix)
                atomicAdd(&h[(r.w >> shift) & bins], 1);
        };
        if (pass == 0) {  // four rounds' loads at a time
            for (int base = t0 + threadIdx.x * 4; base < t1; base += THREADS * 16) {
                int blk[4];
                float4 v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int at = base + u * THREADS * 4;
                    blk[u] = at < t1 ? __ldg(tab + (at >> 4)) : -1;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    v[u] = weights_at(p, blk[u], kvh, base + u * THREADS * 4);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int at = base + u * THREADS * 4;
                    if (at < t1) {
                        const uint4 r = ranks(p, v[u], at, len);
                        if (cached)
                            *reinterpret_cast<uint4 *>(cache + (at - t0)) = r;
                        count(r, at);
                    }
                }
            }
        } else {
            for (int at = t0 + threadIdx.x * 4; at < t1; at += THREADS * 4)
                count(fetch(at), at);
        }
        if constexpr (CTAS > 1) {  // each CTA adds up its share of the bins for all of them
            tc::cluster_sync();
            for (int i = threadIdx.x; i < BINS / CTAS; i += THREADS) {
                const int b = part * (BINS / CTAS) + i;
                int sum = 0;
#pragma unroll
                for (int c = 0; c < CTAS; ++c)
                    sum += remote(&h[b], c);
#pragma unroll
                for (int c = 0; c < CTAS; ++c)
                    set_remote(&totals[b], c, sum);
            }
            tc::cluster_sync();
            h = totals;
        } else {
            __syncthreads();
        }
        // the digit in whose bin the left-th largest lies; bins from the top
        int mine[EACH], sum = 0;
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
            mine[j] = h[BINS - 1 - ((int)threadIdx.x * EACH + j)];
            sum += mine[j];
        }
        int upto = scan_warp(sum, lane);
        if (lane == 31)
            s_warp[warp] = upto;
        __syncthreads();
        int before = upto - sum;
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            before += w < warp ? s_warp[w] : 0;
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
            if (before < left && before + mine[j] >= left) {
                s_digit = BINS - 1 - ((int)threadIdx.x * EACH + j);
                s_left = left - before;
                s_all = mine[j] == left - before;
            }
            before += mine[j];
        }
        __syncthreads();
        prefix |= (uint32_t)s_digit << shift;
        mask |= bins << shift;
        left = s_left;
        if (s_all)  // what has this prefix stays, all of it: its further digits do not matter
            break;
    }
    // all above prefix, and the first `left` that equal it, in the digits looked at
    auto masked = [&](int at) {
        const uint4 r = fetch(at);
        return make_uint4(r.x & mask, r.y & mask, r.z & mask, r.w & mask);
    };
    int done = 0, equal = 0;      // taken, and equals met, before this round
    if constexpr (CTAS > 1) {  // in the pieces before this one
        int above = 0, same = 0;
        for (int at = t0 + threadIdx.x * 4; at < t1; at += THREADS * 4) {
            const uint4 r = masked(at);
            above += (r.x > prefix) + (at + 1 < t1 && r.y > prefix) + (at + 2 < t1 && r.z > prefix) +
                     (at + 3 < t1 && r.w > prefix);
            same += (r.x == prefix) + (at + 1 < t1 && r.y == prefix) + (at + 2 < t1 && r.z == prefix) +
                    (at + 3 < t1 && r.w == prefix);
        }
        above = __reduce_add_sync(0xffffffffu, above);
        same = __reduce_add_sync(0xffffffffu, same);
        if (lane == 0) {
            atomicAdd(&s_count[0], above);
            atomicAdd(&s_count[1], same);
        }
        tc::cluster_sync();
        for (int c = 0; c < part; ++c) {
            done += remote(&s_count[0], c);
            equal += remote(&s_count[1], c);
        }
        done += min(equal, left);
    }
    for (int base = t0; base < t1; base += THREADS * 4) {
        const int at = base + threadIdx.x * 4;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (at < t1)
            v = masked(at);
        const uint32_t r[4] = {v.x, v.y, v.z, v.w};
        int count = 0;  // above in the low half, equal in the high
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (at + j < t1)
                count += r[j] > prefix ? 1 : r[j] == prefix ? 1 << 16 : 0;
        const int upto = scan_warp(count, lane);
        __syncthreads();  // s_warp of the round before is read
        if (lane == 31)
            s_warp[warp] = upto;
        __syncthreads();
        if (warp == 0) {
            const int x = lane < WARPS ? s_warp[lane] : 0, u = scan_warp(x, lane);
            if (lane < WARPS)
                s_warp[lane] = u - x;
            if (lane == 31)
                s_total = u;
        }
        __syncthreads();
        const int before = s_warp[warp] + upto - count, total = s_total;
        int above = before & 0xffff, same = equal + (before >> 16);
        const int met = min(equal, left);  // equals taken before this round
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (at + j < t1) {
                if (r[j] > prefix || (r[j] == prefix && same < left))
                    kept[done + above + (min(same, left) - met)] = at + j;
                above += r[j] > prefix;
                same += r[j] == prefix;
            }
        done += (total & 0xffff) + (min(equal + (total >> 16), left) - met);
        equal += total >> 16;
    }
    if constexpr (CTAS > 1)
        tc::cluster_sync();  // no CTA's shared memory goes while another reads it
}

// Up to 64 tokens: a warp a sequence's kv head.  A token stays if fewer than keep
// others come before it, by rank and then by position: a lane's compares, not
// memory, are its time, and they grow with the square.  us, a CTA of k_evict_select
// and a warp: 720 heads of 30 tokens 7.3 and 4.0, 16 of them 4.6 and 4.1; 5120 of
// 64 tokens 31.6 and 15.3, 720 of them 7.3 and 7.5, 16 of them 4.6 and 7.3.
constexpr int FEW_WARPS = 8, FEW_TOKENS = 64, FEW_ITEMS = 720;

template <int N>  // tokens of a lane
__global__ void __launch_bounds__(FEW_WARPS * 32) k_evict_select_few(const Select p, long long items)
{
    pdl_wait();
    pdl_trigger();
    const long long item = (long long)blockIdx.x * FEW_WARPS + (threadIdx.x >> 5);
    if (item >= items)
        return;
    const int lane = threadIdx.x & 31, seq = (int)(item / p.n_kv), kvh = (int)(item % p.n_kv);
    int len = p.lens[seq];
    if (len < 0 || len > p.max_len)
        len = 0;
    int *kept = p.kept + item * p.keep;
    uint32_t r[N];
    int before[N];
#pragma unroll
    for (int t = 0; t < N; ++t) {
        const int i = t * 32 + lane;
        r[t] = 0u;
        before[t] = 0;
        if (i < len) {
            const int blk = __ldg(p.tables + (size_t)seq * p.stride + (i >> 4));
            if (i < p.first || i >= len - p.recent)
                r[t] = STAYS;
            else if (blk >= 0 && blk < p.num_blocks)
                r[t] = rank_of(p.w[((size_t)blk * p.n_kv + kvh) * 16 + (i & 15)]);
        }
    }
    if (len > p.keep)
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int n = min(32, len - q * 32);
            for (int l = 0; l < n; ++l) {
                const uint32_t x = __shfl_sync(0xffffffffu, r[q], l);
#pragma unroll
                for (int t = 0; t < N; ++t)
                    before[t] += x > r[t] || (x == r[t] && q * 32 + l < t * 32 + lane);
            }
        }
    int done = 0;
#pragma unroll
    for (int t = 0; t < N; ++t) {
        const bool take = t * 32 + lane < len && before[t] < p.keep;
        const uint32_t mask = __ballot_sync(0xffffffffu, take);
        if (take)
            kept[done + __popc(mask & ((1u << lane) - 1u))] = t * 32 + lane;
        done += __popc(mask);
    }
    for (int i = done + lane; i < p.keep; i += 32)
        kept[i] = -1;
}

// --------------------------------------------------------------------- move

struct Move {
    uint8_t *pool[2];
    int num_blocks, n_kv;
    const int *from, *to;
    int from_stride, to_stride;
    const int *kept;
    int keep;
    float *w;             // null: none
    int w_blocks;
    const int *w_from, *w_to;
    int w_from_stride, w_to_stride;
};

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src)
{
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Batches of tokens in shared memory, and where each token goes.  Three CTAs of
// four stages share an SM; in a cluster, of which there are few, a CTA has six.
template <int PIECES, int P, int CTAS>
struct MoveTile {
    static constexpr int STAGES = CTAS > 1 ? 6 : 4;
    static constexpr int TOKENS = P == 4 ? 1024 : 16384 / (PIECES * P);
    static constexpr int BYTES = TOKENS * PIECES * P;
    static constexpr int LAG = CTAS > 1 ? 1 : 0, AHEAD = STAGES - 2 - LAG;  // batches loading beside the one waited for
    // Slots are looked up for all threads' worth of batches at a time: BATCHES of
    // them, PUT groups ahead of the one whose first batch is waited for.
    static constexpr int BATCHES = TOKENS < MOVE_THREADS ? MOVE_THREADS / TOKENS : 1, GROUP = BATCHES * TOKENS;
    static constexpr int PUT = (BATCHES - 1 + AHEAD) / BATCHES + 1, GROUPS = PUT + 2;
    static constexpr int SMEM = STAGES * BYTES + 8 * GROUPS * GROUP;
};

// Rows of PIECES pieces of P bytes, one a token of one kv head: token i from
// slot kept[i].  A cluster of CTAS CTAs goes through the tokens in order, a
// batch for each of them at a time, and stores those only when all of them and
// those before have been loaded: kept[i] >= i, so what they overwrite belongs to
// them or to batches before, and later ones may be on their way already.  In a
// cluster a batch is stored one round after its barrier began.  Slots of a batch
// are looked up while the batches before it load.
//
// Memory bounds it, by rows of 128 or 256 bytes that are gathered: 18 x 40 heads
// that keep 512 of 1025 tokens 62 us, 5.8 TB/s read and written; 8 heads that keep
// 65536 of 131000, 24 streams of 8 CTAs, 110 us, 4.6 TB/s (the same within 5 us with
// clusters of 4 or 16, with 5 to 12 stages, and with no barriers).
template <int PIECES, int P, int CTAS>
__device__ __forceinline__ void move_rows(uint8_t *ring, uint8_t *pool, int num_blocks, int n_kv, int kvh, int rank,
                                          const int *from, int from_stride, const int *to, int to_stride,
                                          const int *kept, int keep)
{
    using T = MoveTile<PIECES, P, CTAS>;
    constexpr int S = T::STAGES, TOKENS = T::TOKENS, PER = TOKENS * PIECES / MOVE_THREADS, ROW = PIECES * P;
    constexpr int LAG = T::LAG, AHEAD = T::AHEAD, GB = T::BATCHES, EACH = T::GROUP / MOVE_THREADS;
    static_assert(PER == 4 && PER * MOVE_THREADS == TOKENS * PIECES && LAG <= GB);
    // where tokens come from and go to, as rows of the pool from this kv head's
    // first on; NONE: not moved
    constexpr uint32_t NONE = 0xffffffffu;
    uint32_t *s_src = reinterpret_cast<uint32_t *>(ring + S * T::BYTES), *s_dst = s_src + T::GROUPS * T::GROUP;
    const int n = (keep + TOKENS * CTAS - 1) / (TOKENS * CTAS);
    const uint32_t page = (uint32_t)n_kv * 16;  // rows
    // a thread has piece c of four neighbouring tokens of a batch
    const int c = threadIdx.x % PIECES, t0 = threadIdx.x / PIECES * PER;
    pool += (size_t)kvh * 16 * ROW + c * P;
    // token of a thread's look-up u in group q of this CTA's batches
    auto token = [&](int q, int u) {
        const int x = u * MOVE_THREADS + (int)threadIdx.x;
        return (((long long)q * GB + x / TOKENS) * CTAS + rank) * TOKENS + x % TOKENS;
    };
    // the slots in two steps, a group apart: a token's position, then its blocks
    auto positions = [&](int q, int (&k)[EACH]) {
#pragma unroll
        for (int u = 0; u < EACH; ++u) {
            const long long i = token(q, u);
            k[u] = i < keep ? __ldg(kept + i) : -1;
        }
    };
    auto blocks = [&](int q, const int (&k)[EACH], int (&b0)[EACH], int (&b1)[EACH]) {
#pragma unroll
        for (int u = 0; u < EACH; ++u) {
            const bool ok = k[u] >= 0 && (k[u] >> 4) < from_stride;
            b0[u] = ok ? __ldg(from + (k[u] >> 4)) : -1;
            b1[u] = ok ? __ldg(to + (token(q, u) >> 4)) : -1;
        }
    };
    auto put = [&](int q, const int (&k)[EACH], const int (&b0)[EACH], const int (&b1)[EACH]) {
#pragma unroll
        for (int u = 0; u < EACH; ++u) {
            const int at = q % T::GROUPS * T::GROUP + u * MOVE_THREADS + (int)threadIdx.x, i = (int)token(q, u);
            const bool ok = b0[u] >= 0 && b0[u] < num_blocks && b1[u] >= 0 && b1[u] < num_blocks &&
                            !(b0[u] == b1[u] && k[u] == i);
            s_src[at] = ok ? b0[u] * page + (k[u] & 15) : NONE;
            s_dst[at] = ok ? b1[u] * page + (i & 15) : NONE;
        }
    };
    auto slots = [&](int b) { return b / GB % T::GROUPS * T::GROUP + b % GB * TOKENS; };  // of batch b
    auto load = [&](int b) {
        if (b < n) {
            const uint32_t at = (uint32_t)__cvta_generic_to_shared(ring + b % S * T::BYTES) + t0 * ROW + c * P;
            const uint4 src = *reinterpret_cast<const uint4 *>(s_src + slots(b) + t0);
            const uint32_t r[PER] = {src.x, src.y, src.z, src.w};
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (r[j] != NONE)
                    copy_async<P>(at + j * ROW, pool + (size_t)r[j] * ROW);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto store = [&](int b) {
        using V = typename std::conditional<P == 16, uint4, uint32_t>::type;
        const uint8_t *at = ring + b % S * T::BYTES + t0 * ROW + c * P;
        const uint4 dst = *reinterpret_cast<const uint4 *>(s_dst + slots(b) + t0);
        const uint32_t r[PER] = {dst.x, dst.y, dst.z, dst.w};
        V v[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j)
            v[j] = *reinterpret_cast<const V *>(at + j * ROW);
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (r[j] != NONE)
                *reinterpret_cast<V *>(pool + (size_t)r[j] * ROW) = v[j];
    };
    // of the group to be put next: positions and blocks; of the one after: positions
    int k[EACH], b0[EACH], b1[EACH], k2[EACH];
    const int groups = (n + GB - 1) / GB;
    {
        int ks[T::PUT][EACH];
#pragma unroll
        for (int q = 0; q < T::PUT; ++q)
            if (q < groups)
                positions(q, ks[q]);
        positions(T::PUT, k);
        positions(T::PUT + 1, k2);
#pragma unroll
        for (int q = 0; q < T::PUT; ++q)
            if (q < groups) {
                blocks(q, ks[q], b0, b1);
                put(q, ks[q], b0, b1);
            }
        blocks(T::PUT, k, b0, b1);
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < AHEAD; ++b)
        load(b);
    for (int b = 0; b < n; ++b) {
        asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
        if constexpr (CTAS > 1) {
            if (b > 0)  // every CTA has batch b - 1
                asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
            // relaxed: this CTA's loads of batch b have returned, and that is all that
            // the others wait for; a release would wait for its stores (1 us a round)
            asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
        } else {
            __syncthreads();  // batch b is here, all of it
        }
        load(b + AHEAD);
        if (b % GB == 0) {
            const int q = b / GB;
            put(q + T::PUT, k, b0, b1);  // the place of a group that is stored
#pragma unroll
            for (int u = 0; u < EACH; ++u)
                k[u] = k2[u];
            blocks(q + T::PUT + 1, k, b0, b1);  // a group's time to come
            positions(q + T::PUT + 2, k2);
        }
        if (b >= LAG)
            store(b - LAG);
        __syncthreads();  // the slots put are there, and the place of the batch just stored is free
    }
    if constexpr (CTAS > 1) {
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        store(n - 1);
    }
}

template <int D, int CTAS>
__global__ void __launch_bounds__(MOVE_THREADS) k_evict_move(const Move p)
{
    extern __shared__ __align__(16) uint8_t ring[];
    pdl_wait();
    pdl_trigger();
    const int seq = blockIdx.y;
    const int rank = blockIdx.x % CTAS, parts = p.w ? 3 : 2;  // K, V, weights
    const int part = blockIdx.x / CTAS % parts, kvh = blockIdx.x / CTAS / parts;
    const int *kept = p.kept + ((size_t)seq * p.n_kv + kvh) * p.keep;
    if (part < 2)
        move_rows<D / 8, 16, CTAS>(ring, p.pool[part], p.num_blocks, p.n_kv, kvh, rank,
                                   p.from + (size_t)seq * p.from_stride, p.from_stride,
                                   p.to + (size_t)seq * p.to_stride, p.to_stride, kept, p.keep);
    else
        move_rows<1, 4, CTAS>(ring, (uint8_t *)p.w, p.w_blocks, p.n_kv, kvh, rank,
                              p.w_from + (size_t)seq * p.w_from_stride, p.w_from_stride,
                              p.w_to + (size_t)seq * p.w_to_stride, p.w_to_stride, kept, p.keep);
}

// Up to 32 tokens: a warp the K, V or weights of a sequence's kv head, all loaded
// before any is stored.  us, a CTA of k_evict_move and a warp: 720 heads of 128
// channels that keep 32 tokens 13.2 and 5.3, 32 of them 4.1 and 3.9, 16 of them
// 2.8 and 3.9; 5120 of them 95 and 43.5, at 3.9 TB/s.
constexpr int MOVE_FEW_ITEMS = 32;

template <int D>
__global__ void __launch_bounds__(FEW_WARPS * 32) k_evict_move_few(const Move p, long long units)
{
    constexpr int PIECES = D / 8, ROW = D * 2;
    pdl_wait();
    pdl_trigger();
    const long long unit = (long long)blockIdx.x * FEW_WARPS + (threadIdx.x >> 5);
    if (unit >= units)
        return;
    const int lane = threadIdx.x & 31, parts = p.w ? 3 : 2;
    const int part = (int)(unit % parts), kvh = (int)(unit / parts % p.n_kv), seq = (int)(unit / parts / p.n_kv);
    const bool weights = part == 2;
    const int *from = (weights ? p.w_from : p.from) + (size_t)seq * (weights ? p.w_from_stride : p.from_stride);
    const int *to = (weights ? p.w_to : p.to) + (size_t)seq * (weights ? p.w_to_stride : p.to_stride);
    const int from_stride = weights ? p.w_from_stride : p.from_stride, blocks = weights ? p.w_blocks : p.num_blocks;
    const int k = lane < p.keep ? __ldg(p.kept + ((size_t)seq * p.n_kv + kvh) * p.keep + lane) : -1;
    bool ok = k >= 0 && (k >> 4) < from_stride;
    const int b0 = ok ? __ldg(from + (k >> 4)) : -1, b1 = ok ? __ldg(to + (lane >> 4)) : -1;
    ok = b0 >= 0 && b0 < blocks && b1 >= 0 && b1 < blocks && !(b0 == b1 && k == lane);
    const long long src = ok ? ((long long)b0 * p.n_kv + kvh) * 16 + (k & 15) : -1;
    const long long dst = ok ? ((long long)b1 * p.n_kv + kvh) * 16 + (lane & 15) : -1;
    if (weights) {
        const float x = ok ? p.w[src] : 0.f;
        __syncwarp();
        if (ok)
            p.w[dst] = x;
        return;
    }
    uint8_t *pool = p.pool[part];
    uint4 v[PIECES];
#pragma unroll
    for (int u = 0; u < PIECES; ++u) {
        const int e = u * 32 + lane;
        const long long row = __shfl_sync(0xffffffffu, src, e / PIECES);
        if (row >= 0)
            v[u] = *reinterpret_cast<const uint4 *>(pool + row * ROW + e % PIECES * 16);
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < PIECES; ++u) {
        const int e = u * 32 + lane;
        const long long row = __shfl_sync(0xffffffffu, dst, e / PIECES);
        if (row >= 0)
            *reinterpret_cast<uint4 *>(pool + row * ROW + e % PIECES * 16) = v[u];
    }
}

// ------------------------------------------------------------------- host

// Whether clusters of sixteen CTAs run, for `items` kv heads of all sequences: they
// need more of an SM group to be free, so that a kernel does not begin while another
// ends.  Choice and move of half of the tokens, 128 channels (us, eight and sixteen):
// 1 head of 6000 tokens 11.9 and 10.6, of 100000 68 and 41; 4 heads of 6000 12.2 and
// 14.0, of 100000 79 and 66; 8 heads of 12000 22.0 and 25.1, of 131000 135 and 138.
bool wide(long long items, int keep) { return items <= 2 || (items <= 4 && keep >= 16384); }

// What a kernel needs once on each device (`done`: a bit for each): its shared
// memory, and leave for clusters of more than eight CTAs.
template <typename P>
cudaError_t allow(void (*kernel)(P), int smem, int ctas, std::atomic<uint64_t> &done)
{
    if (ctas > 8) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess && !(dev < 64 && done.load(std::memory_order_acquire) >> dev & 1))
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess)
            return e;
    }
    return kv4_allow_smem((const void *)kernel, smem, done);
}

// A launch of clusters of CTAS CTAs.
template <int CTAS, typename P>
cudaError_t launch_clusters(void (*kernel)(P), long long gx, int gy, int threads, int smem, cudaStream_t s, const P &p)
{
    const cudaError_t e = max_carveout((const void *)kernel);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)gx, (unsigned)gy);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CTAS;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CTAS > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, int CTAS>
int launch_move(const Move &p, int n_seqs, cudaStream_t s)
{
    static std::atomic<uint64_t> done{0};
    constexpr int smem = MoveTile<D / 8, 16, CTAS>::SMEM;
    static_assert(smem >= MoveTile<1, 4, CTAS>::SMEM);
    auto kernel = k_evict_move<D, CTAS>;
    const long long gx = (long long)p.n_kv * CTAS * (p.w ? 3 : 2);
    if (gx > 0x7fffffffll)
        return HB_ERANGE;
    if (allow(kernel, smem, CTAS, done) != cudaSuccess)
        return HB_ECUDA;
    return launch_clusters<CTAS>(kernel, gx, n_seqs, MOVE_THREADS, smem, s, p) == cudaSuccess ? HB_OK : HB_ECUDA;
}

template <int THREADS, int BITS, int CTAS>
int launch_select(Select p, int n_seqs, cudaStream_t s)
{
    static std::atomic<uint64_t> done{0};
    auto kernel = k_evict_select<THREADS, BITS, CTAS>;
    const long long piece = (((long long)p.max_len + CTAS - 1) / CTAS + 15) & ~15ll;
    const int smem = piece <= MOST_RANKS ? (int)piece * 4 : 0;
    p.room = smem / 4;
    const long long gx = (long long)p.n_kv * CTAS;
    if (gx > 0x7fffffffll)
        return HB_ERANGE;
    if (allow(kernel, MOST_RANKS * 4, CTAS, done) != cudaSuccess)
        return HB_ECUDA;
    return launch_clusters<CTAS>(kernel, gx, n_seqs, THREADS, smem, s, p) == cudaSuccess ? HB_OK : HB_ECUDA;
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
                      max_len,       keep,                n_first,             n_recent,      kept,      0};
    cudaStream_t s = (cudaStream_t)cuda_stream;
    // One CTA, or a cluster that shares the tokens, for a sequence's kv head
    // (us): 1 of them with 12000 tokens 13.7 and 8.6 to 10.0; 16 with 6000 9.1 and
    // 9.6, with 30000 27.8 and 13.9; 64 with 12000 13.8 and 13.7; 256 with 12000
    // 20.3 and 34.7, with 30000 54 and 50.  256 threads for few tokens: 16 with
    // 2000 6.0 and 7.3 (1024 threads).  In a cluster 512 threads and digits of 11
    // bits for few: 8 with 131000 20.6, 30.2 with 256; 64 with 40000 34 and 22.
    const long long items = (long long)n_seqs * weights->n_kv_heads;
    if (max_len <= 32 || (max_len <= FEW_TOKENS && items > FEW_ITEMS)) {
        static_assert(FEW_TOKENS == 64);
        const long long blocks = (items + FEW_WARPS - 1) / FEW_WARPS;
        if (blocks > 0x7fffffffll)
            return HB_ERANGE;
        auto kernel = max_len <= 32 ? k_evict_select_few<1> : k_evict_select_few<2>;
        return launch_kernel(true, kernel, dim3((unsigned)blocks), dim3(FEW_WARPS * 32), 0, s, p, items) == cudaSuccess
                   ? HB_OK
                   : HB_ECUDA;
    }
    if (max_len > 5500 + 78 * items || max_len > MOST_RANKS)
        return max_len > 50000 && wide(items, keep) ? launch_select<512, 11, WIDE>(p, n_seqs, s)
               : items <= 24                        ? launch_select<512, 11, CLUSTER>(p, n_seqs, s)
                                                    : launch_select<256, 8, CLUSTER>(p, n_seqs, s);
    return max_len <= 3000 ? launch_select<256, 8, 1>(p, n_seqs, s) : launch_select<512, 9, 1>(p, n_seqs, s);
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
    if (weights) {
        p.w = weights->data;
        p.w_blocks = weights->num_blocks;
        p.w_from = weight_tables;
        p.w_from_stride = wt_stride;
        p.w_to = new_weight_tables;
        p.w_to_stride = new_wt_stride;
    }
    cudaStream_t s = (cudaStream_t)cuda_stream;
    // a token's row in its pool is counted in 32 bits
    const long long most = weights && weights->num_blocks > p.num_blocks ? weights->num_blocks : p.num_blocks;
    if (most * p.n_kv * 16 > 0xfffffffell)
        return HB_ERANGE;
    const long long items = (long long)n_seqs * p.n_kv;
    if (keep <= 32 && items >= MOVE_FEW_ITEMS) {
        const long long units = items * (p.w ? 3 : 2), blocks = (units + FEW_WARPS - 1) / FEW_WARPS;
        if (blocks > 0x7fffffffll)
            return HB_ERANGE;
        return launch_kernel(true, pool->head_dim == 128 ? k_evict_move_few<128> : k_evict_move_few<64>,
                             dim3((unsigned)blocks), dim3(FEW_WARPS * 32), 0, s, p, units) == cudaSuccess
                   ? HB_OK
                   : HB_ECUDA;
    }
    // One CTA or a cluster of them for a stream (us): 1 kv head that keeps 1000
    // tokens 7.9 and 3.5; 16 that keep 250 3.6 and 5.4, 1000 8.3 and 6.7; 64 that
    // keep 1000 14.2 and 19.8, 3000 42.9 and 40.9
    if ((long long)keep * pool->head_dim <= 128 * (64 + 36 * items))
        return pool->head_dim == 128 ? launch_move<128, 1>(p, n_seqs, s) : launch_move<64, 1>(p, n_seqs, s);
    if (wide(items, keep))
        return pool->head_dim == 128 ? launch_move<128, WIDE>(p, n_seqs, s) : launch_move<64, WIDE>(p, n_seqs, s);
    return pool->head_dim == 128 ? launch_move<128, CLUSTER>(p, n_seqs, s) : launch_move<64, CLUSTER>(p, n_seqs, s);
} catch (...) {
    return HB_ENOMEM;
}
