// paged_attention.cu -- decode attention over the paged bf16 cache: of rows
// behind shared prefixes, and with the weight that each key gets
// (include/hb_paged.h).
//
//   s_t = q . k_t,  p_t = 2^((s_t - m) c2),  o = sum p_t v_t / sum p_t,
//   c2 = log2(e) / sqrt(d)
//
// in one pass over a row's keys with the running maximum m and sum of the
// softmax; rows with many keys are split over CTAs and joined by a second
// kernel.
//
// A warp takes a page (16 keys) at a time and 8 or 16 queries that share the kv
// head as the columns of m16n8k16 MMAs (bf16 in, fp32 sums): S^T = K q, then
// O^T += V^T P with P in two bf16 terms (16 significant bits: one term alone
// would cost as much precision as rounding the result to bf16 does).
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "kv4_host.h"
#include "paged.h"

namespace hb {
namespace {

using namespace paged;

constexpr int WARPS = 4;
constexpr int JOIN_WARPS = 8;
// A warp takes a tile's keys alone up to so many of them, where there are so many
// tiles, and up to more where many tiles share their keys (us, four warps a tile and
// so): 71 rows of 14 to 31 keys, 32 heads, 19.3 and 10.1; 16 rows of 281 behind a
// prefix, 52 heads, 46.4 and 52.8; windows of 16 queries, 58 x 10 kv heads x 8 at
// 260 keys, 160 and 127, 16 x 4 x 12 at 260, 22.1 and 23.8.
constexpr int ALONE_KEYS = 192, ALONE_KEYS_SHARED = 512;
constexpr long long ALONE_UNITS = 456, ALONE_UNITS_SHARED = 1200;
constexpr int SMS = 152;
constexpr int PART_MIN = 2;          // sub-tiles of a CTA of the prefixes' kernel at least
constexpr long long SHARE_BYTES = 24 << 20;  // of all groups
constexpr long long SHARE_GROUP = 1 << 20;   // of one, where others are shared anyway
// Bytes of own keys that an SM streams in a third of a sub-tile's time, halved
// where contexts are taken to be half of max_ctx on average; more beside prefixes
// bound by their products, which leave the memory to the others: 53.1 us so and
// 47.5 with 32768 (1 + 7 + 56 rows, prefixes of 0, 333 and 16389), but 25.6 and
// 27.5 (18 rows over 768 keys).
constexpr int OWN_UNIT = 20480, OWN_UNIT_BESIDE = 32768;
// Sub-tiles from which on a window's keys go to the tensor cores' kernel, with
// many queries of a kv head and with 17 to 48 (us): 4 sequences of 8 kv heads x
// 8 x 16 queries at 200 keys 17.5 against 14.4, at 600 21 and 24, at 3000 41 and
// 93; 4 of 40 kv heads x 32 queries at 600 keys 35 and 29, at 3000 104 and 107.
constexpr int COMMON_MIN = 8, COMMON_MIN_FEW = 24;
constexpr int WEIGH_THREADS = 256;
constexpr int JOIN_CTAS = 2 * SMS;   // CTAs of weights up to which their kernel takes the join along
constexpr float LOG2E = 1.4426950408889634f;

__device__ __forceinline__ float nan_f() { return __int_as_float(0x7fc00000); }

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16 bytes to shared memory, zeros unless ok.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool ok)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// Two fp32 numbers as bf16 pairs hi + lo.
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t &hi, uint32_t &lo)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    const float2 f = __bfloat1622float2(h);
    const __nv_bfloat162 r = __floats2bfloat162_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&r);
}

// A bf16 pair with what is beyond the finite numbers brought back to the largest of
// its sign.  V is multiplied by P = hi + lo, of which lo may be 0 or negative: an
// infinity is the high term's alone.  128 rows' own keys beside a prefix take 103.6 us
// with it and 103.1 without, 4 short rows 4.00 and 3.94.
__device__ __forceinline__ uint32_t finite_pair(uint32_t x)
{
    uint32_t y;
    asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0x7f7f7f7fu));
    return y;
}

// A bf16 pair with an infinity or a NaN in it.
__device__ __forceinline__ bool odd_pair(uint32_t x)
{
    return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}

template <int D>
struct Ring {
    static constexpr int ROW = D * 2;             // bytes of a key
    static constexpr int HALF = 16 * ROW;         // K or V of a page
    static constexpr int PAGE = 2 * HALF;
    static constexpr int DEPTH = D == 128 ? 2 : 3;  // pages of a warp, one of them in use
};

// Shared memory: a ring of pages for each warp, and after the key loop, in the
// same place, the warps' results.
template <int D, int NT>
struct Smem {
    static constexpr int ROW = D + 4;  // floats of a result row, off the banks of the next
    static constexpr int RINGS = WARPS * Ring<D>::DEPTH * Ring<D>::PAGE;
    static constexpr int JOIN = WARPS * 8 * NT * ROW * 4;
    static constexpr int BYTES = RINGS > JOIN ? RINGS : JOIN;
    static constexpr int SCORES = 2048;  // numbers that follow where a CTA keeps its scores: three CTAs an SM still fit
};

// Row chunks of 16 bytes lie at c ^ (key & 7), so that eight keys' chunks are on
// different banks.
template <int D>
__device__ __forceinline__ uint32_t place(int key, int c)
{
    return (uint32_t)(key * Ring<D>::ROW + ((c ^ (key & 7)) << 4));
}

// a[j] += the weight of key j of four, from their scores and a query's m and 1 / l
// (0 where that is not a number: it adds nothing).
__device__ __forceinline__ void add_weights(float (&a)[4], float4 v, float2 ml, float c2)
{
    if (ml.y == 0.f)
        return;
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        a[j] += ex2((x[j] - ml.x) * c2) * ml.y;
}

// Where the weights of keys key .. key + 3 lie (key a multiple of 4), or null.
__device__ __forceinline__ float *weights_of(const Attn &p, int seq, int kvh, int key)
{
    const Weigh &w = p.weigh;
    const int blk = __ldg(w.tables + (size_t)seq * w.stride + (key >> 4));
    return blk < 0 || blk >= w.num_blocks ? nullptr : w.w + ((size_t)blk * p.n_kv + kvh) * 16 + (key & 15);
}

// w = decay w + a there, of the keys up to ctx; the call's own rows' start from 0.
__device__ __forceinline__ void put_weights(const Attn &p, float *to, float4 old, int ctx, int key, const float (&a)[4])
{
    const float decay = p.weigh.decay, o[4] = {old.x, old.y, old.z, old.w};
    float x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        x[j] = decay == 0.f || key + j > ctx - p.nq ? a[j] : a[j] + decay * o[j];
    if (key + 3 <= ctx) {
        *reinterpret_cast<float4 *>(to) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (key + j <= ctx)
                to[j] = x[j];
    }
}

// A tile of 8 NT of a kv head's queries of one sequence, and the keys of one
// split.  KW = WARPS: a CTA has one tile, whose warps take the pages in turn, each
// with a ring and a softmax of its own, and join their results in shared memory.
// KW = 1, for many queries or few keys: each warp has a tile of its own, or a kv
// head, and all pages.  BALANCE: splits go by the rows' lengths.
//
// The keys' stream bounds it: twelve warps an SM with a page of 8 KB each under way
// beside the one in use (18 rows of 1024 keys, 40 heads, with weights: 64.7 us, 0.87
// of a copy's rate; two pages a warp and three CTAs in place of three and two took 7
// of 82 us).  That most of the MMAs' columns are idle for one query costs nothing
// then; for more than eight a page's time is the MMAs' and the softmax's latency.
template <int D, int NT, bool SCORES, int KW, bool BALANCE>
__global__ void __launch_bounds__(WARPS * 32) k_paged_attention(const __grid_constant__ Attn p)
{
    using R = Ring<D>;
    using S = Smem<D, NT>;
    constexpr int KS = D / 16;  // k-steps of S, channel tiles of O
    constexpr int COLS = 8 * NT;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_m[WARPS][COLS], s_l[WARPS][COLS];
    __shared__ float2 s_final[WARPS / KW][COLS];

    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int g = lane >> 2, t = lane & 3;
    const int split = blockIdx.x % p.n_splits;
    const int rest = blockIdx.x / p.n_splits;
    const int unit = rest * (WARPS / KW) + (KW == 1 ? warp : 0), tile = unit % p.col_tiles, kvh = unit / p.col_tiles;
    const int kw = KW == 1 ? 0 : warp;  // this warp's turn among the pages
    const int seq = blockIdx.y;
    const int ncols = p.nq * p.group;
    const int c0 = tile * COLS;

    // Beside the prefixes' kernel, whose CTAs have all passed their wait for what
    // came before when this one starts.  One CTA waits for its end, so that the
    // join, which waits for this kernel, finds both done.
    if (!p.beside)
        pdl_wait();
    pdl_trigger();
    auto leave = [&]() {
        if (p.beside && blockIdx.x == 0 && blockIdx.y == 0)
            pdl_wait();
    };
    const int ctx = p.ctx_lens[seq];
    int from = 0, least = 0;  // first own key, smallest context
    int common = 0, row0 = seq;  // pages that are the group's, found through its first row's table
    if (p.n_groups > 0) {
        const Group gr = p.of(seq);
        from = gr.shared;
        least = gr.prefix > 0 ? gr.prefix - 1 : 0;
        common = gr.prefix >> 4;
        row0 = gr.row0;
    } else if (ctx >= 0 && ctx <= p.max_ctx) {
        from = p.sequence(seq, ctx).shared;
    }
    // where a row's keys start and end is the same for all threads of the CTA
    if (ctx < least || ctx > p.max_ctx) {  // padding: zeros; outside its range: NaN
        if (p.direct && split == 0 && kvh < p.n_kv)
            for (int i = kw * 32 + lane; i < COLS * D; i += KW * 32) {
                const int c = c0 + i / D;
                if (c < ncols)
                    p.out[(long long)(seq * p.nq + c / p.group) * p.out_stride +
                          (size_t)(kvh * p.group + c % p.group) * D + i % D] = f2bf(ctx == -1 ? 0.f : nan_f());
            }
        return leave();
    }
    const int split_len = BALANCE ? p.balanced() : p.split_len;
    const int k0 = from + split * split_len, k1 = min(ctx + 1, k0 + split_len);
    if (k0 >= k1 || (KW == 1 && kvh >= p.n_kv))
        return leave();  // the join knows how many splits a row has

    // ---- this warp's pages: b0 + KW i, i < n
    const int b0 = (k0 >> 4) + kw;
    const int n = max(0, (((k1 + 15) >> 4) - b0 + KW - 1) / KW);
    auto page_id = [&](int i) {
        const int b = b0 + i * KW;
        return __ldg(p.tables + (size_t)(b < common ? row0 : seq) * p.bt_stride + b);
    };
    uint8_t *ring = smem + warp * R::DEPTH * R::PAGE;
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
    int ids = lane < n ? page_id(lane) : 0;  // lane i: page i of the current 32
    bool bad = false;
    auto issue = [&](int i) {
        if (i < n) {
            if ((i & 31) == 0 && i > 0)
                ids = i + lane < n ? page_id(i + lane) : 0;
            const int blk = __shfl_sync(0xffffffffu, ids, i & 31);
            const bool ok = blk >= 0 && blk < p.num_blocks;
            bad |= !ok;
            const size_t at = ((size_t)(ok ? blk : 0) * p.n_kv + kvh) * 16 * D;
            const int left = ok ? k1 - (b0 + i * KW) * 16 : 0;  // keys of the page that count
            const uint32_t dst = ring_at + (i % R::DEPTH) * R::PAGE;
#pragma unroll
            for (int j = 0; j < R::HALF / 512; ++j) {
                const int e = j * 32 + lane, key = e / (D / 8), c = e % (D / 8);
                copy16(dst + place<D>(key, c), p.k + at + (size_t)e * 8, key < left);
                copy16(dst + R::HALF + place<D>(key, c), p.v + at + (size_t)e * 8, key < left);
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < R::DEPTH - 1; ++i)
        issue(i);

    // ---- q as B fragments: (channels 2t, 2t + 1 and 2t + 8, 2t + 9; column g)
    uint32_t qf[NT][KS][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int c = c0 + nt * 8 + g;
        const bool have = c < ncols;
        const bf16 *qr = p.q + (long long)(seq * p.nq + (have ? c / p.group : 0)) * p.q_stride +
                         (size_t)(kvh * p.group + (have ? c % p.group : 0)) * D + 2 * t;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            qf[nt][ks][0] = have ? *reinterpret_cast<const uint32_t *>(qr + 16 * ks) : 0u;
            qf[nt][ks][1] = have ? *reinterpret_cast<const uint32_t *>(qr + 16 * ks + 8) : 0u;
        }
    }
    // keys that this lane's columns see
    int see[NT][2];
    int fewest = ctx + 1;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = min(c0 + nt * 8 + 2 * t + j, ncols - 1);
            see[nt][j] = min(k1, ctx + 1 - (p.nq - 1) + c / p.group);
        }
    if (p.nq > 1)
        fewest = ctx + 1 - (p.nq - 1) + c0 / p.group;

    float m[NT][2], l[NT][2], o[NT][KS][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int i = 0; i < KS; ++i)
            o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    }
    float *score_at = nullptr;  // of column 2t of the first tile, key g
    // scores in shared memory
    const bool keep = SCORES && p.fused && ncols * p.score_stride <= S::SCORES * KW / WARPS;
    float *scores = nullptr;
    if (SCORES) {
        scores = keep ? reinterpret_cast<float *>(smem + S::BYTES) + (KW == 1 ? warp : 0) * (S::SCORES / WARPS)
                      : p.scores + ((size_t)seq * p.n_kv + kvh) * ncols * p.score_stride;
        score_at = scores + (size_t)(c0 + 2 * t) * p.score_stride + g;
    }

    const int mi = lane >> 3;
    for (int i = 0; i < n; ++i) {
        copy_wait<R::DEPTH - 2>();
        __syncwarp();  // every lane's copies of page i are here, and page i - 1 is done with
        issue(i + R::DEPTH - 1);
        const uint32_t page = ring_at + (i % R::DEPTH) * R::PAGE;
        const int key0 = (b0 + i * KW) * 16;

        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t a[4];
            ldmatrix4(a, page + place<D>((lane & 7) + 8 * (mi & 1), 2 * ks + (mi >> 1)));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                mma_bf16(s[nt], a, qf[nt][ks][0], qf[nt][ks][1]);
        }
        if (key0 + 16 > min(fewest, k1))  // keys that a query does not see
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (key0 + g + 8 * (j >> 1) >= see[nt][j & 1])
                        s[nt][j] = -INFINITY;
        if (SCORES)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c0 + nt * 8 + 2 * t + (j & 1) < ncols)
                        score_at[(size_t)(nt * 8 + (j & 1)) * p.score_stride + key0 + 8 * (j >> 1)] = s[nt][j];

        uint32_t hi[NT][2], lo[NT][2];
        float pr[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float corr[2], base[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float mx = fmaxf(s[nt][j], s[nt][j + 2]);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                mx = fmaxf(mx, m[nt][j]);
                base[j] = mx == -INFINITY ? 0.f : mx;
                corr[j] = ex2((m[nt][j] - base[j]) * p.c2);
                m[nt][j] = mx;
            }
            // the difference first: a fused s c2 - m c2 would round a large maximum away
#pragma unroll
            for (int j = 0; j < 4; ++j)
                pr[nt][j] = ex2((s[nt][j] - base[j & 1]) * p.c2);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                l[nt][j] = l[nt][j] * corr[j] + (pr[nt][j] + pr[nt][j + 2]);
            if (corr[0] != 1.f || corr[1] != 1.f)
#pragma unroll
                for (int x = 0; x < KS; ++x)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        o[nt][x][j] *= corr[j & 1];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                split_bf16(pr[nt][2 * h], pr[nt][2 * h + 1], hi[nt][h], lo[nt][h]);
                hi[nt][h] = movmatrix(hi[nt][h]);
                lo[nt][h] = movmatrix(lo[nt][h]);
            }
        }
        const uint32_t vpage = page + R::HALF;
#pragma unroll
        for (int x = 0; x < KS; ++x) {
            uint32_t a[4];
            ldmatrix4_trans(a, vpage + place<D>((lane & 7) + 8 * (mi >> 1), 2 * x + (mi & 1)));
            if (p.nq == 1 || key0 + 16 <= fewest ||
                !__any_sync(0xffffffffu, odd_pair(a[0]) || odd_pair(a[1]) || odd_pair(a[2]) || odd_pair(a[3]))) {
                const uint32_t b[4] = {finite_pair(a[0]), finite_pair(a[1]), finite_pair(a[2]), finite_pair(a[3])};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_bf16(o[nt][x], a, hi[nt][0], hi[nt][1]);
                    mma_bf16(o[nt][x], b, lo[nt][0], lo[nt][1]);
                }
                continue;
            }
            // an infinity or a NaN that not every query sees: key by key
#pragma unroll 1
            for (int key = 0; key < 16; ++key) {
                const bf16 *vr = reinterpret_cast<const bf16 *>(ring + (i % R::DEPTH) * R::PAGE + R::HALF);
                const float v0 = bf2f(vr[(place<D>(key, 2 * x) >> 1) + g]);
                const float v1 = bf2f(vr[(place<D>(key, 2 * x + 1) >> 1) + g]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float a0 = __shfl_sync(0xffffffffu, pr[nt][j], (key & 7) * 4 + t);
                        const float a1 = __shfl_sync(0xffffffffu, pr[nt][j + 2], (key & 7) * 4 + t);
                        const float w = key < 8 ? a0 : a1;
                        if (key0 + key < see[nt][j]) {
                            o[nt][x][j] += w * v0;
                            o[nt][x][j + 2] += w * v1;
                        }
                    }
            }
        }
    }
    copy_wait<0>();
    bad = __any_sync(0xffffffffu, bad);

    // ---- join the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float x = l[nt][j];
            x += __shfl_xor_sync(0xffffffffu, x, 4);
            x += __shfl_xor_sync(0xffffffffu, x, 8);
            x += __shfl_xor_sync(0xffffffffu, x, 16);
            if (g == 0) {
                s_m[warp][nt * 8 + 2 * t + j] = m[nt][j];
                s_l[warp][nt * 8 + 2 * t + j] = bad ? nan_f() : x;
            }
        }
    auto sync = [&]() {
        if constexpr (KW == 1)
            __syncwarp();
        else
            __syncthreads();
    };
    sync();  // also: no warp's ring is in use any more (KW = 1: this warp's)
    const int first = KW == 1 ? warp : 0;  // of the warps that share the tile
    float *so = reinterpret_cast<float *>(KW == 1 ? ring : smem);
    static_assert(COLS * S::ROW * 4 <= R::DEPTH * R::PAGE);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = nt * 8 + 2 * t + j;
            float mx = s_m[first][c];
#pragma unroll
            for (int w = 1; w < KW; ++w)
                mx = fmaxf(mx, s_m[w][c]);
            const float f = KW == 1 ? 1.f : ex2((m[nt][j] - (mx == -INFINITY ? 0.f : mx)) * p.c2);
            float *row = so + (kw * COLS + c) * S::ROW + g;
#pragma unroll
            for (int x = 0; x < KS; ++x) {
                row[x * 16] = o[nt][x][j] * f;
                row[x * 16 + 8] = o[nt][x][j + 2] * f;
            }
        }
    sync();
    for (int i = kw * 32 + lane; i < COLS * (D / 4); i += KW * 32) {
        const int cl = i / (D / 4), e = i % (D / 4) * 4, c = c0 + cl;
        if (c >= ncols)
            break;
        float mx = s_m[first][cl];
#pragma unroll
        for (int w = 1; w < KW; ++w)
            mx = fmaxf(mx, s_m[w][cl]);
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            sum += s_l[first + w][cl] * ex2((s_m[first + w][cl] - (mx == -INFINITY ? 0.f : mx)) * p.c2);
            const float4 a = *reinterpret_cast<const float4 *>(so + (w * COLS + cl) * S::ROW + e);
            acc.x += a.x, acc.y += a.y, acc.z += a.z, acc.w += a.w;
        }
        const long long row = (long long)seq * p.nq + c / p.group;
        const int head = kvh * p.group + c % p.group;
        if (p.direct) {
            const bool none = ctx + 1 - (p.nq - 1) + c / p.group <= 0;
            const float f = none ? 0.f : 1.f / sum;
            uint2 u;
            __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&u);
            h[0] = __floats2bfloat162_rn(none ? 0.f : acc.x * f, none ? 0.f : acc.y * f);
            h[1] = __floats2bfloat162_rn(none ? 0.f : acc.z * f, none ? 0.f : acc.w * f);
            *reinterpret_cast<uint2 *>(p.out + row * p.out_stride + (size_t)head * D + e) = u;
        } else {
            const size_t slot = ((size_t)row * p.n_heads + head) * p.n_slots + p.first_slot + split;
            if (e == 0)
                p.part_ml[slot] = make_float2(mx, sum);
            *reinterpret_cast<float4 *>(p.part_o + slot * D + e) = acc;
        }
        if (SCORES && p.direct && e == 0) {
            const float2 x = make_float2(mx == -INFINITY ? 0.f : mx, sum > 0.f ? 1.f / sum : 0.f);
            if (p.fused)
                s_final[KW == 1 ? warp : 0][cl] = x;
            else
                p.final_ml[(size_t)row * p.n_heads + head] = x;
        }
    }
    if (SCORES && p.fused) {  // the CTA (or warp) has all keys and queries: the weights, four keys a thread
        sync();
        for (int key = (kw * 32 + lane) * 4; key <= ctx; key += KW * 32 * 4) {
            float *to = weights_of(p, seq, kvh, key);
            if (!to)
                continue;
            float4 old = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p.weigh.decay != 0.f)
                old = *reinterpret_cast<const float4 *>(to);
            float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < COLS; ++c)
                if (c < ncols) {
                    const float *s = scores + c * p.score_stride + key;
                    add_weights(a, keep ? *reinterpret_cast<const float4 *>(s) : __ldcg(reinterpret_cast<const float4 *>(s)),
                                s_final[KW == 1 ? warp : 0][c], p.c2);
                }
            put_weights(p, to, old, ctx, key, a);
        }
    }
    leave();
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= FLT_MAX; }

// Infinities and NaN of V in E channels, of a table's first keys (a multiple of 16),
// added up without their weights; 0 where there are none.
template <int D, int E>
__device__ __forceinline__ void odd_values(const Attn &p, const int *table, int kvh, int keys, int channel, float (&s)[E])
{
    constexpr int BATCH = 8;
    using V = typename std::conditional<E == 4, uint2, uint32_t>::type;
#pragma unroll
    for (int e = 0; e < E; ++e)
        s[e] = 0.f;
    int next = __ldg(table);
#pragma unroll 1
    for (int t = 0; t < keys; t += BATCH) {
        const int blk = next;
        next = __ldg(table + (min(t + BATCH, keys - 1) >> 4));
        if (blk < 0 || blk >= p.num_blocks)
            continue;
        const bf16 *at = p.v + (((size_t)blk * p.n_kv + kvh) * 16 + (t & 15)) * D + channel;
        V v[BATCH];
#pragma unroll
        for (int u = 0; u < BATCH; ++u)
            v[u] = *reinterpret_cast<const V *>(at + u * D);
#pragma unroll
        for (int u = 0; u < BATCH; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float x = bf2f(reinterpret_cast<const bf16 *>(&v[u])[e]);
                s[e] += finite(x) ? 0.f : x;
            }
    }
}

// The join of a row's partials, those of the common keys and of its own splits:
// W warps a (row, head), each with every W-th partial.  o = sum 2^((m_i - m) c2) o_i
// / sum 2^((m_i - m) c2) l_i.  Latency bounds it, two reads that follow one another:
// 3 to 4 us behind the attention (64 heads of 57 partials, 128 channels).
template <int D, int W>
__device__ __forceinline__ void join(const Attn &p, int split_len, int block, int n_rows)
{
    constexpr int E = D / 32;
    constexpr int BATCH = 4;  // partials whose loads are under way together
    __shared__ float s_o[W > 1 ? JOIN_WARPS : 1][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w0 = warp % W;
    const long long item = (long long)block * (JOIN_WARPS / W) + warp / W;
    if (W < JOIN_WARPS && item >= (long long)n_rows * p.n_heads)
        return;
    const int row = (int)(item / p.n_heads), head = (int)(item % p.n_heads);
    const int seq = row / p.nq;
    const int ctx = p.ctx_lens[seq];
    int from = 0, least = 0, parts = 0, row0 = seq;
    if (p.n_groups > 0) {
        const Group gr = p.of(seq);
        from = gr.shared;
        least = gr.prefix > 0 ? gr.prefix - 1 : 0;
        parts = gr.parts;
        row0 = gr.row0;
    }
    const bool in = ctx >= least && ctx <= p.max_ctx;
    if (p.n_groups == 0 && in) {
        const Group gr = p.sequence(seq, ctx);
        from = gr.shared;
        parts = gr.parts;
    }
    const bool sees = ctx + 1 - (p.nq - 1) + row % p.nq > 0;
    const int n = in ? parts + (ctx + 1 - from + split_len - 1) / split_len : 0;
    const size_t first = ((size_t)row * p.n_heads + head) * p.n_slots;
    auto slot = [&](int i) { return first + (i < parts ? i : p.first_slot + i - parts); };
    // (m, l) of the first 32 partials, a lane each, and the greatest m of all
    float2 mine = make_float2(-INFINITY, 0.f);
    if (lane < n)
        mine = __ldcg(&p.part_ml[slot(lane)]);
    float mx = mine.x;
    for (int i = lane + 32; i < n; i += 32)
        mx = fmaxf(mx, __ldcg(&p.part_ml[slot(i)]).x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1)
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    const float base = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        acc[e] = 0.f;
    for (int j0 = 0; j0 < n; j0 += 32) {
        if (j0 > 0)
            mine = j0 + lane < n ? __ldcg(&p.part_ml[slot(j0 + lane)]) : make_float2(-INFINITY, 0.f);
        const float f = ex2((mine.x - base) * p.c2);
        float part = j0 + lane < n ? mine.y * f : 0.f;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1)
            part += __shfl_xor_sync(0xffffffffu, part, x);
        sum += part;
        const int upto = min(32, n - j0);
        for (int i0 = w0; i0 < upto; i0 += BATCH * W) {
            float v[BATCH][E];
#pragma unroll
            for (int u = 0; u < BATCH; ++u)
                if (i0 + u * W < upto) {
                    const float *o = p.part_o + slot(j0 + i0 + u * W) * D + lane * E;
                    if constexpr (E == 4)
                        *reinterpret_cast<float4 *>(v[u]) = __ldcg(reinterpret_cast<const float4 *>(o));
                    else
                        *reinterpret_cast<float2 *>(v[u]) = __ldcg(reinterpret_cast<const float2 *>(o));
                }
#pragma unroll
            for (int u = 0; u < BATCH; ++u)
                if (i0 + u * W < upto) {
                    const float x = __shfl_sync(0xffffffffu, f, i0 + u * W);
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        acc[e] += v[u][e] * x;
                }
        }
    }
    if constexpr (W > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            s_o[warp][lane * E + e] = acc[e];
        __syncthreads();
        if (w0 != 0)
            return;
#pragma unroll
        for (int w = 1; w < W; ++w) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                acc[e] += s_o[warp + w][lane * E + e];
        }
    }
    float all = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
        all += acc[e];
    if (all * 0.f != 0.f && sum > 0.f && parts > 0) {
        // An infinity in V: the common keys' products have both terms of P with V as it
        // is, and what they give for it says nothing.  So the infinities themselves, and
        // those of the own keys' results (16 rows x 64 heads behind 60000 keys: 4.5 ms).
        float odd[E];
        odd_values<D>(p, p.tables + (size_t)row0 * p.bt_stride, head / p.group, from, lane * E, odd);
        for (int i = parts; i < n; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float x = __ldcg(p.part_o + slot(i) * D + lane * E + e);
                odd[e] += finite(x) ? 0.f : x;
            }
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = finite(acc[e]) || odd[e] == 0.f ? acc[e] : odd[e];
    }
#pragma unroll
    for (int e = 0; e < E; ++e)  // padding, and a row that sees no key: zeros; outside its range: NaN
        acc[e] = in ? (sees ? acc[e] / sum : 0.f) : ctx == -1 ? 0.f : nan_f();
    bf16 *to = p.out + (long long)row * p.out_stride + (size_t)head * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<__nv_bfloat162 *>(to + e) = __floats2bfloat162_rn(acc[e], acc[e + 1]);
    if (p.final_ml && lane == 0)
        p.final_ml[(size_t)row * p.n_heads + head] = make_float2(base, sum > 0.f ? 1.f / sum : 0.f);
}

template <int D, int W, bool BALANCE>
__global__ void __launch_bounds__(JOIN_WARPS * 32) k_paged_join(const __grid_constant__ Attn p, int n_rows)
{
    const int split_len = BALANCE ? p.balanced() : p.split_len;  // the contexts were there before the kernel before this one
    pdl_wait();
    pdl_trigger();
    join<D, W>(p, split_len, blockIdx.x, n_rows);
}

// The weights of a kv head's keys, summed over its queries' scores: four keys a
// thread, and SHARES threads for the queries of the same keys.  The (m, l) of the
// rows come from the join's kernel before this one, and the first scores are fetched
// while it runs.  JOIN, for few CTAs: the join runs in this kernel's first CTAs,
// and each of the others joins the (m, l) that it needs for itself, so that neither
// waits for the other (us, as chosen and the other way: 2 rows of 30550 keys, 4
// heads, 14.0 and 16.4; one of 131000, 8 x 8 heads, 102.6 and 107.9; 2 x 32
// queries, 8 x 4 heads, 27.7 and 30.0).
template <int SHARES, bool JOIN, int D, int W>
__global__ void __launch_bounds__(WEIGH_THREADS)
    k_paged_weigh(const __grid_constant__ Attn p, int n_rows, int join_blocks, int chunks)
{
    constexpr int QUADS = WEIGH_THREADS / SHARES, BATCH = 8, CHUNK = 256, LANES = 8;
    static_assert(WEIGH_THREADS == JOIN_WARPS * 32);
    __shared__ float2 s_ml[CHUNK];
    __shared__ float4 s_a[SHARES > 1 ? SHARES - 1 : 1][QUADS];
    [[maybe_unused]] int split_len;
    if constexpr (JOIN) {  // at most 16 queries a kv head, no common keys, several splits
        split_len = p.balanced();
        if ((int)blockIdx.x < join_blocks) {
            pdl_wait();
            pdl_trigger();
            return join<D, W>(p, split_len, blockIdx.x, n_rows);
        }
    }
    int seq = blockIdx.y, kvh = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
    if constexpr (JOIN) {  // all in one row of the grid
        const int at = (int)blockIdx.x - join_blocks;
        seq = at / (p.n_kv * chunks), kvh = at / chunks % p.n_kv, chunk = at % chunks;
    }
    // When this kernel starts those before it have passed their waits: what was
    // there before the last of them can be read, old weights and (where that is the
    // join) scores; only its own results not yet
    const int ctx = p.ctx_lens[seq];
    const int quad = threadIdx.x % QUADS, share = threadIdx.x / QUADS;
    const int key = (chunk * QUADS + quad) * 4;
    const bool none = ctx > p.max_ctx || chunk * QUADS * 4 > ctx, some = !none && key <= ctx;
    float *to = nullptr;
    float4 old = make_float4(0.f, 0.f, 0.f, 0.f);
    if (some && share == 0) {
        to = weights_of(p, seq, kvh, key);
        if (to && p.weigh.decay != 0.f)
            old = __ldcg(reinterpret_cast<const float4 *>(to));
    }
    // queries CHUNK at a time, an equal number for each of the shares
    const int ncols = p.nq * p.group;
    const float *s = p.scores + ((size_t)seq * p.n_kv + kvh) * ncols * p.score_stride + key;
    float4 v[BATCH];
    auto load = [&](int c0, int c1) {
        const float *at = s + (size_t)c0 * p.score_stride;
#pragma unroll
        for (int u = 0; u < BATCH; ++u, at += p.score_stride)
            if (c0 + u < c1)
                v[u] = __ldcg(reinterpret_cast<const float4 *>(at));
    };
    const int each0 = (min(CHUNK, ncols) + SHARES - 1) / SHARES;  // of the first chunk
    const bool early = !JOIN && !p.direct;
    if (early && some)
        load(share * each0, min(min(CHUNK, ncols), (share + 1) * each0));
    pdl_wait();
    pdl_trigger();
    if (none)
        return;
    if (!early && some)
        load(share * each0, min(min(CHUNK, ncols), (share + 1) * each0));
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    for (int q0 = 0; q0 < ncols; q0 += CHUNK) {
        const int n = min(CHUNK, ncols - q0), each = (n + SHARES - 1) / SHARES;
        if (q0 > 0)
            __syncthreads();  // the chunk before is done with
        auto row_head = [&](int c) {
            const int i = (q0 + c) / p.group;
            return ((size_t)seq * p.nq + i) * p.n_heads + kvh * p.group + (q0 + c - i * p.group);
        };
        if constexpr (!JOIN) {
            for (int c = threadIdx.x; c < n; c += WEIGH_THREADS)
                s_ml[c] = __ldcg(p.final_ml + row_head(c));
        } else {  // LANES threads a query, each with every LANES-th partial
            const int n_parts = (ctx + split_len) / split_len;
            for (int b = 0; b < n; b += WEIGH_THREADS / LANES) {
                const int c = b + (int)threadIdx.x / LANES;
                const float2 *ml = p.part_ml + row_head(min(c, n - 1)) * p.n_slots;
                float m = -INFINITY, l = 0.f;
                auto add = [&](float m1, float l1) {
                    const float mx = fmaxf(m, m1), base = mx == -INFINITY ? 0.f : mx;
                    l = l * ex2((m - base) * p.c2) + l1 * ex2((m1 - base) * p.c2);
                    m = mx;
                };
#pragma unroll 4
                for (int x = threadIdx.x % LANES; x < n_parts; x += LANES) {
                    const float2 y = __ldcg(ml + x);
                    add(y.x, y.y);
                }
                __syncwarp();
#pragma unroll
                for (int x = 1; x < LANES; x <<= 1)
                    add(__shfl_xor_sync(0xffffffffu, m, x), __shfl_xor_sync(0xffffffffu, l, x));
                if (threadIdx.x % LANES == 0 && c < n)
                    s_ml[c] = make_float2(m == -INFINITY ? 0.f : m, l > 0.f ? 1.f / l : 0.f);
            }
        }
        __syncthreads();
        if (!some)
            continue;
        const int c1 = min(n, (share + 1) * each);
        for (int c0 = share * each; c0 < c1; c0 += BATCH) {
            if (q0 > 0 || c0 > share * each)
                load(q0 + c0, q0 + c1);
#pragma unroll
            for (int u = 0; u < BATCH; ++u)
                if (c0 + u < c1)
                    add_weights(a, v[u], s_ml[c0 + u], p.c2);
        }
    }
    if constexpr (SHARES > 1) {
        if (share > 0)
            s_a[share - 1][quad] = make_float4(a[0], a[1], a[2], a[3]);
        __syncthreads();
        if (share > 0)
            return;
#pragma unroll
        for (int i = 0; i < SHARES - 1; ++i) {
            const float4 b = s_a[i][quad];
            a[0] += b.x, a[1] += b.y, a[2] += b.z, a[3] += b.w;
        }
    }
    if (to)
        put_weights(p, to, old, ctx, key, a);
}

__global__ void k_paged_groups(Group *to, const __grid_constant__ Attn p, int first, int n)
{
    pdl_wait();
    if ((int)threadIdx.x < n)
        to[first + threadIdx.x] = p.few[threadIdx.x];
}

// ------------------------------------------------------------------- host

thread_local bool test_lose = false;  // of this thread's next launch of the common keys' kernel

long long round_up(long long x, long long to) { return (x + to - 1) / to * to; }

// Splits of at most `keys` own keys (a multiple of 64 each) of n_rows rows with
// `tiles` CTAs a split each: as many as the SMs hold at once, three each.  Where
// rows differ, counted are those that there will be: by `sum` of the lengths that
// the caller's prefixes tell, the longest of them `longest`.  A CTA's way through
// its keys is then weighed against the CTAs of the other rows, which find nothing
// to do: ROUND_US a round of 64 keys, for up to eight queries and for more, and
// EMPTY_US.  (33 rows, two of 4000 to 5700 keys among them, 5 kv heads x 12: 62 us
// with splits by the number of rows alone, 33 so; 21 rows, one of 4800, 40 heads:
// 30 and 25, and 49 with splits of 256.)
constexpr double ROUND_US[2] = {0.6, 1.1}, EMPTY_US = 1.55e-3;
void plan_splits(long long n_rows, long long tiles, int keys, long long longest, long long sum, int nt, int *len, int *n)
{
    const long long base = n_rows * tiles, most = keys / SPLIT_MIN;
    long long s = SLOTS / (base > 0 ? base : 1);
    const double least = sqrt((double)base * keys * 64 * EMPTY_US / ROUND_US[nt - 1]);
    if (longest > least && sum < n_rows * keys) {
        const long long w = (long long)((double)SLOTS * keys / ((double)tiles * sum)), fit = (long long)(keys / least);
        s = s > w || s > fit ? s : w < fit ? w : fit;
    }
    s = s < most ? s : most;
    s = s < 1 ? 1 : s;
    const long long each = round_up((keys + s - 1) / s, 64);
    *len = (int)(each > 0 ? each : 64);
    *n = (int)((keys + *len - 1) / *len);
    if (*n < 1)
        *n = 1;
}

// Byte offsets of the workspace, from its first multiple of 32 on: partials and
// scores are stored 32 bytes at a time, and a caller's workspace begins at 16.
constexpr int WORK_ALIGN = 32, WORK_GIVEN = 16;
struct Layout {
    long long ml, o, scores, final_ml, groups, bytes;
    long long score_stride;
};

char *work_base(void *workspace)
{
    return (char *)(((uintptr_t)workspace + WORK_ALIGN - 1) & ~(uintptr_t)(WORK_ALIGN - 1));
}

Layout layout(long long rows, int heads, int d, int slots, bool parts, int groups, bool scores, bool finals, int max_ctx)
{
    Layout w;
    w.ml = 0;
    w.score_stride = scores ? round_up((long long)max_ctx + 1, 64) : 0;
    w.o = w.ml + (parts ? round_up(rows * heads * slots * 8, 256) : 0);
    w.scores = w.o + (parts ? round_up(rows * heads * slots * d * 4, 256) : 0);
    w.final_ml = w.scores + rows * heads * w.score_stride * 4;
    w.groups = w.final_ml + (finals ? round_up(rows * heads * 8, 256) : 0);
    w.bytes = w.groups + (groups > INLINE_GROUPS ? round_up((long long)groups * sizeof(Group), 256) : 0);
    if (w.bytes > 0)
        w.bytes += WORK_ALIGN - WORK_GIVEN;
    return w;
}

int tiles_of(long long cols, int nt) { return (int)((cols + 8 * nt - 1) / (8 * nt)); }

template <int D, int NT, bool SCORES, int KW, bool BALANCE>
int launch_attention(const Attn &p, int n_seqs, cudaStream_t s)
{
    static std::atomic<uint64_t> done{0};
    auto kernel = k_paged_attention<D, NT, SCORES, KW, BALANCE>;
    const long long units = (long long)p.n_kv * p.col_tiles;
    // fits 31 bits: plan_splits() gives at most 3 SMS CTAs, a split a tile, or 2^11 sqrt(keys / tiles) splits
    const long long gx = (units * KW + WARPS - 1) / WARPS * p.n_splits;
    using S = Smem<D, NT>;
    constexpr int most = S::BYTES + (SCORES ? 4 * S::SCORES : 0);
    if (kv4_allow_smem((const void *)kernel, most, done) != cudaSuccess)
        return HB_ECUDA;
    const int smem = p.fused ? most : S::BYTES;
    return launch_kernel(true, kernel, dim3((unsigned)gx, (unsigned)n_seqs), dim3(WARPS * 32), smem, s, p) == cudaSuccess
               ? HB_OK
               : HB_ECUDA;
}

// Whether a warp takes a tile's keys alone.
bool alone(const Attn &p, int n_seqs)
{
    const long long units = (long long)n_seqs * p.n_kv * p.col_tiles;
    const bool shared = p.col_tiles > 1 && units >= ALONE_UNITS_SHARED;
    return units >= ALONE_UNITS && p.split_len <= (shared ? ALONE_KEYS_SHARED : ALONE_KEYS);
}

template <int D, int NT, bool SCORES>
int attention_of(const Attn &p, int n_seqs, cudaStream_t s)
{
    if (p.balance)  // at most SLOTS / 2 tiles: too few for a warp each
        return launch_attention<D, NT, SCORES, WARPS, true>(p, n_seqs, s);
    return alone(p, n_seqs) ? launch_attention<D, NT, SCORES, 1, false>(p, n_seqs, s)
                            : launch_attention<D, NT, SCORES, WARPS, false>(p, n_seqs, s);
}

template <bool SCORES>
int attention(const Attn &p, int d, int nt, int n_seqs, cudaStream_t s)
{
    if (d == 128)
        return nt == 1 ? attention_of<128, 1, SCORES>(p, n_seqs, s) : attention_of<128, 2, SCORES>(p, n_seqs, s);
    return nt == 1 ? attention_of<64, 1, SCORES>(p, n_seqs, s) : attention_of<64, 2, SCORES>(p, n_seqs, s);
}

// Checks that the attention calls share.  rows: of q and out.
int check_attention(const hb_paged_pool *pool, const void *q, long long q_stride, const int32_t *tables, int bt_stride,
                    const int32_t *ctx_lens, long long rows, int n_heads, int max_ctx, const void *out,
                    long long out_stride)
{
    int rc = check_pool(pool);
    if (rc)
        return rc;
    if (!tables || !ctx_lens || n_heads < 1 || n_heads % pool->n_kv_heads || max_ctx < 0)
        return HB_EINVAL;
    if ((uintptr_t)tables % 4 || (uintptr_t)ctx_lens % 4)
        return HB_EINVAL;
    if ((long long)n_heads * pool->head_dim > 0x7fffffffll)
        return HB_ERANGE;
    if ((rc = kv4_check_rows(q, q_stride, (int)rows, n_heads * pool->head_dim)) ||
        (rc = kv4_check_rows(out, out_stride, (int)rows, n_heads * pool->head_dim)))
        return rc;
    if (max_ctx >= MAX_KEYS || bt_stride < max_ctx / 16 + 1 || rows > 65535 || rows * n_heads > 0x7fffffffll)
        return HB_ERANGE;
    return HB_OK;
}

struct Plan {
    int nt, split_len, n_splits, col_tiles, first_slot, n_slots;
    int ctas;  // of the common keys' kernel
    bool balance;
    int seq_parts, seq_part_len;
    bool direct, fused;
    Layout at;
};

// Where all keys are the rows' own, splits go by the lengths that the rows have
// (Attn::balanced), with twice as many of them as rows of one length have, for those
// longer than the others (us): one row of 4000 keys, 8 kv heads x 8, in a call that
// allows 131071, 32 with splits by max_ctx and 10 so; weights of 6 sequences of 2517
// to 40293 keys, 4 kv heads x 5, 47 and 34; of 20 of 5928 keys, 5 kv heads, 55 and 58.
void balance(long long n_seqs, long long tiles, int keys, Plan *pl)
{
    const long long room = 2ll * pl->n_splits, all = SLOTS / tiles, most = keys / SPLIT_MIN;
    const long long n = room < all ? room : all, m = n < most ? n : most;
    static_assert(SLOTS / 2 <= BALANCE_SEQS);  // with two splits each no more of them have room
    pl->balance = true;
    pl->n_splits = n_seqs > 1 && m > pl->n_splits ? (int)m : pl->n_splits;
}

// Bytes that are read once only if a group's whole blocks are shared.
long long saved_bytes(int rows, int prefix, int n_kv, int d) { return (long long)(rows - 1) * (prefix & ~15) * n_kv * 4 * d; }

Group shared_group(int row0, int rows, int prefix, int n_kv, int d, bool share)
{
    Group g = {row0, rows, prefix, 0, 0, 0, 1};
    if (share && saved_bytes(rows, prefix, n_kv, d) >= SHARE_GROUP)
        g.shared = prefix & ~15;
    return g;
}

// CTAs of a group when none is to take more than `most` units (of a sub-tile's
// time: 3 where a CTA has at most 128 rows, 4 with two Q tiles), and their cut.
long long cut_group(Group *g, int heads, int n_kv, long long most)
{
    if (g->shared == 0)
        return 0;
    const long long cols = (long long)g->rows * heads, tiles = (cols + 255) / 256;
    const int subs = (g->shared + 63) / 64;
    const long long fit = most / (cols > 128 ? 4 : 3);
    g->part_len = fit < PART_MIN ? PART_MIN : fit > subs ? subs : (int)fit;
    g->parts = (subs + g->part_len - 1) / g->part_len;
    g->part_len = (subs + g->parts - 1) / g->parts;
    g->parts = (subs + g->part_len - 1) / g->part_len;
    return tiles * n_kv * g->parts;
}

// What hb_decode_shared does with its groups, which `each` receives in order.  HB_OK or an error.
template <typename F>
int plan_shared(int n_rows, int n_heads, int n_kv, int d, int num_blocks, int max_ctx, const int32_t *group_rows,
                const int32_t *prefix_lens, int n_groups, Plan *pl, F each)
{
    if (!group_rows || !prefix_lens || n_groups < 1)
        return HB_EINVAL;
    long long rows = 0;
    int deepest = 0;
    for (int i = 0; i < n_groups; ++i) {
        if (group_rows[i] < 1 || prefix_lens[i] < 0)
            return HB_EINVAL;
        if (prefix_lens[i] > max_ctx + 1)
            return HB_ERANGE;
        rows += group_rows[i];
        deepest = prefix_lens[i] > deepest ? prefix_lens[i] : deepest;
    }
    if (rows != n_rows)
        return HB_EINVAL;
    const int g = n_heads / n_kv;
    // a copy's row coordinate is 32 bits wide, a group's queries are counted in as many
    bool can = (long long)num_blocks * n_kv * 16 <= 0x7fffffffll && (long long)n_rows * g <= 0x7fffffffll;
    // the reads saved have to pay for a second kernel and a join
    long long saved = 0;
    for (int i = 0; i < n_groups; ++i)
        saved += saved_bytes(group_rows[i], prefix_lens[i], n_kv, d);
    can = can && saved >= SHARE_BYTES;
    // the smallest load of a CTA for which all run at once, or else the whole of a prefix
    auto total = [&](long long most) {
        long long n = 0;
        for (int i = 0; i < n_groups; ++i) {
            Group gr = shared_group(0, group_rows[i], prefix_lens[i], n_kv, d, can);
            n += cut_group(&gr, g, n_kv, most);
        }
        return n;
    };
    long long lo = 0, hi = 4ll * (MAX_KEYS / 64 + 1);
    const long long least = total(hi);
    if (least > 0 && least <= SMS)
        while (hi - lo > 1) {  // total(hi) fits
            const long long mid = (lo + hi) / 2;
            if (total(mid) <= SMS)
                hi = mid;
            else
                lo = mid;
        }
    // The rows' own keys run beside: a prefix's CTA has an even share of all the
    // work at least, in units of a third of a sub-tile's time (0.27 us)
    long long units = 0;
    int own_unit = OWN_UNIT;
    int own = max_ctx + 1;  // of a row, by the longest prefix: the others' own keys may be far fewer than max_ctx allows
    for (int i = 0; i < n_groups; ++i) {
        const Group gr = shared_group(0, group_rows[i], prefix_lens[i], n_kv, d, can);
        own = max_ctx + 1 - gr.shared < own ? max_ctx + 1 - gr.shared : own;
        if (gr.shared > 0 && (long long)gr.rows * g > 128)
            own_unit = OWN_UNIT_BESIDE;
    }
    for (int i = 0; i < n_groups; ++i) {
        const Group gr = shared_group(0, group_rows[i], prefix_lens[i], n_kv, d, can);
        const long long cols = (long long)gr.rows * g;
        units += (cols + 255) / 256 * n_kv * ((gr.shared + 63) / 64) * (cols > 128 ? 4 : 3);
        units += (long long)gr.rows * n_kv * (own / 16 + 1) * (64 * d) / own_unit;
    }
    hi = hi > units / SMS ? hi : units / SMS;
    long long ctas = 0;
    int row = 0, parts = 0, most = 0, longest = 0;  // own keys of a row at most, and as the prefixes tell
    long long sum = 0;
    for (int i = 0; i < n_groups; ++i) {
        Group gr = shared_group(row, group_rows[i], prefix_lens[i], n_kv, d, can);
        const long long n = cut_group(&gr, g, n_kv, hi);
        if (ctas + n > 0x7fffffffll)
            return HB_ERANGE;
        gr.cta0 = (int)ctas;
        ctas += n;
        parts = gr.parts > parts ? gr.parts : parts;
        most = max_ctx + 1 - gr.shared > most ? max_ctx + 1 - gr.shared : most;
        const int mine = gr.prefix - gr.shared + max_ctx + 1 - deepest;
        longest = mine > longest ? mine : longest;
        sum += (long long)gr.rows * mine;
        row += gr.rows;
        each(i, gr);
    }
    pl->ctas = (int)ctas;
    pl->nt = g > 8 ? 2 : 1;
    pl->col_tiles = tiles_of(g, pl->nt);
    plan_splits(n_rows, (long long)n_kv * pl->col_tiles, most, longest, sum, pl->nt, &pl->split_len, &pl->n_splits);
    pl->balance = false;  // unless the prefixes tell that some rows are longer
    if (ctas == 0 && pl->n_splits > 1 && sum == (long long)n_rows * most)
        balance(n_rows, (long long)n_kv * pl->col_tiles, most, pl);
    pl->first_slot = parts;
    pl->n_slots = pl->first_slot + pl->n_splits;
    pl->seq_parts = pl->seq_part_len = 0;
    pl->direct = pl->n_slots == 1;
    pl->fused = false;
    pl->at = layout(n_rows, n_heads, d, pl->n_slots, !pl->direct, n_groups, false, false, max_ctx);
    return HB_OK;
}

int plan_weigh(long long n_seqs, int nq, int n_heads, int n_kv, int d, int num_blocks, int max_ctx, Plan *pl)
{
    const int g = n_heads / n_kv;
    const long long cols = (long long)nq * g;
    if (cols > 1 << 24)
        return HB_ERANGE;
    pl->nt = cols > 8 ? 2 : 1;
    pl->col_tiles = tiles_of(cols, pl->nt);
    pl->ctas = pl->seq_parts = pl->seq_part_len = pl->first_slot = 0;
    // the keys that all rows of a sequence see go to the tensor cores' kernel
    // where they are read more than once otherwise, or split in any case
    const long long items = n_seqs * n_kv * ((cols + 255) / 256);
    const int subs = (max_ctx + 64) / 64;
    if ((long long)num_blocks * n_kv * 16 <= 0x7fffffffll && subs >= (pl->col_tiles >= WARPS ? COMMON_MIN : COMMON_MIN_FEW) &&
        pl->col_tiles > 1 && items <= 0xffff) {
        long long parts = items < SMS ? SMS / items : 1;
        if (parts > subs / PART_MIN)
            parts = subs / PART_MIN;
        pl->seq_part_len = (int)((subs + parts - 1) / parts);
        pl->seq_parts = (subs + pl->seq_part_len - 1) / pl->seq_part_len;
        pl->ctas = (int)(items * pl->seq_parts);
        pl->first_slot = pl->seq_parts;
    }
    // what is left with them: the last rows' own positions and less than a block
    const int own = pl->ctas > 0 && nq + 15 < max_ctx + 1 ? nq + 15 : max_ctx + 1;
    plan_splits(n_seqs, (long long)n_kv * pl->col_tiles, own, own, n_seqs * own, pl->nt, &pl->split_len, &pl->n_splits);
    pl->balance = false;
    if (pl->ctas == 0 && pl->n_splits > 1)
        balance(n_seqs, (long long)n_kv * pl->col_tiles, own, pl);
    pl->n_slots = pl->first_slot + pl->n_splits;
    pl->direct = pl->n_slots == 1;
    pl->fused = pl->direct && pl->col_tiles == 1;
    pl->at = layout(n_seqs * nq, n_heads, d, pl->n_slots, !pl->direct, 0, true, !pl->fused, max_ctx);
    return HB_OK;
}

void params(Attn *a, const hb_paged_pool *pool, const void *q, long long q_stride, const int32_t *tables, int bt_stride,
            const int32_t *ctx_lens, int n_heads, int max_ctx, int nq, void *out, long long out_stride, const Plan &pl,
            void *workspace)
{
    Attn &p = *a;
    p.k = (const bf16 *)pool->k;
    p.v = (const bf16 *)pool->v;
    p.num_blocks = pool->num_blocks;
    p.n_kv = pool->n_kv_heads;
    p.n_heads = n_heads;
    p.group = n_heads / pool->n_kv_heads;
    p.q = (const bf16 *)q;
    p.q_stride = q_stride;
    p.tables = tables;
    p.bt_stride = bt_stride;
    p.ctx_lens = ctx_lens;
    p.max_ctx = max_ctx;
    p.nq = nq;
    p.c2 = LOG2E / sqrtf((float)pool->head_dim);
    p.split_len = pl.split_len;
    p.n_splits = pl.n_splits;
    p.balance = pl.balance;
    p.col_tiles = pl.col_tiles;
    p.first_slot = pl.first_slot;
    p.n_slots = pl.n_slots;
    p.direct = pl.direct;
    p.fused = pl.fused;
    p.seq_parts = pl.seq_parts;
    p.seq_part_len = pl.seq_part_len;
    p.out = (bf16 *)out;
    p.out_stride = out_stride;
    char *w = work_base(workspace);
    p.part_ml = (float2 *)(w + pl.at.ml);
    p.part_o = (float *)(w + pl.at.o);
    p.scores = (float *)(w + pl.at.scores);
    p.score_stride = pl.at.score_stride;
}

// All warps of a CTA of the join for a row and head where there are few, with many partials.
bool wide_join(const Attn &p, int rows) { return (long long)rows * p.n_heads < 4 * SMS && p.n_slots > 8; }

long long join_blocks(const Attn &p, int rows, int warps)
{
    return ((long long)rows * p.n_heads * warps + JOIN_WARPS - 1) / JOIN_WARPS;
}

template <int D, int W>
int launch_join(const Attn &p, int rows, cudaStream_t s)
{
    return launch_kernel(true, p.balance ? k_paged_join<D, W, true> : k_paged_join<D, W, false>,
                         dim3((unsigned)join_blocks(p, rows, W)), dim3(JOIN_WARPS * 32), 0, s, p, rows) == cudaSuccess
               ? HB_OK
               : HB_ECUDA;
}

int launch_join(const Attn &p, int d, int rows, cudaStream_t s)
{
    if (d == 128)
        return wide_join(p, rows) ? launch_join<128, JOIN_WARPS>(p, rows, s) : launch_join<128, 1>(p, rows, s);
    return wide_join(p, rows) ? launch_join<64, JOIN_WARPS>(p, rows, s) : launch_join<64, 1>(p, rows, s);
}

// Threads for the queries of the same keys: with more than sixteen queries of a kv head eight.
int weigh_shares(int cols) { return cols > 16 ? 8 : 1; }

template <int SHARES, bool JOIN, int D, int W>
int launch_weigh(const Attn &p, int rows, int chunks, cudaStream_t s)
{
    const long long blocks = (long long)p.n_kv * chunks, first = JOIN ? join_blocks(p, rows, W) : 0;
    const dim3 grid = JOIN ? dim3((unsigned)(first + blocks * p.n_seqs)) : dim3((unsigned)blocks, (unsigned)p.n_seqs);
    return launch_kernel(true, k_paged_weigh<SHARES, JOIN, D, W>, grid, dim3(WEIGH_THREADS), 0, s, p, rows,
                         (int)first, chunks) == cudaSuccess
               ? HB_OK
               : HB_ECUDA;
}

template <int D>
int launch_weigh_and_join(const Attn &p, int rows, int chunks, cudaStream_t s)
{
    return wide_join(p, rows) ? launch_weigh<1, true, D, JOIN_WARPS>(p, rows, chunks, s)
                              : launch_weigh<1, true, D, 1>(p, rows, chunks, s);
}

// The rows' results and the weights after the attention, `chunks` CTAs of weights a
// sequence's kv head.
int finish_weigh(const Attn &p, int d, int rows, int chunks, cudaStream_t s)
{
    const int shares = weigh_shares(p.nq * p.group);
    if (p.balance && shares == 1 && (long long)p.n_seqs * p.n_kv * chunks <= JOIN_CTAS)
        return d == 128 ? launch_weigh_and_join<128>(p, rows, chunks, s)
                        : launch_weigh_and_join<64>(p, rows, chunks, s);
    const int rc = p.direct ? HB_OK : launch_join(p, d, rows, s);
    if (rc)
        return rc;
    return shares > 1 ? launch_weigh<8, false, 0, 0>(p, rows, chunks, s) : launch_weigh<1, false, 0, 0>(p, rows, chunks, s);
}

int check_workspace(const void *workspace, long long bytes, long long need)
{
    if (need > 0 && (!workspace || (uintptr_t)workspace % WORK_GIVEN))
        return HB_EINVAL;
    return bytes < need ? HB_ERANGE : HB_OK;
}

int check_heads(int n_heads, int n_kv, int d, int max_ctx)
{
    if (n_heads < 1 || n_kv < 1 || n_heads % n_kv || (d != 64 && d != 128) || max_ctx < 0)
        return HB_EINVAL;
    return max_ctx >= MAX_KEYS || (long long)n_heads * d > 0x7fffffffll ? HB_ERANGE : HB_OK;
}

}  // namespace

namespace paged {

int check_pool(const hb_paged_pool *p)
{
    if (!p || !p->k || !p->v || (uintptr_t)p->k % 16 || (uintptr_t)p->v % 16 || p->num_blocks < 1 ||
        p->num_blocks >= MAX_KEYS || p->n_kv_heads < 1 || (p->head_dim != 64 && p->head_dim != 128))
        return HB_EINVAL;
    return HB_OK;
}

int check_weight_pool(const hb_weight_pool *p)
{
    return !p || !p->data || (uintptr_t)p->data % 16 || p->num_blocks < 1 || p->num_blocks >= MAX_KEYS ||
                   p->n_kv_heads < 1
               ? HB_EINVAL
               : HB_OK;
}

}  // namespace paged
}  // namespace hb

using namespace hb;
using namespace hb::paged;

extern "C" long long hb_decode_shared_workspace(int n_rows, int n_heads, int n_kv_heads, int head_dim, int max_ctx,
                                                const int32_t *group_rows, const int32_t *prefix_lens, int n_groups)
{
    if (n_rows < 0 || n_groups < 0 || (n_rows == 0) != (n_groups == 0))
        return HB_EINVAL;
    const int rc = check_heads(n_heads, n_kv_heads, head_dim, max_ctx);
    if (rc)
        return rc;
    if (n_rows == 0)
        return 0;
    if (n_rows > 65535 || (long long)n_rows * n_heads > 0x7fffffffll)
        return HB_ERANGE;
    Plan pl;
    auto none = [](int, const Group &) {};
    // with shared prefixes, and without as for a pool too large for them
    const int rp = plan_shared(n_rows, n_heads, n_kv_heads, head_dim, 1, max_ctx, group_rows, prefix_lens, n_groups,
                               &pl, none);
    if (rp)
        return rp;
    const long long bytes = pl.at.bytes;
    plan_shared(n_rows, n_heads, n_kv_heads, head_dim, MAX_KEYS, max_ctx, group_rows, prefix_lens, n_groups, &pl, none);
    return pl.at.bytes > bytes ? pl.at.bytes : bytes;
}

extern "C" int hb_decode_shared(const hb_paged_pool *pool, const void *q, long long q_stride,
                                const int32_t *block_tables, int bt_stride, const int32_t *ctx_lens, int n_rows,
                                int n_heads, int max_ctx, const int32_t *group_rows, const int32_t *prefix_lens,
                                int n_groups, void *out, long long out_stride, void *workspace,
                                long long workspace_bytes, void *cuda_stream)
try {
    if (n_rows < 0 || n_groups < 0 || (n_rows == 0) != (n_groups == 0))
        return HB_EINVAL;
    if (n_rows == 0)
        return check_pool(pool);
    int rc = check_attention(pool, q, q_stride, block_tables, bt_stride, ctx_lens, n_rows, n_heads, max_ctx, out,
                             out_stride);
    if (rc)
        return rc;
    Plan pl;
    Attn p = {};
    rc = plan_shared(n_rows, n_heads, pool->n_kv_heads, pool->head_dim, pool->num_blocks, max_ctx, group_rows,
                     prefix_lens, n_groups, &pl, [&](int i, const Group &g) {
                         if (n_groups <= INLINE_GROUPS)
                             p.few[i] = g;
                     });
    if (rc || (rc = check_workspace(workspace, workspace_bytes, pl.at.bytes)))
        return rc;
    cudaStream_t s = (cudaStream_t)cuda_stream;
    params(&p, pool, q, q_stride, block_tables, bt_stride, ctx_lens, n_heads, max_ctx, 1, out, out_stride, pl, workspace);
    p.n_seqs = n_rows;
    p.n_groups = n_groups;
    if (n_groups > INLINE_GROUPS) {  // the groups go ahead into the workspace
        Group *list = (Group *)(work_base(workspace) + pl.at.groups);
        bool sent = true;
        plan_shared(n_rows, n_heads, pool->n_kv_heads, pool->head_dim, pool->num_blocks, max_ctx, group_rows, prefix_lens,
                    n_groups, &pl, [&](int i, const Group &g) {
                        const int at = i % INLINE_GROUPS;
                        p.few[at] = g;
                        if (at == INLINE_GROUPS - 1 || i == n_groups - 1)
                            sent = sent && launch_kernel(true, k_paged_groups, dim3(1), dim3(32), 0, s, list, p, i - at,
                                                         at + 1) == cudaSuccess;
                    });
        if (!sent)
            return HB_ECUDA;
        p.groups = list;
    }
    if (pl.ctas > 0) {
        p.lose = test_lose;
        test_lose = false;
        if ((rc = launch_prefix(pool, p, pl.ctas, s)))
            return rc;
        p.beside = true;
    }
    rc = attention<false>(p, pool->head_dim, pl.nt, n_rows, s);
    return rc || pl.direct ? rc : launch_join(p, pool->head_dim, n_rows, s);
} catch (...) {
    return HB_ENOMEM;
}

extern "C" long long hb_decode_weigh_workspace(int n_seqs, int n_queries, int n_heads, int n_kv_heads, int head_dim,
                                               int max_ctx)
{
    if (n_seqs < 0 || n_queries < 1)
        return HB_EINVAL;
    const int rc = check_heads(n_heads, n_kv_heads, head_dim, max_ctx);
    if (rc)
        return rc;
    if (n_queries > 1024 || (long long)n_seqs * n_queries > 65535 ||
        (long long)n_seqs * n_queries * n_heads > 0x7fffffffll)
        return HB_ERANGE;
    if (n_seqs == 0)
        return 0;
    Plan pl;
    // with common keys, and without as for a pool too large for them
    const int rp = plan_weigh(n_seqs, n_queries, n_heads, n_kv_heads, head_dim, 1, max_ctx, &pl);
    if (rp)
        return rp;
    const long long bytes = pl.at.bytes;
    plan_weigh(n_seqs, n_queries, n_heads, n_kv_heads, head_dim, MAX_KEYS, max_ctx, &pl);
    return pl.at.bytes > bytes ? pl.at.bytes : bytes;
}

extern "C" int hb_decode_weigh(const hb_paged_pool *pool, const void *q, long long q_stride,
                               const int32_t *block_tables, int bt_stride, const int32_t *ctx_lens, int n_seqs,
                               int n_queries, int n_heads, int max_ctx, const hb_weight_pool *weights,
                               const int32_t *weight_tables, int wt_stride, float decay, void *out,
                               long long out_stride, void *workspace, long long workspace_bytes, void *cuda_stream)
try {
    if (n_seqs < 0 || n_queries < 1 || !(decay >= 0.f && decay <= 1.f))
        return HB_EINVAL;
    int rc = check_pool(pool);
    if (rc || (rc = check_weight_pool(weights)))
        return rc;
    if (weights->n_kv_heads != pool->n_kv_heads)
        return HB_EINVAL;
    if (n_queries > 1024)
        return HB_ERANGE;
    if (n_seqs == 0)
        return HB_OK;
    if ((long long)n_seqs * n_queries > 65535)
        return HB_ERANGE;
    const int rows = n_seqs * n_queries;
    rc = check_attention(pool, q, q_stride, block_tables, bt_stride, ctx_lens, rows, n_heads, max_ctx, out, out_stride);
    if (rc)
        return rc;
    if (!weight_tables || (uintptr_t)weight_tables % 4)
        return HB_EINVAL;
    if (wt_stride < max_ctx / 16 + 1)
        return HB_ERANGE;
    Plan pl;
    if ((rc = plan_weigh(n_seqs, n_queries, n_heads, pool->n_kv_heads, pool->head_dim, pool->num_blocks, max_ctx, &pl)) ||
        (rc = check_workspace(workspace, workspace_bytes, pl.at.bytes)))
        return rc;
    cudaStream_t s = (cudaStream_t)cuda_stream;
    Attn p = {};
    params(&p, pool, q, q_stride, block_tables, bt_stride, ctx_lens, n_heads, max_ctx, n_queries, out, out_stride, pl,
           workspace);
    p.n_seqs = n_seqs;
    p.weigh = Weigh{weights->data, weights->num_blocks, weight_tables, wt_stride, decay};
    const int chunks = max_ctx / (WEIGH_THREADS / weigh_shares(n_queries * p.group) * 4) + 1;
    if ((long long)p.n_kv * chunks > 0x7fffffffll)
        return HB_ERANGE;
    if (!pl.fused)
        p.final_ml = (float2 *)(work_base(workspace) + pl.at.final_ml);
    if (pl.ctas > 0) {
        p.lose = test_lose;
        test_lose = false;
        if ((rc = launch_prefix(pool, p, pl.ctas, s)))
            return rc;
        p.beside = true;
    }
    if ((rc = attention<true>(p, pool->head_dim, pl.nt, n_seqs, s)) || pl.fused)
        return rc;
    return finish_weigh(p, pool->head_dim, rows, chunks, s);
} catch (...) {
    return HB_ENOMEM;
}

extern "C" void hb_paged_test_lost_block(void) { test_lose = true; }
