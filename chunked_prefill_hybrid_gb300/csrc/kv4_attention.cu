// kv4_attention.cu -- attention over the 4-bit paged cache: decode rows and
// prefill chunks (include/hb_cache.h).
//
//   s_j = q . k_j / sqrt(d),  p_j = exp(s_j - m),  o = sum p_j v_j / sum p_j
//
// over the keys a query sees, in one pass with the running maximum m and sum
// of the softmax; rows with many keys are split over CTAs and joined by a
// second kernel.
//
// A warp takes 16 keys at a time and up to eight queries that share a kv head
// as the columns of m16n8k16 MMAs (f16 in, fp32 sums): S^T = K q, then
// O^T += V^T P.  A code times its block's scale has at most six significant
// bits, so it is exact in f16; q is brought to [1, 2) by a power of two per
// query, where f16 holds all eight bits of a component down to 2^-17 of the
// largest; a smaller one is rounded to a multiple of 2^-24 of the power.
#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "hb_cache.h"
#include "kv4.cuh"
#include "kv4_chunk.h"
#include "kv4_host.h"
#include "tc_ptx.cuh"

namespace hb {
namespace {

using namespace kv4;
using namespace tc;

constexpr int WARPS = 4;
constexpr int RING = 4;               // pages a warp has in flight
constexpr int JOIN_WARPS = 8;
constexpr int SMS = 152;
constexpr uint64_t WAIT_NS = 2000000000ull;
constexpr int SPLIT_MIN = 256;        // keys of a split at least
constexpr int MAX_KEYS = 1 << 27;
constexpr int MAX_COLS = 1 << 24;     // queries of a kv head in a chunk

struct Kv4Attn {
    const uint8_t *pool;
    int num_blocks, n_kv, group;      // group: query heads of a kv head
    float ks, vs;
    const bf16 *q;
    long long q_stride;
    const int *tables;
    int bt_stride;
    const int *ctx_lens;              // decode only
    int max_ctx;
    int chunk_offset, chunk_len;      // chunk only (chunk_len 0: decode)
    int n_heads;
    int col_groups;                   // CTAs of eight queries for a kv head
    int split_len, n_splits;
    bf16 *out;
    long long out_stride;
    float2 *part_ml;                  // [row][head][split] (m in log2, l)
    float *part_o;                    // [row][head][split][D]
    bool lose;                        // the first CTA leaves out the copy of its first page (hb_kv4_test_lost_page)
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t x)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// All ones in the bytes of the first n of four tokens.
__device__ __forceinline__ uint32_t first_bytes(int n)
{
    return n >= 4 ? 0xffffffffu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
}

// Row, head and visible keys of query column c of kv head kvh.
struct Col {
    int row, head, nkeys;
};
__device__ __forceinline__ Col column(const Kv4Attn &p, int seq, int kvh, int c)
{
    Col r;
    const int i = c / p.group;
    r.head = kvh * p.group + (c - i * p.group);
    r.row = p.chunk_len > 0 ? i : seq;
    r.nkeys = p.chunk_len > 0 ? p.chunk_offset + i + 1 : p.ctx_lens[seq] + 1;
    return r;
}

// A fragments of V^T for channel blocks 4w..4w+3: the bytes of two tokens
// (channels 2g, 2g + 1) become bytes of two channels, and those f16 pairs of
// tokens.  a[0], a[1]: the first two tokens of rows g and g + 8, a[2], a[3] the
// other two.
template <int KW>
__device__ __forceinline__ void pair_tokens(const uint32_t (&vw)[2][KW], int w, uint32_t (&a)[4][4])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t x = vw[h][w], y = vw[h][KW / 2 + w];
        from_e2m1x8((x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u), a[2 * h]);
        from_e2m1x8(((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u), a[2 * h + 1]);
    }
}

// Shared memory of a CTA: a ring of RING pages for each warp, and after the
// key loop (in the same place) the warps' results.
template <int D, int W>
struct Smem {
    static constexpr int RINGS = W * RING * Layout<D>::BYTES;
    static constexpr int ROW = D + 4;  // floats of a result row, off the banks of the next
    static constexpr int JOIN = W * 8 * ROW * 4;
    static constexpr int BYTES = (RINGS > JOIN ? RINGS : JOIN);
};

// A warp reads pages of its own through a ring of bulk copies, four under way,
// and works on two at a time; the W warps of a CTA join their results in shared
// memory.  128 rows of 128 to 2048 keys, 40 heads of 128, take 97 us (5.3 TB/s,
// 0.79 of the copy rate); 18 rows of 1024 keys 23.4 us; one row of 130999 keys,
// 8 kv heads of 8, 35.9 us with the join.  Bound by the issue of conversions (two
// thirds of the slots) and, where there is one wave of CTAs, by their start.
//
// FEW: one query (d = 128) or two (d = 64) share the kv head.  The eight
// columns are then the (query, scale block) pairs: column (c, i) holds query
// c's block i and zeros elsewhere, so the MMAs give the scores block by block
// and each is scaled once in fp32 instead of each code's value; and in V^T P
// column (c, i) holds P times the scales of block i, for channel block i's MMA
// alone (zeros for the others'), so that one accumulator of four registers
// takes every channel: 128 rows as above take 197 us with a multiplied K and V
// and one page at a time, 97 so.  A small weight times a small scale would
// leave f16's range, so the scales of a column are brought near 1 by a power of
// two, and the accumulator back at the end: 3% of the time of 128 rows.  What a
// key adds is lost only where its weight times its V scale is below 2^-34 of the
// largest weight times the largest scale.
//
// Else the scales multiply V's codes, which is exact, and P is all that a
// column holds: one power of two for each of eight blocks and eight queries
// would cost as much.
//
// Six CTAs an SM of four warps need at most 80 registers, which the compiler
// passes by four unless it is told: 133 us in place of 132.
template <int D, bool FEW, int W>
__global__ void __launch_bounds__(W * 32, (FEW ? (D == 128 && W == WARPS ? 6 : 5) : 4) * WARPS / W)
    k_kv4_attention(const Kv4Attn p)
{
    using L = Layout<D>;
    constexpr int NB = L::NB, KW = NB / 2;  // words of a lane's 8- or 16-byte load
    constexpr int COLS = FEW ? 8 / NB : 8;  // queries of a CTA
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[W][RING];
    __shared__ float s_scale[8], s_m[W][8], s_l[W][8];

    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int g = lane >> 2, t = lane & 3;
    const int split = blockIdx.x % p.n_splits;
    const int rest = blockIdx.x / p.n_splits;
    const int cg = rest % p.col_groups, kvh = rest / p.col_groups;
    const int seq = blockIdx.y;
    const int ncols = p.chunk_len > 0 ? p.chunk_len * p.group : p.group;
    const int c0 = cg * COLS, c1 = min(c0 + COLS, ncols);  // this CTA's queries

    if (lane == 0) {
        for (int i = 0; i < RING; ++i)
            mbar_init(&full[warp][i], 1);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();
    // this warp's pages: b0 + 4 i, i < n_tiles, through its ring.  The first
    // ids are fetched before it is known how many are needed (a table row has
    // bt_stride of them): the context's length comes in the same time.
    const int k0 = split * p.split_len, b0 = (k0 >> 4) + warp;
    const int *tab = p.tables + (size_t)seq * p.bt_stride + b0;
    int ids = b0 + lane * W < p.bt_stride ? __ldg(tab + lane * W) : 0;  // lane i: page of tile i of the current 32
    if (p.chunk_len == 0) {
        const int ctx = p.ctx_lens[seq];
        if (ctx < 0 || ctx > p.max_ctx) {  // padding: zeros; outside what the grid was sized for: NaN
            if (split == 0)
                for (int c = c0; c < c1; ++c) {
                    const Col co = column(p, seq, kvh, c);
                    for (int e = threadIdx.x; e < D; e += W * 32)
                        p.out[co.row * p.out_stride + (size_t)co.head * D + e] =
                            f2bf(ctx == -1 ? 0.f : __int_as_float(0x7fc00000));
                }
            return;
        }
    }
    const int nkeys = column(p, seq, kvh, c1 - 1).nkeys;  // the most any query sees
    const int k1 = min(nkeys, k0 + p.split_len);
    if (k0 >= k1)
        return;
    const int fewest = column(p, seq, kvh, c0).nkeys;  // keys that every query sees

    const int n_tiles = max(0, (((k1 + 15) >> 4) - b0 + W - 1) / W);
    uint8_t *ring = smem + warp * RING * L::BYTES;
    bool bad = false;
    const uint8_t *head = p.pool + (size_t)kvh * L::BYTES;
    // copy pages tile..tile + N - 1 (tile a multiple of N), lane i the i-th
    auto issue = [&](int tile, auto n) {
        constexpr int N = decltype(n)::value;
        if (tile >= n_tiles)
            return;
        if ((tile & 31) == 0 && tile > 0)
            ids = tile + lane < n_tiles ? __ldg(tab + (tile + lane) * W) : 0;
        const int mine = tile + (lane & (N - 1));
        const int blk = __shfl_sync(0xffffffffu, ids, mine & 31);
        const bool ok = blk >= 0 && blk < p.num_blocks;
        const bool lose = N == RING && p.lose && blockIdx.x + blockIdx.y + threadIdx.x == 0;
        if (lane < N && mine < n_tiles && !lose) {
            bad |= !ok;
            uint64_t *bar = &full[warp][mine % RING];
            if (ok) {
                mbar_expect_tx(bar, L::BYTES);
                bulk_load(ring + mine % RING * L::BYTES, head + (size_t)blk * (p.n_kv * L::BYTES), L::BYTES, bar);
            } else {
                mbar_arrive(bar);  // nothing is read there; what the slot holds is not used
            }
        }
    };
    __syncwarp();
    issue(0, std::integral_constant<int, RING>());

    // ---- q as B fragments, and what its scores are scaled by
    uint32_t qf[NB][2];
    {
        const int qi = FEW ? g / NB : g;
        const bool have = c0 + qi < c1;
        const Col co = column(p, seq, kvh, have ? c0 + qi : c0);
        const bf16 *qr = p.q + co.row * p.q_stride + (size_t)co.head * D;
        float x[NB][4];
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const uint2 u = *reinterpret_cast<const uint2 *>(qr + 16 * i + 4 * t);
            const float2 f0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x));
            const float2 f1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y));
            x[i][0] = f0.x, x[i][1] = f0.y, x[i][2] = f1.x, x[i][3] = f1.y;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                a = fmaxf(a, fabsf(x[i][j]));
        }
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
        const int e = query_exponent(a);
        const float down = pow2(-e);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const bool put = have && (!FEW || g % NB == i);
            qf[i][0] = put ? pack_h2(x[i][0] * down, x[i][1] * down) : 0u;
            qf[i][1] = put ? pack_h2(x[i][2] * down, x[i][3] * down) : 0u;
        }
        if (warp == 0 && t == 0)
            s_scale[g] = fminf(p.ks * (rsqrtf((float)D) * LOG2E) * pow2(e), LARGEST_SCALE);
    }
    __syncthreads();

    // Running reference of the softmax (log2).  It moves only when a score
    // passes it by LIFT + RAISE: P stays at 2^15 or below, and a tile costs one
    // vote instead of a maximum over its lanes.  Scores may be so large that
    // their last place is worth more than that: the sum that they are compared
    // with is rounded down, the new reference up, and the products that are
    // compared are those that the exponent is taken of.
    constexpr int Q = FEW ? 1 : 2;  // queries this lane keeps: its own column's, or columns 2t and 2t + 1
    const int myq = FEW ? (2 * t) / NB : 2 * t;
    float sc[Q], m[Q], l[Q];
    int seen[Q];
#pragma unroll
    for (int j = 0; j < Q; ++j) {
        sc[j] = s_scale[FEW ? myq * NB : myq + j];
        seen[j] = column(p, seq, kvh, min(c0 + myq + j, c1 - 1)).nkeys;
        m[j] = LOWEST;
        l[j] = 0.f;
    }
    constexpr int OT = FEW ? 2 : NB;  // accumulators: one for each page in hand, or for each channel block
    float o[OT][4];
#pragma unroll
    for (int i = 0; i < OT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[i][j] = 0.f;

    const int tok0 = 4 * (g >> 1) + (g & 1);  // tokens tok0 and tok0 + 2 are rows g and g + 8 of S^T
    // Keys that the query of column g sees.  A slot that it does not see may
    // hold anything, a NaN scale among it, and is kept out of V by its place;
    // a weight of 0 does not say so, as those of keys that are seen may vanish.
    const int seen_g = FEW ? min(column(p, seq, kvh, min(c0 + g / NB, c1 - 1)).nkeys, k1) : 0;
    // a page that did not come: the rows get NaN, and no copy may land after
    // the CTA has ended
    auto lost = [&](int i) {
        bad = true;
        for (int j = i; j < min(i + RING, n_tiles); ++j)
            mbar_wait(&full[warp][j % RING], (uint32_t)(j / RING) & 1u, nullptr, WAIT_NS / 8);
    };
    // tile i, or tiles i and i + 1: some lanes look at one, some at the other
    auto arrived = [&](int i, bool two) {
        const int mine = i + (two ? lane & 1 : 0);
        return __all_sync(0xffffffffu,
                          mbar_sleep(&full[warp][mine % RING], (uint32_t)(mine / RING) & 1u, nullptr));
    };
    if constexpr (FEW) {
        // two pages at a time: the four lanes of a quad hold the parts of four
        // tokens' scores and end up with one token each (d = 128)
        const int lim = min(seen[0], k1);
        const bool b0_ = t & 1, b1_ = t & 2;
        const int my_x = D == 128 ? t >> 1 : t & 1;  // page whose tokens this lane keeps
        uint32_t only[NB];                           // 1 for a column of block i, 0 for the others
#pragma unroll
        for (int i = 0; i < NB; ++i)
            only[i] = g % NB == i ? 0x3c003c00u : 0u;
        // 2^lift_e that column g's V scales are multiplied by, as an f16 pair;
        // and what carries a byte of a scale past 0x7f if it makes 2 or more.
        // It moves to bring the largest to [1/4, 1/2): with [1, 2) pages whose
        // scales grow a little cost 132 us in place of 129.
        uint32_t lift = 0x58005800u, over = 0x78787878u;  // 2^7: the smallest scale is 2^-9
        auto lift_e = [&]() { return (int)(lift >> 26) - 15; };
        for (int i = 0; i < n_tiles; i += 2) {
            if (!arrived(i, i + 1 < n_tiles)) {
                lost(i);
                break;
            }
            const uint8_t *page = ring + (i % RING) * L::BYTES;
            // ---- S^T = K q, a scale block a column
            float part[2][2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint8_t *pg = page + x * L::BYTES;  // past the last page: whatever the slot holds, masked below
                uint32_t kw[2][KW], ks[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    load_words<KW>(pg + L::k_code(tok0 + 2 * r, t, 0), kw[r]);
                    ks[r] = *reinterpret_cast<const uint16_t *>(pg + L::k_scale(tok0 + 2 * r, (2 * t) % NB));
                }
                float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < KW; ++w) {
                    uint32_t a[2][4];
                    from_e2m1x8(kw[0][w], a[0]);
                    from_e2m1x8(kw[1][w], a[1]);
                    mma_f16(s, a[0][0], a[1][0], a[0][1], a[1][1], qf[2 * w][0], qf[2 * w][1]);
                    mma_f16(s, a[0][2], a[1][2], a[0][3], a[1][3], qf[2 * w + 1][0], qf[2 * w + 1][1]);
                }
                const float2 f0 = h2f2(from_e4m3x2(ks[0])), f1 = h2f2(from_e4m3x2(ks[1]));
                part[x][0] = s[0] * f0.x + s[1] * f0.y;
                part[x][1] = s[2] * f1.x + s[3] * f1.y;
            }
            // ---- sum over the blocks of a query: reduce-scatter over its lanes
            constexpr int M = D == 128 ? 1 : 2;  // tokens this lane ends up with
            float s[M];
            {
                const bool b = my_x != 0;
                float keep[2], send[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    keep[r] = b ? part[1][r] : part[0][r];
                    send[r] = b ? part[0][r] : part[1][r];
                    keep[r] += __shfl_xor_sync(0xffffffffu, send[r], D == 128 ? 2 : 1);
                }
                if constexpr (D == 128) {
                    s[0] = (b0_ ? keep[1] : keep[0]) + __shfl_xor_sync(0xffffffffu, b0_ ? keep[0] : keep[1], 1);
                } else {
                    s[0] = keep[0];
                    s[1] = keep[1];
                }
            }
            // ---- softmax
            const int base = (b0 + (i + my_x) * W) * 16;
            const bool edge = (b0 + (i + 1) * W) * 16 + 16 > min(fewest, k1);
            uint32_t vs[2];
            bool raise = false;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                vs[x] = *reinterpret_cast<const uint32_t *>(page + x * L::BYTES + L::v_scale(4 * t, g % NB));
                if (edge)
                    vs[x] &= first_bytes(seen_g - (b0 + (i + x) * W) * 16 - 4 * t);
                raise |= (((vs[x] & 0x7f7f7f7fu) + over) & 0x80808080u) != 0;
            }
#pragma unroll
            for (int j = 0; j < M; ++j) {
                s[j] = __fmul_rn(s[j], sc[0]);
                if (edge)
                    s[j] = base + tok0 + 2 * (D == 128 ? (int)b0_ : j) < lim ? s[j] : -INFINITY;
                raise |= s[j] > __fadd_rd(m[0], LIFT + RAISE);
            }
            if (__any_sync(0xffffffffu, raise)) {
                float mx = M == 2 ? fmaxf(s[0], s[M - 1]) : s[0];
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                if (D == 128)
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                const float mn = fmaxf(m[0], __fadd_ru(mx, -LIFT)), corr = ex2(m[0] - mn);
                m[0] = mn;
                l[0] *= corr;
                uint32_t top = 0;  // the largest V scale of column g
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t b = vs[j / 4] >> (8 * (j & 3)) & 0x7fu;
                    top = b == 0x7fu ? top : max(top, b);
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = top >= 8 ? 5 - (int)(top >> 3) : top > 0 ? 7 - (31 - __clz(top)) : 7;
                const int had = lift_e(), now = min(had, e);
                lift = (uint32_t)(now + 15) * 0x04000400u;
                over = (uint32_t)max(64 + 8 * now, 0) * 0x01010101u;  // 0x80 less the code of 2^(1 - now)
                const float down = pow2(now - had);
                const float f[2] = {__shfl_sync(0xffffffffu, down, 8 * t), __shfl_sync(0xffffffffu, down, 8 * t + 4)};
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        o[x][j] *= corr * f[j & 1];
            }
#pragma unroll
            for (int j = 0; j < M; ++j) {
                s[j] = ex2(s[j] - m[0]);
                l[0] += s[j];
            }
            // ---- every lane gets the weights of both pages' rows g and g + 8
            uint32_t pr[2];
            if constexpr (D == 128) {
                const uint32_t own = pack_h2(s[0], s[0]);
                const uint32_t pair = __byte_perm(own, __shfl_xor_sync(0xffffffffu, own, 1), b0_ ? 0x3254 : 0x7610);
                const uint32_t far = __shfl_xor_sync(0xffffffffu, pair, 2);
                pr[0] = b1_ ? far : pair;
                pr[1] = b1_ ? pair : far;
            } else {
                const uint32_t own = pack_h2(s[0], s[M - 1]);
                const uint32_t far = __shfl_xor_sync(0xffffffffu, own, 1);
                pr[0] = b0_ ? far : own;
                pr[1] = b0_ ? own : far;
            }
            // ---- O^T += V^T P, P times the scales of a column's block
            uint32_t vw[2][2][KW], pb[2][2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint8_t *pg = page + x * L::BYTES;
                load_words<KW>(pg + L::v_code(4 * t, g, 0), vw[x][0]);
                load_words<KW>(pg + L::v_code(4 * t + 2, g, 0), vw[x][1]);
                const uint32_t p0 = movmatrix(__byte_perm(pr[x], 0, 0x1010));  // tokens 4t, 4t + 1
                const uint32_t p1 = movmatrix(__byte_perm(pr[x], 0, 0x3232));  // tokens 4t + 2, 4t + 3
                pb[x][0] = hmul2(p0, hmul2(from_e4m3x2(vs[x] & 0xffffu), lift));
                pb[x][1] = hmul2(p1, hmul2(from_e4m3x2(vs[x] >> 16), lift));
            }
            __syncwarp();  // the slots are read
            issue(i + RING, std::integral_constant<int, 2>());
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int w = 0; w < KW / 2; ++w) {
                    uint32_t a[4][4];
                    pair_tokens<KW>(vw[x], w, a);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_f16(o[x], a[0][j], a[1][j], a[2][j], a[3][j], hmul2(pb[x][0], only[4 * w + j]),
                                hmul2(pb[x][1], only[4 * w + j]));
                }
        }
        const float down = pow2(-lift_e());
        const float f[2] = {__shfl_sync(0xffffffffu, down, 8 * t), __shfl_sync(0xffffffffu, down, 8 * t + 4)};
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[x][j] *= f[j & 1];
    } else {
        // Slots that some queries see and others do not (a chunk's rows): a NaN
        // scale among them is taken out and put into the sums of those that do.
        auto hidden_nans = [&](uint32_t(&vst)[NB], int base) {
            uint32_t any = 0;
#pragma unroll
            for (int w = 0; w < NB; ++w)
                any |= (vst[w] & 0x7f7f7f7fu) + 0x01010101u;
            if (!__any_sync(0xffffffffu, (any & 0x80808080u) != 0))
                return;
#pragma unroll
            for (int w = 0; w < NB; ++w) {
                const uint32_t nan = ((vst[w] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                vst[w] &= ~((nan >> 7) * 0xffu);
                int first = nan ? base + (__ffs(nan) - 1) / 8 : MAX_KEYS;
                first = min(first, __shfl_xor_sync(0xffffffffu, first, 1));
                first = min(first, __shfl_xor_sync(0xffffffffu, first, 2));
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (first < seen[j])
                        o[w][j] = o[w][2 + j] = __int_as_float(0x7fc00000);
            }
        };
        // two pages at a time, scaled by their blocks' scales
        for (int i = 0; i < n_tiles; i += 2) {
            if (!arrived(i, i + 1 < n_tiles)) {
                lost(i);
                break;
            }
            const uint8_t *page = ring + (i % RING) * L::BYTES;
            // ---- S^T = K q
            float s[2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint8_t *pg = page + x * L::BYTES;  // past the last page: whatever the slot holds, masked below
                uint32_t kw[2][KW], kst[2][NB / 4];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    load_words<KW>(pg + L::k_code(tok0 + 2 * r, t, 0), kw[r]);
                    if constexpr (NB == 8) {
                        const uint2 u = *reinterpret_cast<const uint2 *>(pg + L::k_scale(tok0 + 2 * r, 0));
                        kst[r][0] = u.x, kst[r][NB / 4 - 1] = u.y;
                    } else {
                        kst[r][0] = *reinterpret_cast<const uint32_t *>(pg + L::k_scale(tok0 + 2 * r, 0));
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[x][j] = 0.f;
#pragma unroll
                for (int w = 0; w < KW; ++w) {
                    uint32_t a[2][4];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        from_e2m1x8(kw[r][w], a[r]);
                        const uint32_t two = from_e4m3x2(kst[r][w / 2] >> (16 * (w & 1)));  // blocks 2w, 2w + 1
                        a[r][0] = mul_lo(a[r][0], two);
                        a[r][1] = mul_lo(a[r][1], two);
                        a[r][2] = mul_hi(a[r][2], two);
                        a[r][3] = mul_hi(a[r][3], two);
                    }
                    mma_f16(s[x], a[0][0], a[1][0], a[0][1], a[1][1], qf[2 * w][0], qf[2 * w][1]);
                    mma_f16(s[x], a[0][2], a[1][2], a[0][3], a[1][3], qf[2 * w + 1][0], qf[2 * w + 1][1]);
                }
            }
            // ---- softmax: rows are tokens, columns queries
            const int key = (b0 + i * W) * 16 + tok0;
            const bool edge = (b0 + (i + 1) * W) * 16 + 16 > min(fewest, k1);
            bool raise = false;
#pragma unroll
            for (int j = 0; j < Q; ++j) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    s[x][j] = __fmul_rn(s[x][j], sc[j]);
                    s[x][2 + j] = __fmul_rn(s[x][2 + j], sc[j]);
                    if (edge) {
                        const int lim = min(seen[j], k1) - key - x * W * 16;
                        s[x][j] = lim > 0 ? s[x][j] : -INFINITY;
                        s[x][2 + j] = lim > 2 ? s[x][2 + j] : -INFINITY;
                    }
                }
                raise |= fmaxf(fmaxf(s[0][j], s[0][2 + j]), fmaxf(s[1][j], s[1][2 + j])) > __fadd_rd(m[j], LIFT + RAISE);
            }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int j = 0; j < Q; ++j) {
                    float mx = fmaxf(fmaxf(s[0][j], s[0][2 + j]), fmaxf(s[1][j], s[1][2 + j]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    const float mn = fmaxf(m[j], __fadd_ru(mx, -LIFT)), corr = ex2(m[j] - mn);
                    m[j] = mn;
                    l[j] *= corr;
#pragma unroll
                    for (int w = 0; w < NB; ++w) {
                        o[w][j] *= corr;
                        o[w][2 + j] *= corr;
                    }
                }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int j = 0; j < Q; ++j) {
                    s[x][j] = ex2(s[x][j] - m[j]);
                    s[x][2 + j] = ex2(s[x][2 + j] - m[j]);
                    l[j] += s[x][j] + s[x][2 + j];
                }
            // ---- O^T += V^T P, V scaled
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint8_t *pg = page + x * L::BYTES;
                uint32_t vw[2][KW], vst[NB];
                load_words<KW>(pg + L::v_code(4 * t, g, 0), vw[0]);
                load_words<KW>(pg + L::v_code(4 * t + 2, g, 0), vw[1]);
#pragma unroll
                for (int w = 0; w < NB; ++w)
                    vst[w] = *reinterpret_cast<const uint32_t *>(pg + L::v_scale(4 * t, w));
                if (x == 1) {
                    __syncwarp();  // the slots are read
                    issue(i + RING, std::integral_constant<int, 2>());
                }
                const uint32_t p0 = movmatrix(pack_h2(s[x][0], s[x][Q - 1]));      // column g, tokens 4t, 4t + 1
                const uint32_t p1 = movmatrix(pack_h2(s[x][2], s[x][2 + Q - 1]));  // tokens 4t + 2, 4t + 3
                if (edge) {
                    const int base = (b0 + (i + x) * W) * 16 + 4 * t;
                    const uint32_t z = first_bytes(k1 - base);
#pragma unroll
                    for (int w = 0; w < NB; ++w)
                        vst[w] &= z;  // slots that no query sees
                    if (fewest < k1)
                        hidden_nans(vst, base);
                }
#pragma unroll
                for (int w = 0; w < KW / 2; ++w) {
                    uint32_t a[4][4];
                    pair_tokens<KW>(vw, w, a);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t s0 = from_e4m3x2(vst[4 * w + j]), s1 = from_e4m3x2(vst[4 * w + j] >> 16);
                        mma_f16(o[4 * w + j], hmul2(a[0][j], s0), hmul2(a[1][j], s0), hmul2(a[2][j], s1),
                                hmul2(a[3][j], s1), p0, p1);
                    }
                }
            }
        }
    }

    // ---- join the warps
    bad = __any_sync(0xffffffffu, bad);
    __syncthreads();  // the rings are done with
    float(*s_o)[8][Smem<D, W>::ROW] = reinterpret_cast<float(*)[8][Smem<D, W>::ROW]>(smem);
#pragma unroll
    for (int j = 0; j < Q; ++j) {
        if (FEW)
            l[j] += __shfl_xor_sync(0xffffffffu, l[j], 1);
        if (FEW && D == 128)
            l[j] += __shfl_xor_sync(0xffffffffu, l[j], 2);
        l[j] += __shfl_xor_sync(0xffffffffu, l[j], 4);
        l[j] += __shfl_xor_sync(0xffffffffu, l[j], 8);
        l[j] += __shfl_xor_sync(0xffffffffu, l[j], 16);
        if (bad) {  // a block id outside the pool poisons every query
            l[j] = __int_as_float(0x7fc00000);
            m[j] = 0.f;
        }
        if (g == 0 && (!FEW || (2 * t) % NB == 0)) {
            s_m[warp][myq + j] = m[j];
            s_l[warp][myq + j] = l[j];
        }
    }
    if constexpr (FEW) {
        // columns 2t and 2t + 1 are two channel blocks of this lane's query
#pragma unroll
        for (int j = 0; j < 2; ++j)
            *reinterpret_cast<float2 *>(&s_o[warp][myq][16 * ((2 * t) % NB + j) + 2 * g]) =
                make_float2(o[0][j] + o[1][j], o[0][2 + j] + o[1][2 + j]);
    } else {
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                *reinterpret_cast<float2 *>(&s_o[warp][2 * t + j][16 * i + 2 * g]) = make_float2(o[i][j], o[i][2 + j]);
    }
    __syncthreads();
    for (int c = c0 + warp; c < c1; c += W) {
        const Col co = column(p, seq, kvh, c);
        float M = LOWEST, lsum = 0.f, f[W];
#pragma unroll
        for (int w = 0; w < W; ++w)
            M = fmaxf(M, s_m[w][c - c0]);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            f[w] = ex2(s_m[w][c - c0] - M);
            lsum += s_l[w][c - c0] * f[w];
        }
        const bool whole = co.nkeys <= p.split_len;  // this split holds every key the query sees
        const float inv = p.vs / lsum;
        const size_t at = ((size_t)co.row * p.n_heads + co.head) * p.n_splits + split;
        if (whole && split > 0)
            continue;
        for (int e = 2 * lane; e < D; e += 64) {
            float v0 = 0.f, v1 = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float2 x = *reinterpret_cast<const float2 *>(&s_o[w][c - c0][e]);
                v0 += x.x * f[w];
                v1 += x.y * f[w];
            }
            if (whole)
                *reinterpret_cast<__nv_bfloat162 *>(p.out + co.row * p.out_stride + (size_t)co.head * D + e) =
                    __floats2bfloat162_rn(v0 * inv, v1 * inv);
            else
                *reinterpret_cast<float2 *>(p.part_o + at * D + e) = make_float2(v0, v1);
        }
        if (!whole && lane == 0)
            p.part_ml[at] = make_float2(M, lsum);
    }
}

// Joins the splits of one (row, head): each warp some of them, eight loads of
// a lane under way at a time, then the warps in order.  Bound by the loads'
// latency: 57 splits of 64 heads (one row of 130999 keys) 1 us less than with
// one load after the other.
template <int D>
__global__ void __launch_bounds__(JOIN_WARPS * 32) k_kv4_join(const Kv4Attn p)
{
    constexpr int E = D / 32, BATCH = 8;
    __shared__ float s_m[JOIN_WARPS], s_l[JOIN_WARPS], s_o[JOIN_WARPS][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int row = blockIdx.x / p.n_heads, head = blockIdx.x - row * p.n_heads;
    const int nkeys = p.chunk_len > 0 ? p.chunk_offset + row + 1 : p.ctx_lens[row] + 1;
    if (nkeys <= p.split_len || (p.chunk_len == 0 && nkeys > p.max_ctx + 1))
        return;  // written by the first kernel
    const int n = (nkeys + p.split_len - 1) / p.split_len;
    const float2 *ml = p.part_ml + (size_t)blockIdx.x * p.n_splits;
    const float *po = p.part_o + (size_t)blockIdx.x * p.n_splits * D + lane * E;
    float M = LOWEST, l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        o[e] = 0.f;
    for (int s0 = warp; s0 < n; s0 += JOIN_WARPS * BATCH) {
        float2 x[BATCH];
        float v[BATCH][E];
        float top = M;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int s = min(s0 + i * JOIN_WARPS, n - 1);
            x[i] = ml[s];
            if constexpr (E == 4)
                *reinterpret_cast<float4 *>(v[i]) = *reinterpret_cast<const float4 *>(po + (size_t)s * D);
            else
                *reinterpret_cast<float2 *>(v[i]) = *reinterpret_cast<const float2 *>(po + (size_t)s * D);
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            top = fmaxf(top, x[i].x);
        const float corr = ex2(M - top);
        M = top;
        l *= corr;
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] *= corr;
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            if (s0 + i * JOIN_WARPS < n) {
                const float f = ex2(x[i].x - M);
                l += x[i].y * f;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    o[e] += v[i][e] * f;
            }
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        s_o[warp][lane * E + e] = o[e];
    if (lane == 0) {
        s_m[warp] = M;
        s_l[warp] = l;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < D; e += JOIN_WARPS * 32) {
        float top = LOWEST, v = 0.f, lsum = 0.f;
#pragma unroll
        for (int w = 0; w < JOIN_WARPS; ++w)
            top = fmaxf(top, s_m[w]);
#pragma unroll
        for (int w = 0; w < JOIN_WARPS; ++w) {
            const float f = ex2(s_m[w] - top);
            v += s_o[w][e] * f;
            lsum += s_l[w] * f;
        }
        p.out[row * p.out_stride + (size_t)head * D + e] = f2bf(v * (p.vs / lsum));
    }
}

struct Split {
    int len, n;
};

// Keys of a split (a multiple of 16 WARPS) and the number of splits: the one
// with the least estimated time.  An SM shares its throughput among its CTAs
// and is taken to need three of them (FULL) to reach it; joining splits counts
// as much as an SM's time for 64 pages of a head (JOIN), however many they are,
// and a CTA's start and end nothing.  So a little better rounding may buy
// hundreds of CTAs: of one row with 8 kv heads of 8, 130999 keys take 36 us in 57
// splits, but 115000 keys 57 us in 360, 132000 46 and 155000 56; with FULL 3.5,
// 4 or 5 it is 115000 keys that take 37, and 130999 that take 50.  Of one row
// (and of a chunk) the keys are known, and CTAs beyond those that an SM holds
// run when others have ended; several rows are mostly shorter than max_ctx, and
// what is left over at the end is not counted (54 rows of 4000 to 8000 keys, 4
// heads: 40.0 us, counted 40.3).
Split plan_split(long long ctas, int resident, int max_keys)
{
    constexpr int UNIT = 16 * WARPS;
    constexpr double FULL = 3, JOIN = 64;
    Split best{0, 1};
    double least = 0;
    const long long most = (max_keys + SPLIT_MIN - 1) / SPLIT_MIN;
    for (long long s = 1; s <= most; s += s < 16 ? 1 : s / 8) {
        const long long len = ((max_keys + s - 1) / s + UNIT - 1) / UNIT * UNIT, n = (max_keys + len - 1) / len;
        const long long per_sm = (ctas * n + SMS - 1) / SMS, last = per_sm % resident;
        const double shares = (double)(per_sm - last) + (last == 0 ? 0 : last > FULL ? last : FULL);
        const double t = shares * (len / 16) + (n > 1 ? JOIN : 0);
        if (best.len == 0 || t < least) {
            best = Split{(int)len, (int)n};
            least = t;
        }
        if (ctas * n > 16ll * SMS)
            break;
    }
    return best;
}

long long workspace_bytes_of(long long rows, int n_heads, int d, int n_splits)
{
    return n_splits > 1 ? rows * n_heads * n_splits * (8 + 4ll * d) : 0;
}

bool dims_ok(int n_heads, int n_kv, int d)
{
    return n_kv >= 1 && n_heads >= 1 && n_heads % n_kv == 0 && n_heads <= 65535 && (d == 64 || d == 128);
}

long long ctas_of(int cols, int n_kv, int seqs) { return (long long)((cols + 7) / 8) * n_kv * seqs; }

thread_local bool test_lose = false;  // of this thread's next attention launch

bool take_lose()
{
    const bool lose = test_lose;
    test_lose = false;
    return lose;
}

// Queries a CTA takes: see k_kv4_attention.
bool few(int cols, int d) { return cols <= (d == 128 ? 1 : 2); }

// CTAs of the attention kernel that an SM holds (registers), for plan_split.
int resident(int rows, int cols, int d) { return rows > 1 ? 1 << 30 : d == 64 ? 5 : few(cols, d) ? 6 : 4; }

template <int D, bool FEW, int W>
cudaError_t launch_w(const Kv4Attn &p, dim3 grid, cudaStream_t s)
{
    // Six CTAs fit an SM.  Where five on each hold the whole grid they lie
    // more evenly with no room for a sixth: 720 CTAs (18 rows of 1024 keys, 40
    // heads) take 23.5 us so and 26.3 with room; 5120 (128 rows of 128 to 2048
    // keys, evenly spread) 131.5 and 129.4.
    constexpr int PAD = FEW && D == 128 && W == WARPS ? 1024 : 0;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = kv4_allow_smem((const void *)k_kv4_attention<D, FEW, W>, Smem<D, W>::BYTES + PAD, done);
    if (e != cudaSuccess)
        return e;
    const int bytes = Smem<D, W>::BYTES + ((long long)grid.x * grid.y <= 5 * SMS ? PAD : 0);
    return launch_kernel(true, k_kv4_attention<D, FEW, W>, grid, dim3(W * 32), bytes, s, p);
}

// Short contexts of more rows than run at once: one warp a CTA, which has no
// others to wait for and to join, and four times as many rows are under way.
// 40 heads: 85 rows of 5 keys 7.3 us against 14.0 with four warps, 128 rows of
// 61 keys 15.7 against 29.1, of 255 keys 35.5 against 41.3, but 64 rows of 1001
// keys 78.2 against 61.5; 8 kv heads of 8: 128 rows of 121 keys 10.4 against
// 11.2, of 501 keys 24.6 against 24.7.
template <int D, bool FEW>
cudaError_t launch_d(const Kv4Attn &p, dim3 grid, cudaStream_t s)
{
    if (p.chunk_len == 0 && p.max_ctx < (FEW ? 256 : 128) && (long long)grid.x * grid.y > 6 * SMS)
        return launch_w<D, FEW, 1>(p, grid, s);
    return launch_w<D, FEW, WARPS>(p, grid, s);
}

int launch(Kv4Attn &p, int d, int seqs, int rows, cudaStream_t s)
{
    const int cols = p.chunk_len > 0 ? p.chunk_len * p.group : p.group;
    const bool f = few(cols, d);
    p.col_groups = f ? 1 : (cols + 7) / 8;
    const long long gx = (long long)p.n_splits * p.col_groups * p.n_kv;
    const long long joins = (long long)rows * p.n_heads;
    if (gx > 0x7fffffff || (p.n_splits > 1 && joins > 0x7fffffff))
        return HB_ERANGE;
    const dim3 grid((unsigned)gx, (unsigned)seqs);
    const cudaError_t e = d == 128 ? (f ? launch_d<128, true>(p, grid, s) : launch_d<128, false>(p, grid, s))
                                   : (f ? launch_d<64, true>(p, grid, s) : launch_d<64, false>(p, grid, s));
    if (e != cudaSuccess)
        return HB_ECUDA;
    if (p.n_splits > 1) {
        auto join = d == 128 ? k_kv4_join<128> : k_kv4_join<64>;
        if (launch_kernel(true, join, dim3((unsigned)joins), dim3(JOIN_WARPS * 32), 0, s, p) != cudaSuccess)
            return HB_ECUDA;
    }
    return HB_OK;
}

}  // namespace
}  // namespace hb

using namespace hb;

extern "C" long long hb_kv4_decode_workspace(int n_decodes, int n_heads, int n_kv_heads, int head_dim, int max_ctx)
{
    if (n_decodes < 0 || n_decodes > 65535 || !dims_ok(n_heads, n_kv_heads, head_dim) || max_ctx < 0 ||
        max_ctx >= MAX_KEYS)
        return HB_EINVAL;
    if (n_decodes == 0)
        return 0;
    const Split sp = plan_split(ctas_of(n_heads / n_kv_heads, n_kv_heads, n_decodes), resident(n_decodes, n_heads / n_kv_heads, head_dim),
                                max_ctx + 1);
    return workspace_bytes_of(n_decodes, n_heads, head_dim, sp.n);
}

extern "C" int hb_kv4_decode(const hb_kv4_pool *pool, const void *q, long long q_stride, const int32_t *block_tables,
                             int bt_stride, const int32_t *ctx_lens, int n_decodes, int n_heads, int max_ctx,
                             void *out, long long out_stride, void *workspace, long long workspace_bytes,
                             void *cuda_stream)
try {
    int rc = kv4_check_pool(pool);
    if (rc)
        return rc;
    const int d = pool->head_dim;
    if (n_decodes < 0 || !dims_ok(n_heads, pool->n_kv_heads, d) || max_ctx < 0)
        return HB_EINVAL;
    if (n_decodes == 0)
        return HB_OK;
    const int width = n_heads * d;
    if (!block_tables || !ctx_lens || kv4_check_rows(q, q_stride, n_decodes, width) ||
        kv4_check_rows(out, out_stride, n_decodes, width))
        return HB_EINVAL;
    if (n_decodes > 65535 || max_ctx >= MAX_KEYS || bt_stride < max_ctx / 16 + 1)
        return HB_ERANGE;
    Kv4Attn p{};
    p.pool = (const uint8_t *)pool->data;
    p.num_blocks = pool->num_blocks;
    p.n_kv = pool->n_kv_heads;
    p.group = n_heads / p.n_kv;
    p.ks = pool->k_scale;
    p.vs = pool->v_scale;
    p.q = (const bf16 *)q;
    p.q_stride = q_stride;
    p.tables = block_tables;
    p.bt_stride = bt_stride;
    p.ctx_lens = ctx_lens;
    p.max_ctx = max_ctx;
    p.n_heads = n_heads;
    const Split sp = plan_split(ctas_of(p.group, p.n_kv, n_decodes), resident(n_decodes, p.group, d), max_ctx + 1);
    p.split_len = sp.len;
    p.n_splits = sp.n;
    p.out = (bf16 *)out;
    p.out_stride = out_stride;
    const long long need = workspace_bytes_of(n_decodes, n_heads, d, sp.n);
    if (need > 0) {
        if (workspace_bytes < need)
            return HB_ERANGE;
        if (!workspace || (uintptr_t)workspace % 16)
            return HB_EINVAL;
        p.part_o = (float *)workspace;
        p.part_ml = (float2 *)(p.part_o + (size_t)n_decodes * n_heads * sp.n * d);
    }
    p.lose = take_lose();
    return launch(p, d, n_decodes, n_decodes, (cudaStream_t)cuda_stream);
} catch (...) {
    return HB_ENOMEM;
}

// Microseconds that a chunk takes as columns of the decode kernel, for the
// choice between it and the tcgen05 kernel, whose plan has an estimate of its
// own: 0.7 to 2.8 of the time over 196 shapes, nearest where the two are close,
// so that the choice costs at most 1.3 of the better one.  With 40 heads of 128
// and 1000 cached keys, 16 rows take 10.6 us against 12.1 on the tcgen05
// kernel, 64 rows 20.7 against 12.7; with 16000 keys, 16 rows 53 against 56, 32
// rows 82 against 56.
static double decode_kernel_us(int offset, int len, int group, int n_kv)
{
    const double pages = (offset + 0.5 * len) / 16 + 1;
    return 5 + n_kv * (double)(((long long)len * group + 7) / 8) * pages / 1500;
}
// Plan a chunk: 0, `p` filled, as columns of the decode kernel; 1, `c` filled,
// on the tcgen05 kernel; -1: too large.
static int plan_chunk(Kv4Attn &p, Kv4Chunk &c, int offset, int len, int n_heads, int n_kv, int d, long long *need)
{
    const int group = n_heads / n_kv;
    c.n_kv = n_kv;
    c.group = group;
    c.n_heads = n_heads;
    c.offset = offset;
    const double few = decode_kernel_us(offset, len, group, n_kv);
    const bool tensor = (long long)len * group > 8 && few > 8;  // below, no plan is much faster
    if (tensor && !kv4_chunk_plan(c, len, d))
        return -1;
    if (tensor && c.us < few) {
        *need = kv4_chunk_workspace_bytes(c, d);
        return 1;
    }
    p.n_kv = n_kv;
    p.group = group;
    p.n_heads = n_heads;
    p.chunk_offset = offset;
    p.chunk_len = len;
    const Split sp = plan_split(ctas_of(len * group, n_kv, 1), resident(1, len * group, d), offset + len);
    p.split_len = sp.len;
    p.n_splits = sp.n;
    *need = workspace_bytes_of(len, n_heads, d, sp.n);
    return 0;
}

extern "C" long long hb_kv4_chunk_workspace(int chunk_offset, int chunk_len, int n_heads, int n_kv_heads, int head_dim)
{
    if (chunk_offset < 0 || chunk_len < 0 || !dims_ok(n_heads, n_kv_heads, head_dim) ||
        (long long)chunk_offset + chunk_len > MAX_KEYS)
        return HB_EINVAL;
    if (chunk_len == 0)
        return 0;
    if ((long long)chunk_len * (n_heads / n_kv_heads) > MAX_COLS)
        return HB_EINVAL;
    Kv4Attn p{};
    Kv4Chunk c;
    long long need = 0;
    return plan_chunk(p, c, chunk_offset, chunk_len, n_heads, n_kv_heads, head_dim, &need) < 0 ? HB_EINVAL : need;
}

extern "C" int hb_kv4_chunk(const hb_kv4_pool *pool, const void *q, long long q_stride, const int32_t *block_table,
                            int n_blocks, int chunk_offset, int chunk_len, int n_heads, void *out,
                            long long out_stride, void *workspace, long long workspace_bytes, void *cuda_stream)
try {
    int rc = kv4_check_pool(pool);
    if (rc)
        return rc;
    const int d = pool->head_dim;
    if (chunk_offset < 0 || chunk_len < 0 || !dims_ok(n_heads, pool->n_kv_heads, d))
        return HB_EINVAL;
    if (chunk_len == 0)
        return HB_OK;
    const int width = n_heads * d;
    if (!block_table || kv4_check_rows(q, q_stride, chunk_len, width) ||
        kv4_check_rows(out, out_stride, chunk_len, width))
        return HB_EINVAL;
    const long long keys = (long long)chunk_offset + chunk_len;
    if (keys > MAX_KEYS || n_blocks < (keys + 15) / 16 ||
        (long long)chunk_len * (n_heads / pool->n_kv_heads) > MAX_COLS)
        return HB_ERANGE;
    Kv4Attn p{};
    Kv4Chunk c;
    long long need = 0;
    const int which = plan_chunk(p, c, chunk_offset, chunk_len, n_heads, pool->n_kv_heads, d, &need);
    if (which < 0)
        return HB_ERANGE;
    if (need > 0) {
        if (workspace_bytes < need)
            return HB_ERANGE;
        if (!workspace || (uintptr_t)workspace % 16)
            return HB_EINVAL;
    }
    if (which == 1) {
        c.pool = (const uint8_t *)pool->data;
        c.num_blocks = pool->num_blocks;
        c.ks = pool->k_scale;
        c.vs = pool->v_scale;
        c.q = (const bf16 *)q;
        c.q_stride = q_stride;
        c.table = block_table;
        c.out = (bf16 *)out;
        c.out_stride = out_stride;
        c.part_o = (float *)workspace;
        c.part_ml = (float2 *)(c.part_o + (size_t)2 * c.ctas * KC_ROWS * d);
        c.lose = take_lose();
        return launch_kv4_chunk(c, d, (cudaStream_t)cuda_stream) == cudaSuccess ? HB_OK : HB_ECUDA;
    }
    p.pool = (const uint8_t *)pool->data;
    p.num_blocks = pool->num_blocks;
    p.ks = pool->k_scale;
    p.vs = pool->v_scale;
    p.q = (const bf16 *)q;
    p.q_stride = q_stride;
    p.tables = block_table;
    p.bt_stride = n_blocks;
    p.out = (bf16 *)out;
    p.out_stride = out_stride;
    p.part_o = (float *)workspace;
    p.part_ml = (float2 *)(p.part_o + (size_t)chunk_len * n_heads * p.n_splits * d);
    p.lose = take_lose();
    return launch(p, d, 1, chunk_len, (cudaStream_t)cuda_stream);
} catch (...) {
    return HB_ENOMEM;
}

extern "C" void hb_kv4_test_lost_page(void) { test_lose = true; }
