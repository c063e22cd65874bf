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
// query (bf16 fits f16 then), and P is formed as 2^(s - m + 7), which keeps
// weights of 2^-21 normal in f16 and P times a V scale (at most 448) finite.
#include <cuda_runtime.h>

#include "common.cuh"
#include "hb_cache.h"
#include "kv4.cuh"
#include "kv4_host.h"

namespace hb {
namespace {

using namespace kv4;

constexpr float LOG2E = 1.4426950408889634f;
constexpr float P_SHIFT = 7.f;
constexpr int WARPS = 4;
constexpr int SPLIT_MIN = 256;        // keys of a split at least
constexpr int MAX_KEYS = 1 << 27;

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

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// All ones in each half of x that is not 0.
__device__ __forceinline__ uint32_t nonzero_mask(uint32_t x)
{
    return ((x & 0x00007fffu) ? 0x0000ffffu : 0u) | ((x & 0x7fff0000u) ? 0xffff0000u : 0u);
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[N])
{
    if constexpr (N == 4) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        w[0] = u.x, w[1] = u.y;
    }
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

template <int D>
__global__ void __launch_bounds__(WARPS * 32) k_kv4_attention(const Kv4Attn p)
{
    using L = Layout<D>;
    constexpr int NB = L::NB, KW = NB / 2;  // words of a lane's 8- or 16-byte load
    __shared__ float s_scale[8];
    __shared__ float s_m[WARPS][8], s_l[WARPS][8];
    __shared__ float s_o[WARPS][8][D + 4];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int split = blockIdx.x % p.n_splits;
    const int rest = blockIdx.x / p.n_splits;
    const int cg = rest % p.col_groups, kvh = rest / p.col_groups;
    const int seq = blockIdx.y;
    const int ncols = p.chunk_len > 0 ? p.chunk_len * p.group : p.group;
    const int c0 = cg * 8, c1 = min(c0 + 8, ncols);  // this CTA's columns

    if (p.chunk_len == 0) {
        const int ctx = p.ctx_lens[seq];
        if (ctx < 0 || ctx > p.max_ctx) {  // padding: zeros; outside what the grid was sized for: NaN
            if (split == 0)
                for (int c = c0; c < c1; ++c) {
                    const Col co = column(p, seq, kvh, c);
                    for (int e = threadIdx.x; e < D; e += WARPS * 32)
                        p.out[co.row * p.out_stride + (size_t)co.head * D + e] =
                            f2bf(ctx == -1 ? 0.f : __int_as_float(0x7fc00000));
                }
            return;
        }
    }
    const int nkeys = column(p, seq, kvh, c1 - 1).nkeys;  // the most any column sees
    const int k0 = split * p.split_len, k1 = min(nkeys, k0 + p.split_len);
    if (k0 >= k1)
        return;
    const int fewest = column(p, seq, kvh, c0).nkeys;  // keys that every column sees

    // q of column c0 + g as B fragments, and what its scores are scaled by
    uint32_t qf[NB][2];
    {
        const int c = c0 + g;
        float x[NB][4];
        float a = 0.f;
        const bool have = c < c1;
        const Col co = column(p, seq, kvh, have ? c : c0);
        const bf16 *qr = p.q + co.row * p.q_stride + (size_t)co.head * D;
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
        const int e = a > 0.f ? ilogbf(a) : 0;
        const int ec = min(max(e, -126), 127);
        const float down = ldexpf(1.f, -ec);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            qf[i][0] = have ? pack_h2(x[i][0] * down, x[i][1] * down) : 0u;
            qf[i][1] = have ? pack_h2(x[i][2] * down, x[i][3] * down) : 0u;
        }
        if (warp == 0 && t == 0)
            s_scale[g] = ldexpf(p.ks * (rsqrtf((float)D) * LOG2E), ec);
    }
    __syncthreads();
    // columns 2t and 2t + 1 are this lane's in S and O
    float sc[2], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int seen[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int c = min(c0 + 2 * t + j, c1 - 1);
        sc[j] = s_scale[2 * t + j];
        seen[j] = column(p, seq, kvh, c).nkeys;
    }
    float o[NB][4];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[i][j] = 0.f;

    const int *tab = p.tables + (size_t)seq * p.bt_stride;
    const int tok0 = 4 * (g >> 1) + (g & 1);  // tokens tok0 and tok0 + 2 are rows g and g + 8 of S^T
    bool bad = false;
    for (int b = (k0 >> 4) + warp; b * 16 < k1; b += WARPS) {
        const int blk = tab[b];
        if (blk < 0 || blk >= p.num_blocks) {
            bad = true;
            continue;
        }
        const uint8_t *page = p.pool + ((size_t)blk * p.n_kv + kvh) * L::BYTES;
        // ---- S^T = K q
        uint32_t kw[2][KW], kst[2][NB / 2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            load_words<KW>(page + L::k_code(tok0 + 2 * r, t, 0), kw[r]);
#pragma unroll
            for (int i = 0; i < NB; i += 2)
                kst[r][i / 2] =
                    from_e4m3x2(*reinterpret_cast<const uint16_t *>(page + L::k_scale(tok0 + 2 * r, i)));
        }
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            uint32_t a[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                from_e2m1x8(kw[r][w], a[r]);
                const uint32_t lo = __byte_perm(kst[r][w], 0, 0x1010), hi = __byte_perm(kst[r][w], 0, 0x3232);
                a[r][0] = hmul2(a[r][0], lo);
                a[r][1] = hmul2(a[r][1], lo);
                a[r][2] = hmul2(a[r][2], hi);
                a[r][3] = hmul2(a[r][3], hi);
            }
            mma_f16(s, a[0][0], a[1][0], a[0][1], a[1][1], qf[2 * w][0], qf[2 * w][1]);
            mma_f16(s, a[0][2], a[1][2], a[0][3], a[1][3], qf[2 * w + 1][0], qf[2 * w + 1][1]);
        }
        // ---- softmax over the 16 keys: rows are tokens, columns queries
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int k = b * 16 + tok0;
            const float s0 = k < seen[j] ? s[j] * sc[j] : -INFINITY;
            const float s1 = k + 2 < seen[j] ? s[2 + j] * sc[j] : -INFINITY;
            float mx = fmaxf(s0, s1);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float mn = fmaxf(m[j], mx);
            const float ref = mn == -INFINITY ? 0.f : mn;
            const float corr = exp2f(m[j] - ref);
            s[j] = exp2f(s0 - ref + P_SHIFT);
            s[2 + j] = exp2f(s1 - ref + P_SHIFT);
            l[j] = l[j] * corr + s[j] + s[2 + j];
            m[j] = mn;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                o[i][j] *= corr;
                o[i][2 + j] *= corr;
            }
        }
        // ---- O^T += V^T P, a V scale times P in place of a scaled V
        const uint32_t p0 = movmatrix(pack_h2(s[0], s[1]));  // column g, tokens 4t, 4t + 1
        const uint32_t p1 = movmatrix(pack_h2(s[2], s[3]));  // tokens 4t + 2, 4t + 3
        uint32_t vw[2][KW];
        load_words<KW>(page + L::v_code(4 * t, g, 0), vw[0]);
        load_words<KW>(page + L::v_code(4 * t + 2, g, 0), vw[1]);
        // a slot that a query does not see may hold anything, a NaN scale
        // among it: where P is 0 its product with the scale is 0 too
        const bool edge = b * 16 + 16 > fewest;
        const uint32_t z0 = edge ? nonzero_mask(p0) : 0xffffffffu, z1 = edge ? nonzero_mask(p1) : 0xffffffffu;
#pragma unroll
        for (int w = 0; w < KW / 2; ++w) {
            // bytes of two tokens (channels 2g, 2g + 1) to bytes of two channels
            uint32_t a[4][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t x = vw[h][w], y = vw[h][KW / 2 + w];
                from_e2m1x8((x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u), a[2 * h]);
                from_e2m1x8(((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u), a[2 * h + 1]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t vs = *reinterpret_cast<const uint32_t *>(page + L::v_scale(4 * t, 4 * w + i));
                const uint32_t b0 = hmul2(p0, from_e4m3x2(vs & 0xffffu)) & z0;
                const uint32_t b1 = hmul2(p1, from_e4m3x2(vs >> 16)) & z1;
                mma_f16(o[4 * w + i], a[0][i], a[1][i], a[2][i], a[3][i], b0, b1);
            }
        }
    }

    // ---- join the warps
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        l[j] += __shfl_xor_sync(0xffffffffu, l[j], 4);
        l[j] += __shfl_xor_sync(0xffffffffu, l[j], 8);
        l[j] += __shfl_xor_sync(0xffffffffu, l[j], 16);
        if (bad) {  // a block id outside the pool poisons every column
            l[j] = __int_as_float(0x7fc00000);
            m[j] = 0.f;
        }
        if (g == 0) {
            s_m[warp][2 * t + j] = m[j];
            s_l[warp][2 * t + j] = l[j];
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            s_o[warp][2 * t + j][16 * i + 2 * g] = o[i][j];
            s_o[warp][2 * t + j][16 * i + 2 * g + 1] = o[i][2 + j];
        }
    }
    __syncthreads();
    for (int c = c0 + warp; c < c1; c += WARPS) {
        const Col co = column(p, seq, kvh, c);
        float M = -INFINITY, lsum = 0.f, f[WARPS];
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            M = fmaxf(M, s_m[w][c - c0]);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            f[w] = s_m[w][c - c0] == -INFINITY ? 0.f : exp2f(s_m[w][c - c0] - M);
            lsum += s_l[w][c - c0] * f[w];
        }
        const bool whole = co.nkeys <= p.split_len;  // this split holds every key the query sees
        const float inv = p.vs / lsum;
        const size_t at = ((size_t)co.row * p.n_heads + co.head) * p.n_splits + split;
        if (whole && split > 0)
            continue;
        for (int e = lane; e < D; e += 32) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w)
                v += s_o[w][c - c0][e] * f[w];
            if (whole)
                p.out[co.row * p.out_stride + (size_t)co.head * D + e] = f2bf(v * inv);
            else
                p.part_o[at * D + e] = v;
        }
        if (!whole && lane == 0)
            p.part_ml[at] = make_float2(M, lsum);
    }
}

// Joins the splits of one (row, head) per warp, in order.
template <int D>
__global__ void __launch_bounds__(128) k_kv4_join(const Kv4Attn p, int n_rows)
{
    const int lane = threadIdx.x & 31;
    const long long idx = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    pdl_wait();
    if (idx >= (long long)n_rows * p.n_heads)
        return;
    const int row = (int)(idx / p.n_heads), head = (int)(idx - (long long)row * p.n_heads);
    const int nkeys = p.chunk_len > 0 ? p.chunk_offset + row + 1 : p.ctx_lens[row] + 1;
    if (nkeys <= p.split_len || (p.chunk_len == 0 && nkeys > p.max_ctx + 1))
        return;  // written by the first kernel
    const int n = (nkeys + p.split_len - 1) / p.split_len;
    const float2 *ml = p.part_ml + (size_t)idx * p.n_splits;
    const float *po = p.part_o + (size_t)idx * p.n_splits * D;
    float M = -INFINITY;
    for (int s = 0; s < n; ++s)
        M = fmaxf(M, ml[s].x);
    float l = 0.f, o[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e)
        o[e] = 0.f;
    for (int s = 0; s < n; ++s) {
        const float2 x = ml[s];
        const float f = x.x == -INFINITY ? 0.f : exp2f(x.x - M);
        l += x.y * f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
            o[e] += po[(size_t)s * D + e * 32 + lane] * f;
    }
    const float inv = p.vs / l;
    bf16 *orow = p.out + row * p.out_stride + (size_t)head * D;
#pragma unroll
    for (int e = 0; e < D / 32; ++e)
        orow[e * 32 + lane] = f2bf(o[e] * inv);
}

struct Split {
    int len, n;
};

// Keys of a split: as many splits as give every SM work, but at least
// SPLIT_MIN keys each, a multiple of 16 WARPS.
Split plan_split(long long ctas, int max_keys)
{
    const int sms = 152;
    long long want = (4ll * sms + ctas - 1) / ctas;
    const long long most = (max_keys + SPLIT_MIN - 1) / SPLIT_MIN;
    if (want > most)
        want = most;
    if (want < 1)
        want = 1;
    long long len = (max_keys + want - 1) / want;
    len = (len + 16 * WARPS - 1) / (16 * WARPS) * (16 * WARPS);
    return Split{(int)len, (int)((max_keys + len - 1) / len)};
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

int launch(Kv4Attn &p, int d, int seqs, int rows, cudaStream_t s)
{
    const long long gx = (long long)p.n_splits * p.col_groups * p.n_kv;
    if (gx > 0x7fffffff)
        return HB_ERANGE;
    auto kern = d == 128 ? k_kv4_attention<128> : k_kv4_attention<64>;
    if (launch_kernel(false, kern, dim3((unsigned)gx, (unsigned)seqs), dim3(WARPS * 32), 0, s, p) != cudaSuccess)
        return HB_ECUDA;
    if (p.n_splits > 1) {
        auto join = d == 128 ? k_kv4_join<128> : k_kv4_join<64>;
        const long long warps = (long long)rows * p.n_heads;
        if (launch_kernel(true, join, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, s, p, rows) != cudaSuccess)
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
    const Split sp = plan_split(ctas_of(n_heads / n_kv_heads, n_kv_heads, n_decodes), max_ctx + 1);
    return workspace_bytes_of(n_decodes, n_heads, head_dim, sp.n);
}

extern "C" int hb_kv4_decode(const hb_kv4_pool *pool, const void *q, long long q_stride, const int32_t *block_tables,
                             int bt_stride, const int32_t *ctx_lens, int n_decodes, int n_heads, int max_ctx,
                             void *out, long long out_stride, void *workspace, long long workspace_bytes,
                             void *cuda_stream)
{
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
    p.col_groups = (p.group + 7) / 8;
    const Split sp = plan_split(ctas_of(p.group, p.n_kv, n_decodes), max_ctx + 1);
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
    return launch(p, d, n_decodes, n_decodes, (cudaStream_t)cuda_stream);
}

extern "C" long long hb_kv4_chunk_workspace(int chunk_offset, int chunk_len, int n_heads, int n_kv_heads, int head_dim)
{
    if (chunk_offset < 0 || chunk_len < 0 || !dims_ok(n_heads, n_kv_heads, head_dim) ||
        (long long)chunk_offset + chunk_len > MAX_KEYS)
        return HB_EINVAL;
    if (chunk_len == 0)
        return 0;
    if ((long long)chunk_len * (n_heads / n_kv_heads) > 0x7fffffff)
        return HB_EINVAL;
    const Split sp = plan_split(ctas_of(chunk_len * (n_heads / n_kv_heads), n_kv_heads, 1), chunk_offset + chunk_len);
    return workspace_bytes_of(chunk_len, n_heads, head_dim, sp.n);
}

extern "C" int hb_kv4_chunk(const hb_kv4_pool *pool, const void *q, long long q_stride, const int32_t *block_table,
                            int n_blocks, int chunk_offset, int chunk_len, int n_heads, void *out,
                            long long out_stride, void *workspace, long long workspace_bytes, void *cuda_stream)
{
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
    if (keys > MAX_KEYS || n_blocks < (keys + 15) / 16 || (long long)chunk_len * (n_heads / pool->n_kv_heads) > 0x7fffffff)
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
    p.tables = block_table;
    p.bt_stride = n_blocks;
    p.chunk_offset = chunk_offset;
    p.chunk_len = chunk_len;
    p.n_heads = n_heads;
    const int cols = chunk_len * p.group;
    p.col_groups = (cols + 7) / 8;
    const Split sp = plan_split(ctas_of(cols, p.n_kv, 1), (int)keys);
    p.split_len = sp.len;
    p.n_splits = sp.n;
    p.out = (bf16 *)out;
    p.out_stride = out_stride;
    const long long need = workspace_bytes_of(chunk_len, n_heads, d, sp.n);
    if (need > 0) {
        if (workspace_bytes < need)
            return HB_ERANGE;
        if (!workspace || (uintptr_t)workspace % 16)
            return HB_EINVAL;
        p.part_o = (float *)workspace;
        p.part_ml = (float2 *)(p.part_o + (size_t)chunk_len * n_heads * sp.n * d);
    }
    return launch(p, d, 1, chunk_len, (cudaStream_t)cuda_stream);
}
