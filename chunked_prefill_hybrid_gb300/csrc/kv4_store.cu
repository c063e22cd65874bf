// kv4_store.cu -- writing rows of K and V into the 4-bit paged cache, and
// reading them back (include/hb_cache.h).
#include <cuda_runtime.h>

#include "common.cuh"
#include "hb_cache.h"
#include "kv4.cuh"
#include "kv4_host.h"

namespace hb {
namespace {

using namespace kv4;

// A row's head is 8 (d = 128) or 4 (d = 64) lanes, lane i with the 16 channels
// of scale block i, of K and of V.  The pool keeps a token's codes in another
// order (kv4.cuh), so the lanes of a head exchange bytes and each then stores,
// or has loaded, eight that lie together: 4 stores a lane in place of 14.

// 4 x 4 transpose of 16-bit units over four lanes: lane a holds units 0..3
// (w0, w1) and gets unit a of the four lanes.
__device__ __forceinline__ void transpose_half4(uint32_t &w0, uint32_t &w1, int a)
{
    const bool b = a & 2, c = a & 1;
    const uint32_t r = __shfl_xor_sync(0xffffffffu, b ? w0 : w1, 2);
    w0 = b ? r : w0;
    w1 = b ? w1 : r;
    const uint32_t s = __shfl_xor_sync(0xffffffffu, __byte_perm(w0, w1, c ? 0x5410 : 0x7632), 1);
    w0 = c ? __byte_perm(s, w0, 0x7610) : __byte_perm(w0, s, 0x5410);
    w1 = c ? __byte_perm(s, w1, 0x7632) : __byte_perm(w1, s, 0x7610);
}

// 8 x 8 transpose of bytes over eight lanes.
__device__ __forceinline__ void transpose_byte8(uint32_t &w0, uint32_t &w1, int a)
{
    const bool b = a & 4, c = a & 2, d = a & 1;
    const uint32_t r = __shfl_xor_sync(0xffffffffu, b ? w0 : w1, 4);
    w0 = b ? r : w0;
    w1 = b ? w1 : r;
    const uint32_t s = __shfl_xor_sync(0xffffffffu, __byte_perm(w0, w1, c ? 0x5410 : 0x7632), 2);
    w0 = c ? __byte_perm(s, w0, 0x7610) : __byte_perm(w0, s, 0x5410);
    w1 = c ? __byte_perm(s, w1, 0x7632) : __byte_perm(w1, s, 0x7610);
    const uint32_t mine = __byte_perm(w0, w1, d ? 0x7531 : 0x6420);
    const uint32_t t = __shfl_xor_sync(0xffffffffu, __byte_perm(w0, w1, d ? 0x6420 : 0x7531), 1);
    const uint32_t even = d ? t : mine, odd = d ? mine : t;
    w0 = __byte_perm(even, odd, 0x5140);
    w1 = __byte_perm(even, odd, 0x7362);
}

// A lane's codes of V, byte g = channels 2g, 2g + 1 of its block, to the eight
// bytes that it stores: all blocks of g = i (d = 128), or of g = 2i and 2i + 1.
template <int D>
__device__ __forceinline__ void exchange_v(uint32_t &w0, uint32_t &w1, int i)
{
    if constexpr (D == 128) {
        transpose_byte8(w0, w1, i);
    } else {
        transpose_half4(w0, w1, i);
        const uint32_t x = __byte_perm(w0, w1, 0x6420), y = __byte_perm(w0, w1, 0x7531);
        w0 = x;
        w1 = y;
    }
}
template <int D>
__device__ __forceinline__ void exchange_v_back(uint32_t &w0, uint32_t &w1, int i)
{
    if constexpr (D == 128) {
        transpose_byte8(w0, w1, i);
    } else {
        const uint32_t x = __byte_perm(w0, w1, 0x5140), y = __byte_perm(w0, w1, 0x7362);
        w0 = x;
        w1 = y;
        transpose_half4(w0, w1, i);
    }
}

// Codes of 8 channels whose quotients may be out of range.
__device__ __noinline__ uint32_t saturated8(uint4 u, float s, float inv)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t r = 0;
    for (int i = 0; i < 4; ++i) {
        float e[2] = {__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)};
        for (int j = 0; j < 2; ++j) {
            const float q = e[j] * inv;
            e[j] = fabsf(q) < 8.f ? fmaf(fmaf(-q, s, e[j]), inv, q) : q;
        }
        r |= to_e2m1x2(e[0], e[1]) << (8 * i);
    }
    return r;
}

// 16 channels of one token, bf16: the e4m3 scale byte, and the codes two a byte.
//
// scale = e4m3(max|x| / (6 ps)), code = e2m1(x / (scale ps)).  Bf16 values
// divided by a scale of four significant bits lie on e2m1's rounding borders
// often (one in twenty), so a product with a reciprocal would send ties the
// wrong way; each quotient is therefore corrected once by its exact remainder
// (Markstein's correction step), which returns the quotient itself wherever it
// is representable, every tie among them.  r6 is 1 / (6 ps).
__device__ __forceinline__ uint32_t quantise16(const uint4 (&u)[2], float ps, float r6, uint32_t (&codes)[2])
{
    const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
    __nv_bfloat162 mx = __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[0]));
#pragma unroll
    for (int i = 1; i < 8; ++i)
        mx = __hmax2_nan(mx, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i])));
    const uint32_t both = *reinterpret_cast<const uint32_t *>(&mx);
    const uint32_t a = max(both & 0xffffu, both >> 16);  // magnitudes of bf16 order like their bits, NaNs last
    const float av = __uint_as_float(a << 16);
    float q = av * r6;
    if (q < 1024.f)  // else it saturates, and may have no remainder
        q = fmaf(fmaf(-q, 6.f * ps, av), r6, q);
    const uint32_t sb = a > 0x7f80u ? 0x7fu : to_e4m3(q);
    const float s = h2f2(from_e4m3x2(sb)).x * ps;
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    if (sb == 0)
        inv = 0.f;
    const uint64_t s2 = pack_f2(-s, -s), inv2 = pack_f2(inv, inv);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = w[4 * h + i];
            const uint64_t v = pack_f2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
            const uint64_t q0 = mul_f2(v, inv2);
            float e0, e1;
            unpack_f2(fma_f2(fma_f2(q0, s2, v), inv2, q0), e0, e1);
            c[i] = to_e2m1x2(e0, e1);
        }
        codes[h] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    }
    // with a scale that saturated (or an infinity or NaN) a quotient may be
    // out of range, where it has no remainder
    if (a >= 0x7f80u || sb == 0x7eu) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            codes[h] = saturated8(u[h], s, inv);
    }
    return sb;
}

// What a thread of the store kernels works on.  A block takes 16 rows of two
// (d = 128) or four (d = 64) heads: rows that follow one another usually lie in
// one page, whose 32-byte sectors are then shared inside the SM.
constexpr int ROWS = 16, THREADS = 256;
template <int D>
struct Place {
    static constexpr int NB = D / 16, HEADS = THREADS / (ROWS * NB);
    int i, h;
    long long row;
    int tok;
    bool ok;       // row and head exist and the slot lies in the pool
    size_t page;   // (block, kv head)

    __device__ Place(int num_blocks, int n_kv, int head_groups, const int *slots, int n_tokens)
    {
        const int rb = blockIdx.x / head_groups, hg = blockIdx.x - rb * head_groups;
        i = threadIdx.x % NB;
        const long long r = (long long)rb * ROWS + threadIdx.x / NB % ROWS;
        const int head = hg * HEADS + threadIdx.x / (NB * ROWS);
        // lanes without a row or a head go along for the exchanges
        row = min(r, (long long)n_tokens - 1);
        h = min(head, n_kv - 1);
        const int slot = slots[row];
        ok = r < n_tokens && head < n_kv && slot >= 0 && (slot >> 4) < num_blocks;
        tok = slot & 15;
        page = (size_t)(ok ? slot >> 4 : 0) * n_kv + h;
    }
};

// One thread per (row, kv head, 16 channels), K and V.  With k_kv4_read 3565
// rows of 40 heads of 128 take 38.1 us, of which the 187 MB that the two move
// would take 27.6 at the copy rate; 274 rows 5.1 us; 18 rows 3.4 (two launches).
// A byte store for each two channels took 51.4 us, 7.8 and 5.2.  Of a prompt this
// kernel takes 22 us against 14 for its bytes: warps mostly wait for their loads
// (8.3 cycles an instruction, the next stall 2.1; 60% of the issue slots taken),
// as a thread has one item and nothing to do until it is there.
template <int D>
__global__ void __launch_bounds__(THREADS, 6)
    k_kv4_append(uint8_t *pool, int num_blocks, int n_kv, int head_groups, float ks, float vs, float k6, float v6,
                 const bf16 *k, long long k_stride, const bf16 *v, long long v_stride, const int *slots, int n_tokens)
{
    using L = Layout<D>;
    pdl_wait();
    pdl_trigger();
    const Place<D> p(num_blocks, n_kv, head_groups, slots, n_tokens);
    uint4 ku[2], vu[2];
    const size_t at = (size_t)p.h * D + p.i * 16;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        ku[j] = __ldg(reinterpret_cast<const uint4 *>(k + p.row * k_stride + at) + j);
        vu[j] = __ldg(reinterpret_cast<const uint4 *>(v + p.row * v_stride + at) + j);
    }
    uint8_t *page = pool + p.page * L::BYTES;
    uint32_t c[2];
    uint32_t sb = quantise16(ku, ks, k6, c);
    transpose_half4(c[0], c[1], p.i & 3);
    if (p.ok) {
        page[L::k_scale(p.tok, p.i)] = (uint8_t)sb;
        *reinterpret_cast<uint2 *>(page + L::k_code(p.tok, p.i & 3, p.i & 4)) = make_uint2(c[0], c[1]);
    }
    sb = quantise16(vu, vs, v6, c);
    exchange_v<D>(c[0], c[1], p.i);
    if (p.ok) {
        page[L::v_scale(p.tok, p.i)] = (uint8_t)sb;
        if constexpr (D == 128) {
            *reinterpret_cast<uint2 *>(page + L::v_code(p.tok, p.i, 0)) = make_uint2(c[0], c[1]);
        } else {
            *reinterpret_cast<uint32_t *>(page + L::v_code(p.tok, 2 * p.i, 0)) = c[0];
            *reinterpret_cast<uint32_t *>(page + L::v_code(p.tok, 2 * p.i + 1, 0)) = c[1];
        }
    }
}

// bf16 of code * scale * ps for 8 channels.
__device__ __forceinline__ uint4 values8(uint32_t codes, float s)
{
    uint32_t hf[4];
    from_e2m1x8(codes, hf);
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = h2f2(hf[j]);
        x[2 * j] = f.x * s;
        x[2 * j + 1] = f.y * s;
    }
    return pack8_bf16(x);
}

// The same the other way: a thread per (row, kv head, 16 channels), figures above.
template <int D>
__global__ void __launch_bounds__(THREADS, 8)
    k_kv4_read(const uint8_t *pool, int num_blocks, int n_kv, int head_groups, float ks, float vs, const int *slots,
               int n_tokens, bf16 *k, long long k_stride, bf16 *v, long long v_stride)
{
    using L = Layout<D>;
    pdl_wait();
    pdl_trigger();
    const Place<D> p(num_blocks, n_kv, head_groups, slots, n_tokens);
    const uint8_t *page = pool + p.page * L::BYTES;  // where !ok, some page that exists
    const uint2 ku = *reinterpret_cast<const uint2 *>(page + L::k_code(p.tok, p.i & 3, p.i & 4));
    uint32_t kc[2] = {ku.x, ku.y}, vc[2];
    if constexpr (D == 128) {
        const uint2 u = *reinterpret_cast<const uint2 *>(page + L::v_code(p.tok, p.i, 0));
        vc[0] = u.x, vc[1] = u.y;
    } else {
        vc[0] = *reinterpret_cast<const uint32_t *>(page + L::v_code(p.tok, 2 * p.i, 0));
        vc[1] = *reinterpret_cast<const uint32_t *>(page + L::v_code(p.tok, 2 * p.i + 1, 0));
    }
    const uint32_t sb = page[L::k_scale(p.tok, p.i)] | (uint32_t)page[L::v_scale(p.tok, p.i)] << 8;
    transpose_half4(kc[0], kc[1], p.i & 3);
    exchange_v_back<D>(vc[0], vc[1], p.i);
    // two neighbouring lanes share their two blocks, so that together they
    // write whole 32-byte sectors: first the lower block, then the upper
    const bool up = p.i & 1;
    const uint32_t other = __shfl_xor_sync(0xffffffffu, sb, 1);
    const uint32_t kx = __shfl_xor_sync(0xffffffffu, up ? kc[0] : kc[1], 1);
    const uint32_t vx = __shfl_xor_sync(0xffffffffu, up ? vc[0] : vc[1], 1);
    const uint32_t s0 = from_e4m3x2(up ? other : sb), s1 = from_e4m3x2(up ? sb : other);  // (K, V) of the two blocks
    if (p.ok) {
        const size_t at = (size_t)p.h * D + (p.i & ~1) * 16 + (up ? 8 : 0);
        bf16 *ko = k + p.row * k_stride + at, *vo = v + p.row * v_stride + at;
        const float2 f0 = h2f2(s0), f1 = h2f2(s1);
        *reinterpret_cast<uint4 *>(ko) = values8(up ? kx : kc[0], f0.x * ks);
        *reinterpret_cast<uint4 *>(ko + 16) = values8(up ? kc[1] : kx, f1.x * ks);
        *reinterpret_cast<uint4 *>(vo) = values8(up ? vx : vc[0], f0.y * vs);
        *reinterpret_cast<uint4 *>(vo + 16) = values8(up ? vc[1] : vx, f1.y * vs);
    }
}

template <int D>
long long store_blocks(int n_kv, int n_tokens, int *head_groups)
{
    *head_groups = (n_kv + Place<D>::HEADS - 1) / Place<D>::HEADS;
    return (long long)*head_groups * ((n_tokens + (long long)ROWS - 1) / ROWS);
}

}  // namespace

int kv4_check_pool(const hb_kv4_pool *p)
{
    if (!p || !p->data || (uintptr_t)p->data % 16 ||
        hb_kv4_pool_bytes(p->num_blocks, p->n_kv_heads, p->head_dim) < 0)
        return HB_EINVAL;
    // also false for NaN
    const float lo = 0x1p-60f, hi = 0x1p60f;
    if (!(p->k_scale >= lo && p->k_scale <= hi && p->v_scale >= lo && p->v_scale <= hi))
        return HB_EINVAL;
    return HB_OK;
}

int kv4_check_rows(const void *p, long long stride, int n, int width)
{
    if (!p || (uintptr_t)p % 16)
        return HB_EINVAL;
    if (n > 1 && (stride % 8 || stride < width || stride > (1ll << 40)))
        return HB_EINVAL;
    return HB_OK;
}

}  // namespace hb

using namespace hb;

extern "C" long long hb_kv4_pool_bytes(int num_blocks, int n_kv_heads, int head_dim)
{
    // slots are int32: 16 num_blocks must stay below 2^31
    if (num_blocks < 1 || num_blocks > (1 << 27) - 1 || n_kv_heads < 1 || n_kv_heads > 65535 ||
        (head_dim != 64 && head_dim != 128))
        return HB_EINVAL;
    return (long long)num_blocks * n_kv_heads * 18 * head_dim;
}

extern "C" int hb_kv4_append(const hb_kv4_pool *pool, const void *k, long long k_stride, const void *v,
                             long long v_stride, const int32_t *slots, int n_tokens, void *cuda_stream)
try {
    int rc = kv4_check_pool(pool);
    if (rc)
        return rc;
    if (n_tokens < 0)
        return HB_EINVAL;
    if (n_tokens == 0)
        return HB_OK;
    const int width = pool->n_kv_heads * pool->head_dim;
    if (!slots || kv4_check_rows(k, k_stride, n_tokens, width) || kv4_check_rows(v, v_stride, n_tokens, width))
        return HB_EINVAL;
    int hg = 0;
    const long long grid = pool->head_dim == 128 ? store_blocks<128>(pool->n_kv_heads, n_tokens, &hg)
                                                 : store_blocks<64>(pool->n_kv_heads, n_tokens, &hg);
    if (grid > 0x7fffffff)
        return HB_ERANGE;
    auto kern = pool->head_dim == 128 ? k_kv4_append<128> : k_kv4_append<64>;
    return launch_kernel(true, kern, dim3((unsigned)grid), dim3(THREADS), 0, (cudaStream_t)cuda_stream,
                         (uint8_t *)pool->data, pool->num_blocks, pool->n_kv_heads, hg, pool->k_scale, pool->v_scale,
                         1.f / (6.f * pool->k_scale), 1.f / (6.f * pool->v_scale), (const bf16 *)k, k_stride,
                         (const bf16 *)v, v_stride, (const int *)slots, n_tokens) == cudaSuccess
               ? HB_OK
               : HB_ECUDA;
} catch (...) {
    return HB_ENOMEM;
}

extern "C" int hb_kv4_read(const hb_kv4_pool *pool, const int32_t *slots, int n_tokens, void *k, long long k_stride,
                           void *v, long long v_stride, void *cuda_stream)
try {
    int rc = kv4_check_pool(pool);
    if (rc)
        return rc;
    if (n_tokens < 0)
        return HB_EINVAL;
    if (n_tokens == 0)
        return HB_OK;
    const int width = pool->n_kv_heads * pool->head_dim;
    if (!slots || kv4_check_rows(k, k_stride, n_tokens, width) || kv4_check_rows(v, v_stride, n_tokens, width))
        return HB_EINVAL;
    int hg = 0;
    const long long grid = pool->head_dim == 128 ? store_blocks<128>(pool->n_kv_heads, n_tokens, &hg)
                                                 : store_blocks<64>(pool->n_kv_heads, n_tokens, &hg);
    if (grid > 0x7fffffff)
        return HB_ERANGE;
    auto kern = pool->head_dim == 128 ? k_kv4_read<128> : k_kv4_read<64>;
    return launch_kernel(true, kern, dim3((unsigned)grid), dim3(THREADS), 0, (cudaStream_t)cuda_stream,
                         (const uint8_t *)pool->data, pool->num_blocks, pool->n_kv_heads, hg, pool->k_scale,
                         pool->v_scale, (const int *)slots, n_tokens, (bf16 *)k, k_stride, (bf16 *)v,
                         v_stride) == cudaSuccess
               ? HB_OK
               : HB_ECUDA;
} catch (...) {
    return HB_ENOMEM;
}
