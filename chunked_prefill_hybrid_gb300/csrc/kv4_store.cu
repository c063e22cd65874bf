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

// 16 channels x of one token: the e4m3 scale byte, and the codes two a byte.
//
// scale = e4m3(max|x| / (6 ps)), code = e2m1(x / (scale ps)).  Bf16 values
// divided by a scale of four significant bits lie on e2m1's rounding borders
// often (one in twenty), so a product with the rounded reciprocal would send
// ties the wrong way; each quotient is therefore corrected once by its exact
// remainder (Markstein's correction step), which returns the quotient itself
// wherever it is representable, every tie among them.
__device__ __forceinline__ uint32_t quantise16(const float (&x)[16], float ps, uint8_t (&codes)[8])
{
    float a = 0.f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        a = fmaxf(a, fabsf(x[i]));
        nan |= x[i] != x[i];
    }
    const uint32_t sb = nan ? 0x7fu : to_e4m3(__fdiv_rn(a, 6.f * ps));
    const float s = h2f2(from_e4m3x2(sb)).x * ps;
    const bool zero = sb == 0;
    const float inv = zero ? 0.f : __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float q[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float v = x[2 * i + j];
            const float q0 = v * inv;
            const float q1 = fmaf(fmaf(-q0, s, v), inv, q0);
            q[j] = fabsf(q0) < 8.f ? q1 : q0;  // infinities have no remainder
        }
        codes[i] = (uint8_t)to_e2m1x2(q[0], q[1]);
    }
    return sb;
}

__device__ __forceinline__ void unpack8(uint4 u, float *x)
{
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(h[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// One thread per (row, kv head, 16 channels), K and V.
template <int D>
__global__ void __launch_bounds__(256)
    k_kv4_append(uint8_t *pool, int num_blocks, int n_kv, float ks, float vs, const bf16 *k, long long k_stride,
                 const bf16 *v, long long v_stride, const int *slots, int n_tokens)
{
    using L = Layout<D>;
    const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const int i = (int)(idx % L::NB);
    const long long r = idx / L::NB;
    const int h = (int)(r % n_kv);
    const long long row = r / n_kv;
    if (row >= n_tokens)
        return;
    const int slot = slots[row];
    if (slot < 0 || (slot >> 4) >= num_blocks)
        return;
    const int tok = slot & 15;
    uint8_t *page = pool + ((size_t)(slot >> 4) * n_kv + h) * L::BYTES;
    const bf16 *kr = k + row * k_stride + (size_t)h * D + i * 16;
    const bf16 *vr = v + row * v_stride + (size_t)h * D + i * 16;
    float x[16];
    uint8_t c[8];
    unpack8(reinterpret_cast<const uint4 *>(kr)[0], x);
    unpack8(reinterpret_cast<const uint4 *>(kr)[1], x + 8);
    page[L::k_scale(tok, i)] = (uint8_t)quantise16(x, ks, c);
#pragma unroll
    for (int t = 0; t < 4; ++t)
        *reinterpret_cast<uint16_t *>(page + L::k_code(tok, t, i)) = (uint16_t)(c[2 * t] | (c[2 * t + 1] << 8));
    unpack8(reinterpret_cast<const uint4 *>(vr)[0], x);
    unpack8(reinterpret_cast<const uint4 *>(vr)[1], x + 8);
    page[L::v_scale(tok, i)] = (uint8_t)quantise16(x, vs, c);
#pragma unroll
    for (int g = 0; g < 8; ++g)
        page[L::v_code(tok, g, i)] = c[g];
}

// bf16 of code * scale * ps for 16 channels given as 8 bytes of codes.
__device__ __forceinline__ void write16(bf16 *out, const uint32_t (&w)[2], uint32_t sb, float ps)
{
    const float s = h2f2(from_e4m3x2(sb)).x * ps;
    uint4 u[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        uint32_t hf[4];
        from_e2m1x8(w[p], hf);
        float x[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = h2f2(hf[j]);
            x[2 * j] = f.x * s;
            x[2 * j + 1] = f.y * s;
        }
        u[p] = pack8_bf16(x);
    }
    reinterpret_cast<uint4 *>(out)[0] = u[0];
    reinterpret_cast<uint4 *>(out)[1] = u[1];
}

template <int D>
__global__ void __launch_bounds__(256)
    k_kv4_read(const uint8_t *pool, int num_blocks, int n_kv, float ks, float vs, const int *slots, int n_tokens,
               bf16 *k, long long k_stride, bf16 *v, long long v_stride)
{
    using L = Layout<D>;
    const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const int i = (int)(idx % L::NB);
    const long long r = idx / L::NB;
    const int h = (int)(r % n_kv);
    const long long row = r / n_kv;
    if (row >= n_tokens)
        return;
    const int slot = slots[row];
    if (slot < 0 || (slot >> 4) >= num_blocks)
        return;
    const int tok = slot & 15;
    const uint8_t *page = pool + ((size_t)(slot >> 4) * n_kv + h) * L::BYTES;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int t = 0; t < 4; ++t)
        w[t >> 1] |= (uint32_t) * reinterpret_cast<const uint16_t *>(page + L::k_code(tok, t, i)) << (16 * (t & 1));
    write16(k + row * k_stride + (size_t)h * D + i * 16, w, page[L::k_scale(tok, i)], ks);
    w[0] = w[1] = 0;
#pragma unroll
    for (int g = 0; g < 8; ++g)
        w[g >> 2] |= (uint32_t)page[L::v_code(tok, g, i)] << (8 * (g & 3));
    write16(v + row * v_stride + (size_t)h * D + i * 16, w, page[L::v_scale(tok, i)], vs);
}

// Whether a row operand (k, v, q, out) is one the kernels can read or write.
int check_rows(const void *p, long long stride, int n, int width)
{
    if (!p || (uintptr_t)p % 16)
        return HB_EINVAL;
    if (n > 1 && (stride % 8 || stride < width || stride > (1ll << 40)))
        return HB_EINVAL;
    return HB_OK;
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

int kv4_check_rows(const void *p, long long stride, int n, int width) { return check_rows(p, stride, n, width); }

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
{
    int rc = kv4_check_pool(pool);
    if (rc)
        return rc;
    if (n_tokens < 0)
        return HB_EINVAL;
    if (n_tokens == 0)
        return HB_OK;
    const int width = pool->n_kv_heads * pool->head_dim;
    if (!slots || check_rows(k, k_stride, n_tokens, width) || check_rows(v, v_stride, n_tokens, width))
        return HB_EINVAL;
    const long long threads = (long long)n_tokens * pool->n_kv_heads * (pool->head_dim / 16);
    const long long grid = (threads + 255) / 256;
    if (grid > 0x7fffffff)
        return HB_ERANGE;
    auto kern = pool->head_dim == 128 ? k_kv4_append<128> : k_kv4_append<64>;
    return launch_kernel(false, kern, dim3((unsigned)grid), dim3(256), 0, (cudaStream_t)cuda_stream,
                         (uint8_t *)pool->data, pool->num_blocks, pool->n_kv_heads, pool->k_scale, pool->v_scale,
                         (const bf16 *)k, k_stride, (const bf16 *)v, v_stride, (const int *)slots,
                         n_tokens) == cudaSuccess
               ? HB_OK
               : HB_ECUDA;
}

extern "C" int hb_kv4_read(const hb_kv4_pool *pool, const int32_t *slots, int n_tokens, void *k, long long k_stride,
                           void *v, long long v_stride, void *cuda_stream)
{
    int rc = kv4_check_pool(pool);
    if (rc)
        return rc;
    if (n_tokens < 0)
        return HB_EINVAL;
    if (n_tokens == 0)
        return HB_OK;
    const int width = pool->n_kv_heads * pool->head_dim;
    if (!slots || check_rows(k, k_stride, n_tokens, width) || check_rows(v, v_stride, n_tokens, width))
        return HB_EINVAL;
    const long long threads = (long long)n_tokens * pool->n_kv_heads * (pool->head_dim / 16);
    const long long grid = (threads + 255) / 256;
    if (grid > 0x7fffffff)
        return HB_ERANGE;
    auto kern = pool->head_dim == 128 ? k_kv4_read<128> : k_kv4_read<64>;
    return launch_kernel(false, kern, dim3((unsigned)grid), dim3(256), 0, (cudaStream_t)cuda_stream,
                         (const uint8_t *)pool->data, pool->num_blocks, pool->n_kv_heads, pool->k_scale,
                         pool->v_scale, (const int *)slots, n_tokens, (bf16 *)k, k_stride, (bf16 *)v,
                         v_stride) == cudaSuccess
               ? HB_OK
               : HB_ECUDA;
}
