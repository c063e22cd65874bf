// pages.cu -- copying pages inside paged pools (include/hb_cache.h), for a
// fork's copy-on-write and for compaction.
#include <cuda_runtime.h>

#include <algorithm>
#include <vector>

#include "common.cuh"
#include "hb_cache.h"
#include "runtime_internal.h"

namespace hb {
namespace {

constexpr int CP_VECS = 4;                   // 16-byte loads in flight per lane
constexpr int CP_UNIT = 32 * CP_VECS * 16;   // bytes a warp copies at a time
constexpr int CP_WARPS = 8;
constexpr long long MAX_BYTES = 1ll << 47;   // keeps the kernel's arithmetic inside 64 bits

// The page pairs travel as kernel parameters: nothing to stage, to keep
// alive after the call, or to free, and a captured launch holds its own copy.
template <int CAP>
struct PagePairs {
    int32_t src[CAP], dst[CAP];
};

// One warp copies 2 KB of one page of one pool at a time, four 16-byte loads a
// lane under way (with 2, 6, 8 or 16, or streaming hints, no faster).  Bound by
// memory: 97 pages of 33 KB in 80 pools take 84 us, 0.89 of the copy rate; one
// page of 164 KB in 80 pools 4.0 us.
template <int CAP>
__global__ void __launch_bounds__(CP_WARPS * 32)
    k_copy_pages(const __grid_constant__ PagePairs<CAP> pairs, uint8_t *data, long long pool_stride, int n_pools,
                 long long page_bytes, int segs, long long units)
{
    const int lane = threadIdx.x & 31;
    const long long warps = (long long)gridDim.x * CP_WARPS;
    pdl_wait();
    pdl_trigger();
    for (long long u = (long long)blockIdx.x * CP_WARPS + (threadIdx.x >> 5); u < units; u += warps) {
        const long long r = u / segs;
        const long long at = (u - r * segs) * CP_UNIT + lane * 16;
        const int pair = (int)(r / n_pools), pool = (int)(r - (long long)pair * n_pools);
        uint8_t *base = data + pool * pool_stride + at;
        const uint8_t *s = base + pairs.src[pair] * page_bytes;
        uint8_t *d = base + pairs.dst[pair] * page_bytes;
        uint4 v[CP_VECS];
#pragma unroll
        for (int i = 0; i < CP_VECS; ++i)
            if (at + i * 512 < page_bytes)
                v[i] = *reinterpret_cast<const uint4 *>(s + i * 512);
#pragma unroll
        for (int i = 0; i < CP_VECS; ++i)
            if (at + i * 512 < page_bytes)
                *reinterpret_cast<uint4 *>(d + i * 512) = v[i];
    }
}

template <int CAP>
cudaError_t launch_copy(const int32_t *src, const int32_t *dst, int n, uint8_t *data, long long pool_stride,
                        int n_pools, long long page_bytes, cudaStream_t s)
{
    PagePairs<CAP> pp;
    for (int i = 0; i < n; ++i) {
        pp.src[i] = src[i];
        pp.dst[i] = dst[i];
    }
    const int segs = (int)((page_bytes + CP_UNIT - 1) / CP_UNIT);
    const long long units = (long long)n * n_pools * segs;
    const long long want = (units + CP_WARPS - 1) / CP_WARPS;
    const unsigned grid = (unsigned)(want < (1 << 20) ? want : (1 << 20));
    return launch_kernel(true, k_copy_pages<CAP>, dim3(grid), dim3(CP_WARPS * 32), 0, s, pp, data, pool_stride,
                         n_pools, page_bytes, segs, units);
}

// HB_OK, or what is wrong with the page pairs (text to *why).
int check_pairs(const int32_t *src, const int32_t *dst, int n, int num_blocks, const char **why)
{
    for (int i = 0; i < n; ++i)
        if (src[i] < 0 || src[i] >= num_blocks || dst[i] < 0 || dst[i] >= num_blocks) {
            *why = "a page lies outside the pool";
            return HB_ERANGE;
        }
    try {
        std::vector<int32_t> to(dst, dst + n);
        std::sort(to.begin(), to.end());
        bool bad = std::adjacent_find(to.begin(), to.end()) != to.end();
        for (int i = 0; i < n && !bad; ++i)
            bad = std::binary_search(to.begin(), to.end(), src[i]);
        if (bad) {
            *why = "a destination page is repeated, or is also a source";
            return HB_EINVAL;
        }
    } catch (...) {
        *why = "no host memory";
        return HB_ENOMEM;
    }
    return HB_OK;
}

cudaError_t copy_pages(uint8_t *data, long long pool_stride, int n_pools, long long page_bytes, const int32_t *src,
                       const int32_t *dst, int n, cudaStream_t s, int *launches)
{
    constexpr int SMALL = 32, LARGE = 1500;  // 256 and 12000 bytes of parameters
    for (int i = 0; i < n; i += LARGE) {
        const int m = n - i < LARGE ? n - i : LARGE;
        const cudaError_t e = m <= SMALL
                                  ? launch_copy<SMALL>(src + i, dst + i, m, data, pool_stride, n_pools, page_bytes, s)
                                  : launch_copy<LARGE>(src + i, dst + i, m, data, pool_stride, n_pools, page_bytes, s);
        ++*launches;
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace
}  // namespace hb

using namespace hb;

extern "C" int hb_copy_pages(void *data, long long pool_stride, int n_pools, long long page_bytes, int num_blocks,
                             const int32_t *src, const int32_t *dst, int n, void *cuda_stream)
try {
    if (!data || n < 0 || n_pools < 1 || num_blocks < 1 || page_bytes < 16 || page_bytes % 16 || pool_stride % 16 ||
        (uintptr_t)data % 16 || (n > 0 && (!src || !dst)))
        return HB_EINVAL;
    // no pool is larger than the address space, and none overlaps the next
    if (page_bytes > MAX_BYTES / num_blocks ||
        (n_pools > 1 && (pool_stride < page_bytes * num_blocks || pool_stride > MAX_BYTES / n_pools)))
        return HB_EINVAL;
    const char *why = nullptr;
    const int rc = check_pairs(src, dst, n, num_blocks, &why);
    if (rc)
        return rc;
    int launches = 0;
    return copy_pages((uint8_t *)data, pool_stride, n_pools, page_bytes, src, dst, n, (cudaStream_t)cuda_stream,
                      &launches) == cudaSuccess
               ? HB_OK
               : HB_ECUDA;
} catch (...) {
    return HB_ENOMEM;
}

extern "C" int hb_copy_blocks(hb_ctx *ctx, const int32_t *src, const int32_t *dst, int n)
try {
    if (!ctx)
        return HB_EINVAL;
    if (n < 0 || (n > 0 && (!src || !dst)))
        return ctx->set_error(HB_EINVAL, "hb_copy_blocks: n < 0 or a NULL pointer");
    const hb_model_config &c = ctx->cfg;
    const char *why = nullptr;
    const int rc = check_pairs(src, dst, n, c.num_blocks, &why);
    if (rc)
        return ctx->set_error(rc, "hb_copy_blocks: %s", why);
    int launches = 0;
    const cudaError_t e = copy_pages((uint8_t *)ctx->kv, (long long)(ctx->kv_elems_per_pool * sizeof(bf16)),
                                     2 * c.n_layers, (long long)c.n_kv_heads * 16 * c.head_dim * sizeof(bf16), src,
                                     dst, n, ctx->stream, &launches);
    ctx->n_launches += launches;
    if (e != cudaSuccess)
        return ctx->set_error(HB_ECUDA, "hb_copy_blocks: %s", cudaGetErrorString(e));
    return HB_OK;
} catch (...) {
    return HB_ENOMEM;
}
