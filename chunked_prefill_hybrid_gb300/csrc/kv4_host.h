// kv4_host.h -- what the calls on the 4-bit cache share on the host.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "hb_cache.h"

namespace hb {

// HB_OK or HB_EINVAL.
int kv4_check_pool(const hb_kv4_pool *p);
// A bf16 row operand of n rows of `width` values: aligned to 16 bytes, rows
// apart by a multiple of 8 values that is at least the width.
int kv4_check_rows(const void *p, long long stride, int n, int width);

// Let a kernel have `bytes` of dynamic shared memory on the current device.
// The limit is kept for each device: done has a bit for those that have it.
inline cudaError_t kv4_allow_smem(const void *kernel, int bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_acquire) & bit)
        return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        done.fetch_or(bit, std::memory_order_release);
    return e;
}

}  // namespace hb
