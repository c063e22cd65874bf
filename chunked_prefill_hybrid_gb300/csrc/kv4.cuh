// kv4.cuh -- the 4-bit paged KV cache (include/hb_cache.h): where things lie
// in a pool, and the conversions of its codes and scales.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace hb {
namespace kv4 {

// Byte offsets inside one (block, kv head) of 16 tokens.  The order of the
// codes is the order in which the lanes of an m16n8k16 MMA hold its A (or, of
// two n8 tiles, its B) fragment: lane 4 g + t reads its share of K for two
// tokens, and of V for four tokens, as 16-byte words (8-byte for d = 64), 32
// lanes side by side.
template <int D>
struct Layout {
    static constexpr int NB = D / 16;        // scale blocks of a token
    static constexpr int K = 0;              // [token 16][t 4][NB][2]
    static constexpr int V = 8 * D;          // [h 2][g 8][t 4][u 2][NB]
    static constexpr int KS = 16 * D;        // [token 16][NB]
    static constexpr int VS = 17 * D;        // [NB][token 16]
    static constexpr int BYTES = 18 * D;
    __host__ __device__ static constexpr int k_code(int tok, int t, int i) { return K + (tok * 4 + t) * 2 * NB + 2 * i; }
    __host__ __device__ static constexpr int v_code(int tok, int g, int i)
    {
        return V + ((((tok >> 1) & 1) * 8 + g) * 4 + (tok >> 2)) * 2 * NB + (tok & 1) * NB + i;
    }
    __host__ __device__ static constexpr int k_scale(int tok, int i) { return KS + tok * NB + i; }
    __host__ __device__ static constexpr int v_scale(int tok, int i) { return VS + i * 16 + tok; }
};

// Two fp32 to a byte of two e2m1 codes, lo in the low four bits (nearest
// even, at most 6).
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi)
{
    uint32_t r;
    asm("{\n"
        ".reg .b8 b;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n"
        "cvt.u32.u8 %0, b;\n"
        "}\n"
        : "=r"(r)
        : "f"(lo), "f"(hi));
    return r;
}

// The four bytes of w (eight e2m1 codes) as four f16 pairs, low code first.
__device__ __forceinline__ void from_e2m1x8(uint32_t w, uint32_t (&r)[4])
{
    asm("{\n"
        ".reg .b8 b0, b1, b2, b3;\n"
        "mov.b32 {b0, b1, b2, b3}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n"
        "}\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}

// fp32 to e4m3 (nearest even, at most 448; NaN to 0x7f).
__device__ __forceinline__ uint32_t to_e4m3(float x)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return r & 0xffu;
}

// Two e4m3 bytes to an f16 pair (exact).
__device__ __forceinline__ uint32_t from_e4m3x2(uint32_t two)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}

__device__ __forceinline__ float2 h2f2(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2 *>(&h)); }

}  // namespace kv4
}  // namespace hb
