// kv4.cuh -- the 4-bit paged KV cache (include/hb_cache.h): where things lie
// in a pool, and the conversions of its codes and scales.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "tc_ptx.cuh"

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

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack_f2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack_f2(uint64_t x, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma_f2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_f2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul_f2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// x times the low (high) half of s.
__device__ __forceinline__ uint32_t mul_lo(uint32_t x, uint32_t s)
{
    const __half2 r = __hmul2(*reinterpret_cast<__half2 *>(&x), __low2half2(*reinterpret_cast<__half2 *>(&s)));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t mul_hi(uint32_t x, uint32_t s)
{
    const __half2 r = __hmul2(*reinterpret_cast<__half2 *>(&x), __high2half2(*reinterpret_cast<__half2 *>(&s)));
    return *reinterpret_cast<const uint32_t *>(&r);
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

// Power of two e that brings a query whose largest magnitude is a into [1, 2)
// (0 for a = 0), and 2^e itself, e in [-126, 126].
__device__ __forceinline__ int query_exponent(float a)
{
    const int e = (int)(__float_as_uint(a) >> 23) - 127;
    return a > 0.f ? min(max(e, -126), 126) : 0;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Wait for the phase of the given parity, asleep inside try_wait (up to some 20
// us at a time), so that the issue slots are left to others.  Gives up after
// WAIT_TRIES looks, two seconds or less, or when *abort is set.
constexpr int WAIT_TRIES = 100000;
__device__ __forceinline__ bool mbar_sleep(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    const uint32_t addr = tc::smem_u32(bar);
#pragma unroll 1
    for (int i = 0; i < WAIT_TRIES; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n"
            ".reg .pred p;\n"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
            "selp.u32 %0, 1, 0, p;\n"
            "}\n"
            : "=r"(ok)
            : "r"(addr), "r"(parity), "r"(20000u)
            : "memory");
        if (ok)
            return true;
        if (abort && *abort)
            return false;
    }
    return false;
}

// 2^x to about 2 ulp (results below 2^-126 are 0).
__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LARGEST_SCALE = 3e38f;  // of scores: 0 times an infinite one (k_scale 2^60, queries of 2^70) would be NaN
constexpr float LOWEST = -3e38f;  // below every score, and finite: differences with it are too

// The weights P = 2^(s - m) go to the tensor cores in f16, as V does (an MMA
// takes one type): 11 bits, an error of 2^-12 a weight, some 2^-3 of a bf16
// result's own rounding.  Where they lie in f16's range of 2^-24 (a subnormal's
// last bit) to 2^16: the reference m is 2^LIFT below the largest
// score when it moves, and moves when a score passes it by LIFT + RAISE.  So P
// is at most 2^15, and a key of 2^-36 of the largest weight still counts; with
// the reference at the largest score, keys behind an attention sink (2^-25 of
// the largest weight) left the sum of V and stayed in the sum of P.  512 rows at
// 15872 keys take 130 us so, 135 with 13 and 2 (the reference moves oftener),
// and 130 with 8 and 7.
constexpr float LIFT = 11.f, RAISE = 4.f;

}  // namespace kv4
}  // namespace hb
