// kv4_chunk.cu -- a prefill chunk's attention over the 4-bit paged cache on
// the tcgen05 tensor cores.
//
//   S = Q K^T,  P = 2^(S c - m),  O += P V,  o = O / sum P
//
// For one kv head the chunk's (row, head) pairs are the columns of an item,
// 128 or 256 at a time; an item's keys come in tiles of 128.  A CTA works
// through (item, key tile) units that follow one another; an item that several
// CTAs share leaves fp32 partials, which a second kernel joins.
//
//   warps 0..7    softmax, one thread per query: S from tensor memory, P back
//                 into it as f16, at most 2^15; O is rescaled only when a
//                 maximum has risen by more than 2^4 (RAISE)
//   warps 8..19   three groups of four, a group a sub-tile of 64 keys, a warp a
//                 page: codes and scales -> f16 rows of the K and V tiles
//                 (128-byte swizzle); code x scale is exact in f16
//   warps 20, 21  issue the MMAs of the two halves of 128 columns: S, and
//                 O += P V with P read from tensor memory
//   warp 22       loader: one bulk copy per page (16 keys) into a ring
//
// S comes in sub-tiles of 64 keys, two for each half, each in tensor memory of
// its own: while one is in the softmax the tensor pipe fills the other.  With
// items of 128 columns ("dual") both halves have the same columns and take the
// sub-tiles in turn; the CTA joins their two results.  The softmax warps take
// the registers that the others do not need.
//
// What bounds it: at 512 rows over 15872 keys, 40 heads of 128 (169 GFLOP in
// 130 us, 1.3 PFLOP/s of f16), two thirds of the issue slots and 61% of the
// tensor pipe's time are taken: the softmax warps, whose exponentials and
// conversions share the schedulers with the conversion of K and V, are the
// longest way.  Small chunks (256 rows at 768 keys, 14.5 us) spend 3 us until
// the first scores and 2.5 us on the last result.  Two groups of converting
// warps in place of three: 14.7 us there, 132 above; one warp issuing for both
// halves where they share the sub-tiles: 151 in place of 139; no maximum unless
// a sum shows that one is needed: 145 in place of 128.
//
// Every wait is bounded; when one runs out, the CTA writes NaN for the rows
// it has left, drains and returns.
#include <cuda.h>
#include <cuda_runtime.h>

#include "kv4.cuh"
#include "kv4_chunk.h"
#include "kv4_host.h"
#include "tc_ptx.cuh"

namespace hb {
namespace {

using namespace kv4;
using namespace tc;

constexpr int GROUPS = 3;                // of four warps that convert sub-tiles of K and V
constexpr int MMA_WARP = 8 + 4 * GROUPS;
constexpr int THREADS = (MMA_WARP + 4) * 32;
// Of 256 and 512 threads: 61440 registers, 80 for each thread at launch.  512
// rows at 15872 keys take 2% longer with 128 and 56, 15% with 112 and 64.
constexpr int REGS_SOFTMAX = 144, REGS_OTHER = 48;
constexpr int RING = 24;                 // pages in flight
constexpr int STAGES = 3;                // sub-tiles of 64 keys of K, and of V, in f16
constexpr int STAGES_DUAL = 4;           // the same where both halves share one Q tile
constexpr float HUGE_SCORE = 1 << 20;    // up to it v sc - m may be fused: m is rounded by 2^-4 at most, for all P alike
constexpr uint64_t WAIT_NS = 2000000000ull;  // after which a wait is given up

template <int D>
struct Ck {
    static constexpr int CB = D / 64;                 // column blocks of 64 channels
    static constexpr int BLK = 128 * 128;             // one column block of a 128-row tile
    static constexpr int TILE = CB * BLK;
    static constexpr int SBLK = 64 * 128;             // the same of a 64-key sub-tile
    static constexpr int SUB = CB * SBLK;
    static constexpr int RAW = Layout<D>::BYTES;
    static constexpr int Q = 0, K = 2 * TILE, R = K + 2 * STAGES * SUB;
    static constexpr int K_DUAL = TILE;               // one Q tile less, one stage of K and of V more
    static_assert(K_DUAL + 2 * STAGES_DUAL * SUB <= R);
    static constexpr int BAR = R + RING * RAW;
    static constexpr int BYTES = BAR + 1024 + 2048 + 1024 + 1024;  // barriers, (m, l) pairs, exponents, alignment
    static constexpr uint32_t S_COL = 128, O0 = 256, O_COL = D;  // S: 64 columns for each (half, buffer)
};

// byte offset of (row, 16-byte chunk c) in a 128-byte-swizzled column block
__device__ __forceinline__ uint32_t swz(int row, int c)
{
    return (uint32_t)((row >> 3) * 1024 + (row & 7) * 128 + ((c ^ (row & 7)) << 4));
}

// MN-major operand, 128-byte swizzle: 64-element column blocks block_stride
// bytes apart, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, uint32_t block_stride)
{
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((block_stride >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

// f16 A and B, fp32 D, A K-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn)
{
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Four k-steps of D (+)= A B, both operands in shared memory: a and b advance
// by 32 bytes a step.  One elected lane issues.
__device__ __forceinline__ void mma_ss4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n"
        ".reg .pred p, t, e;\n"
        ".reg .b64 a1, a2, a3, b1, b2, b3;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "setp.eq.b32 t, 0, 0;\n"
        "add.s64 a1, %1, 2;\n"
        "add.s64 b1, %2, 2;\n"
        "add.s64 a2, %1, 4;\n"
        "add.s64 b2, %2, 4;\n"
        "add.s64 a3, %1, 6;\n"
        "add.s64 b3, %2, 6;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n"
        "}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Four k-steps of D (+)= A B with A in tensor memory (8 columns a step) and B
// MN-major in shared memory (16 rows of 128 bytes a step).
__device__ __forceinline__ void mma_ts4(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n"
        ".reg .pred p, t, e;\n"
        ".reg .b64 b1, b2, b3;\n"
        ".reg .b32 a1, a2, a3;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "setp.eq.b32 t, 0, 0;\n"
        "add.s32 a1, %1, 8;\n"
        "add.s64 b1, %2, 128;\n"
        "add.s32 a2, %1, 16;\n"
        "add.s64 b2, %2, 256;\n"
        "add.s32 a3, %1, 24;\n"
        "add.s64 b3, %2, 384;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n"
        "}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, float (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
          "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
          "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, float (&r)[16])
{
    tmem_ld_32x32b_x16(taddr, reinterpret_cast<uint32_t(&)[16]>(r));
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ------------------------------------------------------------------- work

// Key tiles of item qt.
__host__ __device__ inline int item_tiles(const Kv4Chunk &p, int qt)
{
    const long long last = (long long)(qt + 1) * p.rows < p.cols ? (long long)(qt + 1) * p.rows : p.cols;
    return (p.offset + (int)((last - 1) / p.group)) / KC_KEYS + 1;
}

// The segments of a CTA: the parts of items in its range, in order.
struct Segments {
    int left;         // units of the range still to come
    int kvh, qt, kt0, kt1, n_tiles;
    bool first;       // the segment starts with the range

    __device__ Segments(const Kv4Chunk &p, int cta)
    {
        const KcStart s = p.start[cta];
        kvh = s.kvh;
        qt = s.qt;
        kt0 = s.kt0;
        left = s.units;
        first = true;
        size(p);
    }
    __device__ void size(const Kv4Chunk &p)
    {
        n_tiles = item_tiles(p, qt);
        kt1 = min(n_tiles, kt0 + left);
    }
    __device__ bool more() const { return left > 0; }
    __device__ void next(const Kv4Chunk &p)
    {
        left -= kt1 - kt0;
        kt0 = 0;
        first = false;
        if (++qt == p.n_qt) {
            qt = 0;
            ++kvh;
        }
        if (left > 0)
            size(p);
    }
    // 64-key sub-tiles: of the segment, and of half h: all of them, or (both
    // halves on the same columns) every other one
    __device__ int subs() const { return 2 * (kt1 - kt0); }
    __device__ int subs_of(const Kv4Chunk &p, int h) const
    {
        if (p.rows == 128)
            return kt1 - kt0;
        return h == 0 || p.cols - (long long)qt * KC_ROWS > 128 ? subs() : 0;
    }
    // keys that the item's last column sees
    __device__ int keys(const Kv4Chunk &p) const
    {
        const long long last = min((long long)(qt + 1) * p.rows, (long long)p.cols) - 1;
        return p.offset + (int)(last / p.group) + 1;
    }
};

// A place in a ring of n stages: the stage, and the parity of its full barrier.
struct Place {
    uint32_t st = 0, ph = 0;
    __device__ __forceinline__ void next(uint32_t n)
    {
        if (++st == n) {
            st = 0;
            ph ^= 1u;
        }
    }
};

// ---------------------------------------------------------------- dequant

// The largest of eight bf16 magnitudes, as bits (above 0x7f80 with a NaN).
__device__ __forceinline__ uint32_t largest_bits(uint4 u)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[0]));
#pragma unroll
    for (int i = 1; i < 4; ++i)
        m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i])));
    const uint32_t b = *reinterpret_cast<const uint32_t *>(&m);
    return max(b & 0xffffu, b >> 16);
}

// K of one page into rows row0.. (a multiple of 16) of a tile.  Lane 4 g + t:
// tokens tok and tok + 8, channels 4t..4t+3 of every block.  The four chunks
// that a lane writes in a row lie at four lane constants; everything else is
// an immediate.  A half-warp's 8-byte stores go to four rows whose swizzles
// differ (tokens 0, 2, 4, 6 or 1, 3, 5, 7): no bank conflict.
template <int D>
__device__ __forceinline__ void page_k(const uint8_t *raw, uint8_t *tile, int row0, int lane)
{
    using L = Layout<D>;
    constexpr int KW = L::NB / 2;
    const int g = lane >> 2, t = lane & 3, tok = ((g & 3) << 1) | (g >> 2);
    uint8_t *base = tile + row0 * 128 + tok * 128 + 8 * (t & 1);
    uint8_t *at[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        at[k] = base + (((2 * k + (t >> 1)) ^ tok) << 4);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        uint32_t w[KW], sb[L::NB / 4];
        load_words<KW>(raw + L::k_code(tok + 8 * r, t, 0), w);
#pragma unroll
        for (int i = 0; i < L::NB / 4; ++i)
            sb[i] = *reinterpret_cast<const uint32_t *>(raw + L::k_scale(tok + 8 * r, 4 * i));
#pragma unroll
        for (int i = 0; i < KW; ++i) {  // blocks 2i, 2i + 1
            uint32_t a[4];
            from_e2m1x8(w[i], a);
            const uint32_t two = from_e4m3x2(sb[i / 2] >> (16 * (i & 1)));
            const int off = (i / 2) * Ck<D>::SBLK + r * 1024;
            *reinterpret_cast<uint2 *>(at[2 * (i & 1)] + off) = make_uint2(mul_lo(a[0], two), mul_lo(a[1], two));
            *reinterpret_cast<uint2 *>(at[2 * (i & 1) + 1] + off) = make_uint2(mul_hi(a[2], two), mul_hi(a[3], two));
        }
    }
}

// V of one page.  Lane 4 g + t: channels 2g, 2g + 1 of every block, tokens
// 4t..4t+3, two at a time in an order that keeps the four t on different
// banks of the swizzle.  NaN scales become 0 when scrub is set (what they
// hide is found again at the end of the segment).
template <int D>
__device__ __forceinline__ void page_v(const uint8_t *raw, uint8_t *tile, int row0, int lane, bool scrub)
{
    using L = Layout<D>;
    constexpr int KW = L::NB / 2;
    const int g = lane >> 2, t = lane & 3;
    const int h0 = t >> 1;  // lanes of the upper tokens start with the other two
    // token 4t + 2h + u is row 4t + 2h + u: 8-row group t / 2, row 4 (t & 1) + 2h + u in it
    uint8_t *base = tile + row0 * 128 + (t >> 1) * 1024 + (t & 1) * 512 + 4 * (g & 3);
    const int r4 = 4 * (t & 1) + 2 * h0;
    uint8_t *at[2][4];  // [u][j]: chunk 2j + g / 4 of row 4t + 2 h0 + u
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            at[u][j] = base + (((2 * j + (g >> 2)) ^ (r4 + u)) << 4) + u * 128;
    uint32_t sb[L::NB];
#pragma unroll
    for (int i = 0; i < L::NB; ++i) {
        sb[i] = *reinterpret_cast<const uint32_t *>(raw + L::v_scale(4 * t, i));
        if (scrub)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if ((sb[i] >> (8 * k) & 0x7fu) == 0x7fu)
                    sb[i] &= ~(0xffu << (8 * k));
        if (h0)
            sb[i] = __byte_perm(sb[i], 0, 0x1032);  // the two tokens taken first in the low half
    }
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        const int h = h0 ^ hh;
        uint32_t w[KW];
        load_words<KW>(raw + L::v_code(4 * t + 2 * h, g, 0), w);
#pragma unroll
        for (int i4 = 0; i4 < L::NB / 4; ++i4) {
            uint32_t a[2][4];
            from_e2m1x8(w[i4], a[0]);
            from_e2m1x8(w[KW / 2 + i4], a[1]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t two = from_e4m3x2(hh ? sb[4 * i4 + j] >> 16 : sb[4 * i4 + j]);
                // the other two rows have chunk c where these have c ^ 2
                const int off = i4 * Ck<D>::SBLK + h * 256;
                *reinterpret_cast<uint32_t *>(at[0][j ^ hh] + off) = mul_lo(a[0][j], two);
                *reinterpret_cast<uint32_t *>(at[1][j ^ hh] + off) = mul_hi(a[1][j], two);
            }
        }
    }
}

// The rare page with NaN scales, kept out of the way of the others' code.
template <int D>
__device__ __noinline__ void page_v_scrub(const uint8_t *raw, uint8_t *tile, int row0, int lane)
{
    page_v<D>(raw, tile, row0, lane, true);
}

// Channel blocks of kv head kvh whose V is NaN at some key in [k0, k1): slow,
// run only when the CTA met a NaN scale.
template <int D>
__device__ __noinline__ uint32_t nan_blocks(const Kv4Chunk &p, int kvh, int k0, int k1)
{
    using L = Layout<D>;
    uint32_t m = 0;
    for (int key = k0; key < k1; ++key) {
        const int blk = p.table[key >> 4];
        if (blk < 0 || blk >= p.num_blocks)
            continue;
        const uint8_t *page = p.pool + ((size_t)blk * p.n_kv + kvh) * L::BYTES;
        for (int i = 0; i < L::NB; ++i)
            if ((page[L::v_scale(key & 15, i)] & 0x7f) == 0x7f)
                m |= 1u << i;
    }
    return m;
}

// 32 bytes to one place: at once where it is the start of a sector.
__device__ __forceinline__ void store_sector(bf16 *at, uint4 a, uint4 b, bool aligned)
{
    if (aligned) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(a.x), "r"(a.y), "r"(a.z),
                     "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(at)[0] = a;
        reinterpret_cast<uint4 *>(at)[1] = b;
    }
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1) k_kv4_chunk(const __grid_constant__ Kv4Chunk p)
{
    using C = Ck<D>;
    using L = Layout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // not by a cast, which would lose that it is shared memory
    uint64_t *raw_full = (uint64_t *)(smem + C::BAR);
    uint64_t *raw_empty = raw_full + RING;
    uint64_t *k_full = raw_empty + RING, *k_empty = k_full + STAGES_DUAL, *v_full = k_empty + STAGES_DUAL;
    uint64_t *v_empty = v_full + STAGES_DUAL, *s_full = v_empty + STAGES_DUAL, *p_full = s_full + 4, *pv_done = p_full + 4;  // [half][sub-tile]
    uint64_t *q_full = pv_done + 4, *drain = q_full + 2;                          // [half]
    uint32_t *tmem_slot = (uint32_t *)(drain + 2);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);
    volatile int *bad_key = abort_flag + 1;   // lowest key met whose page lies outside the pool
    volatile int *nan_seen = bad_key + 1;     // a NaN scale of V was met

    float2 *ml_x = (float2 *)(smem + C::BAR + 1024);  // [half][128]: m and l for the other half
    int *s_exp = (int *)(ml_x + 256);                 // [half][128]: by what power of two a row of Q was scaled down

    const bool dual = p.rows == 128;
    const uint32_t stages = dual ? STAGES_DUAL : STAGES;
    uint8_t *sK = smem + (dual ? C::K_DUAL : C::K), *sV = sK + stages * C::SUB;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < RING; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], 1);
        }
        for (int i = 0; i < STAGES_DUAL; ++i) {
            mbar_init(&k_full[i], 4);
            mbar_init(&k_empty[i], dual ? 1 : 2);
            mbar_init(&v_full[i], 4);
            mbar_init(&v_empty[i], dual ? 1 : 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 4);
            mbar_init(&drain[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&pv_done[i], 1);
        }
        *abort_flag = 0;
        *bad_key = 0x7fffffff;
        *nan_seen = 0;
        fence_mbar_init();
    }
    if (warp == MMA_WARP)
        tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;  // all 512 columns: they begin at 0
    Segments sg(p, blockIdx.x);
    pdl_wait();
    pdl_trigger();

    bool ok = true;
    // A whole warp's wait, short of code: the roles together have to stay in
    // the instruction caches.  Plain looks, each as long as the hardware cares
    // to make it (they hardly ever come to a second one), without a time to
    // sleep: with one for the converting warps alone 148 us in place of 140,
    // for all 158 (512 rows at 15872).  The votes tell the compiler that the
    // warp stays together, so that addresses and descriptors are kept in
    // uniform registers (154 us without).
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        uint32_t looks = 0;
        uint64_t since = 0;
#pragma unroll 1
        while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
            bool over = *abort_flag;
            if ((++looks & 63u) == 0) {
                const uint64_t now = globaltimer_ns();
                since = since ? since : now;
                over |= now - since > WAIT_NS;
            }
            if (__any_sync(0xffffffffu, over)) {
                *abort_flag = 1;
                return ok = false;
            }
        }
        return ok;
    };

    if (warp < 8) {
        // -------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
        const int half = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t sT = lanes + half * C::S_COL, oT = lanes + C::O0 + half * C::O_COL;
        uint32_t n = 0;  // sub-tiles this half has been through
        for (; sg.more(); sg.next(p)) {
            const int own = sg.subs_of(p, half);
            const int col0 = sg.qt * p.rows + (dual ? 0 : half * 128);
            const int valid = min(128, p.cols - col0);  // columns of this half (<= 0 if it has none)
            const int col = min(col0 + r, p.cols - 1);
            const int row = col / p.group, head = sg.kvh * p.group + (col - row * p.group);
            const int seen = p.offset + row + 1;
            uint8_t *q = smem + C::Q + (dual ? 0 : half * C::TILE);
            int *exps = s_exp + (dual ? 0 : half * 128);
            constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes a row, rows a warp-wide access
            const int lr = lane / LPR, lc = lane % LPR;
            if (own > 0) {
                // this warp's 32 rows of Q as f16, or 16 of them where the
                // other half has the same (past the last column, that column's
                // again: their results go nowhere).  Rows of ordinary size go
                // as they are (components below 2^-17 lose bits: an error of
                // 2^-25, at most 2^-19 of the row's largest); if any of a batch
                // has its largest magnitude outside [2^-6, 2^15), each is
                // scaled by a power of two into [1, 2) first
                const long long src = row * p.q_stride + (size_t)head * D;
                constexpr int N = 16 / RPI;  // 16 rows a batch, the next one's loads under way meanwhile
                const int i0 = dual ? half * 16 : 0, i1 = dual ? i0 + 16 : 32;
                auto load = [&](int i) {
                    return __ldg(reinterpret_cast<const uint4 *>(p.q + __shfl_sync(0xffffffffu, src, i + lr)) + lc);
                };
                auto put = [&](uint4 x, int i, float down) {
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[j]));
                        o[j] = pack_h2(f.x * down, f.y * down);
                    }
                    *reinterpret_cast<uint4 *>(q + (lc >> 3) * C::BLK + swz((warp & 3) * 32 + i + lr, lc & 7)) =
                        make_uint4(o[0], o[1], o[2], o[3]);
                };
                uint4 u[N];
#pragma unroll
                for (int k = 0; k < N; ++k)
                    u[k] = load(i0 + k * RPI);
#pragma unroll 1
                for (int i = i0; i < i1; i += N * RPI) {
                    uint4 next[N];
                    if (i + N * RPI < i1)
#pragma unroll
                        for (int k = 0; k < N; ++k)
                            next[k] = load(i + (N + k) * RPI);
                    // bit k: some lane of the k-th row has a value of 2^-6 or
                    // more; bit 16 + k: has one that is not 0
                    uint32_t bits = 0, top = 0;
#pragma unroll
                    for (int k = 0; k < N; ++k) {
                        const uint32_t a = largest_bits(u[k]);
                        top = max(top, a);
                        bits |= (a >= 0x3c80u ? 1u << k : 0u) | (a != 0u ? 0x10000u << k : 0u);
                    }
#pragma unroll
                    for (int x = 1; x < LPR; x *= 2)
                        bits |= __shfl_xor_sync(0xffffffffu, bits, x);
                    const bool plain = top < 0x4700u && (bits & 0xffffu) == bits >> 16;
                    if (__all_sync(0xffffffffu, plain)) {
#pragma unroll
                        for (int k = 0; k < N; ++k)
                            put(u[k], i + k * RPI, 1.f);
                        if (lane < N * RPI)
                            exps[(warp & 3) * 32 + i + lane] = 0;
                    } else {
#pragma unroll 1
                        for (int k = 0; k < N; ++k) {
                            const uint4 x = load(i + k * RPI);
                            uint32_t a = largest_bits(x);
#pragma unroll
                            for (int y = 1; y < LPR; y *= 2)
                                a = max(a, __shfl_xor_sync(0xffffffffu, a, y));
                            const int e = query_exponent(__uint_as_float(a << 16));
                            put(x, i + k * RPI, pow2(-e));
                            if (lc == 0)
                                exps[(warp & 3) * 32 + i + k * RPI + lr] = e;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        u[k] = next[k];
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&q_full[half]);
            } else if (!dual) {
                continue;
            }
            if (dual)  // half of this warp's exponents are the other half's
                asm volatile("bar.sync 1, 256;" ::: "memory");
            // never 0: a masked score stays -inf
            const float sc = fminf(fmaxf(p.ks * (rsqrtf((float)D) * LOG2E) * pow2(exps[r]), 1e-38f), LARGEST_SCALE);
            const int seen0 = p.offset + col0 / p.group + 1;  // of the half's first column
            float m = LOWEST, l = 0.f;
            float raise_at = LOWEST;  // a maximum above it moves m
            bool fresh = true;  // no O yet
#pragma unroll 1
            for (int i = 0; i < own; ++i, ++n) {
                const uint32_t buf = n & 1u;
                if (!wait(&s_full[2 * half + buf], (n >> 1) & 1u))
                    break;
                tc_fence_after();
                const int key = sg.kt0 * KC_KEYS + (dual ? 2 * i + half : i) * 64;
                const int lim = seen - key;          // keys of the 64 this row sees
                const bool edge = seen0 < key + 64;  // some row does not see them all
                float v[2][32];
                tmem_ld_x32(sT + buf * 64, v[0]);
                tmem_ld_x32(sT + buf * 64 + 32, v[1]);
                tmem_ld_wait();
                if (edge)
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        v[0][j] = j < lim ? v[0][j] : -INFINITY;
                        v[1][j] = 32 + j < lim ? v[1][j] : -INFINITY;
                    }
                float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    x[j & 3] = fmaxf(fmaxf(x[j & 3], v[0][j]), v[1][j]);
                const float mx = __fmul_rn(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), sc);
                float by = sc, off = -m;  // P = 2^(v by + off)
                if (__any_sync(0xffffffffu, mx > raise_at)) {
                    const float mn = fmaxf(m, __fadd_ru(mx, -LIFT)), corr = ex2(m - mn);
                    m = mn;
                    l *= corr;
                    raise_at = __fadd_rd(m, LIFT + RAISE);
                    off = -m;
                    if (fabsf(m) > HUGE_SCORE) {
                        // the product rounded as m was, then m off; and here again with every sub-tile
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            v[0][j] = __fmul_rn(v[0][j], sc) - m;
                            v[1][j] = __fmul_rn(v[1][j], sc) - m;
                        }
                        by = 1.f;
                        off = 0.f;
                        raise_at = -INFINITY;
                    }
                    if (!fresh) {  // O holds the products before this one: let the last of them end
                        if (!wait(&pv_done[2 * half + (buf ^ 1u)], ((n - 1) >> 1) & 1u))
                            break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            float y[16];
                            tmem_ld_x16(oT + c, y);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                y[j] *= corr;
                            tmem_st_x16(oT + c, reinterpret_cast<uint32_t(&)[16]>(y));
                        }
                    }
                }
                fresh = false;
                const uint64_t sc2 = pack_f2(by, by), m2 = pack_f2(off, off);
                uint64_t sum2[2] = {0, 0};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t ph[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float a, b;
                        unpack_f2(fma_f2(pack_f2(v[k][2 * j], v[k][2 * j + 1]), sc2, m2), a, b);
                        a = ex2(a);
                        b = ex2(b);
                        sum2[j & 1] = add_f2(sum2[j & 1], pack_f2(a, b));
                        ph[j] = pack_h2(a, b);
                    }
                    tmem_st_x16(sT + buf * 64 + k * 16, ph);  // over S, which is read already
                }
                float a, b;
                unpack_f2(add_f2(sum2[0], sum2[1]), a, b);
                l += a + b;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&p_full[2 * half + buf]);
            }
            // ---- the segment's result
            if (ok && own > 0 && wait(&pv_done[2 * half + ((n - 1) & 1u)], ((n - 1) >> 1) & 1u))
                tc_fence_after();
            // with both halves on the same columns, each takes half of the
            // channels and joins the two O there: f, f2 are their factors
            float f = 1.f, f2 = 0.f;
            const int c0 = dual ? half * (D / 2) : 0, c1 = dual ? c0 + D / 2 : D;
            if (dual) {
                ml_x[half * 128 + r] = make_float2(m, l);
                tc_fence_before();
                asm volatile("bar.sync 1, 256;" ::: "memory");
                tc_fence_after();
                const float2 o = ml_x[(half ^ 1) * 128 + r];
                const float M = fmaxf(m, o.x);
                f = ex2(m - M);
                f2 = ex2(o.x - M);
                l = l * f + o.y * f2;
                m = M;
                if (half == 1) {  // f belongs to the first half's O, f2 to the second's
                    const float x = f;
                    f = f2;
                    f2 = x;
                }
                ok = ok && !__any_sync(0xffffffffu, *abort_flag);
            }
            uint32_t nans = 0;
            if (*nan_seen)  // after the barrier above: the other half's tiles count too
                nans = nan_blocks<D>(p, sg.kvh, sg.kt0 * KC_KEYS, min(seen, sg.kt1 * KC_KEYS));
            __syncwarp();
            if (!ok || *bad_key < seen) {  // one table serves every item, so the key found in any of them counts
                l = __int_as_float(0x7fc00000);
                m = 0.f;
            }
            const bool whole_sectors = ((uintptr_t)p.out | (uintptr_t)(2 * p.out_stride)) % 32 == 0;
            const bool whole = sg.kt0 == 0 && sg.kt1 == sg.n_tiles;
            const size_t part = (size_t)blockIdx.x * 2 + (sg.first ? 0 : 1);
            const int pr = (dual ? 0 : half * 128) + r;  // row of the item's partial
            const float inv = p.vs / l;
            const long long dst = row * p.out_stride + (size_t)head * D;
            const uint32_t oA = dual ? lanes + C::O0 : oT, oB = lanes + C::O0 + C::O_COL;
#pragma unroll 1
            for (int c = c0; c < c1; c += 32) {
                float v[32];
                if (ok) {
                    float y[32];
                    tmem_ld_x32(oA + c, v);
                    if (dual)
                        tmem_ld_x32(oB + c, y);
                    tmem_ld_wait();
                    if (dual)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] = v[j] * f + y[j] * f2;
                } else {  // l is another warp's where both halves have the same columns, and that may not know yet
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = __int_as_float(0x7fc00000);
                }
                if (nans >> (c / 16) & 3u)
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (nans >> (c / 16 + j / 16) & 1u)
                            v[j] = __int_as_float(0x7fc00000);
                if (whole) {
                    if (r < valid)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float x[2][8];
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                x[j / 8][j % 8] = v[16 * k + j] * inv;
                            store_sector(p.out + dst + c + 16 * k, pack8_bf16(x[0]), pack8_bf16(x[1]), whole_sectors);
                        }
                } else if (r < valid) {
                    float4 *po = reinterpret_cast<float4 *>(p.part_o) + (part * (D / 4) + c / 4) * KC_ROWS + pr;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        po[k * KC_ROWS] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                }
                __syncwarp();
            }
            if (!whole && r < valid && (!dual || half == 0)) {
                p.part_ml[part * KC_ROWS + pr] = make_float2(m, l);
            }
            tc_fence_before();  // the next segment's MMAs overwrite O
            if (dual)           // and both halves have read both
                asm volatile("bar.sync 1, 256;" ::: "memory");
        }
    } else if (warp < MMA_WARP) {
        // -------------------------------------------------------- dequant
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
        // each group of four warps takes every third sub-tile, a warp a page
        const int sub = (warp - 8) >> 2, pg = (warp - 8) & 3;
        uint32_t j = sub, base = 0;  // sub-tiles since the start: this group's next, and the segment's first
        Place at;
        for (int i = 0; i < sub; ++i)
            at.next(stages);
        for (; sg.more() && ok; base += 2 * (sg.kt1 - sg.kt0), sg.next(p)) {
            const int keys = sg.keys(p);
            for (; j < base + 2 * (sg.kt1 - sg.kt0) && ok; j += GROUPS) {
                const uint32_t n = j * 4 + pg, slot = n % RING;  // pages since the start
                const uint8_t *raw = smem + C::R + slot * C::RAW;
                if ((j >= stages && !wait(&k_empty[at.st], at.ph ^ 1u)) || !wait(&raw_full[slot], (n / RING) & 1u))
                    break;
                page_k<D>(raw, sK + at.st * C::SUB, pg * 16, lane);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&k_full[at.st]);
                if (j >= stages && !wait(&v_empty[at.st], at.ph ^ 1u))
                    break;
                // NaN scales: four scale bytes a lane (half of the lanes for d = 64)
                const uint32_t sb = lane < D / 4 ? *reinterpret_cast<const uint32_t *>(raw + L::VS + 4 * lane) : 0u;
                uint8_t *V = sV + at.st * C::SUB;
                if (__any_sync(0xffffffffu, (((sb & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0u)) {
                    if (sg.kt0 * KC_KEYS + (int)(j - base) * 64 + pg * 16 < keys)
                        *nan_seen = 1;  // or a slot past the last key: the search will tell
                    page_v_scrub<D>(raw, V, pg * 16, lane);
                    __threadfence_block();
                } else {
                    page_v<D>(raw, V, pg * 16, lane, false);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&raw_empty[slot]);
                    mbar_arrive(&v_full[at.st]);
                }
#pragma unroll
                for (int i = 0; i < GROUPS; ++i)
                    at.next(stages);
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
        if (warp == MMA_WARP || (warp == MMA_WARP + 1 && !dual)) {
            // ---------------------------------------------------- MMA issue
            // a warp for each half; where the halves take the sub-tiles in
            // turn, one for both, so that the stages are let go in order
            const int h = warp - MMA_WARP;
            const uint32_t id_s = idesc_f16(128, 64, false), id_o = idesc_f16(128, D, true);
            const uint64_t dQ = sdesc_kmajor_sw128(smem_u32(smem + C::Q) + (dual ? 0 : h * C::TILE));
            const uint64_t dK = sdesc_kmajor_sw128(smem_u32(sK)), dV = sdesc_mn(smem_u32(sV), C::SBLK);
            const uint32_t turn = dual ? 1 : 0, ahead = 2u << turn;  // S is two sub-tiles of a half ahead of O
            Place k, v;
            uint32_t n_s = 0, n_o = 0, n_q = 0;  // S and O products, and segments with rows for this warp
            auto half_of = [&](uint32_t n) { return dual ? n & 1u : (uint32_t)h; };
            auto slot_of = [&](uint32_t n) { return 2 * half_of(n) + (n >> turn & 1u); };  // half and buffer
            auto issue_s = [&]() {  // S of the sub-tile at k
                const uint32_t slot = slot_of(n_s++);
#pragma unroll
                for (int cb = 0; cb < C::CB; ++cb)
                    mma_ss4(slot * 64, dQ + cb * (C::BLK >> 4), dK + k.st * (C::SUB >> 4) + cb * (C::SBLK >> 4), id_s, cb);
                mma_commit_elect(&s_full[slot]);
                mma_commit_elect(&k_empty[k.st]);
                k.next(stages);
            };
            for (; sg.more() && ok; sg.next(p)) {
                const uint32_t subs = sg.subs();
                if (sg.subs_of(p, h) == 0) {  // the other half's alone: let each stage go as soon as it is filled
                    for (uint32_t t = 0; t < subs && ok; ++t) {
                        if (wait(&k_full[k.st], k.ph) && lane == 0)
                            mbar_arrive(&k_empty[k.st]);
                        if (wait(&v_full[v.st], v.ph) && lane == 0)
                            mbar_arrive(&v_empty[v.st]);
                        k.next(stages);
                        v.next(stages);
                    }
                    continue;
                }
                wait(&q_full[dual ? lane & 1 : h], n_q++ & 1u);
#pragma unroll 1
                for (uint32_t t = 0; t < min(ahead, subs) && ok; ++t) {
                    wait(&k_full[k.st], k.ph);
                    tc_fence_after();
                    issue_s();
                }
#pragma unroll 1
                for (uint32_t t = 0; t < subs && ok; ++t) {
                    // lanes look at several barriers at once: P and V of this
                    // sub-tile, and K of the one whose S comes next
                    const uint32_t slot = slot_of(n_o);
                    uint64_t *bar = &p_full[slot];
                    uint32_t ph = n_o >> (1 + turn) & 1u;
                    if (lane == 1)
                        bar = &v_full[v.st], ph = v.ph;
                    if (lane == 2 && t + ahead < subs)
                        bar = &k_full[k.st], ph = k.ph;
                    if (!wait(bar, ph))
                        break;
                    tc_fence_after();
                    mma_ts4(C::O0 + half_of(n_o) * C::O_COL, slot * 64, dV + v.st * (C::SUB >> 4), id_o, t >> turn);
                    mma_commit_elect(&pv_done[slot]);
                    mma_commit_elect(&v_empty[v.st]);
                    v.next(stages);
                    ++n_o;
                    if (t + ahead < subs)
                        issue_s();
                }
            }
            // no product may be under way, and no arrival, when the CTA ends:
            // the other roles may have given up before this warp's last ones
            mma_commit_elect(&drain[h]);
            mbar_wait(&drain[h], 0, nullptr, WAIT_NS / 4);
        } else if (warp == MMA_WARP + 2) {
            // ---------------------------------------------------- loader
            uint32_t it = 0;
            for (; sg.more() && ok; sg.next(p)) {
                const int keys = sg.keys(p);
                for (int kt = sg.kt0; kt < sg.kt1; ++kt, ++it) {
                    const int pg = kt * 8 + (lane & 7);
                    const uint32_t n = it * 8 + (lane & 7), slot = n % RING;
                    const bool need = lane < 8 && pg * 16 < keys;
                    const int blk = need ? __ldg(p.table + pg) : 0;
                    const bool in = need && blk >= 0 && blk < p.num_blocks;
                    if (need && !in)
                        atomicMin((int *)bad_key, pg * 16);
                    bool got = true;
                    if (lane < 8 && n >= RING)
                        got = mbar_sleep(&raw_empty[slot], (n / RING - 1) & 1u, abort_flag);
                    if (!__all_sync(0xffffffffu, got)) {
                        *abort_flag = 1;
                        ok = false;
                        break;
                    }
                    if (lane < 8 && !(p.lose && blockIdx.x == 0 && n == 0)) {
                        if (in) {
                            mbar_expect_tx(&raw_full[slot], C::RAW);
                            bulk_load(smem + C::R + slot * C::RAW, p.pool + ((size_t)blk * p.n_kv + sg.kvh) * C::RAW,
                                      C::RAW, &raw_full[slot]);
                        } else {
                            mbar_arrive(&raw_full[slot]);  // past the keys or outside the pool: what the slot holds is masked
                        }
                    }
                }
            }
            // no copy may land after the CTA has ended: the last RING pages
            const uint32_t pages = it * 8;
            for (uint32_t n = pages > RING ? pages - RING : 0; n < pages; ++n)
                mbar_wait(&raw_full[n % RING], (n / RING) & 1u, nullptr, ok ? WAIT_NS : WAIT_NS / 8);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the partials of an item, in the order of its keys: 32 columns and 32
// channels a block, four parts at a time.  Block x belongs to the item that
// CTA x + 1 begins inside, unless CTA x did so too (then an earlier block has
// it).  Bound by the partials' traffic: 30 MB for 512 rows at 15872 keys, some
// 7 us of 130.
template <int D>
__global__ void __launch_bounds__(256, 6) k_kv4_chunk_join(const __grid_constant__ Kv4Chunk p)
{
    constexpr int BATCH = 4;
    __shared__ __align__(16) bf16 s_o[32][32 + 8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ca = blockIdx.x;
    const KcStart a = p.start[ca], item = p.start[ca + 1];
    const bool same = a.kvh == item.kvh && a.qt == item.qt;
    pdl_wait();
    pdl_trigger();
    if (item.kt0 == 0 || (same && a.kt0 > 0))
        return;
    int cb = ca + 1;  // the last CTA with a part of the item
    while (cb + 1 < p.ctas && p.start[cb + 1].kvh == item.kvh && p.start[cb + 1].qt == item.qt)
        ++cb;
    // of the CTAs only ca can have come to the item from another one
    const int first = 2 * ca + (same ? 0 : 1);
    const int r = blockIdx.y * 32 + lane;  // this lane's column of the item
    const int valid = (int)min((long long)p.rows, p.cols - (long long)item.qt * p.rows);
    if (blockIdx.y * 32 >= valid)
        return;
    const float2 *ml = p.part_ml + r;
    const float4 *po = reinterpret_cast<const float4 *>(p.part_o) + (size_t)(blockIdx.z * 8 + warp) * KC_ROWS + r;
    float M = LOWEST, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < valid)
        for (int c0 = ca; c0 <= cb; c0 += BATCH) {
            float2 x[BATCH];
            float4 v[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int c = c0 + i;
                const size_t part = c == ca ? first : 2 * c;
                x[i] = make_float2(LOWEST, 0.f);
                v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c <= cb) {
                    x[i] = ml[part * KC_ROWS];
                    v[i] = po[part * (D / 4) * KC_ROWS];
                }
            }
            float top = M;
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                top = fmaxf(top, x[i].x);
            const float corr = ex2(M - top);
            M = top;
            l *= corr;
            o.x *= corr, o.y *= corr, o.z *= corr, o.w *= corr;
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const float f = ex2(x[i].x - M);
                l += x[i].y * f;
                o.x += v[i].x * f, o.y += v[i].y * f, o.z += v[i].z * f, o.w += v[i].w * f;
            }
        }
    const float inv = p.vs / l;
    __nv_bfloat162 *s = reinterpret_cast<__nv_bfloat162 *>(&s_o[lane][warp * 4]);
    s[0] = __floats2bfloat162_rn(o.x * inv, o.y * inv);
    s[1] = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    __syncthreads();
    const int rr = threadIdx.x >> 2, ch = threadIdx.x & 3;
    if (rr < 32 && blockIdx.y * 32 + rr < valid) {
        const int col = item.qt * p.rows + blockIdx.y * 32 + rr;
        const int row = col / p.group, head = item.kvh * p.group + col - row * p.group;
        *reinterpret_cast<uint4 *>(p.out + row * p.out_stride + (size_t)head * D + blockIdx.z * 32 + ch * 8) =
            *reinterpret_cast<const uint4 *>(&s_o[rr][ch * 8]);
    }
}

template <int D>
cudaError_t launch_d(const Kv4Chunk &p, cudaStream_t s)
{
    static std::atomic<uint64_t> done{0};
    cudaError_t e = kv4_allow_smem((const void *)k_kv4_chunk<D>, Ck<D>::BYTES, done);
    if (e != cudaSuccess)
        return e;
    e = launch_kernel(true, k_kv4_chunk<D>, dim3(p.ctas), dim3(THREADS), Ck<D>::BYTES, s, p);
    if (e != cudaSuccess)
        return e;
    if (kv4_chunk_workspace_bytes(p, D) == 0)
        return cudaSuccess;
    return launch_kernel(true, k_kv4_chunk_join<D>, dim3(p.ctas - 1, p.rows / 32, D / 32), dim3(256), 0, s, p);
}

}  // namespace

// How the work of a chunk may be cut, and about how long each way takes: fits
// of measured times, 0.82 to 1.21 of them over 216 shapes.
//
//   parts  an item to one CTA, or to several that share its tiles evenly
//   whole  more items than CTAs: each takes some that follow one another
//   even   every CTA the same load, wherever that ends: most even, but each CTA
//          may leave two partials of 256 x d fp32, written and read at some
//          2.5 MB a microsecond
//
// A load is key tiles, and for each item the tiles' worth of a change of items
// (the queries, the pipeline's start and end, the result).  Items of 256
// columns convert each key once for both halves; items of 128 (both halves on
// them) make twice as many.  With 40 heads of 128, 512 rows at offset 0 take
// 14.6 us as whole items and 17.8 cut evenly, 256 rows at 768 keys 14.3 and
// 18.7; 512 rows at 15872 keys 129 us cut evenly, 1.9 CTAs an item, and 208 as
// whole items, or 164 cut into items of 128.
namespace {

constexpr double SWITCH_US = 5, JOIN_US = 2, PART_US = 0.25, BYTES_PER_US = 2.5e6;
constexpr int MAX_UNITS = 1 << 28;  // of a CTA: the kernel counts pages, eight a unit, in 32 bits
constexpr int MANY_ITEMS = 640;  // from here on an even cut loses little, and a search would cost the host

enum Way { PARTS, WHOLE, EVEN };
struct Cut {
    int rows;
    Way way;
    long long tiles;  // PARTS: of a CTA at most; WHOLE: its load
    double us;
};

// A launch and an item's start and end; a key tile; the tiles' worth of a change of items.
double start_us(int d) { return d == 64 ? 4.5 : 5.5; }
double tile_us(int rows, int d) { return rows == 256 ? (d == 64 ? 1.5 : 1.65) : (d == 64 ? 0.8 : 1.05); }
int change_tiles(int rows, int d) { return (int)(SWITCH_US / tile_us(rows, d)) + 1; }

// Cuts of items of p.rows columns: takes over any that beats best.
void try_cuts(const Kv4Chunk &p, int d, Cut &best)
{
    const double start = start_us(d), tile = tile_us(p.rows, d);
    const int change = change_tiles(p.rows, d);
    const long long items = (long long)p.n_qt * p.n_kv;
    const double part_us = (p.cols < p.rows ? p.cols : p.rows) * (4.0 * d + 8) / BYTES_PER_US;
    auto take = [&](Way way, long long tiles, double us) {
        if (us < best.us)
            best = Cut{p.rows, way, tiles, us};
    };
    const long long ctas = p.units < KC_CTAS ? p.units : KC_CTAS, load = p.units + items * change;
    const double shared = items < ctas ? ctas + items : 2 * ctas;
    take(EVEN, 0, start + (double)load / ctas * tile + shared * part_us + JOIN_US + PART_US * ctas / items);
    if (items > MANY_ITEMS)
        return;
    int n[MANY_ITEMS];
    for (int qt = 0; qt < p.n_qt; ++qt)
        n[qt] = item_tiles(p, qt);
    const int most = n[p.n_qt - 1];
    if (items <= KC_CTAS) {
        for (int k = 1; k <= most; ++k) {  // CTAs of the longest item
            const int tiles = (most + k - 1) / k;
            long long used = 0, parts = 0;
            for (int qt = 0; qt < p.n_qt; ++qt) {
                const int share = (n[qt] + tiles - 1) / tiles;
                used += share;
                parts += share > 1 ? share : 0;
            }
            if (used * p.n_kv > KC_CTAS)
                break;
            take(PARTS, tiles,
                 start + tiles * tile + (parts ? parts * p.n_kv * part_us + JOIN_US + PART_US * k : 0));
        }
    } else {
        // the least load for which the CTAs suffice, to one part in 32
        long long lo = load / KC_CTAS, hi = lo + most + change;
        while (hi - lo > 1 + lo / 32) {
            const long long mid = (lo + hi) / 2;
            long long sum = 0, used = 1;
            for (int kvh = 0; kvh < p.n_kv; ++kvh)
                for (int qt = 0; qt < p.n_qt; ++qt) {
                    if (sum > 0 && sum + n[qt] + change > mid) {
                        ++used;
                        sum = 0;
                    }
                    sum += n[qt] + change;
                }
            (used <= KC_CTAS && most + change <= mid ? hi : lo) = mid;
        }
        take(WHOLE, hi, start + (hi - change) * tile);
    }
}

void count_units(Kv4Chunk &p, int rows)
{
    p.rows = rows;
    p.n_qt = (p.cols + rows - 1) / rows;
    p.units = 0;
    for (int qt = 0; qt < p.n_qt; ++qt)
        p.units += item_tiles(p, qt);
    p.units *= p.n_kv;
}

}  // namespace

bool kv4_chunk_plan(Kv4Chunk &p, int chunk_len, int d)
{
    p.cols = chunk_len * p.group;
    Cut cut{256, EVEN, 0, 1e300};
    count_units(p, 256);
    try_cuts(p, d, cut);
    if (p.units <= 16ll * KC_CTAS) {  // beyond, 256 columns are always better
        count_units(p, 128);
        try_cuts(p, d, cut);
    }
    if (p.rows != cut.rows)
        count_units(p, cut.rows);
    p.us = cut.us;
    p.shared = false;
    p.ctas = 0;
    bool fits = true;
    auto add = [&](int kvh, int qt, int kt0, long long units) {
        fits &= units < MAX_UNITS;
        p.start[p.ctas++] = KcStart{kvh, qt, kt0, (int)units};
        p.shared |= kt0 > 0;
    };
    const int change = change_tiles(p.rows, d);
    if (cut.way == EVEN) {
        const long long ctas = p.units < KC_CTAS ? p.units : KC_CTAS;
        const long long all = p.units + (long long)p.n_qt * p.n_kv * change;
        // the item at hand: its load begins at `from`, its units at `before`
        long long from = 0, before = 0, at = 0;
        int kvh = 0, qt = 0, n = item_tiles(p, 0);
        int at_kvh = 0, at_qt = 0, at_kt = 0;  // where unit `at` lies
        for (long long c = 1; c <= ctas; ++c) {
            const long long to = all * c / ctas;
            while (c < ctas && from + change + n <= to) {
                from += change + n;
                before += n;
                if (++qt == p.n_qt) {
                    qt = 0;
                    ++kvh;
                }
                n = item_tiles(p, qt);
            }
            const int kt = c < ctas && to > from + change ? (int)(to - from - change) : 0;
            const long long next = c < ctas ? before + kt : p.units;
            if (next > at)
                add(at_kvh, at_qt, at_kt, next - at);
            at = next;
            at_kvh = kvh, at_qt = qt, at_kt = kt;
        }
        return fits;
    }
    long long load = 0;
    for (int kvh = 0; kvh < p.n_kv; ++kvh)
        for (int qt = 0; qt < p.n_qt; ++qt) {
            const int n = item_tiles(p, qt);
            if (cut.way == PARTS) {
                const int share = (int)((n + cut.tiles - 1) / cut.tiles);
                for (int i = 0; i < share; ++i) {
                    const int from = (int)((long long)n * i / share), to = (int)((long long)n * (i + 1) / share);
                    add(kvh, qt, from, to - from);
                }
            } else if (load == 0 || load + n + change > cut.tiles) {
                add(kvh, qt, 0, n);
                load = n + change;
            } else {
                p.start[p.ctas - 1].units += n;
                load += n + change;
            }
        }
    return fits;  // WHOLE is for a few hundred items, whose tiles a CTA can always count
}

long long kv4_chunk_workspace_bytes(const Kv4Chunk &p, int d)
{
    return p.shared ? 2ll * p.ctas * KC_ROWS * (8 + 4ll * d) : 0;
}

cudaError_t launch_kv4_chunk(const Kv4Chunk &p, int head_dim, cudaStream_t s)
{
    return head_dim == 128 ? launch_d<128>(p, s) : launch_d<64>(p, s);
}

}  // namespace hb
