// prefix_attention.cu -- attention of a group's rows to the prefix that they
// share, on the tcgen05 tensor cores (include/hb_paged.h).
//
//   S = Q K^T,  P = 2^((S - m) c2),  O += P V;  partials (m, sum P, O)
//
// Q's rows are the group's (row, head) pairs of one kv head, up to 256 of them
// in a CTA, which takes a run of the prefix's whole 16-token blocks: every row
// sees every key, so nothing is masked.  Other CTAs have other runs of the same
// keys; the join of the rows' partials follows with their own keys
// (paged_attention.cu).
//
//   warps 0..15  softmax, two threads a row: S from tensor memory, P back over
//                it in two bf16 terms (16 significant bits, as in
//                paged_attention.cu); O is rescaled only when a maximum has
//                risen by more than 2^8
//   warps 16, 17 issue the MMAs of the two halves of 128 rows
//   warps 18, 19 load sub-tiles of 64 keys of K and of V by TMA, a box per block
//                and 64 channels
//
// Two halves keep the tensor pipe busy: while one is in the softmax the other's
// products run.  A CTA of more than 128 rows has a Q tile for each half; with
// up to 128 ("dual") both have the same tile and take the sub-tiles in turn, and
// the CTA joins their two results.  S has two buffers a half.
//
// What bounds it: for up to 128 rows the stream of K and V (16 rows x 8 heads of 8
// kv heads over 130000 keys: 87 us, 0.90 of a copy's rate; 64 keys are 0.75 us of an
// SM's stream and 0.45 of its products).  For two tiles the products: a tile's S of
// 64 keys and 128 channels takes 384 cycles (Q and K come from shared memory), P V
// in two terms 512, the two in turn 875, the softmax less: 56 rows x 8 heads over
// 16384 keys 46 us, the tensor pipe 70 % busy.  Boxes of 64 keys rather than 128 let
// both halves have two buffers of S beside O in 512 columns.
//
// Every wait is bounded; when one runs out, the CTA writes NaN for its rows,
// drains and returns.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "gemm_tc.h"
#include "kv4.cuh"
#include "kv4_host.h"
#include "paged.h"
#include "tc_ptx.cuh"

namespace hb {
namespace {

using namespace paged;
using namespace tc;
using kv4::add_f2;
using kv4::ex2;
using kv4::fma_f2;
using kv4::pack_f2;
using kv4::unpack_f2;

constexpr int MMA_WARP = 16, LOAD_WARP = 18;
constexpr int THREADS = 20 * 32;
constexpr float LOWEST = -3e38f;         // below every score, and finite: differences with it are too
constexpr float RAISE = 8.f;             // in powers of two: how far a score may pass the maximum used
// Up to it P = 2^(s c2 - m c2) with one fused step a score: m c2 is rounded, by 2^-4
// at most, and the sums have that factor until m changes or they are given out.
constexpr float HUGE_SCORE = 1 << 20;
constexpr uint64_t WAIT_NS = 2000000000ull;  // after which a wait is given up

template <int D>
struct Px {
    static constexpr int CB = D / 64;               // column blocks of 64 channels
    static constexpr int QBLK = 128 * 128;          // one column block of a 128-row tile
    static constexpr int TILE = CB * QBLK;
    static constexpr int BLK = 64 * 128;            // the same of a 64-key sub-tile
    static constexpr int SUB = CB * BLK;            // K or V of a sub-tile
    // of V, one more than of K, which is let go earlier
    static constexpr int STAGES = D == 128 ? 5 : 10, STAGES_DUAL = D == 128 ? 6 : 11;
    static constexpr int BAR = (2 * TILE + (2 * STAGES - 1) * SUB) > (TILE + (2 * STAGES_DUAL - 1) * SUB)
                                   ? 2 * TILE + (2 * STAGES - 1) * SUB
                                   : TILE + (2 * STAGES_DUAL - 1) * SUB;
    static constexpr int BYTES = BAR + 512 + 4096 + 1024;  // barriers, maxima, alignment
    static_assert(BYTES <= 227 * 1024);
    static constexpr uint32_t O0 = 256;             // S: 64 columns for each (half, buffer); then O of the halves
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

// One k-step of D (+)= A B with A (bf16) in tensor memory and B in shared
// memory; one elected lane issues.
__device__ __forceinline__ void mma_ts_elect(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n"
        ".reg .pred p, e;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
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

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// 32 bytes, a whole sector.
__device__ __forceinline__ void store8(float *to, float a, float b, float c, float d, float e, float f, float g, float h)
{
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "f"(a), "f"(b), "f"(c), "f"(d),
                 "f"(e), "f"(f), "f"(g), "f"(h)
                 : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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

template <int D, bool SCORES>
__global__ void __launch_bounds__(THREADS, 1)
    k_prefix_attention(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ Attn p)
{
    using C = Px<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    constexpr int MOST = C::STAGES_DUAL;
    uint64_t *k_full = (uint64_t *)(smem + C::BAR), *v_full = k_full + MOST, *k_empty = v_full + MOST;
    uint64_t *v_empty = k_empty + MOST, *s_full = v_empty + MOST, *p_full = s_full + 4, *pv_done = p_full + 4;  // [half][buffer]
    uint64_t *q_full = pv_done + 4, *drain = q_full + 1;                           // [half]
    uint32_t *tmem_slot = (uint32_t *)(drain + 2);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);
    volatile int *bad = abort_flag + 1;  // a block outside the pool was met
    static_assert((4 * MOST + 15) * 8 + 12 <= 512);
    float *s_max = (float *)(smem + C::BAR + 512);  // [buffer][half][sub][128]

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    // ---- this CTA's group (or sequence), kv head, rows and keys
    Group gr;
    int local, table;
    if (SCORES) {
        pdl_wait();
        const int each = (int)gridDim.x / p.n_seqs;
        table = (int)blockIdx.x / each;
        local = (int)blockIdx.x % each;
        const int ctx = p.ctx_lens[table];
        gr = p.sequence(table, ctx < 0 || ctx > p.max_ctx ? -1 : ctx);
        if (local % p.seq_parts >= gr.parts) {
            pdl_trigger();
            return;  // the join knows how many parts a sequence has
        }
    } else {
        if (p.groups)
            pdl_wait();  // a kernel before this one puts them there
        int gi = 0, hi = p.n_groups - 1;  // the last group that starts at or before this CTA
        while (gi < hi) {
            const int mid = (gi + hi + 1) >> 1;
            if (p.at(mid).cta0 <= (int)blockIdx.x)
                gi = mid;
            else
                hi = mid - 1;
        }
        gr = p.at(gi);
        local = (int)blockIdx.x - gr.cta0;
        table = gr.row0;
    }
    const int parts = SCORES ? p.seq_parts : gr.parts;
    const int part = local % parts, kvh = local / parts % p.n_kv, tile = local / parts / p.n_kv;
    const int c0 = tile * 256, cols = min(256, gr.rows * p.group - c0);
    const bool dual = cols <= 128;
    const uint32_t stages = dual ? C::STAGES_DUAL : C::STAGES;  // of V
    const int t0 = part * gr.part_len, subs = min((gr.shared + 63) / 64, t0 + gr.part_len) - t0;
    auto blocks_of = [&](int t) { return min(4, (gr.shared >> 4) - (t0 + t) * 4); };  // of sub-tile t
    uint8_t *sK = smem + (dual ? C::TILE : 2 * C::TILE), *sV = sK + (stages - 1) * C::SUB;

    if (threadIdx.x == 0) {
        for (int i = 0; i < (int)stages; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&k_empty[i], dual ? 1 : 2);
            mbar_init(&v_empty[i], dual ? 1 : 2);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 8);
            mbar_init(&pv_done[i], 1);
        }
        mbar_init(q_full, 16);
        mbar_init(&drain[0], 1);
        mbar_init(&drain[1], 1);
        *abort_flag = 0;
        *bad = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (warp == MMA_WARP)
        tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;  // all 512 columns: they begin at 0
    pdl_wait();
    pdl_trigger();

    bool ok = true;
    // A whole warp's wait (the votes tell the compiler that the warp stays
    // together).
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

    if (warp < MMA_WARP) {
        // -------------------------------------------------------- softmax
        // Q: the CTA's rows of (row, head) pairs, zeros past the last
        {
            constexpr int LANES = D / 8, STEP = MMA_WARP * 32 / LANES, N = 128 / STEP;  // threads a row, rows a round
            const int ch = threadIdx.x % LANES, r0 = threadIdx.x / LANES;
#pragma unroll 1
            for (int t = 0; t < (dual ? 1 : 2); ++t) {
                uint4 v[N];
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const int c = c0 + t * 128 + r0 + k * STEP, row = c / p.group;
                    v[k] = make_uint4(0, 0, 0, 0);
                    if (c - c0 < cols)
                        v[k] = __ldg(reinterpret_cast<const uint4 *>(p.q + (long long)(gr.row0 + row) * p.q_stride +
                                                                     (size_t)(kvh * p.group + c - row * p.group) * D) +
                                     ch);
                }
#pragma unroll
                for (int k = 0; k < N; ++k)
                    *reinterpret_cast<uint4 *>(smem + t * C::TILE + (ch >> 3) * C::QBLK + swz(r0 + k * STEP, ch & 7)) = v[k];
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0)
            mbar_arrive(q_full);

        // two threads a row, each with 32 of a sub-tile's 64 keys
        const int half = warp >> 3, sub = (warp >> 2) & 1, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t sT = lanes + half * 128, oT = lanes + C::O0 + half * D;
        const int own = dual ? (subs + 1 - half) / 2 : subs;  // sub-tiles of this half
        const int valid = min(128, cols - (dual ? 0 : half * 128));
        const bool idle = (warp & 3) * 32 >= valid;  // no row in this warp
        float *my_max = s_max + (half * 2 + sub) * 128 + r, *its_max = s_max + (half * 2 + (sub ^ 1)) * 128 + r;
        auto pair_sync = [&]() {  // the two warps of 32 rows
            asm volatile("bar.sync %0, 64;" ::"r"(2 + half * 4 + (warp & 3)) : "memory");
        };
        float m = LOWEST, l = 0.f;
        float raise_at = LOWEST;  // a maximum above it moves m
        // P = 2^(s c2 + offset(m)), or of the difference where that is huge; sums of it
        // times 2^residue(m) are those of 2^((s - m) c2)
        auto offset = [&](float max) { return __fmul_rn(-max, p.c2); };
        auto residue = [&](float max) {
            const float off = offset(max);
            return fabsf(off) > HUGE_SCORE ? 0.f : __fmaf_rn(-max, p.c2, -off);
        };
        float *score_at = nullptr;
        if (SCORES)
            score_at = p.scores + (((size_t)table * p.n_kv + kvh) * (gr.rows * p.group) + c0 + (dual ? 0 : half * 128) + r) *
                                      p.score_stride + sub * 32;
#pragma unroll 1
        for (int i = 0; i < own; ++i) {
            const uint32_t buf = i & 1u;
            if (ok)
                wait(&s_full[2 * half + buf], (uint32_t)(i >> 1) & 1u);
            if (!ok) {  // a wait ran out: no more work, but as many barriers as the other warp of the rows
                if (!idle)
                    pair_sync();
                continue;
            }
            if (idle) {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&p_full[2 * half + buf]);
                continue;
            }
            tc_fence_after();
            float v[32];
            tmem_ld_x32(sT + buf * 64 + sub * 32, v);
            tmem_ld_wait();
            const int t = dual ? 2 * i + half : i, n = blocks_of(t) - 2 * sub;  // blocks of this thread's two
            if (SCORES) {
                float *to = score_at + (size_t)(t0 + t) * 64;
                if (r < valid)
#pragma unroll
                    for (int j = 0; j < 32; j += 8)
                        if (j / 16 < n)
                            store8(to + j, v[j], v[j + 1], v[j + 2], v[j + 3], v[j + 4], v[j + 5], v[j + 6], v[j + 7]);
            }
            if (n < 2)  // the last blocks
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    v[j] = j < n * 16 ? v[j] : -INFINITY;
            float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < 32; j += 2)
                x[(j >> 1) & 3] = fmaxf(fmaxf(x[(j >> 1) & 3], v[j]), v[j + 1]);
            float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
            my_max[buf * 512] = mx;
            pair_sync();
            mx = fmaxf(mx, its_max[buf * 512]);
            float off = offset(m);
            if (__any_sync(0xffffffffu, mx > raise_at)) {  // as the other warp finds: it has the same maxima
                const float mn = fmaxf(m, mx), corr = ex2((m - mn) * p.c2 + (residue(m) - residue(mn)));
                m = mn;
                l *= corr;
                raise_at = m + RAISE / p.c2;
                off = offset(m);
                if (fabsf(off) > HUGE_SCORE) {  // the difference first; and here again with every sub-tile
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] -= m;
                    off = 0.f;
                    raise_at = -INFINITY;
                }
                if (i > 0) {  // O holds the products before this one: let the last of them end
                    if (!wait(&pv_done[2 * half + (buf ^ 1u)], (uint32_t)((i - 1) >> 1) & 1u))
                        continue;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = sub * (D / 2); c < (sub + 1) * (D / 2); c += 16) {
                        uint32_t y[16];
                        tmem_ld_32x32b_x16(oT + c, y);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            y[j] = __float_as_uint(__uint_as_float(y[j]) * corr);
                        tmem_st_x16(oT + c, y);
                    }
                }
            }
            const uint64_t c2 = pack_f2(p.c2, p.c2), off2 = pack_f2(off, off), minus = pack_f2(-1.f, -1.f);
            uint64_t sum2[2] = {0, 0};
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                float a, b;
                unpack_f2(fma_f2(pack_f2(v[2 * j], v[2 * j + 1]), c2, off2), a, b);
                a = ex2(a);
                b = ex2(b);
                const uint64_t ab = pack_f2(a, b);
                sum2[j & 1] = add_f2(sum2[j & 1], ab);
                const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
                hi[j] = *reinterpret_cast<const uint32_t *>(&h);
                float ra, rb;
                unpack_f2(fma_f2(pack_f2(__uint_as_float(hi[j] << 16), __uint_as_float(hi[j] & 0xffff0000u)), minus, ab),
                          ra, rb);
                const __nv_bfloat162 q = __floats2bfloat162_rn(ra, rb);
                lo[j] = *reinterpret_cast<const uint32_t *>(&q);
            }
            // over S, which both warps have read: pair_sync() was after that
            tmem_st_x16(sT + buf * 64 + sub * 16, hi);
            tmem_st_x16(sT + buf * 64 + 32 + sub * 16, lo);
            float a, b;
            unpack_f2(add_f2(sum2[0], sum2[1]), a, b);
            l += a + b;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&p_full[2 * half + buf]);
        }
        // ---- the result
        if (ok && own > 0 && wait(&pv_done[2 * half + ((own - 1) & 1)], (uint32_t)((own - 1) >> 1) & 1u))
            tc_fence_after();
        // the row's other threads' m and l, through tensor memory, over this
        // half's S: its products are done
        float2 o[4];  // [half][sub]
        asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(sT + 2 * sub), "f"(m), "f"(l) : "memory");
        tmem_st_wait();
        tc_fence_before();
        if (dual)
            asm volatile("bar.sync 1, %0;" ::"n"(MMA_WARP * 32) : "memory");
        else
            pair_sync();
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t from = lanes + (dual ? k : half) * 128;
            asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];"
                         : "=f"(o[2 * k].x), "=f"(o[2 * k].y)
                         : "r"(from)
                         : "memory");
            asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];"
                         : "=f"(o[2 * k + 1].x), "=f"(o[2 * k + 1].y)
                         : "r"(from + 2)
                         : "memory");
        }
        tmem_ld_wait();
        // f, f2: factors of the two halves' sums, where both are of the same rows
        if (dual)
            m = fmaxf(o[0].x, o[2].x);
        const float f = ex2((o[0].x - m) * p.c2 + residue(o[0].x));
        const float f2 = dual ? ex2((o[2].x - m) * p.c2 + residue(o[2].x)) : 0.f;
        l = (o[0].y + o[1].y) * f;
        if (dual)
            l += (o[2].y + o[3].y) * f2;
        __syncwarp();
        ok = !__any_sync(0xffffffffu, !ok || *abort_flag);
        const int width = dual ? D / 4 : D / 2;  // channels of this thread
        const int e0 = (dual ? 2 * half + sub : sub) * width;
        const bool two = dual && subs > 1;  // the second half has an O
        const int c = c0 + (dual ? 0 : half * 128) + (r < valid ? r : 0);
        const size_t slot =
            ((size_t)(gr.row0 + c / p.group) * p.n_heads + kvh * p.group + c % p.group) * p.n_slots + part;
        if (!idle) {
            if (r < valid && e0 == 0)
                p.part_ml[slot] = make_float2(m, !ok || *bad ? __int_as_float(0x7fc00000) : l);
#pragma unroll 1
            for (int e = e0; e < e0 + width; e += 16) {
                uint32_t x[16], y[16];
                if (ok) {
                    tmem_ld_32x32b_x16((dual ? lanes + C::O0 : oT) + e, x);
                    if (two)
                        tmem_ld_32x32b_x16(lanes + C::O0 + D + e, y);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        x[j] = __float_as_uint(__uint_as_float(x[j]) * f + (two ? __uint_as_float(y[j]) * f2 : 0.f));
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        x[j] = 0;
                }
                if (r < valid)
#pragma unroll
                    for (int j = 0; j < 16; j += 8)
                        store8(p.part_o + slot * D + e + j, __uint_as_float(x[j]), __uint_as_float(x[j + 1]),
                               __uint_as_float(x[j + 2]), __uint_as_float(x[j + 3]), __uint_as_float(x[j + 4]),
                               __uint_as_float(x[j + 5]), __uint_as_float(x[j + 6]), __uint_as_float(x[j + 7]));
                __syncwarp();
            }
        }
    } else if (warp == MMA_WARP || (warp == MMA_WARP + 1 && !dual)) {
        // ---------------------------------------------------- MMA issue
        // a warp for each half; where the halves take the sub-tiles in turn,
        // one for both, so that the stages are let go in order
        const int h = warp - MMA_WARP;
        const uint32_t id_o = idesc_bf16_f32(128, D) | (1u << 16);  // V is MN-major
        const uint64_t dQ = sdesc_kmajor_sw128(smem_u32(smem) + (dual ? 0 : h * C::TILE));
        const uint64_t dK = sdesc_kmajor_sw128(smem_u32(sK)), dV = sdesc_mn(smem_u32(sV), C::BLK);
        const uint32_t turn = dual ? 1 : 0;
        const int ahead = 2 << turn;  // S is two sub-tiles of a half ahead of O
        Place k, v;
        auto half_of = [&](int t) { return dual ? (uint32_t)t & 1u : (uint32_t)h; };
        auto slot_of = [&](int t) { return 2 * half_of(t) + ((uint32_t)t >> turn & 1u); };  // half and buffer
        auto issue_s = [&](int t) {  // S of sub-tile t, which is at k
            const uint32_t slot = slot_of(t), id_s = idesc_bf16_f32(128, 0) | (uint32_t)(2 * blocks_of(t)) << 17;
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
                mma_bf16_elect(tmem + slot * 64, dQ + (j >> 2) * (C::QBLK >> 4) + (j & 3) * 2,
                               dK + k.st * (C::SUB >> 4) + (j >> 2) * (C::BLK >> 4) + (j & 3) * 2, id_s, j);
            mma_commit_elect(&s_full[slot]);
            mma_commit_elect(&k_empty[k.st]);
            k.next(stages - 1);
        };
        wait(q_full, 0);
#pragma unroll 1
        for (int t = 0; t < min(ahead, subs) && ok; ++t) {
            if (!wait(&k_full[k.st], k.ph))
                break;
            tc_fence_after();
            issue_s(t);
        }
#pragma unroll 1
        for (int t = 0; t < subs && ok; ++t) {
            // lanes look at several barriers at once: P and V of this sub-tile,
            // and K of the one whose S comes next
            const uint32_t slot = slot_of(t);
            uint64_t *bar = &p_full[slot];
            uint32_t ph = (uint32_t)t >> (1 + turn) & 1u;
            if (lane == 1)
                bar = &v_full[v.st], ph = v.ph;
            if (lane == 2 && t + ahead < subs)
                bar = &k_full[k.st], ph = k.ph;
            if (!wait(bar, ph))
                break;
            tc_fence_after();
            const int n = blocks_of(t);
            const uint32_t o = tmem + C::O0 + half_of(t) * D, pa = tmem + slot * 64;
            const uint64_t vd = dV + v.st * (C::SUB >> 4);
            if (n == 4) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    mma_ts_elect(o, pa + j * 8, vd + (j & 3) * 128, id_o, (t >> turn) | j);
            } else {
                for (int j = 0; j < n; ++j) {
                    mma_ts_elect(o, pa + j * 8, vd + j * 128, id_o, (t >> turn) | j);
                    mma_ts_elect(o, pa + 32 + j * 8, vd + j * 128, id_o, 1u);
                }
            }
            mma_commit_elect(&pv_done[slot]);
            mma_commit_elect(&v_empty[v.st]);
            v.next(stages);
            if (t + ahead < subs)
                issue_s(t + ahead);
        }
        // no product may be under way, and no arrival, when the CTA ends: the
        // other roles may have given up before this warp's last ones
        mma_commit_elect(&drain[h]);
        mbar_wait(&drain[h], 0, nullptr, WAIT_NS / 4);
    } else if (warp >= LOAD_WARP) {
        // ---------------------------------------------------- loaders
        // one warp for K and one for V, whose stages are let go at other times.
        // The whole warp stays together and one elected lane issues: a box a
        // lane took 97 us for 16 rows x 8 heads over 130000 keys of 8 kv heads, 87 so.
        const bool is_v = warp > LOAD_WARP;
        const int st = is_v ? (int)stages : (int)stages - 1;
        uint8_t *ring = is_v ? sV : sK;
        const CUtensorMap *tm = is_v ? &tm_v : &tm_k;
        uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
        const int *tab = p.tables + (size_t)table * p.bt_stride + (size_t)t0 * 4;
        const int n_blocks = (gr.shared >> 4) - t0 * 4;
        // block ids 32 at a time, eight sub-tiles' of them, the next ones under way
        auto fetch = [&](int chunk) { return chunk * 32 + lane < n_blocks ? __ldg(tab + chunk * 32 + lane) : 0; };
        int ids = fetch(0), next = fetch(1);
        Place at;
        int t = 0;
        for (; t < subs; ++t) {
            if (t > 0 && (t & 7) == 0) {
                ids = next;
                next = fetch((t >> 3) + 1);
            }
            if ((t & 7) == 0 && __any_sync(0xffffffffu, ids < 0 || ids >= p.num_blocks)) {
                *bad = 1;  // not read: the group's rows become NaN
                ids = ids < 0 || ids >= p.num_blocks ? 0 : ids;
            }
            if (t >= st && !wait(&empty[at.st], at.ph ^ 1u))
                break;
            const int n = blocks_of(t);
            mbar_expect_tx_elect(&full[at.st], (uint32_t)(n * C::CB * 2048));
            uint8_t *to = ring + at.st * C::SUB;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j >= n)
                    break;
                const int row = (int)(((long long)__shfl_sync(0xffffffffu, ids, (t & 7) * 4 + j) * p.n_kv + kvh) * 16);
#pragma unroll
                for (int cb = 0; cb < C::CB; ++cb)
                    if (!(p.lose && !is_v && blockIdx.x + t + j + cb == 0))
                        tma_load_2d_elect(to + cb * C::BLK + j * 2048, tm, &full[at.st], cb * 64, row);
            }
            at.next(st);
        }
        // no copy may land after the CTA has ended
        for (int i = max(0, t - st); i < t; ++i)
            mbar_wait(&full[i % st], (uint32_t)(i / st) & 1u, nullptr, ok ? WAIT_NS : WAIT_NS / 8);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

namespace paged {

int launch_prefix(const hb_paged_pool *pool, const Attn &p, int ctas, cudaStream_t s)
{
    static std::atomic<uint64_t> done[4];
    CUtensorMap k, v;
    if (!make_tmap_kv_pool(&k, pool->k, pool->num_blocks, pool->n_kv_heads, pool->head_dim) ||
        !make_tmap_kv_pool(&v, pool->v, pool->num_blocks, pool->n_kv_heads, pool->head_dim))
        return HB_ECUDA;
    const bool wide = pool->head_dim == 128, scores = p.n_groups == 0;
    auto kernel = scores ? (wide ? k_prefix_attention<128, true> : k_prefix_attention<64, true>)
                         : (wide ? k_prefix_attention<128, false> : k_prefix_attention<64, false>);
    const int smem = wide ? Px<128>::BYTES : Px<64>::BYTES;
    if (kv4_allow_smem((const void *)kernel, smem, done[2 * scores + wide]) != cudaSuccess)
        return HB_ECUDA;
    return launch_kernel(true, kernel, dim3((unsigned)ctas), dim3(THREADS), smem, s, k, v, p) == cudaSuccess ? HB_OK
                                                                                                             : HB_ECUDA;
}

}  // namespace paged
}  // namespace hb
