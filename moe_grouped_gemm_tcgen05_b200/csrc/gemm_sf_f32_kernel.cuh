// FP8 GEMM with fp32 block scales for sm_100a.
//
//   D[m, n] = (C[m, n] +) sum_kb sfa[m, kb] sfb[n', kb] P_kb[m, n],
//   P_kb[m, n] = sum over the 128 values k of block kb of A[m, k] B[n, k]
//
// with n' = n / 128 (one scale per 128x128 block of B) or n (one per 1x128
// block of each row). The block-scaled MMA takes power-of-two (UE8M0) scales
// only, so fp32 scales are applied outside it: every 128-K block is multiplied
// without scales into a TMEM buffer of its own (kind::f8f6f4, fp32
// accumulation inside the block), read back with tcgen05.ld and added to fp32
// accumulators in registers with one FMA per element. Only D is rounded.
//
// What bounds it. A 128 x 128 product of one K-block is 4 MMAs of 64 clocks; the
// epilogue's reads and FMAs take as long again next to them (8 warps: ~35 clocks
// to read 64 columns each, ~130 to add them), and the hand-off of a product from
// the MMAs to the epilogue and back ~280 clocks of latency in every warp
// that takes part. The two meet at ~480 clocks a block, against 256 for the MMAs
// alone. What that taught (clocks and times measured on one B200, 4096x7168x16384):
//   - Next to one-wide FMAs the warp that issues MMAs starves: it shares its
//     scheduler with FMAs that fill every issue slot, and 4 MMAs of N = 256 take
//     890 clocks instead of 512. Two-wide FMAs leave every other slot free.
//   - One warp issues 4 MMAs and a commit in ~300 clocks there, and waits for
//     ~200; two warps take turns (647 -> 548 us with everything else equal).
//   - Wider tiles (256 columns: two TMEM buffers) wait for the hand-off of
//     a buffer, narrower ones do not: four buffers of 128 columns fit.
//   - A warp's sums are all that its loop carries from block to block. Reading
//     16 columns ahead across blocks cost ~200 clocks of register moves a block.
//   - Scales loaded by the epilogue's warps themselves, even blocks ahead, held
//     them up for ~300 clocks a block: a warp of its own brings them to shared
//     memory (532 -> 505 us).
//   - Two sets of warps that take every other block with all columns, and swap
//     halves at the end, need 64 KB for the swap and leave too few stages in
//     flight: 580 us.
//   - 16 epilogue warps of 32 columns overlap more but hand a buffer back by twice
//     as many arrivals (503 us on pairs against 467); products handed over two
//     blocks at a time halve the waits and gain nothing (465 on pairs, 500 against
//     480 on single CTAs, where three double stages are too few). The clock falls
//     under the power limit (~1.5 GHz) as the pipes fill up, which eats such gains.
// Measured as it stands (graph of calls, rotating operands): 4096x7168x16384 459-475
// us on pairs (2.0-2.1 PFLOP/s), 468-505 on single CTAs; 4096x4096x7168 113-119 and
// 118-125 us; one row by 4096x7168 11.3 us; 2112x7168x4096 with a bf16 D, an fp32 D,
// and C with an fp32 D 66, 73 and 88 us, with per-row scales 101, 120 and 135-139 (the
// products of two scales per element and block are half of the FMA pipe's work then).
//
// CTA = 12 warps (three warpgroups), one CTA per SM, persistent:
//   warp 0      TMA producer (128-byte swizzle, STAGES-deep ring)
//   warps 1, 2  MMA issue, every other product each; warp 1 allocates TMEM
//   warp 3      scale producer
//   warps 4..   epilogue. Warp w reads TMEM lanes 32 (w % 4) .. + 31 (a row per
//               lane) and owns half of the tile's columns, whose sums stay in its
//               registers over the whole K loop.
// The first warpgroup gives registers to the other two (88 + 2 x 208 of the
// launch's 3 x 168 per lane).
//
// CG = 2 (dense): a cluster of two CTAs computes 256 x 128 (tcgen05 cta_group::2),
// which takes B's loads from 16 to 8 KB a block and SM; the L2 feeds an SM about
// 77 bytes per clock, so a lone CTA's 32 KB take ~425 clocks. No load is multicast.
//
// Split-K (dense, small M): the CTAs of a cluster take K ranges of one tile,
// leave their fp32 partials in their own shared memory (the operand ring, idle
// by then) and add each others' in split order through distributed shared
// memory: no workspace, identical bits on every call.
//
// Scheduling, masks and bounded waits are those of gemm_kernel.cuh.
#pragma once

#include <type_traits>

#include "gemm_kernel.cuh"

namespace dg {

struct SfF32Params : GemmParams {
    const float* sfa32;   // [rows, kb]
    const float* sfb32;   // [groups, nb_sf, kb]
    int sfa_vec4, sfb_vec4;  // 16-byte reads of scale rows: kb % 4 == 0 on 16-byte aligned bases
    int a_box_rows;       // rows of A that a stage's load brings (128, fewer when M is small)
};

// D[tmem] (+)= A[smem] * B[smem]^T for 8-bit operands without scales (kind::f8f6f4, K = 32).
template <int CG>
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
}

// Instruction descriptor of kind::f8f6f4: E4M3 x E4M3 -> F32, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t m, uint32_t n) {
    return (1u << 4)             // D format F32
         | ((n >> 3) << 17)      // N >> 3
         | ((m >> 4) << 24);     // M >> 4
}

// Columns of TMEM (32 lanes x N, N a multiple of 32) into registers, and the
// wait for them; naming the registers keeps their uses behind the wait.
template <int N>
__device__ __forceinline__ void tmem_read(uint32_t taddr, uint32_t (&r)[N]) {
    static_assert(N % 32 == 0, "32 columns at a time");
#pragma unroll
    for (int h = 0; h < N; h += 32) tmem_ld_32x32b_x32(taddr + h, r + h);
}
template <int N>
__device__ __forceinline__ void tmem_read_done(uint32_t (&r)[N]) {
    tc_wait_ld();
#pragma unroll
    for (int h = 0; h < N; h += 16)
        asm volatile("" : "+r"(r[h]), "+r"(r[h + 1]), "+r"(r[h + 2]), "+r"(r[h + 3]), "+r"(r[h + 4]), "+r"(r[h + 5]),
                          "+r"(r[h + 6]), "+r"(r[h + 7]), "+r"(r[h + 8]), "+r"(r[h + 9]), "+r"(r[h + 10]),
                          "+r"(r[h + 11]), "+r"(r[h + 12]), "+r"(r[h + 13]), "+r"(r[h + 14]), "+r"(r[h + 15]));
}

// 16 TMEM lanes x 64 columns into registers, in pairs of columns: register 4 j + 2 u + v of
// lane l holds row 8 u + l / 4, column 8 j + 2 (l % 4) + v.
__device__ __forceinline__ void tmem_ld_16x256b_x8(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
          "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
          "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
          "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
          "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// Scale loads that stay where they are written: left to itself the compiler moves
// them down to their use, a group of blocks later.
__device__ __forceinline__ float ld_scale(const float* p) {
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ void ld_scale4(const float* p, float (&v)[4]) {
    asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "l"(p));
}

__device__ __forceinline__ void mbar_arrive_addr(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_addr(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
template <int CG>
__device__ __forceinline__ void tc_commit_addr(uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
            ::"r"(bar), "h"(static_cast<uint16_t>(0x3)) : "memory");
}

// wait_warp whose first probe is all that a ready barrier costs: the epilogue and
// the MMA warps wait twice per K-block.
__device__ __forceinline__ bool wait_block(uint64_t* bar, uint32_t parity, const GemmParams& p, volatile int* s_abort) {
    if (__builtin_expect(__all_sync(0xffffffffu, mbar_try_wait(bar, parity)) != 0, 1)) return true;
    return wait_warp(bar, parity, p, s_abort);
}

// Registers of the calling warpgroup from here on (per thread).
template <int N>
__device__ __forceinline__ void registers_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Two FMAs in one instruction: a += x * f. It takes the FMA pipe for two cycles
// and the issue slot for one. That matters more than its own speed: with
// one-wide FMAs the epilogue's warps fill the issue slots of their scheduler, and
// the MMA warp that shares it issues a block's MMAs in ~890 clocks instead of
// 512 (microbenchmark, N = 256).
__device__ __forceinline__ void fma2(float& a0, float& a1, float x0, float x1, float f0, float f1) {
    asm("{\n\t.reg .b64 a, x, f;\n\t"
        "mov.b64 a, {%0, %1};\n\t"
        "mov.b64 x, {%2, %3};\n\t"
        "mov.b64 f, {%4, %5};\n\t"
        "fma.rn.f32x2 a, x, f, a;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a0), "+f"(a1) : "f"(x0), "f"(x1), "f"(f0), "f"(f1));
}
__device__ __forceinline__ void mul2(float& y0, float& y1, float x0, float x1, float f0, float f1) {
    asm("{\n\t.reg .b64 y, x, f;\n\t"
        "mov.b64 x, {%2, %3};\n\t"
        "mov.b64 f, {%4, %5};\n\t"
        "mul.rn.f32x2 y, x, f;\n\t"
        "mov.b64 {%0, %1}, y;\n\t}"
        : "=f"(y0), "=f"(y1) : "f"(x0), "f"(x1), "f"(f0), "f"(f1));
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

constexpr int SF_F32_THREADS = 384;
constexpr int SF_F32_ISSUERS = 2;                     // warps that issue MMAs (warps 1 and 2)
constexpr int SF_F32_EPI_WARP0 = 4;                   // first epilogue warp
constexpr int SF_F32_BN = 128;                        // columns of a tile
constexpr int SF_F32_LAUNCH_REGS = 168, SF_F32_EPI_REGS = 208, SF_F32_OTHER_REGS = 88;
static_assert(SF_F32_OTHER_REGS + 2 * SF_F32_EPI_REGS <= 3 * SF_F32_LAUNCH_REGS, "registers of the launch");

// ROWB: B is scaled per row (sfb_gran_n = 1). EPI: D is bf16 (0), fp32 (1), or C is
// added, of D's type (2). (One kernel for all three lost 10% and more in its main
// loop, even where C was not read: its registers are assigned with C's in mind.
// D's rows stored by bulk copies from staging, too, took 96 us instead of 88 with C,
// and 78 instead of 73 without: those copies queue with the operands'.)
template <int CG, int SCHED_INTS, bool ROWB, int EPI>
struct SfF32Config {
    static constexpr int BN = SF_F32_BN;
    static constexpr int EW = 8;                      // epilogue warps
    static constexpr int CW = BN / 2;                 // columns of an epilogue warp
    static constexpr int B_ROWS = BN / CG;            // rows of B in this CTA's shared memory
    static constexpr int A_BYTES = BM * BK;
    static constexpr int B_BYTES = B_ROWS * BK;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int NBUF = 512 / BN;             // TMEM buffers of a block product
    // output staging: 32 rows of 64 bytes per epilogue warp, rows 80 bytes apart (no bank
    // conflicts). With C the whole of the warp's columns, whose C comes in while the
    // K loop runs (a stage or two of the ring less).
    static constexpr int STG_ROW = EPI == 2 ? CW * 4 + 16 : 80;
    static constexpr int STG_BYTES = EW * 32 * STG_ROW;
    // scales of four K-blocks per slot: [4][128 rows] (times B's, when that is one
    // per 128 columns), and with ROWB [4][BN columns]
    static constexpr int SF_SLOTS = !ROWB ? 2 : EPI == 2 ? 3 : 4;
    static constexpr int SF_SLOT_FLOATS = 4 * BM + (ROWB ? 4 * BN : 0);
    static constexpr int SF_BYTES = SF_SLOTS * SF_SLOT_FLOATS * 4;
    static constexpr int SCHED_BYTES = SCHED_INTS * 4;
    static constexpr int FIXED_BYTES = 1024 /*align slack*/ + STG_BYTES + SF_BYTES + 512 /*barriers*/ + SCHED_BYTES;
    static constexpr int STAGES_FIT = (SMEM_LIMIT - FIXED_BYTES) / STAGE_BYTES;
    static constexpr int STAGES = STAGES_FIT > 8 ? 8 : STAGES_FIT;
    static_assert(STAGES >= NBUF, "a stage's barrier completes again only after its product's buffer was handed back");
    static constexpr int SMEM_BYTES = FIXED_BYTES + STAGES * STAGE_BYTES;
    static_assert(SMEM_BYTES <= SMEM_LIMIT, "shared memory of a CTA");
    static constexpr uint32_t IDESC = idesc_e4m3_f32(BM * CG, BN);
    // split-K: a partial tile of fp32 rows, four floats of padding per row
    static constexpr int PART_ROW = BN + 4;
    static_assert(BM * PART_ROW * 4 <= STAGES * STAGE_BYTES, "the partial tile fits the idle ring");
};

// The 128-row share of D that an epilogue warp writes: 32 rows from `row0` of
// D, bit r of `rows` set where row r may be written.
struct StoreRows {
    size_t row0;
    uint32_t rows;
};

// `bytes` (a multiple of 16, on 16-byte boundaries) to shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

// Where a lane's sums are in its warp's 32 rows x CW columns. One scale of B for
// all columns: lane = row, sum i = column i. Per-row scales of B: sum
// 32 h + 4 j + 2 u + v is row 16 h + 8 u + lane / 4, column 8 j + 2 (lane % 4) + v, so
// that a lane needs 4 scales of A and 16 of B a block instead of 1 and 64. (Read as
// 16-byte broadcasts, those 64 keep the path from shared memory busy for 512 clocks
// a block and SM: 2112x7168x4096 with a bf16 D took 116-127 us, with this layout 101.)

// CW columns of a warp's 32 rows, from registers to D through the warp's staging rows, 64 bytes of every row at a time: written back, four
// lanes take the 64 bytes of a row. (Row-wise 16-byte stores straight from the
// registers touch 32 rows per instruction and slow the operand loads.)
template <int CW, int STG_ROW, int EPI, bool ROWB>
__device__ __forceinline__ void store_rows(const GemmParams& p, const float (&acc)[CW], const StoreRows& to,
                                           int col0, uint8_t* stg, int lane) {
    const int sub = lane >> 2, piece = lane & 3;
    if constexpr (EPI == 0) {
#pragma unroll
        for (int u = 0; u < CW; u += 32) {
            __syncwarp();
            if constexpr (ROWB) {
#pragma unroll
                for (int i = 0; i < 32; i += 2) {  // i = 16 h + 4 j + 2 u of these 32 columns
                    const int h = i >> 4, j = (i >> 2) & 3, a = 32 * h + u / 2 + 4 * j + (i & 2);
                    *reinterpret_cast<__nv_bfloat162*>(stg + (16 * h + 4 * (i & 2) + sub) * STG_ROW + 16 * j + 4 * piece) =
                        __floats2bfloat162_rn(acc[a], acc[a + 1]);
                }
            }
#pragma unroll
            for (int q = 0; !ROWB && q < 4; ++q) {  // 16-byte pieces of eight bf16 columns
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(acc[u + 8 * q + 2 * i], acc[u + 8 * q + 2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&b);
                }
                *reinterpret_cast<uint4*>(stg + lane * STG_ROW + 16 * q) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
            const int col = col0 + u + 8 * piece;  // N % 8 == 0: a piece is wholly inside or outside D
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 8 * i + sub;
                if (col < p.n && ((to.rows >> r) & 1u))
                    *reinterpret_cast<uint4*>(p.d + (to.row0 + r) * p.n + col) =
                        *reinterpret_cast<const uint4*>(stg + r * STG_ROW + 16 * piece);
            }
        }
    } else {
        // 16 fp32 columns at a time. C's part of the tile is in staging already, 4 (bf16: 2)
        // bytes a column; 16 columns of it go to registers and sums take their place (bf16:
        // stand behind the row's C).
#pragma unroll
        for (int u = 0; u < CW; u += 16) {
            float4 c[4];
            uint8_t* part = stg;
            if constexpr (EPI == 2) {
                if (p.out_f32) {
                    part += 4 * u;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        c[i] = *reinterpret_cast<const float4*>(part + (8 * i + sub) * STG_ROW + 16 * piece);
                } else {
                    part += 2 * CW;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint2 x = *reinterpret_cast<const uint2*>(stg + (8 * i + sub) * STG_ROW + 2 * u + 8 * piece);
                        c[i] = make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xFFFF0000u),
                                           __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xFFFF0000u));
                    }
                }
            }
            __syncwarp();
            if constexpr (ROWB) {
#pragma unroll
                for (int i = 0; i < 16; i += 2) {  // i = 8 h + 4 j + 2 u of these 16 columns
                    const int h = i >> 3, j = (i >> 2) & 1, a = 32 * h + u / 2 + 4 * j + (i & 2);
                    *reinterpret_cast<float2*>(part + (16 * h + 4 * (i & 2) + sub) * STG_ROW + 32 * j + 8 * piece) =
                        make_float2(acc[a], acc[a + 1]);
                }
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<float4*>(part + lane * STG_ROW + 16 * q) =
                        make_float4(acc[u + 4 * q], acc[u + 4 * q + 1], acc[u + 4 * q + 2], acc[u + 4 * q + 3]);
            }
            __syncwarp();
            const int col = col0 + u + 4 * piece;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 8 * i + sub;
                if (col >= p.n || !((to.rows >> r) & 1u)) continue;
                const size_t at = (to.row0 + r) * p.n + col;
                float4 v = *reinterpret_cast<const float4*>(part + r * STG_ROW + 16 * piece);
                if constexpr (EPI == 2) {
                    v.x += c[i].x;
                    v.y += c[i].y;
                    v.z += c[i].z;
                    v.w += c[i].w;
                }
                if (EPI == 1 || p.out_f32) {
                    *reinterpret_cast<float4*>(p.d32 + at) = v;
                } else {
                    const __nv_bfloat162 b0 = __floats2bfloat162_rn(v.x, v.y), b1 = __floats2bfloat162_rn(v.z, v.w);
                    *reinterpret_cast<uint2*>(p.d + at) = make_uint2(*reinterpret_cast<const uint32_t*>(&b0),
                                                                     *reinterpret_cast<const uint32_t*>(&b1));
                }
            }
        }
    }
}

template <int KIND, int CG, bool ROWB, int EPI>
__global__ void __launch_bounds__(SF_F32_THREADS, 1) fp8_gemm_sf_f32_kernel(const __grid_constant__ SfF32Params p) {
    static_assert(CG == 1 || KIND == kDense, "CTA pairs are built for the dense form");
    static_assert((!ROWB && EPI == 0) || KIND == kDense, "per-row scales of B, C and an fp32 D: dense form");
    using Cfg = SfF32Config<CG, sched_ints<KIND>(), ROWB, EPI>;
    constexpr int BN = Cfg::BN;
    constexpr int CW = Cfg::CW;
    constexpr int NBUF = Cfg::NBUF;
    constexpr int STAGES = Cfg::STAGES;
    constexpr bool kCanSplit = KIND == kDense && CG == 1;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* smem_a = smem;
    uint8_t* smem_b = smem_a + STAGES * Cfg::A_BYTES;
    uint8_t* smem_stg = smem_b + STAGES * Cfg::B_BYTES;
    float* smem_sf = reinterpret_cast<float*>(smem_stg + Cfg::STG_BYTES);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem_stg + Cfg::STG_BYTES + Cfg::SF_BYTES);
    uint64_t* full_bar = bars;                   // A/B bytes landed (the leader's counts both CTAs)
    uint64_t* done_bar = full_bar + STAGES;      // block product ready; its stage is read
    uint64_t* tempty_bar = done_bar + STAGES;    // TMEM buffer read back
    uint64_t* sfull_bar = tempty_bar + NBUF;     // scales of four K-blocks are in shared memory
    uint64_t* sempty_bar = sfull_bar + Cfg::SF_SLOTS;   // ... and used by every epilogue warp
    uint64_t* drain_bar = sempty_bar + Cfg::SF_SLOTS;         // all MMAs issued for this CTA finished
    uint64_t* c_bar = drain_bar + 1;             // an epilogue warp's part of C is in staging (EPI 2)
    static_assert((2 * STAGES + NBUF + 2 * Cfg::SF_SLOTS + 1 + Cfg::EW) * 8 + 16 <= 512, "barrier space");
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(c_bar + Cfg::EW);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    int* s_prefix = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + 512);
    int* s_mm = s_prefix + MAX_MASKED_GROUPS + 4;

    const uint32_t warp = threadIdx.x / 32;
    const uint32_t lane = lane_id();
    const uint32_t rank = (CG == 1) ? 0u : cluster_ctarank();
    const bool leader = rank == 0;
    const int unit = static_cast<int>(blockIdx.x) / CG;
    const int units = static_cast<int>(gridDim.x) / CG;
    const bool split = kCanSplit && p.split_mode == SPLIT_CLUSTER;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&done_bar[s], 1);
        }
        for (int i = 0; i < NBUF; ++i) mbar_init(&tempty_bar[i], Cfg::EW * CG);
        for (int i = 0; i < Cfg::SF_SLOTS; ++i) {
            mbar_init(&sfull_bar[i], 1);
            mbar_init(&sempty_bar[i], Cfg::EW);
        }
        mbar_init(drain_bar, SF_F32_ISSUERS);
        for (int i = 0; i < Cfg::EW; ++i) mbar_init(&c_bar[i], 1);
        *s_abort = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&p.tma_a);
        tma_prefetch_desc(&p.tma_b);
    }
    if (warp == 1) {
        tmem_alloc<CG>(s_tmem, 512);
        tmem_relinquish<CG>();
    }
    griddep_launch_dependents();
    griddep_wait();
    prepare_schedule<KIND, CG, SF_F32_THREADS>(p, s_prefix, s_mm, warp, lane);
    tc_fence_before();
    __syncthreads();
    if (CG == 2 || split) cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *s_tmem;
    const int my_rows = BM * static_cast<int>(rank);

    if (warp < SF_F32_EPI_WARP0) {
        registers_dec<SF_F32_OTHER_REGS>();
        if (warp == 0) {
            // -------------------------------------------------------- TMA producer --
            [[maybe_unused]] uint32_t full_leader0 = 0;
            if constexpr (CG == 2) full_leader0 = mapa_shared(smem_u32(&full_bar[0]), 0);
            int stage = 0, issued = 0, gcur = first_cursor<KIND, CG>(p, s_prefix);
            uint32_t phase = 0;
            Tile cur;
            bool aborted = false;
            const uint32_t tx = static_cast<uint32_t>(CG * (p.a_box_rows * BK + Cfg::B_BYTES));
            for (int t = unit; !aborted && next_tile<KIND, CG, true, true>(p, s_prefix, s_mm, t, units, gcur, cur, lane);
                 t += units) {
                const int a_row = cur.m_blk * BM * CG + my_rows;
                const int b_row = cur.n_blk * BN + Cfg::B_ROWS * static_cast<int>(rank);
                const int kb1 = min(4 * cur.kg1, p.kb);
                for (int kb = 4 * cur.kg0; kb < kb1; ++kb) {
                    if (issued >= STAGES && !wait_warp(&done_bar[stage], phase ^ 1u, p, s_abort)) { aborted = true; break; }
                    // (the failure-path hook withholds CTA 0's first load)
                    if (elect_one() && !(p.test_mode == 1 && blockIdx.x == 0 && issued == 0)) {
                        uint8_t* a_dst = smem_a + stage * Cfg::A_BYTES;
                        uint8_t* b_dst = smem_b + stage * Cfg::B_BYTES;
                        const int kx = kb * BK;
                        if constexpr (CG == 1) {
                            mbar_arrive_expect_tx(&full_bar[stage], tx);
                            if constexpr (KIND == kMasked) tma_load_3d(a_dst, &p.tma_a, &full_bar[stage], kx, a_row, cur.g);
                            else tma_load_2d(a_dst, &p.tma_a, &full_bar[stage], kx, a_row);
                            if constexpr (KIND == kDense) tma_load_2d(b_dst, &p.tma_b, &full_bar[stage], kx, b_row);
                            else tma_load_3d(b_dst, &p.tma_b, &full_bar[stage], kx, b_row, cur.g);
                        } else {
                            // both CTAs' loads complete on the leader's barrier
                            if (leader) mbar_arrive_expect_tx(&full_bar[stage], tx);
                            const uint32_t fb = full_leader0 + 8u * static_cast<uint32_t>(stage);
                            tma_load_2d_pair(a_dst, &p.tma_a, fb, kx, a_row);
                            tma_load_2d_pair(b_dst, &p.tma_b, fb, kx, b_row);
                        }
                    }
                    __syncwarp();
                    ++issued;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            if (aborted) {
                // let the loads already issued land before shared memory goes away
                if constexpr (CG == 1) {
                    int s = stage;
                    uint32_t ph = phase;
                    for (int i = 0; i < STAGES && i < issued; ++i) {
                        if (--s < 0) { s = STAGES - 1; ph ^= 1u; }
                        wait_quiet(&full_bar[s], ph, p.wait_limit_ns / 16);
                    }
                } else {
                    sleep_ns(p.wait_limit_ns / 16);
                }
            }
        } else if (warp <= SF_F32_ISSUERS) {
            // --------------------------------------------------------- MMA issuers --
            // Block products are dealt out in turn: two waits, four MMAs and two
            // commits take a lone warp ~450 clocks next to the epilogue's warps,
            // longer than the MMAs run.
            if (CG == 1 || leader) {
                const uint32_t mine = warp - 1;
                const uint64_t adesc0 = smem_desc_sw128(smem_u32(smem_a));
                const uint64_t bdesc0 = smem_desc_sw128(smem_u32(smem_b));
                const uint32_t full0 = smem_u32(full_bar), tempty0 = smem_u32(tempty_bar), done0 = smem_u32(done_bar);
                int gcur = first_cursor<KIND, CG>(p, s_prefix);
                uint32_t item0 = 0;   // block products before this tile
                uint32_t stage = mine, par = 0;   // of this warp's next product
                Tile c;
                bool aborted = false;
                for (int t = unit; !aborted && next_tile<KIND, CG, false, true>(p, s_prefix, s_mm, t, units, gcur, c, lane);
                     t += units) {
                    const uint32_t n = static_cast<uint32_t>(min(4 * c.kg1, p.kb) - 4 * c.kg0);
                    // the products whose number has this warp's parity
                    for (uint32_t it = item0 + ((item0 ^ mine) & 1u); it < item0 + n; it += 2) {
                        // operands landed, and the buffer's last product read back: both probes at once
                        const uint32_t buf = it % NBUF, buf_par = ((it / NBUF) & 1u) ^ 1u;
                        const bool ready = mbar_try_wait_addr(full0 + 8 * stage, par) & mbar_try_wait_addr(tempty0 + 8 * buf, buf_par);
                        if (!__all_sync(0xffffffffu, ready) && !(wait_warp(&full_bar[stage], par, p, s_abort) &&
                                                                wait_warp(&tempty_bar[buf], buf_par, p, s_abort))) {
                            aborted = true;
                            break;
                        }
                        tc_fence_after();  // the epilogue's reads of this buffer precede the MMAs below
                        const uint64_t adesc = adesc0 + stage * (Cfg::A_BYTES >> 4), bdesc = bdesc0 + stage * (Cfg::B_BYTES >> 4);
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tc_mma_f8<CG>(tmem_base + buf * BN, adesc + 2 * k, bdesc + 2 * k, Cfg::IDESC, k > 0 ? 1u : 0u);
                            tc_commit_addr<CG>(done0 + 8 * stage);
                        }
                        __syncwarp();
                        stage += 2;
                        if (stage >= STAGES) { stage -= STAGES; par ^= 1u; }
                    }
                    item0 += n;
                }
                if (elect_one()) tc_commit<CG>(drain_bar);
                __syncwarp();
            }
            wait_quiet(drain_bar, 0, p.wait_limit_ns);
        } else {
            // ------------------------------------------------------ scale producer --
            // Gathers the scales of four K-blocks of every row (lane l: rows l, l + 32,
            // ...) into shared memory, the next four K-blocks' loads in flight. (Read
            // by the epilogue's warps from global memory, even several blocks ahead,
            // the scales held them up for ~300 clocks a block.)
            float a[2][4][4], b[2][ROWB ? 4 : 1][4];   // [set][row][K-block]
            auto load4 = [&](const float* row, int kb0, bool vec, float (&v)[4]) {
                if (vec) {
                    ld_scale4(row + kb0, v);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = ld_scale(row + min(kb0 + i, p.kb - 1));
                }
            };
            uint32_t stored = 0;
            auto store = [&](int set) {
                const uint32_t slot = stored % Cfg::SF_SLOTS;
                if (!wait_block(&sempty_bar[slot], ((stored / Cfg::SF_SLOTS) & 1u) ^ 1u, p, s_abort)) return false;
                float* dst = smem_sf + slot * Cfg::SF_SLOT_FLOATS + lane;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        dst[i * BM + 32 * j] = ROWB ? a[set][j][i] : a[set][j][i] * b[set][0][i];
                        if constexpr (ROWB) dst[4 * BM + i * BN + 32 * j] = b[set][j][i];
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sfull_bar[slot]);
                ++stored;
                return true;
            };
            int gcur = first_cursor<KIND, CG>(p, s_prefix);
            Tile c;
            bool aborted = false;
            for (int t = unit; !aborted && next_tile<KIND, CG, true, true>(p, s_prefix, s_mm, t, units, gcur, c, lane);
                 t += units) {
                // rows and columns clamped into the operands (those past them are never stored)
                const size_t a_base = KIND == kMasked ? static_cast<size_t>(c.g) * p.rows : 0;
                const int row0 = c.m_blk * BM * CG + my_rows + static_cast<int>(lane);
                const float* sfb = p.sfb32 + static_cast<size_t>(KIND == kDense ? 0 : c.g) * p.nb_sf * p.kb;
                auto load = [&](int set, int kg) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        load4(p.sfa32 + (a_base + min(row0 + 32 * j, p.rows - 1)) * p.kb, 4 * kg, p.sfa_vec4 != 0, a[set][j]);
#pragma unroll
                    for (int j = 0; j < (ROWB ? 4 : 1); ++j) {
                        const int row = ROWB ? min(c.n_blk * BN + 32 * j + static_cast<int>(lane), p.n - 1) : c.n_blk;
                        load4(sfb + static_cast<size_t>(row) * p.kb, 4 * kg, p.sfb_vec4 != 0, b[set][j]);
                    }
                };
                load(0, c.kg0);
                for (int kg = c.kg0; kg < c.kg1; kg += 2) {
                    if (kg + 1 < c.kg1) load(1, kg + 1);
                    if (!store(0)) { aborted = true; break; }
                    if (kg + 1 >= c.kg1) break;
                    if (kg + 2 < c.kg1) load(0, kg + 2);
                    if (!store(1)) { aborted = true; break; }
                }
            }
        }
    } else {
        registers_inc<SF_F32_EPI_REGS>();
        // ------------------------------------------------------------ epilogue --
        const int q = static_cast<int>(warp & 3);              // TMEM lanes 32q .. 32q + 31
        const int grp = static_cast<int>(warp - SF_F32_EPI_WARP0) / 4;  // columns CW grp ...
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + grp * CW;
        uint8_t* stg = smem_stg + (warp - SF_F32_EPI_WARP0) * 32 * Cfg::STG_ROW;
        const uint32_t done0 = smem_u32(done_bar);
        const uint32_t tempty0 = CG == 1 ? smem_u32(tempty_bar) : mapa_shared(smem_u32(tempty_bar), 0);
        int gcur = first_cursor<KIND, CG>(p, s_prefix);
        uint32_t stage = 0, par = 0, buf = 0;
        uint32_t sf_group = 0;       // groups of four K-blocks before this one
        [[maybe_unused]] uint64_t* const my_c_bar = c_bar + (warp - SF_F32_EPI_WARP0);
        [[maybe_unused]] uint32_t c_par = 0;
        [[maybe_unused]] bool c_pending = false;
        bool aborted = false;
        Tile c;
        for (int t = unit; !aborted && next_tile<KIND, CG, false, true>(p, s_prefix, s_mm, t, units, gcur, c, lane);
             t += units) {
            // (contiguous: the tile is placed when its sums are complete)
            int mloc = KIND == kContiguous ? 0 : c.m_blk * BM * CG + my_rows + 32 * q + static_cast<int>(lane);
            const size_t a_base = KIND == kMasked ? static_cast<size_t>(c.g) * p.rows : 0;
            const int kb1 = min(4 * c.kg1, p.kb);
            // A warp without a row that D takes hands everything back unread: 32 experts of
            // 1-20 rows, 4096x7168, 190 us a call under load instead of 200 (the power limit),
            // 67-124 rows the same 204. (Boxes of 32 rows of A, as many as the expert has rows
            // in, took 200 and 225.)
            // (Contiguous: only the last block can have such warps.)
            if (KIND != kContiguous && !__any_sync(0xffffffffu, KIND == kMasked ? mloc < s_mm[c.g] : mloc < p.rows)) {
                for (int kb = 4 * c.kg0; kb < kb1; kb += 4) {
                    const uint32_t slot = sf_group % Cfg::SF_SLOTS;
                    if (!wait_block(&sfull_bar[slot], (sf_group / Cfg::SF_SLOTS) & 1u, p, s_abort)) { aborted = true; break; }
                    if (lane == 0) mbar_arrive(&sempty_bar[slot]);
                    ++sf_group;
                    const int n = min(4, kb1 - kb);
                    for (int i = 0; i < n; ++i) {
                        if (!wait_block(&done_bar[stage], par, p, s_abort)) { aborted = true; break; }
                        if (lane == 0) {
                            if (CG == 1) mbar_arrive_addr(tempty0 + 8 * buf);
                            else mbar_arrive_cluster(tempty0 + 8 * buf);
                        }
                        buf = (buf + 1) % NBUF;
                        if (++stage == STAGES) { stage = 0; par ^= 1u; }
                    }
                    if (aborted) break;
                }
                if (aborted) break;
                continue;
            }
            if constexpr (EPI == 2) {
                // C's part of the tile, a K loop ahead of its use: a row per lane
                if (!split) {
                    const int col0 = c.n_blk * BN + grp * CW, size = p.out_f32 ? 4 : 2;
                    const int bytes = max(0, min(CW, p.n - col0)) * size;  // N % 8 == 0: whole 16 bytes
                    const bool has = mloc < p.rows && bytes > 0;
                    const uint32_t lanes = __ballot_sync(0xffffffffu, has);
                    fence_proxy_async_smem();  // the last tile's accesses to staging precede the copies
                    __syncwarp();
                    if (lane == 0) mbar_arrive_expect_tx(my_c_bar, static_cast<uint32_t>(__popc(lanes) * bytes));
                    __syncwarp();
                    if (has)
                        bulk_load(stg + lane * Cfg::STG_ROW,
                                  static_cast<const char*>(p.c) + (static_cast<size_t>(mloc) * p.n + col0) * size,
                                  static_cast<uint32_t>(bytes), my_c_bar);
                    c_pending = true;
                }
            }
            float acc[CW];
#pragma unroll
            for (int i = 0; i < CW; ++i) acc[i] = 0.f;

            for (int kb = 4 * c.kg0; kb < kb1; kb += 4) {
                const uint32_t slot = sf_group % Cfg::SF_SLOTS;
                if (!wait_block(&sfull_bar[slot], (sf_group / Cfg::SF_SLOTS) & 1u, p, s_abort)) { aborted = true; break; }
                const float* sf = smem_sf + slot * Cfg::SF_SLOT_FLOATS + 32 * q + (ROWB ? lane / 4 : lane);
                [[maybe_unused]] const float* sfb_cols =
                    smem_sf + slot * Cfg::SF_SLOT_FLOATS + 4 * BM + grp * CW + 2 * (lane % 4);
                const int n = min(4, kb1 - kb);
#pragma unroll 2
                for (int i = 0; i < n; ++i) {
                    float f[ROWB ? 4 : 1];
#pragma unroll
                    for (int h = 0; h < (ROWB ? 4 : 1); ++h) f[h] = sf[i * BM + 8 * h];
                    if (!__all_sync(0xffffffffu, mbar_try_wait_addr(done0 + 8 * stage, par)) &&
                        !wait_warp(&done_bar[stage], par, p, s_abort)) {
                        aborted = true;
                        break;
                    }
                    tc_fence_after();
                    // The whole product is read and its buffer handed back before
                    // anything is added, and nothing is carried to the next block
                    // but the sums.
                    uint32_t r[CW];
                    if constexpr (ROWB) {
                        tmem_ld_16x256b_x8(t_row + buf * BN, r);
                        tmem_ld_16x256b_x8(t_row + (16u << 16) + buf * BN, r + 32);
                    } else {
                        tmem_read<CW>(t_row + buf * BN, r);
                    }
                    tmem_read_done<CW>(r);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (CG == 1) mbar_arrive_addr(tempty0 + 8 * buf);
                        else mbar_arrive_cluster(tempty0 + 8 * buf);
                    }
                    buf = (buf + 1) % NBUF;
                    if (++stage == STAGES) { stage = 0; par ^= 1u; }
                    if constexpr (ROWB) {
#pragma unroll
                        for (int j = 0; j < CW / 8; ++j) {
                            const float2 g = *reinterpret_cast<const float2*>(sfb_cols + i * BN + 8 * j);
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                const int a = 32 * (h / 2) + 4 * j + 2 * (h % 2);
                                float s0, s1;
                                mul2(s0, s1, g.x, g.y, f[h], f[h]);
                                fma2(acc[a], acc[a + 1], __uint_as_float(r[a]), __uint_as_float(r[a + 1]), s0, s1);
                            }
                        }
                    } else {
#pragma unroll
                        for (int a = 0; a < CW; a += 2)
                            fma2(acc[a], acc[a + 1], __uint_as_float(r[a]), __uint_as_float(r[a + 1]), f[0], f[0]);
                    }
                }
                if (aborted) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sempty_bar[slot]);
                ++sf_group;
            }
            if (aborted) break;

            if (kCanSplit && split) {
                // this K range's partial, for the cluster's sum below (the ring is
                // idle: every MMA of the one tile has been read back)
                float* part = reinterpret_cast<float*>(smem_a) + (32 * q + (ROWB ? lane / 4 : lane)) * Cfg::PART_ROW + grp * CW;
                if constexpr (ROWB) {
#pragma unroll
                    for (int a = 0; a < CW; a += 2)
                        *reinterpret_cast<float2*>(part + (16 * (a / 32) + 8 * (a / 2 % 2)) * Cfg::PART_ROW + 8 * (a / 4 % 8) +
                                                   2 * (lane % 4)) = make_float2(acc[a], acc[a + 1]);
                } else if (mloc < p.rows) {
#pragma unroll
                    for (int i = 0; i < CW; i += 4)
                        *reinterpret_cast<float4*>(part + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
                }
                continue;  // one tile per CTA
            }
            if constexpr (KIND == kContiguous) {
                place_tile<KIND, CG>(p, s_prefix, c);
                mloc = c.m_blk * BM + 32 * q + static_cast<int>(lane);
            }
            bool valid;
            StoreRows to;
            to.row0 = a_base + static_cast<size_t>(mloc - static_cast<int>(lane));
            if constexpr (KIND == kDense) {
                valid = mloc < p.rows;
            } else if constexpr (KIND == kMasked) {
                valid = mloc < s_mm[c.g];
            } else {
                const int id = mloc < p.rows ? __ldg(p.meta + mloc) : -1;
                const bool in_range = id >= 0 && id < p.groups;
                valid = in_range && id == c.g;
                if (in_range && id != c.g) atomicOr(p.status, DEVERR_MIXED_EXPERT_BLOCK);
            }
            to.rows = __ballot_sync(0xffffffffu, valid);
            if constexpr (EPI == 2) {
                if (!wait_block(my_c_bar, c_par, p, s_abort)) { aborted = true; break; }
                c_pending = false;
                c_par ^= 1u;
            }
            if (to.rows != 0)
                store_rows<CW, Cfg::STG_ROW, EPI, ROWB>(p, acc, to, c.n_blk * BN + grp * CW, stg, static_cast<int>(lane));
        }
        // (a wait gave up: the copies land before shared memory goes away)
        if (EPI == 2 && c_pending) wait_quiet(my_c_bar, c_par, p.wait_limit_ns / 16);
    }

    tc_fence_before();
    __syncthreads();
    if constexpr (kCanSplit) {
        if (split) {
            cluster_sync();  // every partial of the tile is in its CTA's shared memory
            Tile c;
            if (raster_tile(p, p.num_m_blocks, static_cast<int>(blockIdx.x), c) && *s_abort == 0) {
                // CTA r of S adds up the 8-column pieces [r NP / S, (r + 1) NP / S) of every row
                const int S = p.splits, NP = BN / 8;
                const int r = static_cast<int>(cluster_ctarank());
                const int p0 = r * NP / S, np = (r + 1) * NP / S - p0;
                const int rows = min(BM, p.rows - c.m_blk * BM);
                const uint32_t ring = smem_u32(smem_a);
                for (int i = static_cast<int>(threadIdx.x); i < rows * np; i += SF_F32_THREADS) {
                    const int row = i / np, pc = p0 + i % np;
                    const int col = c.n_blk * BN + 8 * pc;
                    if (col >= p.n) continue;
                    float sum[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[j] = 0.f;
                    for (int sp = 0; sp < S; ++sp) {
                        const uint32_t at = mapa_shared(ring + (row * Cfg::PART_ROW + 8 * pc) * 4, static_cast<uint32_t>(sp));
                        const float4 lo = ld_cluster_f32x4(at), hi = ld_cluster_f32x4(at + 16);
                        sum[0] += lo.x; sum[1] += lo.y; sum[2] += lo.z; sum[3] += lo.w;
                        sum[4] += hi.x; sum[5] += hi.y; sum[6] += hi.z; sum[7] += hi.w;
                    }
                    cluster_store8<EPI != 0 ? 1 : 0>(p, sum, (static_cast<size_t>(c.m_blk) * BM + row) * p.n + col);
                }
            }
        }
    }
    // neither CTA of a pair frees TMEM while the pair still uses it; no CTA of a
    // split exits while peers read its partial
    if (CG == 2 || split) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<CG>(tmem_base, 512);
    }
}

}  // namespace dg
