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
// What bounds it: the tensor core needs 4 x BN/2 clocks per 128-K block of a
// 128 x BN tile (M = 128 rows per SM); reading the block back and the FMAs take
// 128 x BN / 128 clocks each (128 lanes per SM), half of that, next to it. So
// the tensor core stays the bound as long as the hand-offs between the two are
// hidden, and the TMEM buffers (512 columns) are as many as fit.
//
// CTA = 12 warps (three warpgroups), one CTA per SM, persistent:
//   warp 0      TMA producer (128-byte swizzle, STAGES-deep ring)
//   warp 1      TMEM allocation and MMA issue
//   warps 2, 3  idle; they complete the first warpgroup, whose registers go to
//               the epilogue (56 + 2 x 224 of the launch's 3 x 168 per lane)
//   warps 4..   epilogue. Warp w reads TMEM lanes 32 (w % 4) .. + 31 (a row per
//               lane) and owns half of the tile's columns, CW = BN / 2, whose
//               accumulators stay in its registers over the whole K loop. 32
//               columns are read from TMEM while the 32 before are added.
// The tile's columns are NSUB sub-tiles with rings of TMEM buffers and barriers
// of their own, so that a sub-tile's buffer is refilled NBUF blocks later while
// the other sub-tiles' MMAs run.
//
// CG = 2: a cluster of two CTAs computes 256 x BN (tcgen05 cta_group::2), which
// halves the B bytes per SM: a lone CTA's 128 x 256 tile needs 48 KB of loads
// per 512 clocks of math, more than the ~77 bytes per clock the L2 feeds an SM.
// No load is multicast.
//
// Split-K (dense, small M): the CTAs of a cluster take K ranges of one tile,
// leave their fp32 partials in their own shared memory (the operand ring, idle
// by then) and add each others' in split order through distributed shared
// memory: no workspace, identical bits on every call.
//
// Scheduling, masks and bounded waits are those of gemm_kernel.cuh.
#pragma once

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

// Wait for the TMEM loads into r; naming the registers keeps their uses behind the wait.
__device__ __forceinline__ void tc_wait_ld16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])
                 :: "memory");
}

// Scale loads that stay where they are written: left to itself the compiler moves
// them down to their use, four K-blocks later, and the warp waits for L2 there.
__device__ __forceinline__ float ld_scale(const float* p) {
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ void ld_scale4(const float* p, float (&v)[4]) {
    asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "l"(p));
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

// ROWB: B is scaled per row (sfb_gran_n = 1).
constexpr int SF_F32_THREADS = 384;
constexpr int SF_F32_EPI_WARP0 = 4;                   // first epilogue warp
constexpr int SF_F32_LAUNCH_REGS = 168, SF_F32_EPI_REGS = 224, SF_F32_OTHER_REGS = 56;
static_assert(SF_F32_OTHER_REGS + 2 * SF_F32_EPI_REGS <= 3 * SF_F32_LAUNCH_REGS, "registers of the launch");

template <int BN, int CG, int NSUB, int SCHED_INTS, bool ROWB>
struct SfF32Config {
    static constexpr int EW = 8;                      // epilogue warps
    static constexpr int GROUPS = EW / 4;             // column groups of epilogue warps
    static constexpr int CW = BN / GROUPS;            // columns of an epilogue warp
    static constexpr int SUB = BN / NSUB;             // columns of a sub-tile (one MMA's N)
    static constexpr int B_ROWS = BN / CG;            // rows of B in this CTA's shared memory
    static constexpr int SUB_B_ROWS = SUB / CG;
    static_assert(BN % GROUPS == 0 && CW % 16 == 0 && SUB % CW == 0, "columns of an epilogue warp");
    static_assert(SUB % 16 == 0 && SUB <= 256 && SUB_B_ROWS % 8 == 0, "N of an MMA");
    static_assert(!ROWB || BN % 128 == 0, "per-row scales: one column per lane and K-block");
    static constexpr int A_BYTES = BM * BK;
    static constexpr int B_BYTES = B_ROWS * BK;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    // columns between TMEM buffers; all 512 columns are used
    static constexpr int TMEM_STRIDE = SUB > 128 ? 256 : (SUB > 64 ? 128 : 64);
    static constexpr int NBUF = 512 / (NSUB * TMEM_STRIDE);
    static_assert(NBUF >= 2, "the MMAs of a block run while the last one is read back");
    // output staging: 32 rows of 64 bytes per epilogue warp, rows 80 bytes apart (no bank conflicts)
    static constexpr int STG_ROW = 80;
    static constexpr int STG_BYTES = EW * 32 * STG_ROW;
    static constexpr int SFB_BYTES = ROWB ? 2 * 4 * BN * 4 : 0;  // two groups of four K-blocks' column scales
    static constexpr int SCHED_BYTES = SCHED_INTS * 4;
    static constexpr int FIXED_BYTES = 1024 /*align slack*/ + STG_BYTES + SFB_BYTES + 512 /*barriers*/ + SCHED_BYTES;
    static constexpr int STAGES_FIT = (SMEM_LIMIT - FIXED_BYTES) / STAGE_BYTES;
    static constexpr int STAGES = STAGES_FIT > 8 ? 8 : STAGES_FIT;
    static_assert(STAGES >= 3, "pipeline too shallow");
    static constexpr int SMEM_BYTES = FIXED_BYTES + STAGES * STAGE_BYTES;
    static constexpr uint32_t IDESC = idesc_e4m3_f32(BM * CG, SUB);
    // split-K: a partial tile of fp32 rows, four floats of padding per row
    static constexpr int PART_ROW = BN + 4;
    static_assert(BM * PART_ROW * 4 <= STAGES * STAGE_BYTES || CG == 2, "the partial tile fits the idle ring");
};

// The 128-row share of D that an epilogue warp writes: 32 rows from `row0` of
// D, bit r of `rows` set where row r may be written.
struct StoreRows {
    size_t row0;
    uint32_t rows;
};

// CW columns of a warp's 32 rows, from registers (lane = row) to D through the
// warp's staging rows, 64 bytes of every row at a time: written back, four
// lanes take the 64 bytes of a row. (Row-wise 16-byte stores straight from the
// registers touch 32 rows per instruction and slow the operand loads.)
template <int CW, int STG_ROW>
__device__ __forceinline__ void store_rows(const GemmParams& p, const float (&acc)[CW], const StoreRows& to,
                                           int col0, uint8_t* stg, int lane) {
    const int sub = lane >> 2, piece = lane & 3;
    if (p.c == nullptr && !p.out_f32) {
#pragma unroll
        for (int u = 0; u < CW; u += 32) {
            const int pieces = (CW - u < 32 ? CW - u : 32) / 8;  // 16-byte pieces of eight bf16 columns
            __syncwarp();
#pragma unroll
            for (int q = 0; q < pieces; ++q) {
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
                if (piece < pieces && col < p.n && ((to.rows >> r) & 1u))
                    *reinterpret_cast<uint4*>(p.d + (to.row0 + r) * p.n + col) =
                        *reinterpret_cast<const uint4*>(stg + r * STG_ROW + 16 * piece);
            }
        }
        return;
    }
    // C and / or an fp32 D: 16 fp32 columns at a time
#pragma unroll
    for (int u = 0; u < CW; u += 16) {
        const int pieces = (CW - u < 16 ? CW - u : 16) / 4;
        __syncwarp();
#pragma unroll
        for (int q = 0; q < pieces; ++q) {
            const int j = u + 4 * q;
            *reinterpret_cast<float4*>(stg + lane * STG_ROW + 16 * q) =
                make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
        }
        __syncwarp();
        const int col = col0 + u + 4 * piece;
        const bool in = piece < pieces && col < p.n;
        float4 c[4];
        if (p.c != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 8 * i + sub;
                if (!in || !((to.rows >> r) & 1u)) continue;
                const size_t at = (to.row0 + r) * p.n + col;
                if (p.out_f32) {
                    c[i] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.c) + at);
                } else {
                    const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.c) + at);
                    c[i] = make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xFFFF0000u),
                                       __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xFFFF0000u));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + sub;
            if (!in || !((to.rows >> r) & 1u)) continue;
            const size_t at = (to.row0 + r) * p.n + col;
            float4 v = *reinterpret_cast<const float4*>(stg + r * STG_ROW + 16 * piece);
            if (p.c != nullptr) {
                v.x += c[i].x;
                v.y += c[i].y;
                v.z += c[i].z;
                v.w += c[i].w;
            }
            if (p.out_f32) {
                *reinterpret_cast<float4*>(p.d32 + at) = v;
            } else {
                const __nv_bfloat162 b0 = __floats2bfloat162_rn(v.x, v.y), b1 = __floats2bfloat162_rn(v.z, v.w);
                *reinterpret_cast<uint2*>(p.d + at) = make_uint2(*reinterpret_cast<const uint32_t*>(&b0),
                                                                 *reinterpret_cast<const uint32_t*>(&b1));
            }
        }
    }
}

template <int BN, int KIND, int CG, int NSUB, bool ROWB>
__global__ void __launch_bounds__(SF_F32_THREADS, 1) fp8_gemm_sf_f32_kernel(const __grid_constant__ SfF32Params p) {
    static_assert(CG == 1 || KIND != kMasked, "CTA pairs are built for the dense and contiguous forms");
    static_assert(!ROWB || KIND == kDense, "per-row scales of B: dense form");
    using Cfg = SfF32Config<BN, CG, NSUB, sched_ints<KIND>(), ROWB>;
    constexpr int STAGES = Cfg::STAGES;
    constexpr int NBUF = Cfg::NBUF;
    constexpr int CW = Cfg::CW;
    constexpr int BUFS = NBUF * NSUB;
    constexpr bool kCanSplit = KIND == kDense && CG == 1;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* smem_a = smem;
    uint8_t* smem_b = smem_a + STAGES * Cfg::A_BYTES;
    uint8_t* smem_stg = smem_b + STAGES * Cfg::B_BYTES;
    float* smem_sfb = reinterpret_cast<float*>(smem_stg + Cfg::STG_BYTES);    // ROWB: [2][4][BN]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem_stg + Cfg::STG_BYTES + Cfg::SFB_BYTES);
    uint64_t* full_bar = bars;                   // A/B bytes landed (the leader's counts both CTAs)
    uint64_t* empty_bar = full_bar + STAGES;     // MMAs reading the stage finished
    uint64_t* tfull_bar = empty_bar + STAGES;    // [buffer][sub-tile]: block product ready
    uint64_t* tempty_bar = tfull_bar + BUFS;     // [buffer][sub-tile]: read back
    uint64_t* sfb_bar = tempty_bar + BUFS;       // ROWB: a column group's scales are in shared memory
    uint64_t* drain_bar = sfb_bar + Cfg::GROUPS; // all MMAs issued for this CTA finished
    static_assert((2 * STAGES + 2 * BUFS + Cfg::GROUPS + 1) * 8 + 16 <= 512, "barrier space");
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drain_bar + 1);
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
            mbar_init(&empty_bar[s], 1);
        }
        for (int i = 0; i < BUFS; ++i) {
            mbar_init(&tfull_bar[i], 1);
            mbar_init(&tempty_bar[i], Cfg::EW / NSUB * CG);
        }
        for (int i = 0; i < Cfg::GROUPS; ++i) mbar_init(&sfb_bar[i], 4);
        mbar_init(drain_bar, 1);
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
    prepare_schedule<KIND, SF_F32_THREADS>(p, s_prefix, s_mm, warp, lane);
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
        int stage = 0, issued = 0, gcur = 0;
        uint32_t phase = 0;
        Tile cur;
        bool aborted = false;
        const uint32_t tx = static_cast<uint32_t>(CG * (p.a_box_rows * BK + Cfg::B_BYTES));
        for (int t = unit; !aborted && next_tile<KIND, true, CG>(p, s_prefix, s_mm, t, units, gcur, cur, lane);
             t += units) {
            const int a_row = cur.m_blk * BM * CG + my_rows;
            const int b_row = cur.n_blk * BN + Cfg::SUB_B_ROWS * static_cast<int>(rank);
            const int g = max(cur.g, 0);
            const int kb1 = min(4 * cur.kg1, p.kb);
            for (int kb = 4 * cur.kg0; kb < kb1; ++kb) {
                if (issued >= STAGES && !wait_warp(&empty_bar[stage], phase ^ 1u, p, s_abort)) { aborted = true; break; }
                // (the failure-path hook withholds CTA 0's first load)
                if (elect_one() && !(p.test_mode == 1 && blockIdx.x == 0 && issued == 0)) {
                    uint8_t* a_dst = smem_a + stage * Cfg::A_BYTES;
                    uint8_t* b_dst = smem_b + stage * Cfg::B_BYTES;
                    const int kx = kb * BK;
                    if constexpr (CG == 1) {
                        mbar_arrive_expect_tx(&full_bar[stage], tx);
                        if constexpr (KIND == kMasked) tma_load_3d(a_dst, &p.tma_a, &full_bar[stage], kx, a_row, g);
                        else tma_load_2d(a_dst, &p.tma_a, &full_bar[stage], kx, a_row);
                    } else {
                        // both CTAs' loads complete on the leader's barrier
                        if (leader) mbar_arrive_expect_tx(&full_bar[stage], tx);
                        tma_load_2d_pair(a_dst, &p.tma_a, full_leader0 + 8u * static_cast<uint32_t>(stage), kx, a_row);
                    }
#pragma unroll
                    for (int s = 0; s < NSUB; ++s) {
                        // sub-tile s: this CTA's SUB / CG rows of it
                        uint8_t* dst = b_dst + s * Cfg::SUB_B_ROWS * BK;
                        const int row = b_row + s * Cfg::SUB;
                        if constexpr (CG == 1) {
                            if constexpr (KIND == kDense) tma_load_2d(dst, &p.tma_b, &full_bar[stage], kx, row);
                            else tma_load_3d(dst, &p.tma_b, &full_bar[stage], kx, row, g);
                        } else {
                            const uint32_t fb = full_leader0 + 8u * static_cast<uint32_t>(stage);
                            if constexpr (KIND == kDense) tma_load_2d_pair(dst, &p.tma_b, fb, kx, row);
                            else tma_load_3d_pair(dst, &p.tma_b, fb, kx, row, g);
                        }
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
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMA issuer --
        if (CG == 1 || leader) {
            int stage = 0, gcur = 0, buf = 0;
            uint32_t phase = 0, buf_phase = 0;
            Tile c;
            bool aborted = false;
            for (int t = unit; !aborted && next_tile<KIND, CG == 2, CG>(p, s_prefix, s_mm, t, units, gcur, c, lane);
                 t += units) {
                const int kb1 = min(4 * c.kg1, p.kb);
                for (int kb = 4 * c.kg0; kb < kb1 && !aborted; ++kb) {
                    if (!wait_warp(&full_bar[stage], phase, p, s_abort)) { aborted = true; break; }
                    const uint64_t adesc = smem_desc_sw128(smem_u32(smem_a + stage * Cfg::A_BYTES));
                    const uint64_t bdesc = smem_desc_sw128(smem_u32(smem_b + stage * Cfg::B_BYTES));
#pragma unroll
                    for (int s = 0; s < NSUB; ++s) {
                        const int b = buf * NSUB + s;
                        if (!wait_warp(&tempty_bar[b], buf_phase ^ 1u, p, s_abort)) { aborted = true; break; }
                        tc_fence_after();  // the epilogue's reads of this buffer precede the MMAs below
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint64_t koff = static_cast<uint64_t>((k * 32) >> 4);
                                const uint64_t soff = static_cast<uint64_t>((s * Cfg::SUB_B_ROWS * BK) >> 4);
                                tc_mma_f8<CG>(tmem_base + b * Cfg::TMEM_STRIDE, adesc + koff, bdesc + soff + koff,
                                              Cfg::IDESC, k > 0 ? 1u : 0u);
                            }
                            tc_commit<CG>(&tfull_bar[b]);
                            if (s == NSUB - 1) tc_commit<CG>(&empty_bar[stage]);
                        }
                        __syncwarp();
                    }
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    if (++buf == NBUF) { buf = 0; buf_phase ^= 1u; }
                }
            }
            if (elect_one()) tc_commit<CG>(drain_bar);
            __syncwarp();
        }
        wait_quiet(drain_bar, 0, p.wait_limit_ns);
    }
    } else {
        registers_inc<SF_F32_EPI_REGS>();
        // ------------------------------------------------------------ epilogue --
        const int q = static_cast<int>(warp & 3);              // TMEM lanes 32q .. 32q + 31
        const int grp = static_cast<int>(warp - SF_F32_EPI_WARP0) / 4;  // column group
        const int col_in_tile = grp * CW;
        const int s = col_in_tile / Cfg::SUB;                  // sub-tile
        const uint32_t t_off = (static_cast<uint32_t>(32 * q) << 16) + s * Cfg::TMEM_STRIDE + (col_in_tile - s * Cfg::SUB);
        uint8_t* stg = smem_stg + (warp - SF_F32_EPI_WARP0) * 32 * Cfg::STG_ROW;
        [[maybe_unused]] uint32_t tempty_leader0 = 0;
        if constexpr (CG == 2) tempty_leader0 = mapa_shared(smem_u32(&tempty_bar[0]), 0);
        // a warp's columns can lie in two 128-column blocks of B when the tile width is no multiple of 128
        constexpr bool kTwoBlocks = !ROWB && BN % 128 != 0;
        int buf = 0, gcur = 0;
        uint32_t buf_phase = 0;
        [[maybe_unused]] uint32_t sfb_slot = 0, sfb_phase = 0;
        bool aborted = false;
        Tile c;
        for (int t = unit; !aborted && next_tile<KIND, true, CG>(p, s_prefix, s_mm, t, units, gcur, c, lane);
             t += units) {
            const int mloc = c.m_blk * BM * CG + my_rows + 32 * q + static_cast<int>(lane);
            const int col0 = c.n_blk * BN + col_in_tile;
            // scale rows, clamped into the operands (rows and columns past them are never stored)
            const size_t a_base = KIND == kMasked ? static_cast<size_t>(c.g) * p.rows : 0;
            const float* sa = p.sfa32 + (a_base + min(mloc, p.rows - 1)) * p.kb;
            const float* sbg = p.sfb32 + static_cast<size_t>(KIND == kDense ? 0 : max(c.g, 0)) * p.nb_sf * p.kb;
            const float* sb0 = sbg + static_cast<size_t>(min(col0 / 128, p.nb_sf - 1)) * p.kb;
            [[maybe_unused]] const float* sb1 = sbg + static_cast<size_t>(min((col0 + CW - 1) / 128, p.nb_sf - 1)) * p.kb;
            // columns of this warp before the next 128-column block
            [[maybe_unused]] const int first_cols = 128 - (col0 & 127);

            float acc[CW];
#pragma unroll
            for (int i = 0; i < CW; ++i) acc[i] = 0.f;

            // scales of four K-blocks, the next four in flight
            float na[4], nb[4];
            [[maybe_unused]] float nb1[4];
            auto load4 = [&](const float* row, int kb0, bool vec, float (&v)[4]) {
                if (vec) {
                    ld_scale4(row + kb0, v);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = ld_scale(row + min(kb0 + i, p.kb - 1));
                }
            };
            // ROWB: the four warps of a column group share its CW columns' scales:
            // warp q fetches CW / 4 of them (lane = column)
            constexpr int kColLanes = CW / 4;
            static_assert(!ROWB || kColLanes <= 32, "one column per lane");
            auto load_group = [&](int kg) {
                load4(sa, 4 * kg, p.sfa_vec4 != 0, na);
                if constexpr (ROWB) {
                    const int col = min(col0 + q * kColLanes + static_cast<int>(lane) % kColLanes, p.n - 1);
                    load4(sbg + static_cast<size_t>(col) * p.kb, 4 * kg, p.sfb_vec4 != 0, nb);
                } else {
                    load4(sb0, 4 * kg, p.sfb_vec4 != 0, nb);
                    if constexpr (kTwoBlocks) load4(sb1, 4 * kg, p.sfb_vec4 != 0, nb1);
                }
            };
            // The block products, 16 columns at a time in two sets of registers: a
            // chunk's read is issued before the chunk before it is added, across
            // blocks too, so that the reads pass under the FMAs. Eight warps read
            // and add 128 columns each in ~285 clocks (microbenchmark).
            constexpr int NCH = CW / 16;
            uint32_t r[2][16];
            auto block_addr = [&]() { return tmem_base + t_off + buf * NSUB * Cfg::TMEM_STRIDE; };
            auto wait_block = [&]() {
                if (!wait_warp(&tfull_bar[buf * NSUB + s], buf_phase, p, s_abort)) return false;
                tc_fence_after();
                return true;
            };
            const int kb1 = min(4 * c.kg1, p.kb);
            load_group(c.kg0);
            if (!wait_block()) break;
            tmem_ld_32x32b_x16(block_addr(), r[0]);
            for (int kg = c.kg0; kg < c.kg1 && !aborted; ++kg) {
                float s0[4];
                [[maybe_unused]] float s1[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s0[i] = ROWB ? na[i] : na[i] * nb[i];
                    if constexpr (kTwoBlocks) s1[i] = na[i] * nb1[i];
                }
                [[maybe_unused]] const float* sfb_cols = smem_sfb + sfb_slot * 4 * BN + col_in_tile;
                if constexpr (ROWB) {
                    float* dst = smem_sfb + sfb_slot * 4 * BN + col_in_tile;
                    if (static_cast<int>(lane) < kColLanes) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) dst[i * BN + q * kColLanes + lane] = nb[i];
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sfb_bar[grp]);
                    if (!wait_warp(&sfb_bar[grp], sfb_phase, p, s_abort)) { aborted = true; break; }
                    sfb_phase ^= 1u;
                    sfb_slot ^= 1u;  // the other slot's readers have all arrived here
                }
                if (kg + 1 < c.kg1) load_group(kg + 1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (4 * kg + i >= kb1) break;
                    const int b = buf * NSUB + s;
                    const uint32_t taddr = block_addr();
#pragma unroll
                    for (int ch = 0; ch < NCH; ++ch) {
                        const int h = 16 * ch;
                        uint32_t (&v)[16] = r[(i * NCH + ch) & 1];
                        uint32_t (&nxt)[16] = r[(i * NCH + ch + 1) & 1];
                        tc_wait_ld16(v);
                        if (ch + 1 < NCH) {
                            tmem_ld_32x32b_x16(taddr + h + 16, nxt);
                        } else {
                            // last read of this buffer: hand it back to the MMA
                            // warp, and start on the next block's
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) {
                                if (CG == 1 || leader) mbar_arrive(&tempty_bar[b]);
                                else mbar_arrive_cluster(tempty_leader0 + 8u * static_cast<uint32_t>(b));
                            }
                            if (++buf == NBUF) { buf = 0; buf_phase ^= 1u; }
                            if (4 * kg + i + 1 < kb1) {
                                if (!wait_block()) { aborted = true; break; }
                                tmem_ld_32x32b_x16(block_addr(), nxt);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            float sb[4] = {1.f, 1.f, 1.f, 1.f};
                            if constexpr (ROWB) {
                                const float4 f = *reinterpret_cast<const float4*>(sfb_cols + i * BN + h + j);
                                sb[0] = f.x; sb[1] = f.y; sb[2] = f.z; sb[3] = f.w;
                            }
                            float f = s0[i];
                            if constexpr (kTwoBlocks) f = h < first_cols ? s0[i] : s1[i];
#pragma unroll
                            for (int e = 0; e < 4; e += 2) {
                                float x0 = __uint_as_float(v[j + e]), x1 = __uint_as_float(v[j + e + 1]);
                                if constexpr (ROWB) mul2(x0, x1, x0, x1, sb[e], sb[e + 1]);
                                fma2(acc[h + j + e], acc[h + j + e + 1], x0, x1, f, f);
                            }
                        }
                    }
                    if (aborted) break;
                }
            }
            if (aborted) break;
            if constexpr (kCanSplit) {
                if (split) {
                    // this K range's partial, for the cluster's sum below (the ring is
                    // idle: every MMA of the one tile has been read back)
                    float* part = reinterpret_cast<float*>(smem_a) + (32 * q + lane) * Cfg::PART_ROW + col_in_tile;
                    if (mloc < p.rows) {
#pragma unroll
                        for (int i = 0; i < CW; i += 4)
                            *reinterpret_cast<float4*>(part + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
                    }
                    continue;
                }
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
                const int own = rank == 0 ? c.e_own[0] : c.e_own[1];
                if (in_range && id != own) atomicOr(p.status, DEVERR_MIXED_EXPERT_BLOCK);
            }
            to.rows = __ballot_sync(0xffffffffu, valid);
            if (to.rows != 0) store_rows<CW, Cfg::STG_ROW>(p, acc, to, col0, stg, static_cast<int>(lane));
        }
        tc_wait_ld();  // a read in flight when a wait gave up
    }

    tc_fence_before();
    __syncthreads();
    if constexpr (kCanSplit) {
        if (split) {
            cluster_sync();  // every partial of the tile is in its CTA's shared memory
            Tile c;
            if (raster_tile(p, static_cast<int>(blockIdx.x), c) && *s_abort == 0) {
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
                    cluster_store8<1>(p, sum, (static_cast<size_t>(c.m_blk) * BM + row) * p.n + col);
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
