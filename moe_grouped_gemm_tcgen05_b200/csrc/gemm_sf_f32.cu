// Host side of the GEMMs with fp32 block scales (include/dgb200.h: *_sf_f32):
// argument checks, tensor maps, the choice of a tile by the sizes, one launch.
#include <atomic>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "gemm_sf_f32_kernel.cuh"
#include "host.h"

namespace {

using dg::is_aligned;
using dg::SfF32Params;

struct Entry {
    int kind, cg;
    bool rowb;      // B scaled per row
    int epi;        // 0: bf16 D, 1: fp32 D, 2: C added
    int b_rows;     // rows of B in one load (the tensor map's box)
    int threads, smem;
    int stages;
    void* fn;
};

template <int KIND, int CG, bool ROWB, int EPI>
Entry entry() {
    using Cfg = dg::SfF32Config<CG, dg::sched_ints<KIND>(), ROWB, EPI>;
    return {KIND, CG, ROWB, EPI, Cfg::B_ROWS, dg::SF_F32_THREADS, Cfg::SMEM_BYTES, Cfg::STAGES,
            reinterpret_cast<void*>(&dg::fp8_gemm_sf_f32_kernel<KIND, CG, ROWB, EPI>)};
}

const Entry kEntries[] = {
    entry<dg::kDense, 1, false, 0>(), entry<dg::kDense, 2, false, 0>(), entry<dg::kDense, 1, true, 0>(),
    entry<dg::kDense, 2, true, 0>(),  entry<dg::kDense, 1, false, 1>(), entry<dg::kDense, 2, false, 1>(),
    entry<dg::kDense, 1, true, 1>(),  entry<dg::kDense, 2, true, 1>(),  entry<dg::kDense, 1, false, 2>(),
    entry<dg::kDense, 2, false, 2>(), entry<dg::kDense, 1, true, 2>(),  entry<dg::kDense, 2, true, 2>(),
    entry<dg::kContiguous, 1, false, 0>(), entry<dg::kMasked, 1, false, 0>(),
};
constexpr int kNumEntries = sizeof(kEntries) / sizeof(kEntries[0]);

struct Device {
    bool ready = false;
    int units[kNumEntries] = {};                                // co-resident CTAs, or CTA pairs
    int clusters[kNumEntries][dg::MAX_CLUSTER_SPLITS + 1] = {};  // co-resident clusters of s CTAs (dense, single CTAs)
};
constexpr int kMaxDevices = 64;
Device g_devices[kMaxDevices];

cudaLaunchConfig_t cluster_config(const Entry& e, unsigned blocks, unsigned cluster, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(static_cast<unsigned>(e.threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(e.smem);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// ------------------------------------------------------------ pairs and splits --
//
// Every tile has 128 columns. Dense calls run on CTA pairs (256 rows) or single
// CTAs, the grouped forms on single CTAs; K is split on single CTAs when the
// output tiles leave SMs idle. The choice with the least modelled time, in clocks:
//   waves x (K blocks of the longest range x clocks of a block + fixed clocks).
// A block takes ~460 clocks on pairs and ~480 on single CTAs (4096x7168x16384:
// 459-475 and 468-505 us; 4096x4096x7168: 105-119 and 111-125). With one m-tile the weights
// stream from HBM: ~24 bytes per clock at most on one SM, ~2400 on all (as
// measured for the block-scaled GEMMs). These are the clocks of the instance with
// a bf16 D and one scale per 128 columns, used for all: per-row scales take ~700 a
// block, and C is per tile. What is chosen for those is near the best all the same:
// per-row scales without C run 1-5% faster on single CTAs (2112x7168x4096 bf16 95.2
// against 97.1 us on the pairs that are chosen), with C 1% slower (121.7 against
// 120.1), one scale per 128 columns with C 12% slower (93.2 against 83.2); splits of
// M <= 128 are within 7% of the best (128x2112x7168, per-row scales, fp32: 5 splits
// 18.8 us, 4 splits 17.6).
constexpr double kPairBlockClocks = 460.0;
constexpr double kBlockClocks = 480.0;
constexpr double kStreamBytesPerClk = 2400.0;
constexpr double kStreamPerSmBytesPerClk = 24.0;
constexpr double kTileClocks = 2000.0;
constexpr double kSplitClocks = 3000.0;

struct Choice {
    int entry, units, splits;
};

Choice choose(const Device& dev, int kind, bool rowb, int epi, int rows, int n, int kb) {
    int forced_bn = 0, forced_cg = 0, forced_splits = 0;
    dg::host_forced_tile(&forced_bn, &forced_cg, &forced_splits);
    Choice best{-1, 0, 1};
    if (forced_bn != 0 && forced_bn != dg::SF_F32_BN) return best;
    if (kind == dg::kMasked) forced_cg = 0;  // always single CTAs, as the block-scaled form
    if (kind != dg::kDense) forced_splits = 1;
    const int kg = (kb + 3) / 4;
    double best_cost = 1e300;
    for (int i = 0; i < kNumEntries; ++i) {
        const Entry& e = kEntries[i];
        if (e.kind != kind || e.rowb != rowb || e.epi != epi || (forced_cg != 0 && e.cg != forced_cg)) continue;
        if (forced_cg == 0 && e.cg == 2 && rows <= dg::BM) continue;  // half of every pair would idle
        if (dev.units[i] < 1) continue;
        const int64_t mt = (static_cast<int64_t>(rows) + e.cg * dg::BM - 1) / (e.cg * dg::BM);
        const int64_t tiles = mt * ((static_cast<int64_t>(n) + dg::SF_F32_BN - 1) / dg::SF_F32_BN);
        for (int s = 1; s <= dg::MAX_CLUSTER_SPLITS; ++s) {
            if (forced_splits != 0 && s != forced_splits) continue;
            int64_t units = dev.units[i];
            if (s > 1) {
                if (e.cg != 1 || s > kg) break;
                if (forced_splits == 0 && tiles >= units) break;  // the tiles alone fill the GPU
                units = static_cast<int64_t>(dev.clusters[i][s]) * s;
                if (units < s) continue;
            }
            const int64_t work = tiles * s;
            const int64_t waves = (work + units - 1) / units;
            double clocks = e.cg == 2 ? kPairBlockClocks : kBlockClocks;
            if (mt == 1) {
                const double bytes = dg::SF_F32_BN * 128.0;  // of B per tile and block
                const double all = bytes * static_cast<double>(work < units ? work : units) / kStreamBytesPerClk;
                const double one = bytes / e.cg / kStreamPerSmBytesPerClk;
                if (all > clocks) clocks = all;
                if (one > clocks) clocks = one;
            }
            const int blocks = 4 * ((kg + s - 1) / s) < kb ? 4 * ((kg + s - 1) / s) : kb;
            const double cost = static_cast<double>(waves) * (blocks * clocks + kTileClocks + (s > 1 ? kSplitClocks : 0.0));
            if (cost < best_cost * 0.999) {
                best_cost = cost;
                best = {i, static_cast<int>(units), s};
            }
        }
    }
    return best;
}

// ------------------------------------------------------------------- launch --

dg_status launch(int kind, SfF32Params& p, const void* a, const void* b, int64_t m_blocks, int64_t a_mats,
                 int64_t b_mats, int sfb_gran_n, void* stream) {
    dg::HostDevice host;
    const dg_status st = dg::host_device(&host);
    if (st != DG_OK) return st;
    const Device& dev = g_devices[host.device];
    p.status = host.status;
    p.kb = p.k / 128;
    p.kp = 0;
    p.sfb_per_row = sfb_gran_n == 1;
    p.nb_sf = p.sfb_per_row ? p.n : (p.n + 127) / 128;
    p.sfa_vec4 = p.kb % 4 == 0 && is_aligned(p.sfa32, 16);
    p.sfb_vec4 = p.kb % 4 == 0 && is_aligned(p.sfb32, 16);
    p.wait_limit_ns = dg::host_wait_limit_ns();
    p.test_mode = dg::host_test_mode();
    const Choice choice = choose(dev, kind, sfb_gran_n == 1, p.c != nullptr ? 2 : p.out_f32, p.rows, p.n, p.kb);
    if (choice.entry < 0) return DG_ERR_UNSUPPORTED;  // a forced combination that is not built
    const Entry& e = kEntries[choice.entry];
    p.num_n_blocks = (p.n + dg::SF_F32_BN - 1) / dg::SF_F32_BN;
    p.num_m_blocks = (p.rows + e.cg * dg::BM - 1) / (e.cg * dg::BM);
    p.raster_group = 16 / e.cg;  // bands of 2048 rows
    p.raster_shift = e.cg == 2 ? 3 : 4;
    p.inv_band_tiles = 1.0f / static_cast<float>(p.raster_group * p.num_n_blocks);
    p.splits = choice.splits;
    p.split_mode = choice.splits > 1 ? dg::SPLIT_CLUSTER : dg::SPLIT_NONE;
    // a load brings no more rows of A than there are, in whole swizzle atoms of eight
    p.a_box_rows = p.rows >= dg::BM ? dg::BM : (p.rows + 7) / 8 * 8;
    if (!dg::host_encode_kmajor(&p.tma_a, a, kind == dg::kMasked ? 3 : 2, p.k, p.rows, a_mats, p.a_box_rows) ||
        !dg::host_encode_kmajor(&p.tma_b, b, kind == dg::kDense ? 2 : 3, p.k, p.n, b_mats, e.b_rows))
        return DG_ERR_INVALID_ARG;
    // work units: masked tiles are bounded by every group's m-blocks
    const int64_t m_tiles = kind == dg::kMasked ? m_blocks : p.num_m_blocks;
    const int64_t tiles = m_tiles * p.num_n_blocks * choice.splits;
    if (tiles > (int64_t{1} << 30)) return DG_ERR_UNSUPPORTED;
    const bool split = choice.splits > 1;
    const int units = static_cast<int>(split || tiles < choice.units ? tiles : choice.units);
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = dg::host_launch(static_cast<unsigned>(units * e.cg), e.threads, static_cast<size_t>(e.smem),
                                             stream, attr);
    if (e.cg == 2 || split) {
        cudaLaunchAttribute& c = attr[cfg.numAttrs++];
        c.id = cudaLaunchAttributeClusterDimension;
        c.val.clusterDim.x = e.cg == 2 ? 2u : static_cast<unsigned>(choice.splits);
        c.val.clusterDim.y = 1;
        c.val.clusterDim.z = 1;
    }
    if (dg::host_log())
        std::fprintf(stderr, "[dgb200] fp32 scales, form=%d rows=%d N=%d K=%d groups=%d: BN=%d CTA-group=%d splits=%d grid=%d "
                             "smem=%d stages=%d\n",
                     kind, p.rows, p.n, p.k, p.groups, dg::SF_F32_BN, e.cg, choice.splits, units * e.cg, e.smem, e.stages);
    void* args[] = {&p};
    return cudaLaunchKernelExC(&cfg, e.fn, args) == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

dg_status check(const void* a, const float* sfa, const void* b, const float* sfb, const void* d, int rows, int N, int K) {
    if (!a || !sfa || !b || !sfb || !d || rows <= 0 || N <= 0 || K <= 0) return DG_ERR_INVALID_ARG;
    if (K % 128 != 0 || N % 8 != 0) return DG_ERR_INVALID_ARG;
    if (K > (1 << 20) || rows > (1 << 30) || N > (1 << 30)) return DG_ERR_UNSUPPORTED;
    if (!is_aligned(a, 16) || !is_aligned(b, 16) || !is_aligned(d, 16) || !is_aligned(sfa, 4) || !is_aligned(sfb, 4))
        return DG_ERR_ALIGNMENT;
    return DG_OK;
}

SfF32Params params(const float* sfa, const float* sfb, void* d, int rows, int N, int K, int G) {
    SfF32Params p;
    std::memset(static_cast<void*>(&p), 0, sizeof(p));
    p.sfa32 = sfa;
    p.sfb32 = sfb;
    p.d = static_cast<__nv_bfloat16*>(d);
    p.rows = rows;
    p.n = N;
    p.k = K;
    p.groups = G;
    return p;
}

}  // namespace

namespace dg {

dg_status setup_sf_f32(int device, int sms) {
    Device& dev = g_devices[device];
    if (dev.ready) return DG_OK;
    for (int i = 0; i < kNumEntries; ++i) {
        const Entry& e = kEntries[i];
        if (cudaFuncSetAttribute(e.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, e.smem) != cudaSuccess)
            return DG_ERR_CUDA;
        dev.units[i] = sms;
        cudaLaunchAttribute attr[1];
        if (e.cg == 2) {
            const cudaLaunchConfig_t cfg = cluster_config(e, static_cast<unsigned>(2 * (sms / 2)), 2, attr);
            if (cudaOccupancyMaxActiveClusters(&dev.units[i], e.fn, &cfg) != cudaSuccess) return DG_ERR_CUDA;
        } else if (e.kind == dg::kDense) {
            for (int s = 2; s <= MAX_CLUSTER_SPLITS; ++s) {
                const cudaLaunchConfig_t cfg = cluster_config(e, static_cast<unsigned>(s * (sms / s)), s, attr);
                if (cudaOccupancyMaxActiveClusters(&dev.clusters[i][s], e.fn, &cfg) != cudaSuccess) {
                    cudaGetLastError();
                    dev.clusters[i][s] = 0;
                }
            }
        }
    }
    dev.ready = true;
    return DG_OK;
}

}  // namespace dg

extern "C" {

dg_status fp8_gemm_nt_sf_f32(const void* a, const float* sfa, const void* b, const float* sfb, int sfb_gran_n,
                             const void* c, void* d, int M, int N, int K, int out_f32, void* stream) {
    const dg_status s = check(a, sfa, b, sfb, d, M, N, K);
    if (s != DG_OK) return s;
    if ((sfb_gran_n != 1 && sfb_gran_n != 128) || (out_f32 != 0 && out_f32 != 1)) return DG_ERR_INVALID_ARG;
    if (c != nullptr && !is_aligned(c, 16)) return DG_ERR_ALIGNMENT;
    SfF32Params p = params(sfa, sfb, d, M, N, K, 1);
    p.d32 = out_f32 ? static_cast<float*>(d) : nullptr;
    p.out_f32 = out_f32;
    p.c = c;
    return launch(dg::kDense, p, a, b, (static_cast<int64_t>(M) + dg::BM - 1) / dg::BM, 1, 1, sfb_gran_n, stream);
}

dg_status m_grouped_fp8_gemm_nt_contiguous_sf_f32(const void* a, const float* sfa, const void* b, const float* sfb,
                                                  void* d, const int32_t* m_indices, int M_total, int N, int K, int G,
                                                  void* stream) {
    const dg_status s = check(a, sfa, b, sfb, d, M_total, N, K);
    if (s != DG_OK) return s;
    if (G <= 0 || m_indices == nullptr) return DG_ERR_INVALID_ARG;
    if (!is_aligned(m_indices, 4)) return DG_ERR_ALIGNMENT;
    SfF32Params p = params(sfa, sfb, d, M_total, N, K, G);
    p.meta = m_indices;
    return launch(dg::kContiguous, p, a, b, (static_cast<int64_t>(M_total) + dg::BM - 1) / dg::BM, 1, G, 128, stream);
}

dg_status m_grouped_fp8_gemm_nt_masked_sf_f32(const void* a, const float* sfa, const void* b, const float* sfb, void* d,
                                              const int32_t* masked_m, int G, int max_m, int N, int K, void* stream) {
    const dg_status s = check(a, sfa, b, sfb, d, max_m, N, K);
    if (s != DG_OK) return s;
    if (G <= 0 || masked_m == nullptr) return DG_ERR_INVALID_ARG;
    if (G > dg::MAX_MASKED_GROUPS) return DG_ERR_UNSUPPORTED;
    if (!is_aligned(masked_m, 4)) return DG_ERR_ALIGNMENT;
    SfF32Params p = params(sfa, sfb, d, max_m, N, K, G);
    p.meta = masked_m;
    const int64_t per_group = (static_cast<int64_t>(max_m) + dg::BM - 1) / dg::BM;
    return launch(dg::kMasked, p, a, b, G * per_group, G, G, 128, stream);
}

}  // extern "C"
