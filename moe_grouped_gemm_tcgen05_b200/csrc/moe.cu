// Host side of the calls around the experts' products (include/dgb200.h:
// moe_route and its gradient, moe_rows_*, moe_dispatch_fp8,
// quantize_fp8_1x128_sf_f32, moe_combine and its gradient): checks of the
// scalars and pointers, the choice of an instantiation by the sizes, one
// launch on the caller's stream. No call allocates, synchronises or reads a
// device value.
#include "host.h"
#include "moe_kernels.cuh"

namespace {

using dg::is_aligned;

constexpr int64_t kMaxInt = 0x7FFFFFFF;
constexpr int64_t kMaxValues = int64_t{1} << 40;  // of an operand

dg_status launched(cudaError_t err) { return err == cudaSuccess ? DG_OK : DG_ERR_CUDA; }

// Registers per lane for E experts: the smallest of the built ones that hold
// them. (A group of experts then fills whole lanes more often than with powers
// of two alone: 160 experts in 8 groups of 20 are 4 lanes of 5.)
constexpr int kLaneExperts[] = {1, 2, 3, 4, 5, 6, 8, 12, 16, 32};

int lane_experts(int E) {
    for (int v : kLaneExperts)
        if (32 * v >= E) return v;
    return 0;
}

template <typename Params>
using RouteFn = void (*)(Params);

template <bool F32>
RouteFn<dg::RouteParams> route_fn(int v) {
    switch (v) {
        case 1: return dg::moe_route_kernel<1, F32>;
        case 2: return dg::moe_route_kernel<2, F32>;
        case 3: return dg::moe_route_kernel<3, F32>;
        case 4: return dg::moe_route_kernel<4, F32>;
        case 5: return dg::moe_route_kernel<5, F32>;
        case 6: return dg::moe_route_kernel<6, F32>;
        case 8: return dg::moe_route_kernel<8, F32>;
        case 12: return dg::moe_route_kernel<12, F32>;
        case 16: return dg::moe_route_kernel<16, F32>;
        default: return dg::moe_route_kernel<32, F32>;
    }
}

template <bool F32, bool EXACT_REST>
RouteFn<dg::RouteBackwardParams> route_backward_fn(int v) {
    switch (v) {
        case 1: return dg::moe_route_backward_kernel<1, F32, EXACT_REST>;
        case 2: return dg::moe_route_backward_kernel<2, F32, EXACT_REST>;
        case 3: return dg::moe_route_backward_kernel<3, F32, EXACT_REST>;
        case 4: return dg::moe_route_backward_kernel<4, F32, EXACT_REST>;
        case 5: return dg::moe_route_backward_kernel<5, F32, EXACT_REST>;
        case 6: return dg::moe_route_backward_kernel<6, F32, EXACT_REST>;
        case 8: return dg::moe_route_backward_kernel<8, F32, EXACT_REST>;
        case 12: return dg::moe_route_backward_kernel<12, F32, EXACT_REST>;
        case 16: return dg::moe_route_backward_kernel<16, F32, EXACT_REST>;
        default: return dg::moe_route_backward_kernel<32, F32, EXACT_REST>;
    }
}

bool flag(int v) { return v == 0 || v == 1; }

// T tokens of E experts, k of them chosen.
dg_status check_route_sizes(int T, int E, int k) {
    if (T <= 0 || E <= 0 || k <= 0 || k > E) return DG_ERR_INVALID_ARG;
    if (E > dg::MOE_MAX_EXPERTS || k > dg::MOE_MAX_TOPK || T > (1 << 30)) return DG_ERR_UNSUPPORTED;
    return DG_OK;
}

// A warp per token; `cap` bounds the blocks (0: none), whose warps then take several.
unsigned route_blocks(int T, int64_t cap) {
    const int per = dg::ROUTE_THREADS / 32;
    const int64_t n = (static_cast<int64_t>(T) + per - 1) / per;
    return static_cast<unsigned>(cap > 0 && n > cap ? cap : n);
}

// One cluster for n choices: a single CTA while its warps have little to count,
// else 16, or as many as the device has a place for (65536 choices of 256
// experts 9.4 us, with 8 CTAs 12.0).
constexpr int kRowsOneCta = 4096;
constexpr int kMaxDevices = 64;
unsigned g_rows_cluster[kMaxDevices];

cudaLaunchConfig_t rows_config(unsigned ctas, int smem, void* stream, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = dg::host_launch(ctas, dg::ROWS_THREADS, static_cast<size_t>(smem), stream, attr);
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = ctas;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
    return cfg;
}

dg_status rows_launch(dg::RowsParams& p, void* stream) {
    dg::HostDevice dev;
    const dg_status s = dg::host_device(&dev);
    if (s != DG_OK) return s;
    unsigned ctas = p.n <= kRowsOneCta ? 1 : g_rows_cluster[dev.device];
    if (dg::host_test_mode() == 2 && ctas > 8) ctas = 8;  // (the hook of a device with no place for more)
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = rows_config(ctas, dg::rows_smem_bytes(p.groups), stream, attr);
    return launched(cudaLaunchKernelEx(&cfg, dg::moe_rows_kernel, p));
}

dg_status check_rows(const int32_t* ids, const int32_t* row_of, const int32_t* meta, const int32_t* counts, int T,
                     int k, int G) {
    if (!ids || !row_of || !meta || !counts || T <= 0 || k <= 0 || G <= 0) return DG_ERR_INVALID_ARG;
    if (G > dg::MOE_MAX_EXPERTS || k > dg::MOE_MAX_TOPK) return DG_ERR_UNSUPPORTED;
    if (!is_aligned(ids, 4) || !is_aligned(row_of, 4) || !is_aligned(meta, 4) || !is_aligned(counts, 4))
        return DG_ERR_ALIGNMENT;
    return DG_OK;
}

// The rows that T*k choices can take in whole 128-row blocks, however they fall.
int64_t row_bound(int64_t T, int64_t k, int64_t G) {
    const int64_t n = T * k;
    return (n + (G < n ? G : n) * 127 + 127) / 128 * 128;
}

dg_status dispatch_launch(const dg::DispatchParams& p, int x_f32, int sf_f32, void* stream) {
    dg::HostDevice dev;
    const dg_status s = dg::host_device(&dev);
    if (s != DG_OK) return s;
    const int64_t warps = static_cast<int64_t>(p.tokens) * p.kp;
    const int64_t blocks = (warps + dg::DISPATCH_THREADS / 32 - 1) / (dg::DISPATCH_THREADS / 32);
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg =
        dg::host_launch(static_cast<unsigned>(blocks), dg::DISPATCH_THREADS, 0, stream, attr);
    if (x_f32)
        return launched(sf_f32 ? cudaLaunchKernelEx(&cfg, dg::moe_dispatch_fp8_kernel<true, true>, p)
                               : cudaLaunchKernelEx(&cfg, dg::moe_dispatch_fp8_kernel<true, false>, p));
    return launched(sf_f32 ? cudaLaunchKernelEx(&cfg, dg::moe_dispatch_fp8_kernel<false, true>, p)
                           : cudaLaunchKernelEx(&cfg, dg::moe_dispatch_fp8_kernel<false, false>, p));
}

// y [rows, H], row_of / w [T, k], token-shaped [T, H]
dg_status check_combine(const void* y, const int32_t* row_of, const float* w, const void* tokens, int64_t rows, int T,
                        int k, int H) {
    if (!y || !row_of || !tokens || rows <= 0 || T <= 0 || k <= 0 || H <= 0) return DG_ERR_INVALID_ARG;
    if (H % 8 != 0) return DG_ERR_INVALID_ARG;
    if (k > dg::MOE_MAX_TOPK || rows > kMaxInt || rows * H >= kMaxValues || static_cast<int64_t>(T) * H >= kMaxValues)
        return DG_ERR_UNSUPPORTED;
    if (!is_aligned(y, 16) || !is_aligned(tokens, 16) || !is_aligned(row_of, 4) || !is_aligned(w, 4))
        return DG_ERR_ALIGNMENT;
    return DG_OK;
}

// One warp's step and an index past the end stay below 2^31.
constexpr int64_t kMaxChoices = int64_t{1} << 30;

}  // namespace

namespace dg {

dg_status setup_moe(int device) {
    if (g_rows_cluster[device] != 0) return DG_OK;
    // (one value for every call: calls on several threads share the attribute)
    if (cudaFuncSetAttribute(moe_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             rows_smem_bytes(MOE_MAX_EXPERTS)) != cudaSuccess ||
        cudaFuncSetAttribute(moe_rows_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return DG_ERR_CUDA;
    // the largest cluster that the device can hold (a part of a GPU may lack a place for 16 CTAs)
    unsigned ctas = ROWS_MAX_CLUSTER;
    for (; ctas > 1; ctas /= 2) {
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = rows_config(ctas, rows_smem_bytes(MOE_MAX_EXPERTS), nullptr, attr);
        int places = 0;
        if (cudaOccupancyMaxActiveClusters(&places, moe_rows_kernel, &cfg) == cudaSuccess && places > 0) break;
        cudaGetLastError();
    }
    g_rows_cluster[device] = ctas;
    return DG_OK;
}

}  // namespace dg

extern "C" {

dg_status moe_route(const void* logits, int logits_f32, const float* bias, int32_t* ids, float* weights, int T, int E,
                    int k, int score, int n_groups, int top_groups, int group_top, int renormalize, float scale,
                    void* stream) {
    if (!logits || !ids || !weights || !flag(logits_f32) || !flag(renormalize)) return DG_ERR_INVALID_ARG;
    dg_status s = check_route_sizes(T, E, k);
    if (s != DG_OK) return s;
    if (score != DG_SCORE_SOFTMAX && score != DG_SCORE_SIGMOID) return DG_ERR_INVALID_ARG;
    if (n_groups <= 0 || E % n_groups != 0 || top_groups <= 0 || top_groups > n_groups) return DG_ERR_INVALID_ARG;
    if (group_top != 1 && group_top != 2) return DG_ERR_INVALID_ARG;
    if (n_groups > dg::MOE_MAX_EXPERT_GROUPS) return DG_ERR_UNSUPPORTED;
    const int size = E / n_groups;
    if (k > top_groups * size) return DG_ERR_INVALID_ARG;  // fewer experts stay than are to be chosen
    if (!is_aligned(logits, logits_f32 ? 4 : 2) || !is_aligned(bias, 4) || !is_aligned(ids, 4) ||
        !is_aligned(weights, 4))
        return DG_ERR_ALIGNMENT;
    dg::HostDevice dev;
    if ((s = dg::host_device(&dev)) != DG_OK) return s;
    const dg::RouteParams p{logits, bias, ids, weights, T, E, k, n_groups, top_groups,
                            group_top < size ? group_top : size, score == DG_SCORE_SOFTMAX ? 1 : 0, renormalize, scale};
    const int v = lane_experts(E);
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg =
        dg::host_launch(route_blocks(T, static_cast<int64_t>(dev.sms) * 4), dg::ROUTE_THREADS, 0, stream, attr);
    return launched(cudaLaunchKernelEx(&cfg, logits_f32 ? route_fn<true>(v) : route_fn<false>(v), p));
}

dg_status moe_route_backward(const void* logits, int logits_f32, const int32_t* ids, const float* d_weights,
                             void* d_logits, int T, int E, int k, int score, int renormalize, float scale,
                             void* stream) {
    if (!logits || !ids || !d_weights || !d_logits || !flag(logits_f32) || !flag(renormalize))
        return DG_ERR_INVALID_ARG;
    dg_status s = check_route_sizes(T, E, k);
    if (s != DG_OK) return s;
    if (score != DG_SCORE_SOFTMAX && score != DG_SCORE_SIGMOID) return DG_ERR_INVALID_ARG;
    if (logits == d_logits) return DG_ERR_INVALID_ARG;  // the row is written before the choices are done with it
    const uintptr_t size = logits_f32 ? 4 : 2;
    if (!is_aligned(logits, size) || !is_aligned(d_logits, size) || !is_aligned(ids, 4) || !is_aligned(d_weights, 4))
        return DG_ERR_ALIGNMENT;
    dg::HostDevice dev;
    if ((s = dg::host_device(&dev)) != DG_OK) return s;
    const dg::RouteBackwardParams p{logits, ids, d_weights, d_logits, T, E, k, score == DG_SCORE_SOFTMAX ? 1 : 0,
                                    renormalize, scale};
    const int v = lane_experts(E);
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = dg::host_launch(route_blocks(T, 0), dg::ROUTE_THREADS, 0, stream, attr);
    if (p.softmax && !p.renorm)
        return launched(cudaLaunchKernelEx(
            &cfg, logits_f32 ? route_backward_fn<true, true>(v) : route_backward_fn<false, true>(v), p));
    return launched(cudaLaunchKernelEx(
        &cfg, logits_f32 ? route_backward_fn<true, false>(v) : route_backward_fn<false, false>(v), p));
}

int64_t moe_rows_bound(int T, int k, int G) {
    if (T <= 0 || k <= 0 || G <= 0) return 0;
    return row_bound(T, k, G);
}

dg_status moe_rows_contiguous(const int32_t* ids, int32_t* row_of, int32_t* m_indices, int32_t* counts, int T, int k,
                              int G, int64_t m_rows, void* stream) {
    const dg_status s = check_rows(ids, row_of, m_indices, counts, T, k, G);
    if (s != DG_OK) return s;
    if (m_rows < row_bound(T, k, G)) return DG_ERR_INVALID_ARG;
    if (m_rows > kMaxInt - 128 || static_cast<int64_t>(T) * k > kMaxChoices) return DG_ERR_UNSUPPORTED;
    dg::RowsParams p{ids, row_of, m_indices, counts, T * k, G, static_cast<int>(m_rows), 0};
    return rows_launch(p, stream);
}

dg_status moe_rows_masked(const int32_t* ids, int32_t* row_of, int32_t* masked_m, int32_t* counts, int T, int k, int G,
                          int max_m, void* stream) {
    const dg_status s = check_rows(ids, row_of, masked_m, counts, T, k, G);
    if (s != DG_OK) return s;
    if (max_m <= 0) return DG_ERR_INVALID_ARG;
    if (static_cast<int64_t>(T) * k > kMaxChoices || static_cast<int64_t>(G) * max_m > kMaxInt - kMaxChoices)
        return DG_ERR_UNSUPPORTED;
    dg::RowsParams p{ids, row_of, masked_m, counts, T * k, G, 0, max_m};
    return rows_launch(p, stream);
}

dg_status moe_dispatch_fp8(const void* x, int x_f32, const int32_t* row_of, void* q, void* sf, int sf_f32,
                           int64_t rows, int T, int k, int H, void* stream) {
    if (!x || !row_of || !q || !sf || !flag(x_f32) || !flag(sf_f32)) return DG_ERR_INVALID_ARG;
    if (rows <= 0 || T <= 0 || k <= 0 || H <= 0 || H % 128 != 0) return DG_ERR_INVALID_ARG;
    if (k > dg::MOE_MAX_TOPK || rows > kMaxInt || H > (1 << 20) || rows * H >= kMaxValues ||
        static_cast<int64_t>(T) * H >= kMaxValues)
        return DG_ERR_UNSUPPORTED;
    if (!is_aligned(x, 16) || !is_aligned(q, 16) || !is_aligned(row_of, 4) || !is_aligned(sf, 4))
        return DG_ERR_ALIGNMENT;
    const int kb = H / 128;
    return dispatch_launch({x, row_of, static_cast<uint4*>(q), sf, rows, T, k, kb, (kb + 3) / 4}, x_f32, sf_f32,
                           stream);
}

dg_status quantize_fp8_1x128_sf_f32(const void* x, int x_f32, void* q, float* sf, int64_t rows, int K, void* stream) {
    if (!x || !q || !sf || rows <= 0 || K <= 0 || !flag(x_f32) || K % 128 != 0) return DG_ERR_INVALID_ARG;
    if (rows > kMaxInt || K > (1 << 20) || rows * K >= kMaxValues) return DG_ERR_UNSUPPORTED;
    if (!is_aligned(x, 16) || !is_aligned(q, 16) || !is_aligned(sf, 4)) return DG_ERR_ALIGNMENT;
    const int kb = K / 128;
    return dispatch_launch({x, nullptr, static_cast<uint4*>(q), sf, rows, static_cast<int>(rows), 1, kb, (kb + 3) / 4},
                           x_f32, 1, stream);
}

dg_status moe_combine(const void* y, const int32_t* row_of, const float* weights, void* out, int64_t rows, int T, int k,
                      int H, void* stream) {
    dg_status s = check_combine(y, row_of, weights, out, rows, T, k, H);
    if (s != DG_OK) return s;
    dg::HostDevice dev;
    if ((s = dg::host_device(&dev)) != DG_OK) return s;
    const dg::CombineParams p{static_cast<const uint4*>(y), row_of, weights, static_cast<uint4*>(out), rows, T, k,
                              H / 8};
    const int64_t blocks = (static_cast<int64_t>(T) * p.vecs + dg::COMBINE_THREADS - 1) / dg::COMBINE_THREADS;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = dg::host_launch(static_cast<unsigned>(blocks), dg::COMBINE_THREADS, 0, stream, attr);
    return launched(cudaLaunchKernelEx(&cfg, dg::moe_combine_kernel, p));
}

dg_status moe_combine_backward(const void* y, const int32_t* row_of, const float* weights, const void* d_out, void* d_y,
                               float* d_weights, int64_t rows, int T, int k, int H, void* stream) {
    if (!d_y || !d_weights || d_y == y) return DG_ERR_INVALID_ARG;
    dg_status s = check_combine(y, row_of, weights, d_out, rows, T, k, H);
    if (s != DG_OK) return s;
    if (!is_aligned(d_y, 16) || !is_aligned(d_weights, 4)) return DG_ERR_ALIGNMENT;
    dg::HostDevice dev;
    if ((s = dg::host_device(&dev)) != DG_OK) return s;
    const dg::CombineBackwardParams p{static_cast<const uint4*>(y), row_of, weights, static_cast<const uint4*>(d_out),
                                      static_cast<uint4*>(d_y), d_weights, rows, T, k, H / 8};
    int threads = (p.vecs + 31) / 32 * 32;
    if (threads > dg::COMBINE_THREADS) threads = dg::COMBINE_THREADS;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = dg::host_launch(static_cast<unsigned>(T), threads, 0, stream, attr);
    return launched(cudaLaunchKernelEx(&cfg, dg::moe_combine_backward_kernel, p));
}

}  // extern "C"
