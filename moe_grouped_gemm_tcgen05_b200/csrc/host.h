// Host-side parts that the library's sources share: the set-up of the current
// device, the process-wide switches and small launch helpers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dgb200.h"

namespace dg {

struct HostDevice {
    int device;        // ordinal
    int sms;           // multiprocessors
    uint32_t* status;  // device status word (DG_DEVERR_* bits)
};

// The current device, set up on its first use (dgb200.cu).
dg_status host_device(HostDevice* out);
// Tensor map of a K-major E4M3 operand [mats, rows, k] in boxes of 128 bytes of K by box_rows rows.
bool host_encode_kmajor(CUtensorMap* map, const void* base, int rank, int64_t k, int64_t rows, int64_t mats,
                        int box_rows);
// The overrides of dgb200_set_block_n, _set_cta_group and _set_splits (0: none).
void host_forced_tile(int* block_n, int* cta_group, int* splits);
uint64_t host_wait_limit_ns();  // bound of every wait inside a kernel
int host_test_mode();           // dgb200_set_test_hooks
bool host_pdl();                // DGB200_PDL
bool host_log();                // DGB200_LOG

// Kernel attributes and co-resident units of the GEMMs with fp32 scales on the
// current device (gemm_sf_f32.cu); part of the device's set-up.
dg_status setup_sf_f32(int device, int sms);

// Kernel attributes and cluster size of the calls around the experts' products on
// the current device (moe.cu).
dg_status setup_moe(int device);

inline bool is_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A launch with programmatic stream serialization (unless switched off) and
// room for a second attribute. `attr` must outlive the launch.
inline cudaLaunchConfig_t host_launch(unsigned blocks, int threads, size_t smem, void* stream,
                                      cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 0;
    if (host_pdl()) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 1;
    }
    return cfg;
}

}  // namespace dg
