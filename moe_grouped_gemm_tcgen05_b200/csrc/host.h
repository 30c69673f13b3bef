// Host-side parts that the library's sources share: the set-up of the current
// device, the process-wide switches and small launch helpers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

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
PFN_cuTensorMapEncodeTiled_v12000 host_tensor_map_encode();
uint64_t host_wait_limit_ns();  // bound of every wait inside a kernel
int host_test_mode();           // dgb200_set_test_hooks
bool host_pdl();                // DGB200_PDL
bool host_log();                // DGB200_LOG

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
