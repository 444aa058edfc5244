// Host-side argument checks and the NVTX range shared by the entry points.
#pragma once

#include <nvtx3/nvToolsExt.h>

#include "common.cuh"

namespace fathom {

// NVTX range over one library call.
struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A pointer the current device can dereference: device or managed memory,
// or page-locked host memory mapped into the device's address space.
inline int check_device_ptr(const void* p)
{
    if (!p) return FATHOM_ERR_INVALID_ARG;
    cudaPointerAttributes attr;
    const cudaError_t e = cudaPointerGetAttributes(&attr, p);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return FATHOM_ERR_INVALID_ARG;
    }
    switch (attr.type) {
        case cudaMemoryTypeDevice:
        case cudaMemoryTypeManaged:
            return FATHOM_OK;
        case cudaMemoryTypeHost:
            return attr.devicePointer == p ? FATHOM_OK : FATHOM_ERR_INVALID_ARG;
        default:
            return FATHOM_ERR_INVALID_ARG;
    }
}

inline bool dims_ok(int D, int G) { return D >= 32 && D <= kMaxD && D % 32 == 0 && G >= 1 && G <= kMaxG; }

}  // namespace fathom
