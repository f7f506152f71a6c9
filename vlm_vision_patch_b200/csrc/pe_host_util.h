// Host-side helpers shared by the translation units of libpe.so: the driver's
// tensor-map encoder, NVTX ranges, the exception barrier of the C ABI, argument
// predicates and the current-device guard.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cstdint>
#include <new>

#include "../../include/pe.h"

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    }
    return fn;
}

// One NVTX range per public call, named after it: visible on Nsight timelines
// and usable as an ncu filter (--nvtx --nvtx-include); without a tool attached
// the push and pop return at once.
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};

// Runs an entry point's body so that no C++ exception crosses the C ABI: a
// failed host allocation (the item tables and chunk plans are std::vectors)
// returns PE_ERR_HOST_MEMORY, anything else PE_ERR_CUDA.
template <class F>
pe_status no_throw(F &&body) {
    try {
        return body();
    } catch (const std::bad_alloc &) {
        return PE_ERR_HOST_MEMORY;
    } catch (...) {
        return PE_ERR_CUDA;
    }
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool valid_dtype(int d) { return d == PE_F32 || d == PE_BF16; }

struct DeviceGuard {
    int prev = -1;
    explicit DeviceGuard(int dev) {
        if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
        if (prev != dev) cudaSetDevice(dev);
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

inline pe_status finish(cudaError_t e) { return e == cudaSuccess ? PE_OK : PE_ERR_CUDA; }

}  // namespace
