// gm_host.cuh - host-side helpers shared by the translation units of the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "../../include/gm.h"

// Every translation unit has its own device error word (gm_common.cuh); this reads and clears
// the one of gm_attn.cu on the current device.
__attribute__((visibility("hidden"))) bool gm_attn_take_errors(unsigned *flag);

namespace {

constexpr int64_t MAX_ROWS = (int64_t)1 << 31;  // edge rows B*n*heads indexed in 32 bits

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline gm_status launched()
{
    return cudaGetLastError() == cudaSuccess ? GM_OK : GM_ERR_CUDA;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (the library does not link
// the driver library itself).
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                                   CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                   CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

}  // namespace
