// Host-side pieces shared by the translation units of the C ABI: error
// reporting, per-device state and the tensor-map encoder.  Defined in
// attn_api.cu; nothing here is exported from the library.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <string.h>

#include <mutex>

#include "../../include/attn.h"

namespace tab_host {

constexpr int kMaxDevices = 64;

// Records the detail text of the calling thread and returns `status`.
attn_status_t fail(attn_status_t status, const char *fmt, ...);
// Clears the detail text and returns ATTN_OK.
attn_status_t ok();

struct DeviceState {
    std::once_flag once;
    cudaError_t init_error = cudaSuccess;
    int *status = nullptr;  // device address of the status word
    int num_sms = 0;
};
// State of the current device, set up on first use.
attn_status_t device_state(DeviceState **out);

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// The driver's cuTensorMapEncodeTiled, or null.
EncodeTiledFn encode_fn();

// Launches `kernel` so that its blocks may start while what stands before it in
// the stream ends; the kernel waits for that end (wait_for_primary()) before
// it touches memory.
template <class... Args>
attn_status_t launch_dependent(void (*kernel)(Args...), dim3 grid, dim3 threads, cudaStream_t stream, size_t smem,
                                const Args &...args) {
    cudaLaunchAttribute attr;
    memset(&attr, 0, sizeof attr);
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config;
    memset(&config, 0, sizeof config);
    config.gridDim = grid;
    config.blockDim = threads;
    config.dynamicSmemBytes = smem;
    config.stream = stream;
    config.attrs = &attr;
    config.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&config, kernel, args...);
    if (e != cudaSuccess) return fail(ATTN_ERR_LAUNCH, "launch: %s", cudaGetErrorString(e));
    return ok();
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace tab_host
