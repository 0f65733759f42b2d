// abi_internal.h -- what the translation units behind the C ABI share: error
// reporting, the per-device state, library-owned workspaces and the driver's
// tensor-map encoder.  Host-side; not installed.
#pragma once

#include "../../include/nvfp4_gemv.h"
#include "internal.h"

namespace nvfp4 {

// Sets the thread's nvfp4_last_error() message and returns `st`.
nvfp4_status fail(nvfp4_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
nvfp4_status cuda_fail(cudaError_t e, const char *what);

struct DeviceState {
    bool ready = false;
    int sms = 0;
    int smem_optin = 0;
    int major = 0, minor = 0;
    unsigned *err_word = nullptr;
};
nvfp4_status device_state(int dev, DeviceState **out);
inline nvfp4_status current_device(int *dev, DeviceState **d) {
    cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    return device_state(*dev, d);
}
inline bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Library-owned workspaces, one per device, stream and kind: the GEMV's and
// the attention's counters and partial results must not share memory.
enum WorkspaceKind { kWsGemv = 0, kWsAttn = 1 };
nvfp4_status stream_workspace(int dev, cudaStream_t stream, WorkspaceKind kind, size_t bytes, void **out);

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
nvfp4_status get_encode_fn(EncodeTiledFn *fn);

}  // namespace nvfp4
