// api_util.h -- host-side helpers shared by the C ABI's source files.
#pragma once

#include <hip/hip_runtime.h>

#include <cstring>
#include <mutex>

#include "../../include/fp8bs.h"

#define FP8BS_EXPORT extern "C" __attribute__((visibility("default")))

namespace fp8bs_api {

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// gfx950 check, cached per device ordinal.
inline int check_device() {
    static std::mutex mu;
    static int cache[64];  // 0 unknown, 1 ok, 2 not ok
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return FP8BS_ERR_DEVICE;
    if (dev < 64) {
        std::lock_guard<std::mutex> lk(mu);
        if (cache[dev] == 1) return FP8BS_OK;
        if (cache[dev] == 2) return FP8BS_ERR_DEVICE;
    }
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return FP8BS_ERR_DEVICE;
    const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    if (dev < 64) {
        std::lock_guard<std::mutex> lk(mu);
        cache[dev] = ok ? 1 : 2;
    }
    return ok ? FP8BS_OK : FP8BS_ERR_DEVICE;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? FP8BS_OK : FP8BS_ERR_HIP; }

}  // namespace fp8bs_api
