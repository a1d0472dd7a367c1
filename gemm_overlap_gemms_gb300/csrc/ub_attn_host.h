// What the host files of the attention and cache operators (ub_attn_api.cu, ub_pages_api.cu)
// share: the device of a call, its timeline range, its pointer and error helpers.
#pragma once

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>
#include <stdint.h>

#include "ub_attn.h"

namespace ubk {
namespace {

struct DeviceScope {
    int prev = -1;
    bool ok = true;
    explicit DeviceScope(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess || (prev != dev && cudaSetDevice(dev) != cudaSuccess)) ok = false;
        if (prev == dev) prev = -1;
    }
    ~DeviceScope()
    {
        if (ok && prev >= 0) cudaSetDevice(prev);
    }
};

struct Range {
    explicit Range(const char *name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int cuda_failed(cudaError_t e, const char *what)
{
    return fail_call(UB_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

}  // namespace
}  // namespace ubk
