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

// A device array of 32-bit words: what a call writes may not overlap what it reads, or what else it
// writes, as its CTAs do both at once.
struct Words {
    const char *name;
    const void *data;
    int64_t n;
};
inline bool overlap(const Words &a, const Words &b)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.data), y = reinterpret_cast<uintptr_t>(b.data);
    return a.n > 0 && b.n > 0 && x < y + 4 * static_cast<uintptr_t>(b.n) && y < x + 4 * static_cast<uintptr_t>(a.n);
}
// Words from a table's first entry to its last.
inline int64_t extent_of(int64_t rows, int64_t row, int64_t width) { return rows > 0 ? (rows - 1) * row + width : 0; }
// `out` against each of `n` others.
inline int check_apart(const char *fn, const Words &out, const Words *others, int n)
{
    for (int i = 0; i < n; ++i)
        if (overlap(out, others[i])) return fail_call(UB_ERR_ARG, "%s: %s overlaps %s", fn, out.name, others[i].name);
    return UB_OK;
}

inline int cuda_failed(cudaError_t e, const char *what)
{
    return fail_call(UB_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

}  // namespace
}  // namespace ubk
