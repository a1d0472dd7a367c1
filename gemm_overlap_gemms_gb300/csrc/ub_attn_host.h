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

// A device array of 32-bit words, or rows of them, `pitch` words apart (as wide or wider, where there
// are several): what a call writes may not overlap what it reads, or what else it writes, as its CTAs
// do both at once.
struct Words {
    const char *name;
    const void *data;
    int64_t width, rows, pitch;
};
inline Words words(const char *name, const void *data, int64_t n) { return {name, data, n, 1, n}; }
inline Words rows_of(const char *name, const void *data, int64_t rows, int64_t pitch, int64_t width)
{
    return {name, data, width, rows, rows > 1 ? pitch : width};
}
// Whether a word belongs to both. Rows of one table may lie between rows of the other.
inline bool overlap(const Words &a, const Words &b)
{
    if (a.rows > b.rows) return overlap(b, a);
    if (a.width <= 0 || a.rows <= 0 || b.width <= 0) return false;
    const int64_t pitch_a = 4 * a.pitch, pitch_b = 4 * b.pitch, wide_a = 4 * a.width, wide_b = 4 * b.width;
    // first byte of a row of `a`, counted from the first of `b`
    int64_t x = static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.data) - reinterpret_cast<uintptr_t>(b.data));
    if (x >= (b.rows - 1) * pitch_b + wide_b || x + (a.rows - 1) * pitch_a + wide_a <= 0) return false;
    for (int64_t r = 0; r < a.rows; ++r, x += pitch_a) {
        if (x + wide_a <= 0) continue;
        const int64_t last = (x + wide_a - 1) / pitch_b;  // the last row of `b` that begins before this one's end
        if ((last < b.rows ? last : b.rows - 1) * pitch_b + wide_b > x) return true;
    }
    return false;
}
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
