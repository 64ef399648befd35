// Host-side checks shared by the C entry points: element types, alignment,
// memory ranges, size bounds, and the device the kernels are built for.
#pragma once

#include "mamba_amd.h"

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <mutex>

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;  // B*D*L bound (keeps every index in int64)

bool valid_dtype(int dt) { return dt == MAMBA_F32 || dt == MAMBA_BF16; }
size_t esize(mamba_dtype dt) { return dt == MAMBA_BF16 ? 2 : 4; }

bool aligned(const void *p, size_t a) { return p == nullptr || (uintptr_t)p % a == 0; }

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};
Range rng(const void *p, size_t bytes) { return {(uintptr_t)p, (uintptr_t)p + bytes}; }
bool overlap(Range a, Range b)
{
    if (a.lo == 0 || b.lo == 0 || a.hi == a.lo || b.hi == b.lo)
        return false;
    return a.lo < b.hi && b.lo < a.hi;
}

// Non-negative sizes; each, and the product of the non-zero ones, at most
// kMaxElems (so an empty dimension leaves the others bounded too).
bool sizes_ok(int64_t a, int64_t b, int64_t c)
{
    if (a < 0 || b < 0 || c < 0)
        return false;
    int64_t p = 1;
    for (const int64_t v : {a, b, c}) {
        if (v == 0)
            continue;
        if (v > kMaxElems || p > kMaxElems / v)
            return false;
        p *= v;
    }
    return true;
}

// The kernels are built for gfx950 only.
mamba_status device_ok()
{
    static std::mutex mu;
    static int checked[64] = {0};  // 0 unknown, 1 ok, 2 bad
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0)
        return MAMBA_ERR_DEVICE;
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 64)
        return MAMBA_ERR_DEVICE;
    if (checked[dev] == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess)
            return MAMBA_ERR_DEVICE;
        checked[dev] = (std::strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
    }
    return checked[dev] == 1 ? MAMBA_OK : MAMBA_ERR_DEVICE;
}

mamba_status launched(hipError_t e) { return e == hipSuccess ? MAMBA_OK : MAMBA_ERR_LAUNCH; }

}  // namespace
