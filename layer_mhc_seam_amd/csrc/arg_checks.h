// arg_checks.h -- what the block and cache operators' entry points share:
// alignment and overlap rules, the current device's compute units.
#pragma once

#include <atomic>
#include <cstdint>
#include <initializer_list>

#include "seam_internal.h"

namespace mhc {
namespace {

constexpr int64_t kMaxElements = int64_t(1) << 40;

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool half_type(int d) { return d == MHC_BF16 || d == MHC_F16; }

int64_t size_of(int d) { return d == MHC_F32 ? 4 : 2; }

struct Range {
    const void *p;
    int64_t bytes;
};

bool overlap(const Range &a, const Range &b)
{
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0)
        return false;
    const uintptr_t al = reinterpret_cast<uintptr_t>(a.p), bl = reinterpret_cast<uintptr_t>(b.p);
    return al < bl + (uintptr_t)b.bytes && bl < al + (uintptr_t)a.bytes;
}

// Whether an output overlaps an input or another output
bool clash(std::initializer_list<Range> outs, std::initializer_list<Range> ins)
{
    for (const Range *o = outs.begin(); o != outs.end(); ++o) {
        for (const Range &i : ins)
            if (overlap(*o, i))
                return true;
        for (const Range *q = outs.begin(); q != o; ++q)
            if (overlap(*o, *q))
                return true;
    }
    return false;
}

// Compute units of the current device, asked for once per device
hipError_t compute_units(int *cus)
{
    static std::atomic<int> known[64];
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return e;
    if (dev >= 0 && dev < 64 && (*cus = known[dev].load(std::memory_order_relaxed)) > 0)
        return hipSuccess;
    e = hipDeviceGetAttribute(cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e == hipSuccess && dev >= 0 && dev < 64)
        known[dev].store(*cus, std::memory_order_relaxed);
    return e;
}

}  // namespace
}  // namespace mhc
