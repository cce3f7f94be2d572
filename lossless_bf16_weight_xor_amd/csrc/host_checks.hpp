// host_checks.hpp -- argument checks shared by the host side of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <vector>

#include "bf16delta.h"

namespace bf16d {

constexpr uint64_t kMaxTiles = 1ull << 24;   // grid limit: tiles * 256 threads < 2^32
constexpr uint64_t kMaxSize = UINT64_MAX >> 2;   // element counts and byte sizes: at most 2^62

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
    uintptr_t lo, hi;   // [lo, hi)
    bool written;
};

// A written range may overlap no other range; read ranges may overlap each other.
inline bool ranges_disjoint(std::vector<Range> &v) {
    v.erase(std::remove_if(v.begin(), v.end(), [](const Range &r) { return r.hi <= r.lo; }),
            v.end());
    std::sort(v.begin(), v.end(), [](const Range &a, const Range &b) { return a.lo < b.lo; });
    // sweep: compare each range with the furthest-reaching earlier written range
    // and the furthest-reaching earlier range of any kind
    uintptr_t reach_any = 0, reach_written = 0;
    for (const Range &r : v) {
        if (r.lo < reach_written) return false;
        if (r.written && r.lo < reach_any) return false;
        reach_any = std::max(reach_any, r.hi);
        if (r.written) reach_written = std::max(reach_written, r.hi);
    }
    return true;
}

inline void add_range(std::vector<Range> &v, const void *p, uint64_t bytes, bool written) {
    v.push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes, written});
}

inline bool device_of(hipStream_t stream, int32_t &out) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) return false;
    out = dev;
    return true;
}

// BF16D_OK if `stream` belongs to the current device
inline int stream_on_current(hipStream_t stream, int32_t &dev) {
    if (!device_of(stream, dev)) return BF16D_EHIP;
    if (stream) {
        hipDevice_t sdev = -1;
        if (hipStreamGetDevice(stream, &sdev) != hipSuccess) return BF16D_EHIP;
        if (sdev != dev) return BF16D_EINVAL;
    }
    return BF16D_OK;
}

}  // namespace bf16d
