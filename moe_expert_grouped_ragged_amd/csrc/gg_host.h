// Host helpers shared by the C-ABI files: the device a call runs on, buffer
// ranges and their overlap, alignment, and the optional check of the offsets.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include "gg.h"

namespace gg {

struct DeviceInfo {
    int checked = 0;      // 0 unknown, 1 gfx950, -1 other
    int num_cu = 0;
    int device = 0;       // device index
};

constexpr int kMaxDevices = 64;
inline DeviceInfo g_dev[kMaxDevices];
inline std::mutex g_dev_mu;

// Properties of the device the work will run on: the stream's device, or the
// current device for the null stream.
inline int device_info(hipStream_t stream, DeviceInfo* out) {
    int dev = 0;
    if (stream == nullptr) {
        if (hipGetDevice(&dev) != hipSuccess) return GG_ERR_HIP;
    } else {
        hipDevice_t d = 0;
        if (hipStreamGetDevice(stream, &d) != hipSuccess) return GG_ERR_HIP;
        dev = static_cast<int>(d);
    }
    if (dev < 0 || dev >= kMaxDevices) return GG_ERR_UNSUPPORTED_DEVICE;
    std::lock_guard<std::mutex> lock(g_dev_mu);
    DeviceInfo& d = g_dev[dev];
    if (d.checked == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return GG_ERR_HIP;
        const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
        d.num_cu = prop.multiProcessorCount;
        d.device = dev;
        d.checked = ok ? 1 : -1;
    }
    if (d.checked != 1) return GG_ERR_UNSUPPORTED_DEVICE;
    *out = d;
    return GG_OK;
}

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};

inline Range range_of(const void* p, size_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Range{a, a + bytes};
}

inline bool overlap(Range a, Range b) {
    return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Outputs must not overlap any input nor each other (an empty range overlaps nothing).
inline int check_aliasing(std::initializer_list<Range> ins, std::initializer_list<Range> outs) {
    for (const Range* o = outs.begin(); o != outs.end(); ++o) {
        for (const Range& r : ins)
            if (overlap(*o, r)) return GG_ERR_ALIASING;
        for (const Range* p = o + 1; p != outs.end(); ++p)
            if (overlap(*o, *p)) return GG_ERR_ALIASING;
    }
    return GG_OK;
}

// Optional synchronous check of the device offsets (GG_DEBUG_VALIDATE=1, read
// at every call so that a process can switch it on and off).
inline int debug_validate_offsets(const int64_t* offsets, int64_t E, int64_t M, hipStream_t stream) {
    const char* v = std::getenv("GG_DEBUG_VALIDATE");
    if (!(v && v[0] == '1')) return GG_OK;
    int64_t h[GG_MAX_EXPERTS + 1];   // E <= GG_MAX_EXPERTS is checked before
    if (hipMemcpyAsync(h, offsets, sizeof(int64_t) * (E + 1), hipMemcpyDeviceToHost, stream) !=
            hipSuccess ||
        hipStreamSynchronize(stream) != hipSuccess)
        return GG_ERR_HIP;
    if (h[0] < 0 || h[E] > M) return GG_ERR_INVALID_ARGUMENT;
    for (int64_t e = 0; e < E; ++e)
        if (h[e + 1] < h[e]) return GG_ERR_INVALID_ARGUMENT;
    return GG_OK;
}

// Slope of the gate activation's sigmoid, or 0 for an unknown activation.
inline float act_slope(int activation) {
    switch (activation) {
        case GG_ACT_SWIGLU: return 1.0f;
        case GG_ACT_QGEGLU: return 1.702f;
        default: return 0.0f;
    }
}

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace gg
