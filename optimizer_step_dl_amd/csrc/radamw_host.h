// radamw_host.h -- host-side checks shared by the C entry points.  Not part
// of the public ABI.
#pragma once

#include "radamw.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>
#include <map>
#include <vector>

namespace radamw {

extern std::atomic<uint64_t> g_launches;  // radamw_launch_count
extern thread_local int g_last_hip;       // radamw_last_hip_error

constexpr int MAX_DEVICES = 64;

inline int hip_status(hipError_t e) {
    if (e == hipSuccess) return RADAMW_OK;
    g_last_hip = static_cast<int>(e);
    return RADAMW_ERR_HIP;
}

// Temporarily make `dev` the calling thread's current device.
struct DeviceScope {
    int prev = -1;
    explicit DeviceScope(int dev) {
        if (hipGetDevice(&prev) != hipSuccess) prev = -1;
        if (prev != dev) (void)hipSetDevice(dev);
    }
    ~DeviceScope() {
        int cur = -1;
        if (prev >= 0 && hipGetDevice(&cur) == hipSuccess && cur != prev) (void)hipSetDevice(prev);
    }
};

// The device of `stream`; a stream being captured into a graph is refused
// (a replay would repeat one step's host-formed coefficients, and a fused
// step waits for its own kernels, which a capture never runs).
inline int stream_device(hipStream_t stream, int *dev) {
    hipDevice_t d = 0;
    hipError_t e = stream ? hipStreamGetDevice(stream, &d) : hipGetDevice(&d);
    hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
    if (e == hipSuccess) e = hipStreamIsCapturing(stream, &capture);
    if (e != hipSuccess) {
        (void)hipGetLastError();
        g_last_hip = static_cast<int>(e);
        return RADAMW_ERR_INVALID;
    }
    if (capture != hipStreamCaptureStatusNone) return RADAMW_ERR_INVALID;
    if (d < 0 || d >= MAX_DEVICES) return RADAMW_ERR_INVALID;
    *dev = static_cast<int>(d);
    return RADAMW_OK;
}

inline bool valid_dtype(int gdt) { return gdt == RADAMW_F32 || gdt == RADAMW_F16 || gdt == RADAMW_BF16; }

inline size_t grad_bytes(int gdt) { return gdt == RADAMW_F32 ? 4 : 2; }

// Element counts above this are rejected (RADAMW_ERR_RANGE) before any byte
// size is formed, so n * element size cannot overflow; any tensor that fits
// in device memory is far below it.
constexpr int64_t MAX_ELEMENTS = int64_t(1) << 48;

// The allocation that holds p, which must be device (or managed) memory of
// device `dev`: its start and end, or 0, 0 when the extent is unknown (e.g.
// managed memory).
inline int query_extent(int dev, const void *p, uintptr_t *lo, uintptr_t *hi) {
    *lo = *hi = 0;
    hipPointerAttribute_t attr;
    std::memset(&attr, 0, sizeof attr);
    hipError_t e = hipPointerGetAttributes(&attr, p);
    if (e != hipSuccess) {
        (void)hipGetLastError();  // leave no sticky error behind for the caller
        return RADAMW_ERR_INVALID;
    }
    if (attr.type != hipMemoryTypeDevice && attr.type != hipMemoryTypeManaged) return RADAMW_ERR_INVALID;
    if (attr.device != dev) return RADAMW_ERR_INVALID;
    hipDeviceptr_t base = nullptr;
    size_t size = 0;
    e = hipMemGetAddressRange(&base, &size, const_cast<void *>(p));
    if (e != hipSuccess || !base || size == 0) {
        (void)hipGetLastError();
        return RADAMW_OK;  // type and device checked
    }
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(base);
    if (a < b || a >= b + size) return RADAMW_OK;
    *lo = b;
    *hi = b + size;
    return RADAMW_OK;
}

// Pointer validation for one call.  A pointer must be device (or managed)
// memory of the stream's device, aligned to its element size, and the bytes
// the call touches must lie inside the allocation that holds it.  Each
// allocation is queried once per call (hipPointerGetAttributes and
// hipMemGetAddressRange); later pointers into an allocation already seen are
// checked against its cached extent, so a list of many tensors carved from
// a few allocations costs a few HIP queries, not one per pointer.
class PtrChecker {
  public:
    explicit PtrChecker(int dev) : dev_(dev) {}

    int check(const void *p, size_t align, int64_t bytes) {
        if (!p) return RADAMW_ERR_INVALID;
        const uintptr_t a = reinterpret_cast<uintptr_t>(p);
        if (a % align != 0) return RADAMW_ERR_ALIGN;
        const uintptr_t end = a + static_cast<uintptr_t>(bytes > 0 ? bytes : 0);
        auto it = known_.upper_bound(a);
        if (it != known_.begin()) {
            --it;
            if (a >= it->first && a < it->second) return end <= it->second ? RADAMW_OK : RADAMW_ERR_INVALID;
        }
        uintptr_t lo = 0, hi = 0;
        const int rc = query_extent(dev_, p, &lo, &hi);
        if (rc != RADAMW_OK || hi == 0) return rc;
        known_[lo] = hi;
        return end <= hi ? RADAMW_OK : RADAMW_ERR_INVALID;
    }

  private:
    int dev_;
    std::map<uintptr_t, uintptr_t> known_;  // allocation base -> end
};

// Byte ranges touched by one call.  Written ranges may overlap nothing;
// read-only ranges may overlap each other.
struct Range {
    uintptr_t lo, hi;
    bool written;
};

inline void add_range(std::vector<Range> &v, const void *p, int64_t bytes, bool written) {
    if (p && bytes > 0) {
        uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        v.push_back({lo, lo + static_cast<uintptr_t>(bytes), written});
    }
}

// Sweep in start order: a written range must start after every earlier
// range ended; a read range must start after every earlier written range.
inline int check_alias(std::vector<Range> &v) {
    std::sort(v.begin(), v.end(), [](const Range &a, const Range &b) { return a.lo < b.lo; });
    uintptr_t end_any = 0, end_written = 0;
    for (const Range &r : v) {
        if (r.written ? r.lo < end_any : r.lo < end_written) return RADAMW_ERR_ALIAS;
        end_any = std::max(end_any, r.hi);
        if (r.written) end_written = std::max(end_written, r.hi);
    }
    return RADAMW_OK;
}

}  // namespace radamw
