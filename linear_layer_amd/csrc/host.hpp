// Host-side argument checks and the device check shared by the entry points of
// the 4-bit products and the residual norms.
#pragma once

#include <hip/hip_runtime.h>

#include <mutex>
#include <stdint.h>
#include <string.h>

#include "linear_layer.h"

namespace ll {
namespace host {

// Bytes from the first element of a rows x cols matrix to its last one's end
// (ld and the row width in elements of `elem` bytes); -1 where 64 bits or the
// address space do not hold them.
inline int64_t span(int64_t rows, int64_t cols, int64_t ld, int64_t elem)
{
    if (rows <= 0 || cols <= 0)
        return 0;
    int64_t reach, total;
    if (__builtin_mul_overflow(rows - 1, ld, &reach) || __builtin_add_overflow(reach, cols, &reach) ||
        __builtin_mul_overflow(reach, elem, &total))
        return -1;
    return total;
}

inline bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p % n) == 0; }

// A range of device memory an entry point reads or writes.
struct Range {
    const void *p;
    int64_t bytes;
};

inline bool overlap(const Range &a, const Range &b)
{
    if (a.p == nullptr || b.p == nullptr || a.bytes <= 0 || b.bytes <= 0)
        return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + (uintptr_t)b.bytes && b0 < a0 + (uintptr_t)a.bytes;
}

// Whether any of the outputs w[0..nw) meets another output or an input r[0..nr).
inline bool any_overlap(const Range *w, int nw, const Range *r, int nr)
{
    for (int i = 0; i < nw; ++i) {
        for (int j = i + 1; j < nw; ++j)
            if (overlap(w[i], w[j]))
                return true;
        for (int j = 0; j < nr; ++j)
            if (overlap(w[i], r[j]))
                return true;
    }
    return false;
}

struct Device {
    int status;
    int cus;
};

// The current device: LL_OK on gfx950, else the status to return. Properties
// are read once per device.
inline Device current_device()
{
    constexpr int kMax = 64;
    static std::once_flag once[kMax];
    static Device info[kMax];
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
        (void)hipGetLastError();
        return Device{LL_ERR_NO_DEVICE, 0};
    }
    const auto probe = [dev] {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
            (void)hipGetLastError();
            return Device{LL_ERR_NO_DEVICE, 0};
        }
        return Device{strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? LL_OK : LL_ERR_UNSUPPORTED_ARCH,
                      prop.multiProcessorCount};
    };
    if (dev >= kMax)
        return probe();
    std::call_once(once[dev], [&] { info[dev] = probe(); });
    return info[dev];
}

inline int status(hipError_t e) { return e == hipSuccess ? LL_OK : LL_ERR_LAUNCH; }

// Bytes of an element of an LL_TYPE_* type; 0 for an unknown one.
inline int type_bytes(int type)
{
    return type == LL_TYPE_F32 ? 4 : type == LL_TYPE_F16 || type == LL_TYPE_BF16 ? 2 : 0;
}

}  // namespace host
}  // namespace ll
