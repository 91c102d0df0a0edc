// checks.hpp -- argument checks that the entry points of the operators around
// the expert GEMM share.  Host code only.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "../../include/ptgg.h"

namespace ptgg {
namespace {

// Whether the current device is gfx950 (asked once per device).
inline bool device_is_gfx950()
{
    static std::atomic<int> state[64] = {};        // 0 unknown, 1 yes, 2 no
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return false;
    int st = state[dev].load(std::memory_order_relaxed);
    if (st == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return false;
        st = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        state[dev].store(st, std::memory_order_relaxed);
    }
    return st == 1;
}

inline bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline int hip_status(hipError_t e) { return e == hipSuccess ? PT_OK : PT_ERR_HIP; }
inline int64_t round256(int64_t x) { return (x + 255) & ~(int64_t)255; }

// Rows of one launch: a workgroup each, and 2^32 threads at most.
constexpr int64_t kMaxRows = (int64_t)1 << 23;

}  // namespace
}  // namespace ptgg
