// checks.hpp -- the argument checks shared by the C entry points: sizes,
// pointers, byte ranges and the device.  Host code only.
#pragma once
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>
#include <vector>

#include "../../include/gemvgemm.h"

namespace gg {

constexpr int64_t kMaxDim = INT32_MAX;   // sizes must be below 2^31
constexpr int kMaxDevices = 64;

// Per-device cache: 0 unknown, else 1 + compute-unit count for a gfx950 and
// -1 for any other device.  Filled without a lock; a race only repeats the
// query and stores the same answer.
inline std::atomic<int> g_device_info[kMaxDevices];

// GG_OK and the current device's CU count, or an error status.
inline int check_device(int *num_cus) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return GG_ERR_NO_DEVICE;
    if (dev < kMaxDevices) {
        const int known = g_device_info[dev].load(std::memory_order_relaxed);
        if (known > 0) {
            *num_cus = known - 1;
            return GG_OK;
        }
        if (known < 0) return GG_ERR_NO_DEVICE;
    }
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return GG_ERR_NO_DEVICE;
    const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    const int cus = prop.multiProcessorCount > 0 ? prop.multiProcessorCount : 1;
    if (dev < kMaxDevices) g_device_info[dev].store(ok ? 1 + cus : -1, std::memory_order_relaxed);
    *num_cus = cus;
    return ok ? GG_OK : GG_ERR_NO_DEVICE;
}

// Byte range [lo, hi) of a rows x cols matrix with leading dimension ld.
struct Span {
    uintptr_t lo, hi;
};

// Bytes from p to the end of the matrix's last element (sizes below 2^31,
// so the product fits in 128 bits).
inline unsigned __int128 extent_bytes(int64_t rows, int64_t cols, int64_t ld, int64_t elem) {
    if (rows <= 0 || cols <= 0) return 0;
    return ((unsigned __int128)(rows - 1) * (uint64_t)ld + (uint64_t)cols) * (uint64_t)elem;
}

// A matrix whose bytes would run past the end of the address space.
inline bool wraps(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t elem) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    return extent_bytes(rows, cols, ld, elem) > (unsigned __int128)(UINTPTR_MAX - b);
}

// Only for matrices that do not wrap.
inline Span span(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t elem) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    return {b, b + (uintptr_t)extent_bytes(rows, cols, ld, elem)};
}

inline bool overlaps(Span a, Span b) {
    return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

inline bool bad_ptr(const void *p, int64_t align) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % (uintptr_t)align) != 0;
}

inline int launch_status(hipError_t e) { return e == hipSuccess ? GG_OK : GG_ERR_LAUNCH; }

// The byte range of one operand of a batch, and whether it is an output.
struct Iv {
    Span s;
    bool out;
};

// True when every output is disjoint from every input and from every other
// output (inputs may overlap each other, e.g. a shared x).  Sorted sweep: an
// interval overlaps an earlier one exactly when its start lies below the
// largest end seen so far.
inline bool outputs_disjoint(std::vector<Iv> &iv) {
    std::sort(iv.begin(), iv.end(), [](const Iv &a, const Iv &b) { return a.s.lo < b.s.lo; });
    uintptr_t end_all = 0, end_out = 0;
    for (const Iv &v : iv) {
        if (v.s.lo >= v.s.hi) continue;
        if (v.out ? end_all > v.s.lo : end_out > v.s.lo) return false;
        end_all = end_all > v.s.hi ? end_all : v.s.hi;
        if (v.out) end_out = end_out > v.s.hi ? end_out : v.s.hi;
    }
    return true;
}

}  // namespace gg
