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

inline bool bad_size(int64_t n) { return n < 0 || n > kMaxDim; }
inline bool bad_act(int act) { return act < GG_ACT_NONE || act > GG_ACT_SILU; }

// The operands of one call, checked as they are added: a pointer that is
// null or misaligned, a short leading dimension or a range past the address
// space makes the call invalid.  Absent operands are not added.
class Operands {
public:
    // An input, or an output, of rows x cols elements of `elem` bytes at p.
    Operands &in(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t elem = 4) {
        return add(INPUT, p, rows, cols, ld, elem);
    }
    Operands &out(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t elem = 4) {
        return add(OUTPUT, p, rows, cols, ld, elem);
    }
    // n matrices of rows x cols elements, `stride` elements apart.
    Operands &in_each(const void *p, int64_t n, int64_t stride, int64_t rows, int64_t cols, int64_t ld,
                      int64_t elem = 4) {
        return add_each(INPUT, p, n, stride, rows, cols, ld, elem);
    }
    Operands &out_each(const void *p, int64_t n, int64_t stride, int64_t rows, int64_t cols, int64_t ld,
                       int64_t elem = 4) {
        return add_each(OUTPUT, p, n, stride, rows, cols, ld, elem);
    }
    // An input that the output `onto` may replace in place, and that output:
    // the same pointer and leading dimension.
    Operands &replaced(const void *p, int64_t rows, int64_t cols, int64_t ld) {
        return add(REPLACED, p, rows, cols, ld, 4);
    }
    Operands &onto(const void *p, int64_t rows, int64_t cols, int64_t ld) {
        return add(ONTO, p, rows, cols, ld, 4);
    }
    // a workspace of `need` bytes (floats in number), 16-byte aligned
    Operands &workspace(const void *p, int64_t bytes, unsigned __int128 need) {
        if (need == 0) return *this;
        const uintptr_t b = reinterpret_cast<uintptr_t>(p);
        if (bytes < 0 || need > (unsigned __int128)bytes || bad_ptr(p, 16) || need > UINTPTR_MAX - b) {
            bad_ = true;
            return *this;
        }
        op_[n_++] = {{b, b + (uintptr_t)need}, OUTPUT, p, 0};
        return *this;
    }
    // GG_OK, or why the call is refused.
    int status() const {
        if (bad_) return GG_ERR_INVALID_ARG;
        for (int i = 0; i < n_; ++i) {
            if (op_[i].kind != OUTPUT && op_[i].kind != ONTO) continue;
            for (int j = 0; j < n_; ++j) {
                if (i == j || !overlaps(op_[i].s, op_[j].s)) continue;
                if (op_[i].kind != ONTO || op_[j].kind != REPLACED || op_[i].p != op_[j].p ||
                    op_[i].ld != op_[j].ld)
                    return GG_ERR_ALIAS;
            }
        }
        return GG_OK;
    }

private:
    enum Kind { INPUT, OUTPUT, REPLACED, ONTO };
    Operands &add(Kind kind, const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t elem) {
        if (rows == 0 || cols == 0) return *this;
        if (ld < cols || ld > kMaxDim || bad_ptr(p, elem) || wraps(p, rows, cols, ld, elem)) {
            bad_ = true;
            return *this;
        }
        op_[n_++] = {span(p, rows, cols, ld, elem), kind, p, ld};
        return *this;
    }
    // Outputs must not overlap each other, and no stride is negative.
    Operands &add_each(Kind kind, const void *p, int64_t n, int64_t stride, int64_t rows, int64_t cols,
                       int64_t ld, int64_t elem) {
        if (n == 0 || rows == 0 || cols == 0) return *this;
        const int before = n_;
        add(kind, p, rows, cols, ld, elem);
        if (n_ == before || n == 1) return *this;
        const unsigned __int128 one = extent_bytes(rows, cols, ld, elem);
        if (stride < 0 || (kind == OUTPUT && (unsigned __int128)stride * (uint64_t)elem < one)) {
            bad_ = true;
            return *this;
        }
        const unsigned __int128 all = (unsigned __int128)(n - 1) * (uint64_t)stride * (uint64_t)elem + one;
        const uintptr_t b = reinterpret_cast<uintptr_t>(p);
        if (all > (unsigned __int128)(UINTPTR_MAX - b)) bad_ = true;
        else op_[before].s = {b, b + (uintptr_t)all};
        return *this;
    }
    struct Op {
        Span s;
        Kind kind;
        const void *p;
        int64_t ld;
    };
    Op op_[20];          // no entry point has more
    int n_ = 0;
    bool bad_ = false;
};

}  // namespace gg
