// kd_check.h -- argument checks shared by the C ABI's entry points (host code).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace kd {

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};

inline Range range_of(const void* p, size_t bytes) {
    Range r;
    r.lo = (uintptr_t)p;
    r.hi = r.lo + bytes;
    return r;
}

inline bool overlap(Range a, Range b) {
    if (a.lo == a.hi || b.lo == b.hi || a.lo == 0 || b.lo == 0) return false;
    return a.lo < b.hi && b.lo < a.hi;
}

inline bool misaligned(const void* p) { return p != nullptr && ((uintptr_t)p & 15u) != 0; }

// Whether a launch of `blocks` workgroups along one dimension is possible: the
// runtime counts its threads in 32 bits.
inline bool grid_fits(int64_t blocks, int threads) { return blocks <= (int64_t)UINT32_MAX / threads; }

inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace kd
