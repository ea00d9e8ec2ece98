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

// Bytes a strided [n0, n1, n2, d] tensor spans from its first element; false
// for a negative stride or one that does not keep 16-byte pieces aligned
// (align16), or an extent beyond 2^62.
inline bool span(const int64_t st[3], int64_t n0, int64_t n1, int64_t n2, int64_t d, size_t es, bool align16, size_t* bytes) {
    const int64_t n[3] = {n0, n1, n2};
    if (n0 == 0 || n1 == 0 || n2 == 0) {
        *bytes = 0;
        return true;
    }
    __int128 last = d;
    for (int i = 0; i < 3; ++i) {
        if (st[i] < 0) return false;
        if (align16 && n[i] > 1 && (st[i] * (int64_t)es) % 16 != 0) return false;
        last += (__int128)st[i] * (n[i] - 1);
    }
    if (last * es > ((__int128)1 << 62)) return false;
    *bytes = (size_t)(last * es);
    return true;
}

// Whether no two elements of a strided [n0, n1, n2, d] tensor share an address
// (an output that is written as such): in the order of their strides, every
// dimension steps over all that the smaller ones span.
inline bool distinct(const int64_t st[3], int64_t n0, int64_t n1, int64_t n2, int64_t d) {
    int64_t n[3] = {n0, n1, n2}, s[3] = {st[0], st[1], st[2]};
    if (n0 == 0 || n1 == 0 || n2 == 0) return true;
    __int128 ext = d;
    for (int k = 0; k < 3; ++k) {
        int at = -1;
        for (int i = 0; i < 3; ++i)
            if (n[i] > 1 && (at < 0 || s[i] < s[at])) at = i;
        if (at < 0) return true;
        if (s[at] < ext) return false;
        ext += (__int128)s[at] * (n[at] - 1);
        n[at] = 1;
    }
    return true;
}

// Whether two tensors of one shape and the same strides, `delta` elements
// apart, share no address although their spans interleave: the shift falls in
// the gap that one dimension's stride leaves behind the smaller dimensions.
inline bool interleaved_apart(const int64_t st[3], int64_t n0, int64_t n1, int64_t n2, int64_t d, int64_t delta) {
    const int64_t n[3] = {n0, n1, n2};
    if (delta < 0) delta = -delta;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        __int128 ext = d;      // what the dimensions of smaller stride span
        for (int j = 0; j < 3; ++j)
            if (j != i && n[j] > 1 && st[j] < st[i]) ext += (__int128)st[j] * (n[j] - 1);
        if (delta >= ext && delta + ext <= st[i]) return true;
    }
    return false;
}

inline bool any_overlap(const Range* outs, int no, const Range* ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlap(outs[i], ins[j])) return true;
        for (int j = i + 1; j < no; ++j)
            if (overlap(outs[i], outs[j])) return true;
    }
    return false;
}

}  // namespace kd
