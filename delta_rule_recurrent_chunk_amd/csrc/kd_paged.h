// kd_paged.h -- launch arguments of the paged cache and of the attention over a
// shared prefix, and what both read of a batch, gfx950.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kd_device.h"

namespace kd {

constexpr int APPEND_TOKENS = 8;      // most tokens of a workgroup
constexpr int APPEND_MAX_D = 256;

struct AppendArgs {
    const void *q, *k, *v;            // [T, H, d], strides over token and head (elements)
    int64_t qs[2], ks[2], vs[2];
    void* qo;                         // [T, Hq, d] contiguous
    void *kc, *vc;                    // pages, strides over page, slot and head
    int64_t kcs[3], vcs[3];
    const int *table, *lens, *cu;
    int64_t ts;                       // table entries from one sequence to the next
    const double* freqs;
    int64_t offset;
    int B, T, Hq, Hkv, d, rot, page, pages, width, interleaved;
    float scale;
    // the launch's own
    int per, perv, tokens;            // items per turned head and per head of v, tokens per workgroup
    unsigned div_row, div_per, div_perv;
};

struct PrefixArgs {
    const void* q;                    // [T, Hq, d], strides over token and head
    int64_t qs[2];
    const void *kc, *vc;
    int64_t kcs[3], vcs[3];
    const int *ptable, *table, *lens, *cu;
    int64_t ts;
    void* o;                          // [T, Hq, d] contiguous
    float* lse;                       // [Hq, T] or null
    float *part, *ml;                 // partial results: o [split][Hkv][T G][d], (m, l) [split][Hkv][T G][2]
    int B, T, Hq, Hkv, page, pages, width, P;
    int sp, so;                       // splits of the prefix and of the own keys
    int blocks, nprefix, nslots;      // row blocks of the prefix, its workgroups, own slots (128 rows)
    float c, scale;                   // c = scale log2(e)
};

// Sequence of packed row `row` as the whole wave finds it: how many of the
// offsets cu[1 ..] are at most it.  B or more: behind the last sequence.
__device__ __forceinline__ int paged_owner(const int* cu, int B, int row) {
    return wave_count(B, [&](int at) { return cu[at + 1] <= row; });
}

}  // namespace kd
