// kd_swa_decode.h -- launch arguments of the decoding step and of the prompt
// store, gfx950.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kd {

constexpr int SWA_DECODE_COUNTERS = 512;    // arrival counters at the start of the workspace
constexpr int SWA_DECODE_SPLITS = 32;       // most splits of a row's keys

struct SwaDecodeArgs {
    const void *q, *k, *v;          // [B, H, d], batch strides qb, kb, vb (elements)
    int64_t qb, kb, vb;
    void *kc, *vc;                  // caches, strides over batch, slot, head
    int64_t kcs[3], vcs[3];
    const int* lens;
    const double* freqs;
    void* o;                        // [B, Hq, d]
    int* count;                     // one word per (b, group of heads), zero between calls
    float* part;                    // partial results of the splits
    int B, Hq, Hkv, cap, W, S, rot, interleaved, nsplit;
    float c, rope_scale;            // c = scale log2(e)
};

struct SwaStoreArgs {
    const void *k, *v;
    int64_t ks[3], vs[3], kcs[3], vcs[3];
    void *kc, *vc;
    const int* lens;
    int T, Hkv, row, es, cap, S;    // row: 16-byte pieces of one head
};

}  // namespace kd
