// kd_rope.h -- rotary positions: launch arguments and the angle, gfx950.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kd {

constexpr int ROPE_MAX_D = 256;
constexpr int ROPE_TOKENS = 8;     // most tokens of a workgroup
constexpr int ROPE_MAX_H = 32767;  // most heads of q and of k (item numbers are divided by multiplication)

// one of the two tensors a launch rotates; strides over batch, token and head
// in elements (the last dimension is contiguous)
struct RopeSide {
    const void* in;
    void* out;
    int64_t is[3], os[3];
    int heads;
};

struct RopeArgs {
    RopeSide side[2];
    const void* pos;        // [T] or [B, T]
    const double* freqs;    // [rot / 2], radians per position
    int B, T, d, rot, pos64, pos_batched, interleaved, inverse;
    float scale;
    // the launch's own
    int per, tokens;                // work items per head, tokens per workgroup
    unsigned div_row, div_per;      // 2^32 / items per token, / items per head, rounded up
};

// scale (cos, sin) of the angle pos * freq (its negative for the inverse):
// the turns are taken in fp64 and only their fraction goes to fp32, so the
// angle's error stays below 2^-24 turns for every position up to 2^28
__device__ __forceinline__ float2 rope_cs(double pos, double freq, float scale, int inverse) {
    double turns = pos * freq * 0.15915494309189533577;   // 1 / (2 pi)
    turns -= rint(turns);
    float s, c;
    sincospif(2.f * (float)turns, &s, &c);
    return make_float2(scale * c, inverse ? -scale * s : scale * s);
}

}  // namespace kd
