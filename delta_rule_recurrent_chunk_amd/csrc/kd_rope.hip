// kd_rope.hip -- rotary positions on queries and keys, gfx950.
//
// Pair j of a head's rotated part (rot elements, rot / 2 pairs) at position p
// turns by the angle p w_j, and is multiplied by `scale`:
//     (a, b) -> scale (a cos - b sin, b cos + a sin)
// with a, b at j and j + rot / 2 (half layout) or 2j and 2j + 1 (interleaved).
// Elements past rot are copied.  The backward pass is the same product with
// the angle negated (the rotation is orthogonal).
//
// The angle is a product in fp64, reduced to its fraction of a turn before
// the sine and cosine in fp32: at position 10^6 an fp32 angle would already
// be off by 0.06 rad.  One wave takes one token: its 64 lanes make the token's
// sines and cosines once, in LDS, for all the heads of q and k.
#include "kd_device.h"
#include "kd_rope.h"

namespace kd {

// One wave per token, one pair (or one element behind the rotated part) per
// lane and step.
template <class E>
__global__ __launch_bounds__(256) void kd_rope_kernel(RopeArgs p)
{
    __shared__ float2 cs[4][ROPE_MAX_D / 2];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t tok = (int64_t)blockIdx.x * 4 + w;
    if (tok >= (int64_t)p.B * p.T) return;      // whole waves leave; no barrier below spans waves
    const int b = (int)(tok / p.T), t = (int)(tok % p.T), n = p.rot / 2;
    const int64_t pi = p.pos_batched ? tok : t;
    const double pos = p.pos64 ? (double)((const int64_t*)p.pos)[pi] : (double)((const int32_t*)p.pos)[pi];
    for (int j = lane; j < n; j += 64) cs[w][j] = rope_cs(pos, p.freqs[j], p.scale, p.inverse);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int per = n + (p.d - p.rot);
    for (int s = 0; s < 2; ++s) {
        const RopeSide& o = p.side[s];
        const E* src = (const E*)o.in + b * o.is[0] + t * o.is[1];
        E* dst = (E*)o.out + b * o.os[0] + t * o.os[1];
        for (int idx = lane; idx < o.heads * per; idx += 64) {
            const int h = idx / per, j = idx % per;
            const E* sp = src + h * o.is[2];
            E* dp = dst + h * o.os[2];
            if (j < n) {
                const int ia = p.interleaved ? 2 * j : j, ib = p.interleaved ? 2 * j + 1 : j + n;
                const float a = (float)sp[ia], bb = (float)sp[ib];
                const float2 c = cs[w][j];
                dp[ia] = (E)fmaf(a, c.x, -bb * c.y);
                dp[ib] = (E)fmaf(bb, c.x, a * c.y);
            } else {
                const int e = p.rot + (j - n);
                dp[e] = sp[e];
            }
        }
    }
}

hipError_t launch_rope(int bf16, const RopeArgs& a, hipStream_t st)
{
    const int64_t blocks = ((int64_t)a.B * a.T + 3) / 4;
    if (bf16)
        kd_rope_kernel<__bf16><<<(unsigned)blocks, 256, 0, st>>>(a);
    else
        kd_rope_kernel<float><<<(unsigned)blocks, 256, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace kd
