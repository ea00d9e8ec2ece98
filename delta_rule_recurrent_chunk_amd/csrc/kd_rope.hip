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
// be off by 0.06 rad.
//
// Bound by memory: every element is read and written once.  A workgroup takes
// up to eight tokens, makes their sines and cosines once in LDS for all heads
// of q and k, and streams the heads in 16-byte pieces, the first ones already
// loading while the angles are made.  8 x 2048 tokens of 16 + 4 heads of 128
// (bf16, half layout, 168 MB): 37 us, 4.5 TB/s (a large copy: 5.1); one wave per
// token and pair by pair it took 77 us.
#include "kd_check.h"
#include "kd_device.h"
#include "kd_rope.h"

namespace kd {

// Work items of one head: VECTOR: 16-byte pieces (half layout: a rotated item
// is a piece of each half); otherwise single pairs and single elements behind
// the rotated part.
template <class E, bool IL, bool VECTOR>
__global__ __launch_bounds__(256) void kd_rope_kernel(RopeArgs p)
{
    constexpr int EPC = VECTOR ? 16 / sizeof(E) : 1;
    typedef E V __attribute__((ext_vector_type(EPC)));
    constexpr int U = VECTOR ? 4 : 8;      // items in flight
    __shared__ float2 cs[ROPE_TOKENS * ROPE_MAX_D / 2];
    const int tid = threadIdx.x, n = p.rot / 2;
    const int tok0 = blockIdx.x * p.tokens;      // (all tokens: below 2^31)
    const int ntok = min(p.tokens, p.B * p.T - tok0);
    const int nrot = VECTOR && IL ? (p.rot + EPC - 1) / EPC : n / EPC;      // rotated items of a head
    const unsigned row = p.per * (p.side[0].heads + p.side[1].heads), total = ntok * row;

    struct Item {
        const E* a;
        E* out;
        int tok, j, second;      // second: offset of the other half's piece
        bool ok, rot;
    };
    auto item = [&](unsigned idx) {
        Item it;
        it.ok = idx < total;
        idx = min(idx, total - 1);
        it.tok = ntok == 1 ? 0 : row > 1 ? (int)__umulhi(idx, p.div_row) : (int)idx;
        const unsigned r = idx - it.tok * row;
        int h = p.per > 1 ? (int)__umulhi(r, p.div_per) : (int)r;
        it.j = (int)(r - h * p.per);
        const unsigned t = tok0 + it.tok, bt = t / (unsigned)p.T;
        const int64_t b = bt, tt = t - bt * p.T;
        const bool isk = h >= p.side[0].heads;
        if (isk) h -= p.side[0].heads;
        const RopeSide& s = p.side[isk];
        it.rot = it.j < nrot;
        // first element of the item within the head
        int e;
        if (IL) e = VECTOR ? it.j * EPC : it.rot ? 2 * it.j : p.rot + (it.j - nrot);
        else e = it.rot ? it.j * EPC : p.rot + (it.j - nrot) * EPC;
        it.second = IL ? (VECTOR ? 0 : 1) : n;
        it.a = (const E*)s.in + b * s.is[0] + tt * s.is[1] + h * s.is[2] + e;
        it.out = (E*)s.out + b * s.os[0] + tt * s.os[1] + h * s.os[2] + e;
        return it;
    };
    V xa[U], xb[U];
    auto load = [&](unsigned i0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Item it = item(i0 + u * 256 + tid);
            if (it.ok) {
                xa[u] = *(const V*)it.a;
                if (it.rot && !(IL && VECTOR)) xb[u] = *(const V*)(it.a + it.second);
            }
        }
    };
    load(0);
    for (int i = tid; i < ntok * n; i += 256) {
        const int t = i / n, j = i - t * n;
        const int at = tok0 + t, pi = p.pos_batched ? at : (int)((unsigned)at % (unsigned)p.T);
        const double pos = p.pos64 ? (double)((const int64_t*)p.pos)[pi] : (double)((const int32_t*)p.pos)[pi];
        cs[i] = rope_cs(pos, p.freqs[j], p.scale, p.inverse);
    }
    __syncthreads();
    for (unsigned i0 = 0; i0 < total; i0 += U * 256) {
        if (i0 > 0) load(i0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Item it = item(i0 + u * 256 + tid);
            if (!it.ok) continue;
            V ya = xa[u], yb = xb[u];
            if (it.rot) {
                const float2* c = cs + it.tok * n;
                if (IL && VECTOR) {
#pragma unroll
                    for (int e = 0; e < EPC / 2; ++e) {
                        const int j = it.j * (EPC / 2) + e;
                        const float2 cj = c[min(j, n - 1)];
                        const float a = (float)xa[u][2 * e], b = (float)xa[u][2 * e + 1];
                        if (j < n) {      // (a piece may hold elements behind the rotated part)
                            ya[2 * e] = (E)fmaf(a, cj.x, -b * cj.y);
                            ya[2 * e + 1] = (E)fmaf(b, cj.x, a * cj.y);
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < EPC; ++e) {
                        const float2 cj = c[it.j * EPC + e];
                        const float a = (float)xa[u][e], b = (float)xb[u][e];
                        ya[e] = (E)fmaf(a, cj.x, -b * cj.y);
                        yb[e] = (E)fmaf(b, cj.x, a * cj.y);
                    }
                    *(V*)(it.out + it.second) = yb;
                }
            }
            *(V*)it.out = ya;
        }
    }
}

static bool rope_aligned(const RopeArgs& a, int64_t es)
{
    for (const RopeSide& s : a.side) {
        if (s.heads == 0) continue;
        if (((uintptr_t)s.in | (uintptr_t)s.out) % 16) return false;
        for (int i = 0; i < 3; ++i)
            if (s.is[i] * es % 16 || s.os[i] * es % 16) return false;
    }
    return true;
}

// Sixteen bytes at a time where addresses, strides and (half layout) the two
// halves allow it (vec); pair by pair otherwise.  Returns the workgroups.
static int64_t rope_plan(RopeArgs& a, int es, bool& vec)
{
    const int epc = 16 / es, H = a.side[0].heads + a.side[1].heads;
    vec = rope_aligned(a, es) && a.d % epc == 0 && (a.interleaved || a.rot / 2 % epc == 0);
    a.per = vec ? (a.interleaved ? a.d / epc : a.rot / 2 / epc + (a.d - a.rot) / epc) : a.rot / 2 + (a.d - a.rot);
    const int64_t row = (int64_t)a.per * H;
    // about 1280 items per workgroup, so that small calls spread over the chip
    // and the angles of a token are made once
    a.tokens = (int)max((int64_t)1, min((int64_t)ROPE_TOKENS, 1280 / row));
    a.div_row = (unsigned)(((1ull << 32) + row - 1) / row);
    a.div_per = (unsigned)(((1ull << 32) + a.per - 1) / a.per);
    return ((int64_t)a.B * a.T + a.tokens - 1) / a.tokens;
}

template <class E>
static hipError_t rope(RopeArgs a, hipStream_t st)
{
    bool vec;
    const dim3 grid((unsigned)rope_plan(a, sizeof(E), vec));
    if (a.interleaved) {
        if (vec) kd_rope_kernel<E, true, true><<<grid, 256, 0, st>>>(a);
        else kd_rope_kernel<E, true, false><<<grid, 256, 0, st>>>(a);
    } else {
        if (vec) kd_rope_kernel<E, false, true><<<grid, 256, 0, st>>>(a);
        else kd_rope_kernel<E, false, false><<<grid, 256, 0, st>>>(a);
    }
    return hipGetLastError();
}

bool rope_fits(int bf16, RopeArgs a)
{
    bool vec;
    return grid_fits(rope_plan(a, bf16 ? 2 : 4, vec), 256);
}

hipError_t launch_rope(int bf16, const RopeArgs& a, hipStream_t st) { return bf16 ? rope<__bf16>(a, st) : rope<float>(a, st); }

}  // namespace kd
