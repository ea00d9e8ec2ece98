// kd_paged.hip -- new keys and values into a paged cache, turned to their
// positions on the way, gfx950.
//
// Own token i of sequence b lies in slot i % page of page table[b][i / page].
// The rows of a call go on from lens[b]: row r of sequence b is own token
// p = lens[b] + r.  Its key (and its queries, when they are given) turn to
// position offset + p as in kd_rope.hip, its value is copied.
//
// Bound by memory: every element is read and written once (13050 rows of 16
// queries, 4 keys and 4 values of 128, bf16: 160 MB in 34 us, 4.7 TB/s; a large
// copy reaches 4.9).  A workgroup takes up to eight rows; sines and cosines are
// made once for a row's heads; the first pieces load while its waves look the
// rows' sequences and pages up.
#include "kd_check.h"
#include "kd_device.h"
#include "kd_paged.h"
#include "kd_rope.h"

namespace kd {

enum { APPEND_PAIRS, APPEND_PIECES, APPEND_SPLIT };

// What an item is: APPEND_PAIRS: 16 bytes of each half of a turned head (half
// layout); APPEND_PIECES: 16 bytes that hold their own pairs (interleaved, or
// nothing turned); APPEND_SPLIT: 16 bytes whose partners are read one by one
// (half layout with halves that are not whole pieces).  Behind the turned part
// an item is a plain piece in all of them.
template <class E, int MODE>
__global__ __launch_bounds__(256) void kd_append_kernel(AppendArgs a)
{
    constexpr int EPC = 16 / sizeof(E), U = 4;
    typedef E V __attribute__((ext_vector_type(EPC)));
    __shared__ float2 cs[APPEND_TOKENS * APPEND_MAX_D / 2];
    __shared__ struct {
        int64_t k, v;      // where the row's key and value go
        int64_t pos;
        int state;         // 0: no sequence, 1: an unused one, 2: no page, 3: all there
    } at[APPEND_TOKENS];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), n = a.rot / 2;
    const int tok0 = blockIdx.x * a.tokens, ntok = min(a.tokens, a.T - tok0);
    const int nrot = MODE == APPEND_PAIRS ? n / EPC : (a.rot + EPC - 1) / EPC;
    const unsigned turned = a.per * (a.Hq + a.Hkv), row = turned + a.perv * a.Hkv, total = ntok * row;

    struct Item {
        const E* in;
        int tok, h, e, side;
        bool ok, rot;
    };
    auto item = [&](unsigned idx) {
        Item it;
        it.ok = idx < total;
        idx = min(idx, total - 1);
        it.tok = ntok == 1 ? 0 : row > 1 ? (int)__umulhi(idx, a.div_row) : (int)idx;
        unsigned r = idx - it.tok * row;
        int j;
        it.rot = false;
        if (r < turned) {
            it.h = a.per > 1 ? (int)__umulhi(r, a.div_per) : (int)r;
            j = (int)(r - it.h * a.per);
            it.rot = j < nrot;
            it.e = MODE == APPEND_PAIRS && !it.rot ? a.rot + (j - nrot) * EPC : j * EPC;
            it.side = it.h >= a.Hq;
            if (it.side) it.h -= a.Hq;
        } else {
            r -= turned;
            it.h = a.perv > 1 ? (int)__umulhi(r, a.div_perv) : (int)r;
            it.e = (int)(r - it.h * a.perv) * EPC;
            it.side = 2;
        }
        const int64_t t = tok0 + it.tok;
        it.in = it.side == 0   ? (const E*)a.q + t * a.qs[0] + it.h * a.qs[1]
                : it.side == 1 ? (const E*)a.k + t * a.ks[0] + it.h * a.ks[1]
                               : (const E*)a.v + t * a.vs[0] + it.h * a.vs[1];
        return it;
    };
    V xa[U], xb[U];
    auto load = [&](unsigned i0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Item it = item(i0 + u * 256 + tid);
            if (!it.ok) continue;
            xa[u] = *(const V*)(it.in + it.e);
            if (it.rot && MODE == APPEND_PAIRS) xb[u] = *(const V*)(it.in + it.e + n);
            if (it.rot && MODE == APPEND_SPLIT) {
#pragma unroll
                for (int e = 0; e < EPC; ++e) {
                    const int i = it.e + e;
                    xb[u][e] = it.in[i < n ? i + n : i < a.rot ? i - n : i];
                }
            }
        }
    };
    load(0);
    for (int t = w; t < ntok; t += 4) {
        const int r = tok0 + t;
        int b = r, first = r;
        bool in = true;
        if (a.cu) {
            b = paged_owner(a.cu, a.B, r);
            in = b < a.B;
            if (in) first = a.cu[b];
            in = in && first <= r;
        }
        if (lane == 0) {
            int state = 0;
            int64_t pos = 0, ko = 0, vo = 0;
            if (in) {
                const int len = a.lens[b];
                state = 1;
                if (len >= 0) {
                    pos = (int64_t)len + ((int64_t)r - first);
                    state = 2;
                    const int64_t i = pos / a.page;
                    if (i < a.width) {
                        const int64_t pg = a.table[b * a.ts + i], slot = pos - i * a.page;
                        if (pg >= 0 && pg < a.pages) {
                            state = 3;
                            ko = pg * a.kcs[0] + slot * a.kcs[1];
                            vo = pg * a.vcs[0] + slot * a.vcs[1];
                        }
                    }
                }
            }
            at[t].k = ko;
            at[t].v = vo;
            at[t].pos = pos;
            at[t].state = state;
        }
    }
    __syncthreads();
    for (int i = tid; i < ntok * n; i += 256) {
        const int t = i / n, j = i - t * n;
        cs[i] = rope_cs((double)(at[t].pos + a.offset), a.freqs[j], a.scale, 0);
    }
    __syncthreads();
    for (unsigned i0 = 0; i0 < total; i0 += U * 256) {
        if (i0 > 0) load(i0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Item it = item(i0 + u * 256 + tid);
            if (!it.ok) continue;
            const int state = at[it.tok].state;
            if (it.side == 0 ? state == 0 : state != 3) continue;
            V ya = xa[u], yb = xb[u];
            const float2* c = cs + it.tok * n;
            if (it.rot) {
#pragma unroll
                for (int e = 0; e < EPC; ++e) {
                    if (MODE == APPEND_PAIRS) {
                        const float2 cj = c[it.e + e];
                        const float x = (float)xa[u][e], y = (float)xb[u][e];
                        ya[e] = (E)fmaf(x, cj.x, -y * cj.y);
                        yb[e] = (E)fmaf(y, cj.x, x * cj.y);
                    } else {
                        const int i = it.e + e;      // (a piece may hold elements behind the turned part)
                        const bool second = MODE == APPEND_PIECES ? e & 1 : i >= n;
                        const float2 cj = c[min(MODE == APPEND_PIECES ? i >> 1 : second ? i - n : i, n - 1)];
                        const float x = (float)xa[u][e], y = MODE == APPEND_PIECES ? (float)xa[u][e ^ 1] : (float)xb[u][e];
                        if (i < a.rot) ya[e] = (E)(second ? fmaf(x, cj.x, y * cj.y) : fmaf(x, cj.x, -y * cj.y));
                    }
                }
            }
            E* out;
            if (it.side == 0) {
                out = (E*)a.qo + ((int64_t)(tok0 + it.tok) * a.Hq + it.h) * a.d;
                if (state == 1) {
#pragma unroll
                    for (int e = 0; e < EPC; ++e) ya[e] = (E)0.f, yb[e] = (E)0.f;
                }
            } else {
                out = it.side == 1 ? (E*)a.kc + at[it.tok].k + it.h * a.kcs[2] : (E*)a.vc + at[it.tok].v + it.h * a.vcs[2];
            }
            *(V*)(out + it.e) = ya;
            if (it.rot && MODE == APPEND_PAIRS) *(V*)(out + it.e + n) = yb;
        }
    }
}

// A workgroup takes as many rows as leave 1024 workgroups, eight at most: the
// angles' parts are read once for them, and small calls spread over the chip
// (13050 rows of 20 + 4 heads of 128: 34 us with eight, 38 with five, 40 with
// one; 32 rows: 5.9 us with one, 9.2 with three).  Returns the workgroups.
static int64_t append_plan(AppendArgs& a, int es, int& mode)
{
    const int epc = 16 / es;
    mode = a.rot == 0 || a.interleaved ? APPEND_PIECES : a.rot / 2 % epc == 0 ? APPEND_PAIRS : APPEND_SPLIT;
    a.perv = a.d / epc;
    a.per = mode == APPEND_PAIRS ? a.rot / 2 / epc + (a.d - a.rot) / epc : a.perv;
    const int64_t row = (int64_t)a.per * (a.Hq + a.Hkv) + (int64_t)a.perv * a.Hkv;
    // (16384 pieces: what the divisions by multiplication are exact for)
    a.tokens = (int)max((int64_t)1, min((int64_t)min(APPEND_TOKENS, a.T / 1024), 16384 / row));
    a.div_row = (unsigned)(((1ull << 32) + row - 1) / row);
    a.div_per = (unsigned)(((1ull << 32) + a.per - 1) / a.per);
    a.div_perv = (unsigned)(((1ull << 32) + a.perv - 1) / a.perv);
    return ((int64_t)a.T + a.tokens - 1) / a.tokens;
}

bool append_fits(int bf16, AppendArgs a)
{
    int mode;
    return grid_fits(append_plan(a, bf16 ? 2 : 4, mode), 256);
}

template <class E>
static hipError_t append(AppendArgs a, hipStream_t st)
{
    int mode;
    const dim3 grid((unsigned)append_plan(a, sizeof(E), mode));
    if (mode == APPEND_PAIRS) kd_append_kernel<E, APPEND_PAIRS><<<grid, 256, 0, st>>>(a);
    else if (mode == APPEND_PIECES) kd_append_kernel<E, APPEND_PIECES><<<grid, 256, 0, st>>>(a);
    else kd_append_kernel<E, APPEND_SPLIT><<<grid, 256, 0, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_append(int bf16, const AppendArgs& a, hipStream_t st) { return bf16 ? append<__bf16>(a, st) : append<float>(a, st); }

}  // namespace kd
