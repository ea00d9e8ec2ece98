// kd_swa_fwd.hip -- sliding-window attention with sinks, forward, gfx950.
//
// One workgroup of four waves takes 128 query rows of one head, one wave 32 of
// them; tiles of BN keys and values pass through LDS.  Per tile a wave forms
//     St = K Qt   (rows = keys, columns = the lane's query)
// so a query's scores lie in one lane (and its partner 32 lanes away): the
// running maximum m and sum l of its softmax are per-lane scalars.  The
// weights exp2(c s - m) are packed to the input type (bf16: off by at most
// 2^-8 of each weight, whose sum is kept in fp32) and go straight back in as
// the B operand of Ot += Vt Pt.
//
// 1 x 32768, 16 query and 4 key heads of 128, window 2048, 4 sinks, bf16: 600 us,
// 890 TFLOP/s of visible pairs (a large library product: 1222).  Bound by
// instructions: per 64 keys a wave issues 32 matrix products and about 160
// vector instructions, 32 of them exponentials; of a SIMD's cycles the matrix
// units are busy in 47% and vector instructions issue in 44%, LDS is active in
// 24% without conflicts.  Tiles of 64 keys, two in LDS: two workgroups per
// compute unit; eight waves per block of queries were 4% slower.
#include "kd_check.h"
#include "kd_swa.h"

namespace kd {

// o of a wave's queries (positions wp0 .. wp0 + 31) again (rare, see its call):
// keys 0 .. S - 1 and first .. last, 32 at a time where all queries see all of
// them, the others one after the other, each for the queries that see it.
template <class E, int D>
__device__ __forceinline__ void swa_fwd_single(floatx16* o, const typename SwaT<E>::Frag* q, const E* k, int64_t krs,
                                               const E* v, int64_t vrs, int last, int first, int wp0, int W, int S,
                                               float c, float mu, int lane)
{
    typedef SwaT<E> T;
    typedef E E4 __attribute__((ext_vector_type(4)));
    constexpr int NK = D / T::KC, ND = D / 32, NP = 16 / T::PR;
    const int g = lane >> 5, pos = wp0 + (lane & 31);
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] = 0.f;
#pragma unroll 1
    for (int key = S > 0 ? 0 : first; key <= last; ++key) {
        if (key >= S && key < first) key = first;
        if (key + 31 <= min(wp0, last) && (wp0 + 31 - key < W || key + 32 <= S)) {
            floatx16 sc;
#pragma unroll
            for (int r = 0; r < 16; ++r) sc[r] = 0.f;
#pragma unroll
            for (int ks = 0; ks < NK; ++ks) sc = T::mma(swa_ld_mem<E>(k + (int64_t)(key + (lane & 31)) * krs, ks, g), q[ks], sc);
#pragma unroll
            for (int r = 0; r < 16; ++r) sc[r] = __builtin_amdgcn_exp2f(fmaf(sc[r], c, -mu));
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const typename T::Frag p = T::pack(sc, j);
#pragma unroll
                for (int i = 0; i < ND; ++i)
                    o[i] = T::mma(swa_ld_col_mem<E>(v + 32 * i + (lane & 31), vrs, key + (32 / NP) * j, g), p, o[i]);
            }
            key += 31;
            continue;
        }
        float s = 0.f;
#pragma unroll
        for (int ks = 0; ks < NK; ++ks) s += SwaT<E>::dot(q[ks], swa_ld_mem<E>(k + key * krs, ks, g));
        s += swa_swap(s);
        const bool sees = (key <= pos) & ((pos - key < W) | (key < S));
        const float p = sees ? __builtin_amdgcn_exp2f(fmaf(s, c, -mu)) : 0.f;
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const E4 x = *reinterpret_cast<const E4*>(v + key * vrs + 32 * i + 8 * j + 4 * g);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][4 * j + e] = fmaf(p, sees ? (float)x[e] : 0.f, o[i][4 * j + e]);
            }
    }
}

template <class E, int D, int BN>
__global__ __launch_bounds__(256, sizeof(E) * D > 256 ? 1 : 2) void kd_swa_fwd_kernel(SwaArgs a, int nslots)
{
    typedef SwaT<E> T;
    typedef typename T::Frag Frag;
    constexpr int NK = D / T::KC, NS = BN / 32, ND = D / 32, NP = 16 / T::PR;
    __shared__ __align__(16) E kt[2][BN * D];
    __shared__ __align__(16) E vt[2][BN * D];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 5;
    const int G = a.Hq / a.Hkv;
    int64_t item;
    if (!swa_item((int64_t)nslots * a.Hq * a.B, item)) return;
    const int hg = item % G;
    item /= G;
    const int slot = nslots - 1 - item % nslots;    // the rows that see most first
    item /= nslots;
    const int hk = item % a.Hkv, b = item / a.Hkv, h = hk * G + hg;
    SwaSeq s;
    if (!swa_locate(a, slot, 128, false, s)) return;
    const int r0 = s.blk * 128, row = r0 + 32 * w + (lane & 31), pos = s.past + row;

    const E* qrow = (const E*)a.q + b * a.qs[0] + (int64_t)(s.q0 + min(row, s.nq - 1)) * a.qs[1] + h * a.qs[2];
    Frag q[NK];
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) q[ks] = swa_ld_mem<E>(qrow, ks, g);
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) swa_arrive(q[ks]);
    const SwaFetch<E, D, BN, 256> kf((const E*)a.k + b * a.ks[0] + (int64_t)s.q0 * a.ks[1] + hk * a.ks[2], a.ks[1], s.nk, tid);
    const SwaFetch<E, D, BN, 256> vf((const E*)a.v + b * a.vs[0] + (int64_t)s.q0 * a.vs[1] + hk * a.vs[2], a.vs[1], s.nk, tid);

    floatx16 o[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] = 0.f;
    float m = -INFINITY, l = 0.f;

    // tiles: the sinks' tiles in front of the window, then lo .. hi - 1
    const int pmax = min(s.past + r0 + 127, s.nk - 1);
    const int lo = max(0, s.past + r0 - a.W + 1) / BN, hi = pmax < 0 ? 0 : pmax / BN + 1;
    const int sk = min((a.S + BN - 1) / BN, lo), nt = sk + max(hi - lo, 0);
    const int wp0 = s.past + r0 + 32 * w, wp1 = wp0 + 31;      // this wave's positions
    auto key0 = [&](int i) { return (i < sk ? i : lo + (i - sk)) * BN; };
    auto fetch = [&](int i) {
        kf(kt[i & 1], 0, key0(i), w);
        vf(vt[i & 1], 0, key0(i), w);
    };
    if (nt > 0) fetch(0);
    // (one copy of the loop's body per buffer, whose LDS addresses are then constants)
    auto tile = [&](int i, const E* kl, const E* vl) {
        // tile i is here; the buffer of tile i - 1 is free
        swa_landed();
        if (i + 1 < nt) fetch(i + 1);
        const int k0 = key0(i);
        if (k0 > wp1 || (k0 + BN - 1 <= wp0 - a.W && k0 >= a.S)) return;   // nothing visible to the wave
        floatx16 sc[NS];
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int n = 0; n < NS; ++n) {
#pragma unroll
            for (int r = 0; r < 16; ++r) sc[n][r] = 0.f;
#pragma unroll
            for (int ks = 0; ks < NK; ++ks)
                sc[n] = T::mma(swa_ld_row<E, D>(kl, 32 * n + (lane & 31), ks, g), q[ks], sc[n]);
        }
        __builtin_amdgcn_s_setprio(0);
        // every pair of the tile visible: no mask
        const bool full = k0 + BN - 1 <= wp0 && (wp1 - k0 < a.W || k0 + BN <= a.S);
        if (!full) {
#pragma unroll
            for (int n = 0; n < NS; ++n) swa_mask_keys(sc[n], k0 + 32 * n + 4 * g, pos, a.W, a.S);
        }
        float mx = sc[0][0];
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int r = 0; r < 16; ++r) mx = fmaxf(mx, sc[n][r]);
        mx = fmaxf(mx, swa_swap(mx)) * a.c;
        // The reference of the exponents follows the maximum only when some row
        // of the wave outgrows it by 2^8: weights up to 2^8 lose nothing in
        // fp32 sums or in the type's relative rounding, and o is rescaled rarely.
        if (__any(mx > m + 8.f)) {
            const float mn = fmaxf(m, mx), alpha = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.f : mn));
            m = mn;
            l *= alpha;
#pragma unroll
            for (int dt = 0; dt < ND; ++dt) o[dt] *= alpha;
        }
        const float mu = m == -INFINITY ? 0.f : m;
        float ls = 0.f;
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                sc[n][r] = __builtin_amdgcn_exp2f(fmaf(sc[n][r], a.c, -mu));
                ls += sc[n][r];
            }
        l += ls;
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const Frag p = T::pack(sc[n], j);
#pragma unroll
                for (int dt = 0; dt < ND; ++dt)
                    o[dt] = T::mma(T::template ld_col<D>(vl, 32 * n + (32 / NP) * j, 32 * dt, lane), p, o[dt]);
            }
        __builtin_amdgcn_s_setprio(0);
    };
    for (int i = 0; i < nt; i += 2) {
        tile(i, kt[0], vt[0]);
        if (i + 1 < nt) tile(i + 1, kt[1], vt[1]);
    }
    l += swa_swap(l);
    // A hidden key has weight 0, and 0 times an infinity or a NaN in its values
    // would still reach the queries of its tile.  A wave with an output that is
    // not finite makes its outputs again from the maxima and sums it has, over
    // the keys that each query sees.
    float sum = 0.f;      // (0 times what is not finite is a NaN)
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) sum = fmaf(o[i][r], 0.f, sum);
    if (__any(!(sum == 0.f)))
        swa_fwd_single<E, D>(o, q, kf.base, a.ks[1], vf.base, a.vs[1], min(wp1, s.nk - 1), max(0, wp0 - a.W + 1), wp0, a.W,
                             a.S, a.c, m == -INFINITY ? 0.f : m, lane);
    if (row >= s.nq) return;
    // a row that sees nothing: o = 0, lse = -infinity
    const bool none = m == -INFINITY && l == 0.f;
    swa_store_row<E, D>((E*)a.o + (((int64_t)b * a.Tq + s.q0 + row) * a.Hq + h) * D, o, none ? 0.f : 1.f / l, g);
    if (a.lse && g == 0)
        a.lse[((int64_t)b * a.Hq + h) * a.Tq + s.q0 + row] = none ? -INFINITY : 0.6931471805599453f * (m + __log2f(l));
}

bool swa_fwd_fits(const SwaArgs& a) { return grid_fits(swa_grid(swa_slots(a.cu, a.N, a.Tq, 128) * a.Hq * a.B), 256); }

template <class E, int D>
static hipError_t swa_fwd(const SwaArgs& a, hipStream_t st)
{
    const int64_t nslots = swa_slots(a.cu, a.N, a.Tq, 128), grid = swa_grid(nslots * a.Hq * a.B);
    kd_swa_fwd_kernel<E, D, sizeof(E) == 2 ? 64 : 32><<<(unsigned)grid, 256, 0, st>>>(a, (int)nslots);
    return hipGetLastError();
}

hipError_t launch_swa_fwd(int bf16, int d, const SwaArgs& a, hipStream_t st)
{
    if (bf16) return d == 32 ? swa_fwd<__bf16, 32>(a, st) : d == 64 ? swa_fwd<__bf16, 64>(a, st) : swa_fwd<__bf16, 128>(a, st);
    return d == 32 ? swa_fwd<float, 32>(a, st) : d == 64 ? swa_fwd<float, 64>(a, st) : swa_fwd<float, 128>(a, st);
}

}  // namespace kd
