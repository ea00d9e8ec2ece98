// kd_swa_bwd.hip -- sliding-window attention with sinks, backward, gfx950.
//
// With P = exp(scale s - lse) recomputed from the saved lse and
// delta_t = sum_s P_ts dP_ts (= sum_i dO_ti o_ti):
//     dV = Pt dO;  dP = dO Vt;  dS = P (dP - delta);  dQ = scale dS K;  dK = scale dSt Q
// Every gradient is summed in registers in a fixed order, no atomics:
//   1. over query blocks: dQ, and delta for the other two;
//   2. where queries lie beyond the window of the first 128 keys: the sinks'
//      dK and dV from those queries, in partial sums over chunks of queries;
//   3. over key blocks: dK and dV from the queries whose window holds them,
//      also summed over the query heads of a group; the first block adds the
//      partial sums of 2.  Where key blocks are few, workgroups share the heads
//      of a group and a last pass adds their fp32 sums.
#include "kd_check.h"
#include "kd_swa.h"

namespace kd {

constexpr float LOG2E = 1.4426950408889634f;

// first query beyond the window of keys 0 .. 127
__device__ __forceinline__ int swa_far(const SwaArgs& a, int past) { return max(0, 127 + a.W - past); }

// dQ and delta of 128 query rows of one head: the forward's layout, with the
// scores' gradient in the weights' place and K in V's.
//
// 4 x 4096, 16/4 heads of 128, window 1024, bf16: 280 us for three products
// (181 GFLOP of visible pairs, 650 TFLOP/s), bound like the forward (matrix
// units 41% of the cycles, vector issue 42%).
//
// dS is rounded to the type before its product with K.  Its delta comes from
// the rounded o there (the sum of P dP is only known at the end, when it goes
// to the other kernels): for queries that see few keys the two roundings
// together would double the error of dQ, so waves whose queries see fewer than
// 512 keys take the rounding's remainder of dS through a second product.  The
// error that o's rounding leaves in delta falls with the root of the number of
// keys against that of dQ; waves whose queries see at most 32 first take the
// sum of P dP from memory, in a pass of its own.
//
// That pass: delta plus the sum of P (dP - delta) over the keys k0 .. k1 - 1
// that the wave's queries see, 32 at a time.
template <class E, int D>
__device__ __forceinline__ float swa_dq_near(float delta, const typename SwaT<E>::Frag* q, const typename SwaT<E>::Frag* dO,
                                             const E* k, int64_t krs, const E* v, int64_t vrs, int k0, int k1, int nk,
                                             int pos, int W, int S, float c, float lse2, int lane)
{
    typedef SwaT<E> T;
    constexpr int NK = D / T::KC;
    const int g = lane >> 5;
    float sum = 0.f;
#pragma unroll 1
    for (; k0 < k1; k0 += 32) {
        const int64_t key = min(k0 + (lane & 31), nk - 1);
        floatx16 sc, dp;
#pragma unroll
        for (int r = 0; r < 16; ++r) sc[r] = 0.f, dp[r] = -delta;
#pragma unroll
        for (int ks = 0; ks < NK; ++ks) {
            sc = T::mma(swa_ld_mem<E>(k + key * krs, ks, g), q[ks], sc);
            dp = T::mma(swa_ld_mem<E>(v + key * vrs, ks, g), dO[ks], dp);
        }
        swa_mask_keys(sc, k0 + 4 * g, pos, W, S);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const float x = __builtin_amdgcn_exp2f(fmaf(sc[r], c, -lse2)) * dp[r];
            sum += sc[r] == -INFINITY ? 0.f : x;      // (a hidden key's dP may be anything)
        }
    }
    return sum;
}

// dQ (before its scale) of a wave's queries (positions wp0 .. wp0 + 31) and the
// sum of P (dP - delta) again (rare, see its call): keys 0 .. S - 1 and first ..
// last, 32 at a time where all queries see all of them, the others one after
// the other, each for the queries that see it.
template <class E, int D>
__device__ __forceinline__ float swa_dq_single(floatx16* acc, const E* q, const E* dO,
                                               const E* k, int64_t krs, const E* v, int64_t vrs, int last, int first,
                                               int wp0, int W, int S, float c, float lse2, float delta, bool few, int lane)
{
    typedef SwaT<E> T;
    typedef E E4 __attribute__((ext_vector_type(4)));
    constexpr int NK = D / T::KC, ND = D / 32, NP = 16 / T::PR;
    const int g = lane >> 5, pos = wp0 + (lane & 31);
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;
    float dsum = 0.f, part = 0.f;      // (part: of this lane's keys alone)
#pragma unroll 1
    for (int key = S > 0 ? 0 : first; key <= last; ++key) {
        if (key >= S && key < first) key = first;
        if (key + 31 <= min(wp0, last) && (wp0 + 31 - key < W || key + 32 <= S)) {
            const int64_t at = key + (lane & 31);
            floatx16 sc, dp;
#pragma unroll
            for (int r = 0; r < 16; ++r) sc[r] = 0.f, dp[r] = -delta;
#pragma unroll
            for (int ks = 0; ks < NK; ++ks) {
                sc = T::mma(swa_ld_mem<E>(k + at * krs, ks, g), swa_ld_mem<E>(q, ks, g), sc);
                dp = T::mma(swa_ld_mem<E>(v + at * vrs, ks, g), swa_ld_mem<E>(dO, ks, g), dp);
                asm volatile("" : "+v"(sc), "+v"(dp) : : "memory");      // (a few loads at a time)
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                sc[r] = __builtin_amdgcn_exp2f(fmaf(sc[r], c, -lse2)) * dp[r];
                part += sc[r];
            }
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const typename T::Frag p = T::pack(sc, j), rest = T::rest(sc, j, p);
#pragma unroll
                for (int i = 0; i < ND; ++i) {
                    const typename T::Frag x = swa_ld_col_mem<E>(k + 32 * i + (lane & 31), krs, key + (32 / NP) * j, g);
                    acc[i] = T::mma(x, p, acc[i]);
                    if (few) acc[i] = T::mma(x, rest, acc[i]);
                    asm volatile("" : "+v"(acc[i]) : : "memory");
                }
            }
            key += 31;
            continue;
        }
        float s = 0.f, dp = 0.f;
#pragma unroll
        for (int ks = 0; ks < NK; ++ks) {
            s += T::dot(swa_ld_mem<E>(q, ks, g), swa_ld_mem<E>(k + key * krs, ks, g));
            dp += T::dot(swa_ld_mem<E>(dO, ks, g), swa_ld_mem<E>(v + key * vrs, ks, g));
            asm volatile("" : "+v"(s), "+v"(dp) : : "memory");
        }
        s += swa_swap(s);
        dp += swa_swap(dp);
        const bool sees = (key <= pos) & ((pos - key < W) | (key < S));
        const float ds = sees && !swa_alone(pos, W, S) ? __builtin_amdgcn_exp2f(fmaf(s, c, -lse2)) * (dp - delta) : 0.f;
        dsum += ds;
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const E4 x = *reinterpret_cast<const E4*>(k + key * krs + 32 * i + 8 * j + 4 * g);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[i][4 * j + e] = fmaf(ds, sees && !swa_alone(pos, W, S) ? (float)x[e] : 0.f, acc[i][4 * j + e]);
            }
    }
    return dsum + part + swa_swap(part);
}

template <int ND>
__device__ __forceinline__ float swa_zero_if_finite(const floatx16* x)
{
    float sum = 0.f;      // (0 times what is not finite is a NaN)
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) sum = fmaf(x[i][r], 0.f, sum);
    return sum;
}

template <class E, int D, int BN>
__global__ __launch_bounds__(256, sizeof(E) * D > 256 ? 1 : 2) void kd_swa_dq_kernel(SwaArgs a, int nslots)
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
    const int slot = nslots - 1 - item % nslots;
    item /= nslots;
    const int hk = item % a.Hkv, b = item / a.Hkv, h = hk * G + hg;
    SwaSeq s;
    if (!swa_locate(a, slot, 128, false, s)) return;
    const int r0 = s.blk * 128, row = r0 + 32 * w + (lane & 31), pos = s.past + row, rc = min(row, s.nq - 1);

    const E* qrow = (const E*)a.q + b * a.qs[0] + (int64_t)(s.q0 + rc) * a.qs[1] + h * a.qs[2];
    const int64_t orow = (((int64_t)b * a.Tq + s.q0 + rc) * a.Hq + h) * D;
    Frag q[NK], dO[NK];
    float delta = 0.f;
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
        q[ks] = swa_ld_mem<E>(qrow, ks, g);
        dO[ks] = swa_ld_mem<E>((const E*)a.dO + orow, ks, g);
        const Frag ov = swa_ld_mem<E>((const E*)a.o + orow, ks, g);
        delta += T::dot(dO[ks], ov);
    }
    delta += swa_swap(delta);
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
        swa_arrive(q[ks]);
        swa_arrive(dO[ks]);
    }
    const int64_t li = ((int64_t)b * a.Hq + h) * a.Tq + s.q0 + rc;
    float lse2 = a.lse[li] * LOG2E, dsum = 0.f;
    if (lse2 == -INFINITY) lse2 = 0.f;      // a row that sees nothing: a masked score has no weight whatever its lse
    asm volatile("" : "+v"(lse2));
    const SwaFetch<E, D, BN, 256> kf((const E*)a.k + b * a.ks[0] + (int64_t)s.q0 * a.ks[1] + hk * a.ks[2], a.ks[1], s.nk, tid);
    const SwaFetch<E, D, BN, 256> vf((const E*)a.v + b * a.vs[0] + (int64_t)s.q0 * a.vs[1] + hk * a.vs[2], a.vs[1], s.nk, tid);

    const int wp0 = s.past + r0 + 32 * w, wp1 = wp0 + 31;
    if (sizeof(E) == 2 && (wp0 < 32 || a.W <= 32 - a.S)) {
        const int first = max(0, wp0 - a.W + 1) & ~31;
        auto near = [&](int k0, int k1) {
            return swa_dq_near<E, D>(delta, q, dO, kf.base, a.ks[1], vf.base, a.vs[1], k0, min(k1, s.nk), s.nk, pos, a.W, a.S,
                                     a.c, lse2, lane);
        };
        float more = near(first, wp1 + 1);
        if (first > 0 && a.S > 0) more += near(0, a.S);
        delta += more + swa_swap(more);
    }

    floatx16 acc[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;

    const int pmax = min(s.past + r0 + 127, s.nk - 1);
    const int lo = max(0, s.past + r0 - a.W + 1) / BN, hi = pmax < 0 ? 0 : pmax / BN + 1;
    const int sk = min((a.S + BN - 1) / BN, lo), nt = sk + max(hi - lo, 0);
    const bool few = sizeof(E) == 2 && (wp0 < 511 || a.W + a.S < 512);
    auto key0 = [&](int i) { return (i < sk ? i : lo + (i - sk)) * BN; };
    auto fetch = [&](int i) {
        kf(kt[i & 1], 0, key0(i), w);
        vf(vt[i & 1], 0, key0(i), w);
    };
    if (nt > 0) fetch(0);
    auto tile = [&](int i, const E* kl, const E* vl) {
        swa_landed();
        if (i + 1 < nt) fetch(i + 1);
        const int k0 = key0(i);
        if (k0 > wp1 || (k0 + BN - 1 <= wp0 - a.W && k0 >= a.S)) return;
        const bool full = k0 + BN - 1 <= wp0 && (wp1 - k0 < a.W || k0 + BN <= a.S);
#pragma unroll 1      // (unrolled, the two halves spill)
        for (int n = 0; n < NS; ++n) {
            // the products of dP start from -delta
            floatx16 sc, dp;
#pragma unroll
            for (int r = 0; r < 16; ++r) sc[r] = 0.f, dp[r] = -delta;
#pragma unroll
            for (int ks = 0; ks < NK; ++ks) {
                sc = T::mma(swa_ld_row<E, D>(kl, 32 * n + (lane & 31), ks, g), q[ks], sc);
                dp = T::mma(swa_ld_row<E, D>(vl, 32 * n + (lane & 31), ks, g), dO[ks], dp);
            }
            if (!full) swa_mask_keys(sc, k0 + 32 * n + 4 * g, pos, a.W, a.S);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                sc[r] = __builtin_amdgcn_exp2f(fmaf(sc[r], a.c, -lse2)) * dp[r];
                dsum += sc[r];
            }
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const Frag p = T::pack(sc, j);
                Frag c[ND];
#pragma unroll
                for (int dt = 0; dt < ND; ++dt) {
                    c[dt] = T::template ld_col<D>(kl, 32 * n + (32 / NP) * j, 32 * dt, lane);
                    acc[dt] = T::mma(c[dt], p, acc[dt]);
                }
                if (few) {
                    const Frag rest = T::rest(sc, j, p);
#pragma unroll
                    for (int dt = 0; dt < ND; ++dt) acc[dt] = T::mma(c[dt], rest, acc[dt]);
                }
            }
        }
    };
    for (int i = 0; i < nt; i += 2) {
        tile(i, kt[0], vt[0]);
        if (i + 1 < nt) tile(i + 1, kt[1], vt[1]);
    }
    dsum += swa_swap(dsum);
    if (swa_alone(pos, a.W, a.S)) {
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;
    }
    // A hidden key's gradient is 0, and 0 times an infinity or a NaN in its key
    // or value would still reach the queries of its tile: a wave with a result
    // that is not finite makes it again over the keys that each query sees.
    if (__any(!(swa_zero_if_finite<ND>(acc) == 0.f)))
        dsum = swa_dq_single<E, D>(acc, qrow, (const E*)a.dO + orow, kf.base, a.ks[1], vf.base, a.vs[1], min(wp1, s.nk - 1), max(0, wp0 - a.W + 1),
                                   wp0, a.W, a.S, a.c, lse2, delta, few, lane);
    if (row >= s.nq) return;
    swa_store_row<E, D>((E*)a.dq + orow, acc, a.scale, g);
    // the sum of P dP: that of P (dP - delta) and delta (P sums to 1).  Queries
    // that see one key are zeros to the dK/dV pass, with lse 0.
    const bool alone = swa_alone(pos, a.W, a.S);
    if (g == 0) a.rows[li] = make_float2(alone ? 0.f : lse2, alone ? 0.f : delta + dsum);
}

// One 32-row piece of a query tile against 32 keys held as B operands (the
// values' either in registers or as rows of an LDS tile): S and dP have the
// queries as rows, so the weights and their gradients are again the B operands
// of the next products (dVt += dOt P, dKt += Qt dS).  few: the keys are seen by
// fewer than 64 queries; P and dS then carry what their rounding left, which
// averages out in longer sums.  rl: lse2 of the tile's
// queries, and RS floats on their -delta.
template <class E, int D, int RS, class VF>
__device__ __forceinline__ void swa_dkv_tile(const E* qt, const E* dt, const float* rl, int r0,
                                             const typename SwaT<E>::Frag* k, const VF& v,
                                             floatx16* dk, floatx16* dv, float c, bool full, bool few, int lane, int key, int p0,
                                             int left, int W, int S)
{
    typedef SwaT<E> T;
    typedef typename T::Frag Frag;
    constexpr int NK = D / T::KC, ND = D / 32, NP = 16 / T::PR;
    // (where registers are short the tile's LDS addresses are formed anew, not kept across the loop)
    if (sizeof(E) * D >= 256) lane += opaque_zero();
    const int g = lane >> 5;
    // lse and -delta of the queries; the products of dP start from -delta
    floatx16 sc, dp, ls;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const floatx4 le = *reinterpret_cast<const floatx4*>(rl + r0 + 8 * j + 4 * g);
        const floatx4 de = *reinterpret_cast<const floatx4*>(rl + RS + r0 + 8 * j + 4 * g);
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[4 * j + e] = 0.f, ls[4 * j + e] = le[e], dp[4 * j + e] = de[e];
    }
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) sc = T::mma(swa_ld_row<E, D>(qt, r0 + (lane & 31), ks, g), k[ks], sc);
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) dp = T::mma(swa_ld_row<E, D>(dt, r0 + (lane & 31), ks, g), v(ks, lane), dp);
    // (rows that see nothing have lse 0 here: a masked score has no weight)
    if (!full) swa_mask_rows(sc, key, p0 + 4 * g, left - 4 * g, W, S);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        sc[r] = __builtin_amdgcn_exp2f(fmaf(sc[r], c, -ls[r]));
        dp[r] *= sc[r];
    }
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        const Frag pv = T::pack(sc, j), pk = T::pack(dp, j);
#pragma unroll
        for (int i = 0; i < ND; ++i) {
            dv[i] = T::mma(T::template ld_col<D>(dt, r0 + (32 / NP) * j, 32 * i, lane), pv, dv[i]);
            dk[i] = T::mma(T::template ld_col<D>(qt, r0 + (32 / NP) * j, 32 * i, lane), pk, dk[i]);
        }
        if (sizeof(E) == 2 && few) {
            const Frag rv = T::rest(sc, j, pv), rk = T::rest(dp, j, pk);
            const int ln = lane + opaque_zero();
#pragma unroll
            for (int i = 0; i < ND; ++i) {
                dv[i] = T::mma(T::template ld_col<D>(dt, r0 + (32 / NP) * j, 32 * i, ln), rv, dv[i]);
                dk[i] = T::mma(T::template ld_col<D>(qt, r0 + (32 / NP) * j, 32 * i, ln), rk, dk[i]);
            }
        }
    }
}

// dK (before its scale) and dV of a wave's keys (wk0 .. wk0 + 31) again (rare,
// see its call): rows t0 .. t1 - 1 of G heads, 32 at a time where all of them
// see all of the keys, the others one after the other.
template <class E, int D, class VF>
__device__ __forceinline__ void swa_dkv_single(floatx16* dk, floatx16* dv, const E* k, const VF& v,
                                               const E* q, int64_t qrs, int64_t qhs, const E* dO, int64_t ors,
                                               const float2* rows, int64_t rhs, int G, int t0, int t1, int past, int wk0,
                                               int W, int S, float c, bool few, int lane)
{
    typedef SwaT<E> T;
    typedef E E4 __attribute__((ext_vector_type(4)));
    constexpr int NK = D / T::KC, ND = D / 32, NP = 16 / T::PR;
    const int g = lane >> 5, key = wk0 + (lane & 31);
    // 32 elements at a time, the scores anew for each: few registers beside k
#pragma unroll
    for (int i = 0; i < ND; ++i) {
        floatx16 x, y;
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] = y[r] = 0.f;
#pragma unroll 1
        for (int h = 0; h < G; ++h)
#pragma unroll 1
            for (int t = t0; t < t1; ++t) {
                if (t + 32 <= t1 && past + t >= wk0 + 31 && (past + t + 31 - wk0 < W || wk0 + 32 <= S)) {
                    const E* qa = q + h * qhs + (int64_t)(t + (lane & 31)) * qrs;
                    const E* ga = dO + h * D + (int64_t)(t + (lane & 31)) * ors;
                    floatx16 sc, dp;
#pragma unroll
                    for (int r = 0; r < 16; ++r) sc[r] = 0.f, dp[r] = -rows[h * rhs + t + 8 * (r / 4) + 4 * g + r % 4].y;
#pragma unroll
                    for (int ks = 0; ks < NK; ++ks) {
                        sc = T::mma(swa_ld_mem<E>(qa, ks, g), swa_ld_mem<E>(k, ks, g), sc);
                        dp = T::mma(swa_ld_mem<E>(ga, ks, g), v(ks, lane), dp);
                        asm volatile("" : "+v"(sc), "+v"(dp) : : "memory");      // (a few loads at a time)
                    }
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        sc[r] = __builtin_amdgcn_exp2f(fmaf(sc[r], c, -rows[h * rhs + t + 8 * (r / 4) + 4 * g + r % 4].x));
                        dp[r] *= sc[r];
                    }
#pragma unroll
                    for (int j = 0; j < NP; ++j) {
                        const typename T::Frag pv = T::pack(sc, j), pk = T::pack(dp, j);
                        const typename T::Frag ge = swa_ld_col_mem<E>(dO + h * D + 32 * i + (lane & 31), ors, t + (32 / NP) * j, g);
                        y = T::mma(ge, pv, y);
                        if (sizeof(E) == 2 && few) y = T::mma(ge, T::rest(sc, j, pv), y);
                        const typename T::Frag qe = swa_ld_col_mem<E>(q + h * qhs + 32 * i + (lane & 31), qrs, t + (32 / NP) * j, g);
                        x = T::mma(qe, pk, x);
                        if (sizeof(E) == 2 && few) x = T::mma(qe, T::rest(dp, j, pk), x);
                        asm volatile("" : "+v"(x), "+v"(y) : : "memory");
                    }
                    t += 31;
                    continue;
                }
                const E* qr = q + h * qhs + t * qrs;
                const E* gr = dO + h * D + t * ors;
                const float2 row = rows[h * rhs + t];
                float s = 0.f, dp = 0.f;
#pragma unroll
                for (int ks = 0; ks < NK; ++ks) {
                    s += SwaT<E>::dot(swa_ld_mem<E>(k, ks, g), swa_ld_mem<E>(qr, ks, g));
                    dp += SwaT<E>::dot(v(ks, lane), swa_ld_mem<E>(gr, ks, g));
                    asm volatile("" : "+v"(s), "+v"(dp) : : "memory");      // (a few loads at a time)
                }
                s += swa_swap(s);
                dp += swa_swap(dp);
                const int pos = past + t;
                const bool sees = (key <= pos) & ((pos - key < W) | (key < S));
                const bool alone = swa_alone(pos, W, S), moves = sees && !alone;
                const float p = !sees ? 0.f : alone ? 1.f : __builtin_amdgcn_exp2f(fmaf(s, c, -row.x));
                const float ds = moves ? p * (dp - row.y) : 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const E4 qe = *reinterpret_cast<const E4*>(qr + 32 * i + 8 * j + 4 * g);
                    const E4 ge = *reinterpret_cast<const E4*>(gr + 32 * i + 8 * j + 4 * g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[4 * j + e] = fmaf(ds, moves ? (float)qe[e] : 0.f, x[4 * j + e]);
                        y[4 * j + e] = fmaf(p, sees ? (float)ge[e] : 0.f, y[4 * j + e]);
                    }
                    asm volatile("" : : : "memory");
                }
            }
        dk[i] = x;
        dv[i] = y;
    }
}

// dK and dV of 128 keys of one key head, 32 per wave: tiles of BQ query rows
// of every head of the group pass through LDS, one tile ahead.  In bf16 the
// values' fragments are read from LDS too: with those of the keys, dK and dV
// in registers (160 of 256) two waves fit a SIMD, and one's products overlap
// the other's exponentials (matrix units 40% of the cycles, vector issue 41%).
// 4 x 4096, 16/4 heads of 128, window 1024, bf16: 355 us for four products (241
// GFLOP of visible pairs, 680 TFLOP/s; with V in registers and one wave per SIMD
// 623 us).
template <class E, int D, int BQ>
__global__ __launch_bounds__(256, sizeof(E) * D <= 256 ? 2 : 1) void kd_swa_dkv_kernel(SwaArgs a, int nslots)
{
    typedef SwaT<E> T;
    typedef typename T::Frag Frag;
    constexpr int NK = D / T::KC, NS = BQ / 32, ND = D / 32;
    constexpr bool VL = sizeof(E) == 2;
    // the tiles first: loads to LDS take destinations in its first 64 KB
    __shared__ __align__(16) struct {
        E q[2][BQ * D], dO[2][BQ * D];
        E v[VL ? 128 * D : 8];
        float rows[2][2][BQ];      // lse2, -delta
    } sm;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 5;
    const int G = a.Hq / a.Hkv;
    int64_t item;
    if (!swa_item((int64_t)nslots * a.nsp * a.Hkv * a.B, item)) return;
    const int slot = item % nslots;
    item /= nslots;
    const int sp = item % a.nsp, g0 = sp * G / a.nsp, GS = (sp + 1) * G / a.nsp - g0;      // its heads of the group
    item /= a.nsp;
    const int hk = item % a.Hkv, b = item / a.Hkv;
    SwaSeq s;
    if (!swa_locate(a, slot, 128, true, s)) return;
    const int k0 = s.blk * 128, key = k0 + 32 * w + (lane & 31), kc = min(key, s.nk - 1);
    const E* krow = (const E*)a.k + b * a.ks[0] + (int64_t)(s.q0 + kc) * a.ks[1] + hk * a.ks[2];
    const E* vrow = (const E*)a.v + b * a.vs[0] + (int64_t)(s.q0 + kc) * a.vs[1] + hk * a.vs[2];
    Frag k[NK], vr[VL ? 1 : NK];
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
        k[ks] = swa_ld_mem<E>(krow, ks, g);
        if (!VL) vr[VL ? 0 : ks] = swa_ld_mem<E>(vrow, ks, g);
    }
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
        swa_arrive(k[ks]);
        if (!VL) swa_arrive(vr[VL ? 0 : ks]);
    }
    if (VL) {
        const SwaFetch<E, D, 128, 256> vf((const E*)a.v + b * a.vs[0] + (int64_t)s.q0 * a.vs[1] + hk * a.vs[2], a.vs[1], s.nk, tid);
        vf(sm.v, 0, k0, w);
    }
    auto v = [&](int ks, int ln) -> Frag {
        if constexpr (VL) return swa_ld_row<E, D>(sm.v, 32 * w + (ln & 31), ks, ln >> 5);
        else return vr[ks];
    };
    floatx16 dk[ND], dv[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) dk[i][r] = dv[i][r] = 0.f;

    // rows whose window holds a key of the block, for every head of the group
    const int t0 = max(0, k0 - s.past) / BQ, t1 = min(s.nq, k0 + 127 + a.W - s.past);
    const int per = max(0, (t1 + BQ - 1) / BQ - t0), nt = per * GS;
    const int wk0 = k0 + 32 * w, wk1 = wk0 + 31;
    const bool few = (int64_t)(min(t1, wk1 + a.W - s.past) - max(0, wk0 - s.past)) * G < 64;
    const SwaFetch<E, D, BQ, 256> qf((const E*)a.q + b * a.qs[0] + (int64_t)s.q0 * a.qs[1] + (hk * G + g0) * a.qs[2], a.qs[1], s.nq, tid);
    const SwaFetch<E, D, BQ, 256> of((const E*)a.dO + (((int64_t)b * a.Tq + s.q0) * a.Hq + hk * G + g0) * D, (int64_t)a.Hq * D, s.nq, tid);
    const float2* rb = a.rows + ((int64_t)b * a.Hq + hk * G + g0) * a.Tq + s.q0;
    int fh = 0, ft = 0;      // head and tile of the next fetch
    float2 next;             // lse and delta of a row of it
    auto fetch = [&](int i) {
        const int t = (t0 + ft) * BQ;
        qf(sm.q[i & 1], fh * a.qs[2], t, w);
        of(sm.dO[i & 1], fh * D, t, w);
        if (tid < BQ) next = rb[(int64_t)fh * a.Tq + min(t + tid, s.nq - 1)];
        if (++ft == per) {
            ft = 0;
            ++fh;
        }
    };
    if (nt > 0) {
        fetch(0);
        if (tid < BQ) sm.rows[0][0][tid] = next.x, sm.rows[0][1][tid] = -next.y;
    }
    int ct = 0;
    for (int i = 0; i < nt; ++i) {
        swa_landed();
        if (i + 1 < nt) fetch(i + 1);
        const int t = (t0 + ct) * BQ;
        if (++ct == per) ct = 0;
        const int p0 = s.past + t, p1 = p0 + BQ - 1;
        // Queries that see one key become zeros: their score is 0, their weight
        // exp2(0 - 0) = 1, and dK takes nothing from them, with no test per pair.
        if (p0 <= 0 || a.W + a.S == 1) {
            typedef SwaTile<E, D> TL;
            for (int x = tid; x < BQ * TL::CPR; x += 256)
                if (swa_alone(p0 + x / TL::CPR, a.W, a.S))
                    *reinterpret_cast<Frag*>(sm.q[i & 1] + x * TL::EPC) = swa_zero<E>();
            __syncthreads();
        }
        if (!(p1 < wk0 || (p0 - wk1 >= a.W && wk0 >= a.S))) {
            const bool full = p0 >= wk1 && (p1 - wk0 < a.W || wk1 < a.S) && t + BQ <= t1;   // (rows from t1 on: the sinks' pass)
#pragma unroll
            for (int n = 0; n < NS; ++n)
                swa_dkv_tile<E, D, BQ>(sm.q[i & 1], sm.dO[i & 1], sm.rows[i & 1][0], 32 * n, k, v, dk, dv, a.c, full, few, lane,
                                   key, p0 + 32 * n, t1 - t - 32 * n, a.W, a.S);
        }
        if (i + 1 < nt && tid < BQ) sm.rows[(i + 1) & 1][0][tid] = next.x, sm.rows[(i + 1) & 1][1][tid] = -next.y;
    }
    // queries that do not see a key, as in dQ
    if (__any(!(swa_zero_if_finite<ND>(dk) + swa_zero_if_finite<ND>(dv) == 0.f)))
        swa_dkv_single<E, D>(dk, dv, krow, v, qf.base, a.qs[1], a.qs[2], of.base, (int64_t)a.Hq * D, rb, a.Tq, GS,
                             max(0, wk0 - s.past), t1, s.past, wk0, a.W, a.S, a.c, few, lane);
    // the sinks' part from the queries beyond the window: all threads add the
    // chunks' partial sums, the lanes that hold the keys take them from LDS
    if (s.blk == 0 && a.pslots > 0 && swa_far(a, s.past) < s.nq) {
        const int first = s.slot0 + swa_far(a, s.past) / a.chunk, last = s.slot0 + (s.nq - 1) / a.chunk;
        float* sum = reinterpret_cast<float*>(&sm);
        const int64_t step = (int64_t)a.Hq * 2 * a.S * D;      // floats of one chunk
        for (int x = 0; x < 2; ++x) {
            const float* pb = a.part + ((int64_t)b * a.pslots + first) * step + ((int64_t)(hk * G + g0) * 2 + x) * a.S * D;
            __syncthreads();
            for (int i = tid; i < a.S * D / 4; i += 256) {
                floatx4 z = {0.f, 0.f, 0.f, 0.f};
                for (int y = 0; y <= last - first; ++y)
#pragma unroll 4
                    for (int hg = 0; hg < GS; ++hg)
                        z += reinterpret_cast<const floatx4*>(pb + y * step + (int64_t)hg * 2 * a.S * D)[i];
                reinterpret_cast<floatx4*>(sum)[i] = z;
            }
            __syncthreads();
            if (key < a.S) {
#pragma unroll
                for (int i = 0; i < ND; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const floatx4 z = *reinterpret_cast<const floatx4*>(sum + key * D + 32 * i + 8 * j + 4 * g);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (x == 0) dk[i][4 * j + e] += z[e];
                            else dv[i][4 * j + e] += z[e];
                        }
                    }
            }
        }
    }
    if (key >= s.nk) return;
    const int64_t at = (((int64_t)b * a.Tk + s.q0 + key) * a.Hkv + hk) * D;
    if (a.nsp > 1) {
        const int64_t n = (int64_t)a.B * a.Tk * a.Hkv * D;
        swa_store_row<float, D>(a.shared + 2 * sp * n + at, dk, a.scale, g);
        swa_store_row<float, D>(a.shared + (2 * sp + 1) * n + at, dv, 1.f, g);
        return;
    }
    swa_store_row<E, D>((E*)a.dk + at, dk, a.scale, g);
    swa_store_row<E, D>((E*)a.dv + at, dv, 1.f, g);
}

// The sum of the workgroups' parts of dK (y = 0) and dV, in their order: n / 4
// pieces of four elements, still in the caches.
template <class E>
__global__ __launch_bounds__(256) void kd_swa_sum_kernel(SwaArgs a, int64_t n)
{
    typedef E E4 __attribute__((ext_vector_type(4)));
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    const float* p = a.shared + blockIdx.y * n + i;
    floatx4 z = *reinterpret_cast<const floatx4*>(p);
    for (int sp = 1; sp < a.nsp; ++sp) z += *reinterpret_cast<const floatx4*>(p + 2 * sp * n);
    E4 x;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = (E)z[e];
    *reinterpret_cast<E4*>((E*)(blockIdx.y ? a.dv : a.dk) + i) = x;
}

// Partial dK and dV of 32 sinks from one chunk of one head's queries beyond the
// window: the waves share the rows (32 each of a tile), their sums are joined in LDS
// one wave after the other.  4 x 4096 queries of 16 heads beyond a window of 1024:
// 34 us, bound by reading Q and dO tile by tile (matrix units 11% of the cycles).
template <class E, int D, int NW>
__global__ __launch_bounds__(64 * NW, 1) void kd_swa_sink_kernel(SwaArgs a)
{
    typedef SwaT<E> T;
    typedef typename T::Frag Frag;
    constexpr int NK = D / T::KC, ND = D / 32, BQ = 32 * NW;
    __shared__ __align__(16) struct {
        E q[BQ * D], dO[BQ * D];
        float rows[2][BQ];
    } sm;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 5;
    const int ng = (a.S + 31) / 32;
    const int slot = blockIdx.x / ng, k0 = blockIdx.x % ng * 32, h = blockIdx.y, hk = h / (a.Hq / a.Hkv), b = blockIdx.z;
    SwaSeq s;
    if (!swa_locate(a, slot, a.chunk, false, s, a.apart)) return;
    const int ta = max(s.blk * a.chunk, swa_far(a, s.past)), tb = min(s.blk * a.chunk + a.chunk, s.nq);
    if (ta >= tb) return;
    const int key = k0 + (lane & 31), kc = min(key, s.nk - 1);
    const E* krow = (const E*)a.k + b * a.ks[0] + (int64_t)(s.q0 + kc) * a.ks[1] + hk * a.ks[2];
    const E* vrow = (const E*)a.v + b * a.vs[0] + (int64_t)(s.q0 + kc) * a.vs[1] + hk * a.vs[2];
    Frag k[NK], v[NK];
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
        k[ks] = swa_ld_mem<E>(krow, ks, g);
        v[ks] = swa_ld_mem<E>(vrow, ks, g);
    }
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
        swa_arrive(k[ks]);
        swa_arrive(v[ks]);
    }
    floatx16 dk[ND], dv[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) dk[i][r] = dv[i][r] = 0.f;
    const bool all = k0 + 32 <= a.S, few = (int64_t)(s.nq - swa_far(a, s.past)) * (a.Hq / a.Hkv) < 64;
    auto vf = [&](int ks, int) -> Frag { return v[ks]; };
    const SwaFetch<E, D, BQ, 64 * NW> qf((const E*)a.q + b * a.qs[0] + (int64_t)s.q0 * a.qs[1] + h * a.qs[2], a.qs[1], s.nq, tid);
    const SwaFetch<E, D, BQ, 64 * NW> of((const E*)a.dO + (((int64_t)b * a.Tq + s.q0) * a.Hq + h) * D, (int64_t)a.Hq * D, s.nq, tid);
    const float2* rb = a.rows + ((int64_t)b * a.Hq + h) * a.Tq + s.q0;
    for (int t = ta; t < tb; t += BQ) {
        __syncthreads();
        qf(sm.q, 0, t, w);
        of(sm.dO, 0, t, w);
        if (tid < BQ) {
            const float2 x = rb[min(t + tid, s.nq - 1)];
            sm.rows[0][tid] = x.x;
            sm.rows[1][tid] = -x.y;
        }
        swa_landed();
        // beyond the window a row sees the sinks alone: window 1 leaves their mask
        swa_dkv_tile<E, D, BQ>(sm.q, sm.dO, sm.rows[0], 32 * w, k, vf, dk, dv, a.c, all && t + BQ <= tb, few, lane, key,
                           s.past + t + 32 * w, tb - t - 32 * w, 1, a.S);
    }
    __syncthreads();
    constexpr int DP = D + 4;                        // (a row's stride: the lanes' rows start in different banks)
    float* sum = reinterpret_cast<float*>(&sm);      // 32 keys by D, dK then dV
    float* out = a.part + ((((int64_t)b * a.pslots + slot) * a.Hq + h) * 2 * a.S + k0) * D;
    for (int x = 0; x < 2; ++x) {
        for (int y = 0; y < NW; ++y) {
            if (w == y && key < a.S) {
#pragma unroll
                for (int i = 0; i < ND; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        floatx4* p = reinterpret_cast<floatx4*>(sum + (lane & 31) * DP + 32 * i + 8 * j + 4 * g);
                        floatx4 z;
#pragma unroll
                        for (int e = 0; e < 4; ++e) z[e] = x == 0 ? dk[i][4 * j + e] : dv[i][4 * j + e];
                        *p = y == 0 ? z : *p + z;
                    }
            }
            __syncthreads();
        }
        for (int i = tid; i < min(32, a.S - k0) * D / 4; i += 64 * NW)
            reinterpret_cast<floatx4*>(out + x * a.S * D)[i] =
                *reinterpret_cast<const floatx4*>(sum + i / (D / 4) * DP + i % (D / 4) * 4);
        __syncthreads();
    }
}

// Rows of a chunk of the sinks' pass: about 256 workgroups over all heads, so
// that the start of each is paid for, and chunks of 256 to 4096 rows.
static int swa_chunk(int64_t rows, int Hq, int S) {
    const int64_t n = rows * Hq * ((S + 31) / 32) / 256;
    return (int)min((int64_t)4096, max((int64_t)256, (n + 127) / 128 * 128));
}

// Rows by which the sinks' pass numbers packed sequences: those of 128 + W rows
// or more have queries beyond the window of their first 128 keys.  0 (one by
// one) where that needs fewer slots.
static int swa_apart(bool packed, int N, int T, int W) {
    const int64_t least = 128 + (int64_t)W;
    return packed && T / least < N ? (int)min(least, (int64_t)INT32_MAX) : 0;
}

// Chunks of the sinks' partial sums; none where every query lies within the
// window of the first 128 keys.
static int64_t swa_part_slots(bool packed, int N, int Tq, int Tk, int W, int S, int chunk) {
    if (S == 0 || Tq == 0 || Tk <= 127 + (int64_t)W) return 0;
    const int apart = swa_apart(packed, N, Tq, W);
    return swa_slots(packed, apart > 0 ? Tq / apart : N, Tq, chunk);
}

static size_t swa_rows_bytes(int B, int Tq, int Hq) { return ((size_t)B * Tq * Hq * 8 + 255) & ~(size_t)255; }

static size_t swa_part_bytes(int64_t slots, int B, int Hq, int S, int d) { return (size_t)slots * B * Hq * 2 * S * d * 4; }

// Workgroups that share the heads of a group in the dK/dV pass: so that there
// is one for each of the chip's 256 compute units, or two where a group's rows
// are many (1536: 48 tiles; the parts, 128 KB of each workgroup's, are written
// and read once more); none share below 512 rows (16 tiles).  Packed calls bring
// their own blocks.  The heads' sums are added in another order then, so the last
// bits differ from an unshared call's.  The whole backward, bf16, heads of 128, one workgroup per block and
// shared: 1 x 820, 32/8 heads: 199 and 94 us; 1 x 4096, 16/1 heads, window 1024:
// 970 and 190 us; 1 x 4096, 16/8 heads (256 blocks), window 1024: 191 and 174 us,
// window 256: 90 and, shared against the rule, 98 us; 1 x 200, 8/2: 45 and 31 us.
static int swa_head_splits(bool packed, int B, int Tq, int Tk, int Hq, int Hkv, int W) {
    const int64_t blocks = swa_slots(false, B, Tk, 128) * Hkv * B;
    const int64_t rows = min((int64_t)Tq, (int64_t)min(W, Tk) + 127) * (Hq / Hkv);
    if (packed || blocks == 0 || rows < 512) return 1;
    return (int)max((int64_t)1, min((int64_t)(Hq / Hkv), (rows < 1536 ? 256 : 512) / blocks));
}

size_t swa_bwd_workspace_bytes(bool packed, int B, int Tq, int Tk, int Hq, int Hkv, int d, int W, int S) {
    const int nb = packed ? 1 : B, nsp = swa_head_splits(packed, B, Tq, Tk, Hq, Hkv, W);
    return swa_rows_bytes(nb, Tq, Hq) +
           swa_part_bytes(swa_part_slots(packed, B, Tq, Tk, W, S, swa_chunk((int64_t)nb * Tq, Hq, S)), nb, Hq, S, d) +
           (nsp > 1 ? (size_t)nsp * 2 * B * Tk * Hkv * d * 4 : 0);
}

// Whether the grids of all passes are possible.
bool swa_bwd_fits(bool packed, int N, int B, int Tq, int Tk, int Hq, int Hkv, int d, int W, int S) {
    const int64_t ks = swa_slots(packed, N, Tk, 128) * swa_head_splits(packed, B, Tq, Tk, Hq, Hkv, W);
    const int64_t np = swa_part_slots(packed, N, Tq, Tk, W, S, swa_chunk((int64_t)B * Tq, Hq, S));
    return grid_fits(swa_grid(swa_slots(packed, N, Tq, 128) * Hq * B), 256) && grid_fits(swa_grid(ks * Hkv * B), 256) &&
           grid_fits(np * ((S + 31) / 32), 256) && grid_fits(((int64_t)B * Tk * Hkv * d / 4 + 255) / 256, 256);
}

template <class E, int D>
static hipError_t swa_bwd(SwaArgs a, void* ws, hipStream_t st)
{
    constexpr int BN = sizeof(E) == 2 ? 64 : 32;
    const int64_t nq = swa_slots(a.cu, a.N, a.Tq, 128), nk = swa_slots(a.cu, a.N, a.Tk, 128);
    const int64_t gq = swa_grid(nq * a.Hq * a.B);
    a.nsp = swa_head_splits(a.cu, a.B, a.Tq, a.Tk, a.Hq, a.Hkv, a.W);
    const int64_t gk = swa_grid(nk * a.nsp * a.Hkv * a.B);
    a.chunk = swa_chunk((int64_t)a.B * a.Tq, a.Hq, a.S);
    const int64_t np = swa_part_slots(a.cu, a.N, a.Tq, a.Tk, a.W, a.S, a.chunk);
    a.apart = swa_apart(a.cu, a.N, a.Tq, a.W);
    a.rows = (float2*)ws;
    a.part = (float*)((char*)ws + swa_rows_bytes(a.B, a.Tq, a.Hq));
    a.pslots = (int)np;
    a.shared = (float*)((char*)a.part + swa_part_bytes(np, a.B, a.Hq, a.S, D));
    if (a.Tq > 0) {
        kd_swa_dq_kernel<E, D, BN><<<(unsigned)gq, 256, 0, st>>>(a, (int)nq);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (np > 0) {
        constexpr int NW = sizeof(E) == 2 ? 4 : 2;
        kd_swa_sink_kernel<E, D, NW><<<dim3((unsigned)(np * ((a.S + 31) / 32)), a.Hq, a.B), 64 * NW, 0, st>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (nk == 0) return hipSuccess;
    kd_swa_dkv_kernel<E, D, sizeof(E) * D <= 128 ? 64 : 32><<<(unsigned)gk, 256, 0, st>>>(a, (int)nk);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.nsp == 1) return e;
    const int64_t n = (int64_t)a.B * a.Tk * a.Hkv * D;
    kd_swa_sum_kernel<E><<<dim3((unsigned)((n / 4 + 255) / 256), 2), 256, 0, st>>>(a, n);
    return hipGetLastError();
}

hipError_t launch_swa_bwd(int bf16, int d, const SwaArgs& a, void* ws, hipStream_t st)
{
    if (bf16) return d == 32 ? swa_bwd<__bf16, 32>(a, ws, st) : d == 64 ? swa_bwd<__bf16, 64>(a, ws, st) : swa_bwd<__bf16, 128>(a, ws, st);
    return d == 32 ? swa_bwd<float, 32>(a, ws, st) : d == 64 ? swa_bwd<float, 64>(a, ws, st) : swa_bwd<float, 128>(a, ws, st);
}

}  // namespace kd
