// kd_swa_bwd.hip -- sliding-window attention with sinks, backward, gfx950.
//
// With P = exp(scale s - lse) recomputed from the saved lse and
// delta_t = sum_i dO_ti o_ti:
//     dV = Pt dO;  dP = dO Vt;  dS = P (dP - delta);  dQ = scale dS K;  dK = scale dSt Q
// Two kernels, so that every gradient is summed in registers in a fixed order
// (no atomics): one over query blocks for dQ (and delta), one over key blocks
// for dK and dV, which also sums over the query heads that share a key head.
#include "kd_swa.h"

namespace kd {

// dQ and delta of 128 query rows of one head: the forward's layout, with the
// scores' gradient in the weights' place and K in V's.
template <class E, int D, int BN>
__global__ __launch_bounds__(256) void kd_swa_dq_kernel(SwaArgs a)
{
    typedef SwaT<E> T;
    typedef typename T::Frag Frag;
    constexpr int NK = D / T::KC, NS = BN / 32, ND = D / 32, NP = 16 / T::PR;
    __shared__ __align__(16) E kt[BN * D];
    __shared__ __align__(16) E vt[BN * D];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 5;
    const int h = blockIdx.y, b = blockIdx.z, hk = h / (a.Hq / a.Hkv);
    SwaSeq s;
    if (!swa_locate(a, blockIdx.x, 128, false, s)) return;
    const int r0 = s.blk * 128, row = r0 + 32 * w + (lane & 31), pos = s.past + row, rc = min(row, s.nq - 1);

    const E* qrow = (const E*)a.q + b * a.qs[0] + (int64_t)(s.q0 + rc) * a.qs[1] + h * a.qs[2];
    const int64_t orow = (((int64_t)b * a.Tq + s.q0 + rc) * a.Hq + h) * D;
    Frag q[NK], dO[NK];
    float delta = 0.f;
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
        q[ks] = row < s.nq ? swa_ld_mem<E>(qrow, ks, g) : swa_zero<E>();
        dO[ks] = row < s.nq ? swa_ld_mem<E>((const E*)a.dO + orow, ks, g) : swa_zero<E>();
        const Frag ov = row < s.nq ? swa_ld_mem<E>((const E*)a.o + orow, ks, g) : swa_zero<E>();
        delta += T::dot(dO[ks], ov);
    }
    delta += swa_swap(delta);
    const int64_t li = ((int64_t)b * a.Hq + h) * a.Tq + s.q0 + rc;
    const float lse2 = a.lse[li] * 1.4426950408889634f;
    if (row < s.nq && g == 0) a.delta[li] = delta;
    const E* kb = (const E*)a.k + b * a.ks[0] + (int64_t)s.q0 * a.ks[1] + hk * a.ks[2];
    const E* vb = (const E*)a.v + b * a.vs[0] + (int64_t)s.q0 * a.vs[1] + hk * a.vs[2];

    floatx16 acc[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;

    const int pmax = min(s.past + r0 + 127, s.nk - 1);
    const int lo = max(0, s.past + r0 - a.W + 1) / BN, hi = pmax < 0 ? 0 : pmax / BN + 1;
    const int sk = min((a.S + BN - 1) / BN, lo);
    const int wp0 = s.past + r0 + 32 * w, wp1 = wp0 + 31;
    for (int i = 0; i < sk + max(hi - lo, 0); ++i) {
        const int k0 = (i < sk ? i : lo + (i - sk)) * BN;
        __syncthreads();
        swa_stage<E, D, BN, 256>(kt, kb, a.ks[1], k0, s.nk, tid);
        swa_stage<E, D, BN, 256>(vt, vb, a.vs[1], k0, s.nk, tid);
        __syncthreads();
        if (k0 > wp1 || (k0 + BN - 1 <= wp0 - a.W && k0 >= a.S)) continue;
        const bool full = k0 + BN - 1 <= wp0 && (wp1 - k0 < a.W || k0 + BN <= a.S);
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            floatx16 sc, dp;
#pragma unroll
            for (int r = 0; r < 16; ++r) sc[r] = dp[r] = 0.f;
#pragma unroll
            for (int ks = 0; ks < NK; ++ks) {
                sc = T::mma(swa_ld_row<E, D>(kt, 32 * n + (lane & 31), ks, g), q[ks], sc);
                dp = T::mma(swa_ld_row<E, D>(vt, 32 * n + (lane & 31), ks, g), dO[ks], dp);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float p = __builtin_amdgcn_exp2f(fmaf(sc[r], a.c, -lse2)) * (dp[r] - delta);
                const bool vis = full || swa_visible(k0 + 32 * n + 8 * (r / 4) + 4 * g + r % 4, pos, a.W, a.S);
                sc[r] = vis ? p : 0.f;
            }
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const Frag p = T::pack(sc, j);
#pragma unroll
                for (int dt = 0; dt < ND; ++dt)
                    acc[dt] = T::mma(T::template ld_col<D>(kt, 32 * n + (32 / NP) * j, 32 * dt, lane), p, acc[dt]);
            }
        }
    }
    if (row < s.nq) swa_store_row<E, D>((E*)a.dq + orow, acc, a.scale, g);
}

// dK and dV of 128 keys of one key head, 32 per wave: tiles of BQ query rows
// of every head of the group pass through LDS.  S = Q Kt has the queries as
// rows, so the weights and their gradients are again the B operands of the
// next products (dVt += dOt P, dKt += Qt dS).
template <class E, int D, int BQ>
__global__ __launch_bounds__(256) void kd_swa_dkv_kernel(SwaArgs a)
{
    typedef SwaT<E> T;
    typedef typename T::Frag Frag;
    constexpr int NK = D / T::KC, NS = BQ / 32, ND = D / 32, NP = 16 / T::PR;
    __shared__ __align__(16) E qt[BQ * D];
    __shared__ __align__(16) E dt_[BQ * D];
    __shared__ __align__(16) float ls[BQ], ds[BQ];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 5;
    const int hk = blockIdx.y, b = blockIdx.z, G = a.Hq / a.Hkv;
    SwaSeq s;
    if (!swa_locate(a, blockIdx.x, 128, true, s)) return;
    const int k0 = s.blk * 128, key = k0 + 32 * w + (lane & 31), kc = min(key, s.nk - 1);
    const E* krow = (const E*)a.k + b * a.ks[0] + (int64_t)(s.q0 + kc) * a.ks[1] + hk * a.ks[2];
    const E* vrow = (const E*)a.v + b * a.vs[0] + (int64_t)(s.q0 + kc) * a.vs[1] + hk * a.vs[2];
    Frag k[NK], v[NK];
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
        k[ks] = key < s.nk ? swa_ld_mem<E>(krow, ks, g) : swa_zero<E>();
        v[ks] = key < s.nk ? swa_ld_mem<E>(vrow, ks, g) : swa_zero<E>();
    }
    floatx16 dk[ND], dv[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) dk[i][r] = dv[i][r] = 0.f;

    // rows that see a key of the block
    const int t0 = max(0, k0 - s.past) / BQ * BQ;
    const int t1 = k0 < a.S ? s.nq : min(s.nq, k0 + 127 + a.W - s.past);
    const int wk0 = k0 + 32 * w, wk1 = wk0 + 31;
    for (int hg = 0; hg < G; ++hg) {
        const int h = hk * G + hg;
        const E* qb = (const E*)a.q + b * a.qs[0] + (int64_t)s.q0 * a.qs[1] + h * a.qs[2];
        const E* ob = (const E*)a.dO + (((int64_t)b * a.Tq + s.q0) * a.Hq + h) * D;
        const int64_t li = ((int64_t)b * a.Hq + h) * a.Tq + s.q0;
        for (int t = t0; t < t1; t += BQ) {
            __syncthreads();
            swa_stage<E, D, BQ, 256>(qt, qb, a.qs[1], t, s.nq, tid);
            swa_stage<E, D, BQ, 256>(dt_, ob, (int64_t)a.Hq * D, t, s.nq, tid);
            if (tid < BQ) {
                ls[tid] = t + tid < s.nq ? a.lse[li + t + tid] * 1.4426950408889634f : 0.f;
                ds[tid] = t + tid < s.nq ? a.delta[li + t + tid] : 0.f;
            }
            __syncthreads();
            const int p0 = s.past + t, p1 = p0 + BQ - 1;
            if (p1 < wk0 || (p0 - wk1 >= a.W && wk0 >= a.S)) continue;
            const bool full = p0 >= wk1 && (p1 - wk0 < a.W || wk1 < a.S) && t + BQ <= s.nq;
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                floatx16 sc, dp;
#pragma unroll
                for (int r = 0; r < 16; ++r) sc[r] = dp[r] = 0.f;
#pragma unroll
                for (int ks = 0; ks < NK; ++ks) {
                    sc = T::mma(swa_ld_row<E, D>(qt, 32 * n + (lane & 31), ks, g), k[ks], sc);
                    dp = T::mma(swa_ld_row<E, D>(dt_, 32 * n + (lane & 31), ks, g), v[ks], dp);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int rr = 32 * n + 8 * j + 4 * g;
                    const floatx4 le = *reinterpret_cast<const floatx4*>(ls + rr);
                    const floatx4 de = *reinterpret_cast<const floatx4*>(ds + rr);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int r = 4 * j + e;
                        const bool vis = full || (t + rr + e < s.nq && swa_visible(key, p0 + rr + e, a.W, a.S));
                        const float p = __builtin_amdgcn_exp2f(fmaf(sc[r], a.c, -le[e]));
                        sc[r] = vis ? p : 0.f;
                        dp[r] = vis ? p * (dp[r] - de[e]) : 0.f;
                    }
                }
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    const Frag pv = T::pack(sc, j), pk = T::pack(dp, j);
#pragma unroll
                    for (int i = 0; i < ND; ++i) {
                        dv[i] = T::mma(T::template ld_col<D>(dt_, 32 * n + (32 / NP) * j, 32 * i, lane), pv, dv[i]);
                        dk[i] = T::mma(T::template ld_col<D>(qt, 32 * n + (32 / NP) * j, 32 * i, lane), pk, dk[i]);
                    }
                }
            }
        }
    }
    if (key >= s.nk) return;
    const int64_t at = (((int64_t)b * a.Tk + s.q0 + key) * a.Hkv + hk) * D;
    swa_store_row<E, D>((E*)a.dk + at, dk, a.scale, g);
    swa_store_row<E, D>((E*)a.dv + at, dv, 1.f, g);
}

template <class E, int D>
static hipError_t swa_bwd(const SwaArgs& a, hipStream_t st)
{
    constexpr int BN = sizeof(E) == 2 ? 64 : 32;
    const unsigned nq = a.cu ? (unsigned)(a.Tq / 128 + a.N) : (unsigned)(((int64_t)a.Tq + 127) / 128);
    const unsigned nk = a.cu ? nq : (unsigned)(((int64_t)a.Tk + 127) / 128);
    if (a.Tq > 0) {
        kd_swa_dq_kernel<E, D, BN><<<dim3(nq, a.Hq, a.B), 256, 0, st>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (nk == 0) return hipSuccess;
    kd_swa_dkv_kernel<E, D, 32><<<dim3(nk, a.Hkv, a.B), 256, 0, st>>>(a);
    return hipGetLastError();
}

size_t swa_bwd_workspace_bytes(int B, int Tq, int Hq) { return (((size_t)B * Tq * Hq * 4) + 255) & ~(size_t)255; }

hipError_t launch_swa_bwd(int bf16, int d, const SwaArgs& a, hipStream_t st)
{
    if (bf16) return d == 32 ? swa_bwd<__bf16, 32>(a, st) : d == 64 ? swa_bwd<__bf16, 64>(a, st) : swa_bwd<__bf16, 128>(a, st);
    return d == 32 ? swa_bwd<float, 32>(a, st) : d == 64 ? swa_bwd<float, 64>(a, st) : swa_bwd<float, 128>(a, st);
}

}  // namespace kd
