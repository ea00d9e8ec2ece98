// kd_gdr_bwd.hip -- gated delta rule, backward, gfx950.
//
// With S0 the state entering a chunk (kept by the forward pass), dS_C the
// gradient of the one leaving it and the notation of kd_gdr.h:
//     dU  = P^T dO + e^(bC - b) K dS_C^T,   X = A^T dU,   dV = beta X
//     dS0 = e^bC dS_C + (scale e^b dO)^T Q - (beta e^b X)^T K
// is the pass over the chunks, backwards, as the forward's; and per chunk
//     W = V - e^b K S0^T,  U = A beta W
//     E = Gam (scale dO U^T) (s <= r),   F = -beta Gam (X U^T) (s < r)
//     dQ = E K + scale e^b dO S0
//     dK = E^T Q + (F + F^T) K + e^(bC - b) U dS_C - beta e^b X S0
//     dbeta_r = X_r.W_r + sum_s F_rs k_r.k_s / beta_r
// The gradient of b collects what each e^b multiplies (rows minus columns of E
// times Q K^T and of F times K K^T, and dot products of the terms above with q
// and k); dg is its sum from the chunk's end, with that of e^bC.
#include "kd_check.h"
#include "kd_gdr.h"

namespace kd {

int64_t gdr_pass_grid(int64_t items, int& run);

// The pass backwards, two waves for every 16 value columns as in the forward
// pass.  The first has the gradient of the state in registers and makes what the
// next chunk waits for.  The second makes what does not depend on it a chunk
// ahead, P^T dO and (scale e^b dO)^T Q, which the first adds in fp32 from LDS, and
// a chunk behind writes X (and dV from it), which it finds in LDS; it makes the
// loads.  Where LDS holds two chunks' worth of what the second wave reads
// (FAR), the barrier in the middle comes before its products, not behind.
//
// Bound by what a chunk waits for, as the forward pass, with one product more for
// the second wave and two products' results through LDS in fp32: 3.2 us a chunk
// with two groups a workgroup (4 sequences of 2048 tokens, 16 heads of 128: 107
// us; one wave for both parts: 159; without FAR: 121), 6.2 us with four.
template <class E, int DK, int CG>
__global__ __launch_bounds__(128 * CG, CG == 4 ? 2 : 1) void kd_gdr_back_kernel(GdrArgs a, int run)
{
    typedef GdrT<E> T;
    typedef typename T::Frag Frag;
    typedef E E4 __attribute__((ext_vector_type(4)));
    constexpr int NT = 64 * CG, NC0 = 16 * CG, W = T::TWO ? 2 : 1, NK = DK / 32, NBUF = sizeof(E) * DK > 256 ? 1 : 2;
    constexpr bool FAR = sizeof(E) == 2 && (DK == 64 || CG == 2);
    constexpr bool KFIRST = sizeof(E) == 2 && CG == 2;      // the first wave loads K (which waits less where it has a SIMD for itself)
    constexpr int XS = 72, XG = 16 * XS;      // X: a row of tokens per value, elements of a group
    __shared__ __align__(16) struct {
        E k[NBUF][64 * DK], q[FAR ? 2 : 1][64 * DK];
        GdrSide<E, W, NC0> side[FAR ? 2 : 1];      // A and the factors of the chunk, dO of the next
        E p[FAR ? 2 : 1][W * gdr_part<E>()];       // P of the next, with its remainder in front
        float se[FAR ? 2 : 1][64];
        float pq[CG * (4 + 2 * NK) * 256];      // P^T dO and Q^T dO of the next
        E x[CG * W * XG];                       // X of the chunk before
    } sm;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, g = lane >> 4;
    const int cg = w % CG;
    const int slices = (a.dv + NC0 - 1) / NC0;
    const int64_t id = blockIdx.x;
    int64_t item = (id >> 3) / run * 8 * run + (id & 7) * run + (id >> 3) % run;
    if (item >= (int64_t)a.B * a.Hv * slices) return;
    const int slice = item % slices;
    item /= slices;
    const int hv = item % a.Hv, hk = hv / (a.Hv / a.Hk);
    const int64_t seq = item / a.Hv;
    const GdrSeq s = gdr_seq(a, seq);
    const int dv0 = slice * NC0 + 16 * cg, col = min(dv0 + l16, a.dv - 1);
    const bool work = dv0 < a.dv;
    const int NC = __builtin_amdgcn_readfirstlane(gdr_chunks(s.T));
    if (a.dk < DK) {
        floatx4* z = reinterpret_cast<floatx4*>(&sm);
        for (int i = tid; i < (int)((NBUF + (FAR ? 2 : 1)) * 64 * DK * sizeof(E) / 16); i += 2 * NT) z[i] = floatx4{0.f, 0.f, 0.f, 0.f};
        __syncthreads();
    }
    const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
    const char* rec0 = (const char*)a.rec + ((int64_t)s.slot0 * a.Hv + hv) * gdr_rec_bytes<E>();
    const int64_t recs = a.Hv * gdr_rec_bytes<E>();
    const int ltid = tid % NT;
    const E* kb = (const E*)a.k + s.b * a.ks[0] + (int64_t)s.row0 * a.ks[1] + hk * a.ks[2];
    const E* qb = (const E*)a.q + s.b * a.qs[0] + (int64_t)s.row0 * a.qs[1] + hk * a.qs[2];
    const GdrFetch<E, DK, NT> kf(kb, a.ks[1], s.T, a.dk, ltid), qf(qb, a.qs[1], s.T, a.dk, ltid);
    float* const pq = sm.pq + cg * (4 + 2 * NK) * 256 + lane * 4;
    E* const xw = sm.x + cg * W * XG;
    // Steps: in step i the first wave has chunk n = NC - i (none in the first and
    // the last one), the second chunks n - 1 and n + 1.  Barriers as in the forward
    // pass: in the middle both have read what the other is about to write.
    auto end = [&](int n) __attribute__((always_inline)) {
        lds_barrier();
        if (NBUF == 1) {
            if (w >= CG && n >= 1) kf(sm.k[0], (n - 1) * GDR_C, cg);
            swa_landed();
        }
    };
    if (w < CG) {
        floatx4 S[2 * NK];      // dS^T, laid out as the forward's state
        const int64_t state = ((seq * a.Hv + hv) * (int64_t)a.dv + col) * a.dk + 8 * g;
        int hat[NK];
#pragma unroll
        for (int p = 0; p < NK; ++p)
            hat[p] = dv0 + l16 < a.dv && 32 * p + 8 * g < a.dk ? (col * a.dk + 32 * p + 8 * g) * (int)sizeof(E) : GDR_NONE;
#pragma unroll
        for (int x = 0; x < 2 * NK; ++x) {
            S[x] = zero;
            if (a.dST && 32 * (x / 2) + 8 * g < a.dk) S[x] = *reinterpret_cast<const floatx4*>(a.dST + state + 32 * (x / 2) + 4 * (x & 1));
        }
        auto chunk = [&](int i, int buf) __attribute__((always_inline)) {
            const int n = NC - i;
            if (!work || i == 0 || n < 0) {
                lds_barrier();
                if (KFIRST && n >= 1) kf(sm.k[buf ^ (NBUF - 1)], (n - 1) * GDR_C, cg);
                if (KFIRST) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                return end(n);
            }
            const E* kt = sm.k[buf];
            const GdrSide<E, W, NC0>& sd = sm.side[FAR ? buf : 0];
            auto factor = [&](int f, int t) { return *reinterpret_cast<const floatx4*>(sd.vec + 64 * f + 16 * t + 4 * g); };
            Frag sh[NK], sl[NK], x[4], A[6], A2[6], f[2], f2[2], f3[2], kc[2 * NK];
            floatx4 U[4], X[4], bb[4], bc[4], po[4], qo[2 * NK];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                x[t] = T::template ld_row<DK>(kt, 16 * t + l16, 0, g);
                U[t] = X[t] = zero;
            }
#pragma unroll
            for (int p = 0; p < NK; ++p) {
                sh[p] = T::pack(S[2 * p], S[2 * p + 1]);
                sl[p] = T::rest(S[2 * p], S[2 * p + 1], sh[p]);
            }
#pragma unroll
            for (int p = 0; p < NK; ++p) {
                Frag y[4];      // the next ones
                if (p + 1 < NK) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) y[t] = T::template ld_row<DK>(kt, 16 * t + l16, p + 1, g);
                } else {
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        bb[t] = factor(1, t);
                        bc[t] = factor(2, t);
                        po[t] = *reinterpret_cast<const floatx4*>(pq + t * 256);
                    }
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) U[t] = T::mma(x[t], sh[p], U[t]);
                if (T::TWO) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) U[t] = T::mma(x[t], sl[p], U[t]);
                }
                if (p + 1 < NK) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) x[t] = y[t];
                }
            }
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int j = t / 2; j < 2; ++j) {
                    A[gdr_block_t(t, j)] = T::ld_at(sd.rec, t, j, lane);
                    if (T::TWO) A2[gdr_block_t(t, j)] = T::ld_at(sd.rec + (W - 1) * gdr_part<E>(), t, j, lane);
                }
#pragma unroll
            for (int y = 0; y < 2 * NK; ++y) qo[y] = *reinterpret_cast<const floatx4*>(pq + (4 + y) * 256);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) U[t][r] = fmaf(U[t][r], bc[t][r], po[t][r]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                f[j] = T::pack(U[2 * j], U[2 * j + 1]);
                f2[j] = T::rest(U[2 * j], U[2 * j + 1], f[j]);
                f3[j] = T::rest(U[2 * j], U[2 * j + 1], f[j], f2[j]);
            }
            const float eC = sd.vec[256];
            lds_barrier();
            if (KFIRST && n >= 1) kf(sm.k[buf ^ (NBUF - 1)], (n - 1) * GDR_C, cg);
#pragma unroll
            for (int y = 0; y < 2 * NK; ++y) kc[y] = T::template ld_col8<DK>(kt, 0, 32 * (y / 2) + 4 * (y & 1), lane);
#pragma unroll
            for (int j = 1; j >= 0; --j) {
#pragma unroll
                for (int t = 0; t < 2 + 2 * j; ++t) X[t] = T::mma(A[gdr_block_t(t, j)], f[j], X[t]);
                if (T::TWO) {
#pragma unroll
                    for (int t = 0; t < 2 + 2 * j; ++t) X[t] = T::mma(A[gdr_block_t(t, j)], f2[j], X[t]);
#pragma unroll
                    for (int t = 0; t < 2 + 2 * j; ++t) X[t] = T::mma(A2[gdr_block_t(t, j)], f[j], X[t]);
#pragma unroll
                    for (int t = 0; t < 2 + 2 * j; ++t) X[t] = T::mma(A[gdr_block_t(t, j)], f3[j], X[t]);
                }
            }
            const auto ds = gdr_buffer((const E*)a.ds + ((int64_t)(s.slot0 + n) * a.Hv + hv) * a.dv * a.dk, (int64_t)a.dv * a.dk * (int)sizeof(E));
#pragma unroll
            for (int p = 0; p < NK; ++p) gdr_store(ds, hat[p], sh[p]);
#pragma unroll
            for (int y = 0; y < 2 * NK; ++y)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[y][r] = fmaf(eC, S[y][r], qo[y][r]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const Frag h = T::pack(X[2 * j], X[2 * j + 1]);
                E* to = xw + l16 * XS + 32 * j + 4 * g;
                *reinterpret_cast<E4*>(to) = __builtin_shufflevector(h, h, 0, 1, 2, 3);
                *reinterpret_cast<E4*>(to + 16) = __builtin_shufflevector(h, h, 4, 5, 6, 7);
                if (T::TWO) {
                    const Frag r = T::rest(X[2 * j], X[2 * j + 1], h);
                    *reinterpret_cast<E4*>(to + (W - 1) * XG) = __builtin_shufflevector(r, r, 0, 1, 2, 3);
                    *reinterpret_cast<E4*>(to + (W - 1) * XG + 16) = __builtin_shufflevector(r, r, 4, 5, 6, 7);
                }
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) X[t] *= -bb[t];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                f[j] = T::pack(X[2 * j], X[2 * j + 1]);
                f2[j] = T::rest(X[2 * j], X[2 * j + 1], f[j]);
                f3[j] = T::rest(X[2 * j], X[2 * j + 1], f[j], f2[j]);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int y = 0; y < 2 * NK; ++y) S[y] = T::mma(kc[y], f[j], S[y]);
                if (T::TWO) {
#pragma unroll
                    for (int y = 0; y < 2 * NK; ++y) S[y] = T::mma(kc[y], f2[j], S[y]);
#pragma unroll
                    for (int y = 0; y < 2 * NK; ++y) S[y] = T::mma(kc[y], f3[j], S[y]);
                }
                if (j == 0)
#pragma unroll
                    for (int y = 0; y < 2 * NK; ++y) kc[y] = T::template ld_col8<DK>(kt, 1, 32 * (y / 2) + 4 * (y & 1), lane);
            }
            if (KFIRST) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            end(n);
        };
        if (NC > 0) {
            swa_landed();
            for (int i = 0; i < NC + 2; i += 2) {
                chunk(i, 0);
                if (i + 1 < NC + 2) chunk(i + 1, NBUF - 1);
            }
        }
        if (a.dS0 && work && dv0 + l16 < a.dv) {
#pragma unroll
            for (int x = 0; x < 2 * NK; ++x)
                if (32 * (x / 2) + 8 * g < a.dk) *reinterpret_cast<floatx4*>(a.dS0 + state + 32 * (x / 2) + 4 * (x & 1)) = S[x];
        }
        return;
    }

    if (NC == 0) return;
    const int64_t out = ((s.b * a.T + s.row0) * a.Hv + hv) * (int64_t)a.dv;
    const int os = a.Hv * a.dv;
    // where the lane's four values of row 16 t + l16 go in X and in dV
    int xat[4], oat[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        xat[t] = dv0 + 4 * g < a.dv ? ((16 * t + l16) * a.dv + dv0 + 4 * g) * (int)sizeof(E) : GDR_NONE;
        oat[t] = dv0 + 4 * g < a.dv ? ((16 * t + l16) * os + dv0 + 4 * g) * (int)sizeof(E) : GDR_NONE;
    }
    GdrSideAhead<E, W, NC0, NT> ahead((const E*)a.dO + out + slice * NC0, os, a.dv - slice * NC0, s.T, ltid);
    constexpr int PP = W * gdr_part<E>() * (int)sizeof(E) / 16, NP = (PP + NT - 1) / NT;
    floatx4 px[NP], sx;
    auto load = [&](int n) __attribute__((always_inline)) {
        const int n1 = max(min(n - 1, NC - 1), 0), n2 = max(min(n - 2, NC - 1), 0);
        ahead.load(rec0 + n1 * recs, ltid);
        ahead.load_v(n2 * GDR_C);
        const char* r = rec0 + n2 * recs;
        const auto ps = gdr_buffer(r, PP * 16);
#pragma unroll
        for (int i = 0; i < NP; ++i) px[i] = gdr_load(ps, (i * NT + ltid) * 16);
        sx = gdr_load(gdr_buffer(r + gdr_rec_bytes<E>() - GDR_VEC * 4 + 192 * 4, 256), ltid * 16);
    };
    auto store = [&](int b) __attribute__((always_inline)) {
        ahead.store(sm.side[b], ltid);
#pragma unroll
        for (int i = 0; i < NP; ++i)
            if (i < NP - 1 || (NP - 1) * NT + ltid < PP) reinterpret_cast<floatx4*>(sm.p[b])[i * NT + ltid] = px[i];
        if (ltid < 16) reinterpret_cast<floatx4*>(sm.se[b])[ltid] = sx;
    };
    float be[4] = {0.f, 0.f, 0.f, 0.f};
    auto step = [&](int i, int buf) __attribute__((always_inline)) {
        const int n = NC - i;
        const bool before = work && n >= 1, after = work && n <= NC - 2;
        const int fb = FAR ? buf : 0;
        if (NBUF == 2 && !KFIRST && n >= 1) kf(sm.k[buf ^ (NBUF - 1)], (n - 1) * GDR_C, cg);
        if (FAR && n >= 2) qf(sm.q[FAR ? buf ^ 1 : 0], (n - 2) * GDR_C, cg);
        load(n);
        floatx4 X[4], X2[4], PO[4] = {zero, zero, zero, zero}, QO[2 * NK];
        float bn[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) bn[t] = sm.side[fb].vec[16 * t + l16];
#pragma unroll
        for (int y = 0; y < 2 * NK; ++y) QO[y] = zero;
        if (after) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                X[t] = T::template ld_t4<XS>(xw, t, lane);
                if (T::TWO) X2[t] = T::template ld_t4<XS>(xw + (W - 1) * XG, t, lane);
            }
        }
        if (FAR) lds_barrier();
        if (before) {
            floatx4 dO[4];
            Frag d[2], d2[2], d3[2];
#pragma unroll
            for (int t = 0; t < 4; ++t) dO[t] = T::template ld_acc<NC0>(sm.side[fb].v, t, 16 * cg, lane);
#pragma unroll
            for (int j = 0; j < 2; ++j) d[j] = T::pack(dO[2 * j], dO[2 * j + 1]);
#pragma unroll
            for (int j = 1; j >= 0; --j)
#pragma unroll
                for (int p = 0; p < W; ++p)
#pragma unroll
                    for (int t = 0; t < 2 + 2 * j; ++t) PO[t] = T::mma(T::ld_at(sm.p[fb] + p * gdr_part<E>(), t, j, lane), d[j], PO[t]);
#pragma unroll
            for (int t = 0; t < 4; ++t) dO[t] *= *reinterpret_cast<const floatx4*>(sm.se[fb] + 16 * t + 4 * g);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                d[j] = T::pack(dO[2 * j], dO[2 * j + 1]);
                d2[j] = T::rest(dO[2 * j], dO[2 * j + 1], d[j]);
                d3[j] = T::rest(dO[2 * j], dO[2 * j + 1], d[j], d2[j]);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int y0 = 0; y0 < 2 * NK; y0 += 4) {
                    Frag z[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) z[y] = T::template ld_col8<DK>(sm.q[fb], j, 32 * ((y0 + y) / 2) + 4 * (y & 1), lane);
#pragma unroll
                    for (int y = 0; y < 4; ++y) QO[y0 + y] = T::mma(z[y], d[j], QO[y0 + y]);
                    if (T::TWO) {
#pragma unroll
                        for (int y = 0; y < 4; ++y) QO[y0 + y] = T::mma(z[y], d2[j], QO[y0 + y]);
#pragma unroll
                        for (int y = 0; y < 4; ++y) QO[y0 + y] = T::mma(z[y], d3[j], QO[y0 + y]);
                    }
                }
        }
        if (!FAR) {
            lds_barrier();
            if (n >= 2) qf(sm.q[0], (n - 2) * GDR_C, cg);
        }
        if (before) {
#pragma unroll
            for (int t = 0; t < 4; ++t) *reinterpret_cast<floatx4*>(pq + t * 256) = PO[t];
#pragma unroll
            for (int y = 0; y < 2 * NK; ++y) *reinterpret_cast<floatx4*>(pq + (4 + y) * 256) = QO[y];
        }
        // the next chunks are here; the stores that follow need not have been written when they begin
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        store(FAR ? buf ^ 1 : 0);
        if (after) {
            const int c = n + 1;
            const int64_t x0 = ((int64_t)(s.slot0 + c) * a.Hv + hv) * GDR_C * a.dv;
            const auto xb = gdr_buffer((const E*)a.x + x0, (int64_t)GDR_C * a.dv * (int)sizeof(E));
            const auto x2b = gdr_buffer(T::TWO ? (const E*)a.x2 + x0 : nullptr, T::TWO ? (int64_t)GDR_C * a.dv * (int)sizeof(E) : 0);
            const auto vb = gdr_buffer((const E*)a.dv_ + out + (int64_t)c * GDR_C * os, ((int64_t)(min(s.T - c * GDR_C, GDR_C) - 1) * os + a.dv) * (int)sizeof(E));
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                gdr_store(xb, xat[t], X[t], (const E*)nullptr);
                if (T::TWO) {
                    gdr_store(x2b, xat[t], X2[t], (const E*)nullptr);
                    X[t] += X2[t];
                }
                gdr_store(vb, oat[t], X[t] * be[t], (const E*)nullptr);
            }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) be[t] = bn[t];
        end(n);
    };
    load(NC + 1);
    qf(sm.q[0], (NC - 1) * GDR_C, cg);
    store(0);
    swa_landed();
    for (int i = 0; i < NC + 2; i += 2) {
        step(i, 0);
        if (i + 1 < NC + 2) step(i + 1, NBUF - 1);
    }
}

// Natural-order fragments of a row-major LDS tile read by columns: K = rows 32
// j + 8 g + e, row (or column) m of the operand = column c0 + P (m / 4) + m % 4.
// (P = 8: two of them, 4 columns apart, leave a lane eight columns in a row.)
template <int D, int P = 4>
__device__ __forceinline__ bf16x8 gdr_coln(const __bf16* tile, int j, int c0, int lane) {
    typedef SwaTile<__bf16, D> TL;
    typedef __attribute__((__vector_size__(4 * sizeof(short)))) short v4s;
    const int l = lane & 15, r = 32 * j + 8 * (lane >> 4) + (l >> 2), c = c0 + P * (l & 3);
    const __bf16* lo = tile + TL::off(r, c / 8) + c % 8;
    const __bf16* hi = tile + TL::off(r + 4, c / 8) + c % 8;
    const s16x4 x = __builtin_bit_cast(s16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(lo)));
    const s16x4 y = __builtin_bit_cast(s16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(hi)));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
}
template <int D, int P = 4>
__device__ __forceinline__ floatx8 gdr_coln(const float* tile, int j, int c0, int lane) {
    typedef SwaTile<float, D> TL;
    const int l = lane & 15, c = c0 + P * (l >> 2) + (l & 3), r = 32 * j + 8 * (lane >> 4);
    floatx8 f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = tile[TL::off(r + e, c / 4) + c % 4];
    return f;
}

// R rows of D columns on their way to an LDS tile through registers, zero past
// `rows` and `cols`.
template <class E, int D, int R>
struct GdrStage {
    typedef SwaTile<E, D> TL;
    static constexpr int N = R * TL::CPR / 512;
    static_assert(R * TL::CPR % 512 == 0, "whole rounds");
    floatx4 v[N];
    __device__ __forceinline__ void load(const E* src, int64_t rs, int rows, int cols, int tid) {
        const int c = tid % TL::CPR * TL::EPC, step = 512 / TL::CPR * (int)rs * (int)sizeof(E);
        const int at = c < cols ? (tid / TL::CPR * (int)rs + c) * (int)sizeof(E) : GDR_NONE;
        const auto buf = gdr_buffer(src, rows > 0 ? ((rows - 1) * rs + cols) * (int)sizeof(E) : 0);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = gdr_load(buf, at == GDR_NONE ? at : at + i * step);
    }
    __device__ __forceinline__ void store(E* tile, int tid) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = i * 512 + tid;
            *reinterpret_cast<floatx4*>(tile + TL::off(at / TL::CPR, at % TL::CPR)) = v[i];
        }
    }
    // in place of what the tile holds; the sum of both products
    __device__ __forceinline__ float replace(E* tile, int tid) const {
        typedef E EV __attribute__((ext_vector_type(TL::EPC)));
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = i * 512 + tid;
            EV* to = reinterpret_cast<EV*>(tile + TL::off(at / TL::CPR, at % TL::CPR));
            const EV x = __builtin_bit_cast(EV, v[i]), y = *to;
#pragma unroll
            for (int e = 0; e < TL::EPC; ++e) s = fmaf((float)x[e], (float)y[e], s);
            *to = x;
        }
        return s;
    }
};

template <class E, int DK, int DV>
struct GdrGradLds {
    static constexpr bool TWO = GdrT<E>::TWO;
    static constexpr int A = (TWO ? 2 : 1) * GDR_BLOCKS * 512;      // elements of A with its remainder
    union {      // A is done with when U is made
        E u2[TWO ? 64 * DV : 8], a[A];
    };
    E u[64 * DV], s[DV * DK];      // (loads straight to LDS reach this far)
    E k[64 * DK], q[64 * DK], x[64 * DV], x2[TWO ? 64 * DV : 8];
    union {      // dO is done with when E and F are made
        E d[64 * DV];
        struct {
            E e[64 * 64], f[64 * 64];
        };
    };
    float vec[GDR_VEC];
    float rows[4][64], cols[4][64];      // of the two matrices that enter db
    float xu[64], brow[4][64], xw[8][64];
    float dot[4][64], send[4][64];
    float ss[8];
};

// Gradients of a chunk's q, k, g and beta: eight waves per chunk and key head,
// the value heads of the group one after the other, values in blocks of DV.
// bf16: X and U with their remainders, S0, dS, E and F rounded.  As many
// workgroups as compute units go over all chunks: what the next head or chunk
// needs loads beside the last stages of this one, to registers or (bf16: A, V
// and S0) straight to LDS, where their places are free by then.
//
// 17 us a chunk and head of 128 x 128, 133 us for the 2048 of the sequences above
// (350 MB, 2.6 TB/s): bound by its nine stages, each of which reads through LDS
// what the one before has written, and by the two tiles of the triangle that
// eight waves leave over.  With everything through registers, some of which
// were spilled: 160 us.
template <class E, int DK, int DV>
__global__ __launch_bounds__(512, 1) void kd_gdr_grad_kernel(GdrArgs a)
{
    typedef GdrT<E> T;
    typedef typename T::Frag Frag;
    typedef SwaTile<E, DK> TK;
    typedef SwaTile<E, DV> TV;
    typedef SwaTile<E, 64> TC;
    typedef E E4 __attribute__((ext_vector_type(4)));
    constexpr int NK = DK / 32, NV = DV / 32, CG = DK / 32, RT = CG / 2;      // pairs of column tiles of dq, row tiles of a wave
    constexpr bool DIRECT = T::TWO;
    __shared__ __align__(16) GdrGradLds<E, DK, DV> sm;
    const int tid = threadIdx.x, lane0 = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = a.Hv / a.Hk;
    const int items = a.slots * a.Hk;
    const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
    // this wave's tiles of dq^T and dk^T: two columns of tiles from key channel c0 on, row tiles r0 ..
    const int cg = w % CG, c0 = 32 * cg, r0 = w / CG * RT;
    floatx4 dq[2][RT], dk[2][RT];
    // its tiles (i, j), j <= i, of the 64 x 64 matrices: number w and, for the first two waves, 8 + w
    auto tile_i = [](int n) { return n < 1 ? 0 : n < 3 ? 1 : n < 6 ? 2 : 3; };
    // (lane numbers made afresh in every phase: addresses that depend on them would otherwise be kept across all)
#define KD_LANE const int lane = lane0 + opaque_zero(), l16 = lane & 15, g = lane >> 4

    // the chunk after an item, if any
    auto next = [&](int item, GdrChunk& c) {
        for (item += gridDim.x; item < items; item += gridDim.x)
            if (gdr_slot(a, item / a.Hk, c)) return item;
        return items;
    };
    GdrStage<E, DK, 64> lk, lq;
    GdrStage<E, DK, DV> ls;
    GdrStage<E, DV, 64> ld, lx, lx2, lv;
    constexpr int AP = GdrGradLds<E, DK, DV>::A * (int)sizeof(E) / 16, NA = (AP + 511) / 512;      // 16-byte pieces
    floatx4 la[NA], lf;
    // What the next head (or values, or chunk) needs, in three parts.  Without
    // rows nothing is read, but the registers are written all the same, or their
    // old values would have to be kept.
    struct Next {
        GdrChunk c;
        int hk, hv, v0, nv, kr;
        int64_t at;
    };
    auto which = [&](int item, GdrChunk c, int hg, int v0) {
        Next n;
        if (item >= items) item = c.rows = c.first = c.base = 0;
        n.c = c;
        n.hk = item % a.Hk;
        n.hv = n.hk * G + hg;
        n.v0 = v0;
        n.nv = c.rows > 0 ? min(DV, a.dv - v0) : 0;
        n.kr = hg == 0 && v0 == 0 ? c.rows : 0;
        n.at = (int64_t)(item / a.Hk) * a.Hv + n.hv;
        return n;
    };
    // A, V and S0 straight to LDS; what they do not fill is cleared
    auto direct = [&](const Next& n) __attribute__((always_inline)) {
        if (!DIRECT || n.c.rows == 0) return;
        KD_LANE;
        const int t = 64 * w + lane;
        const char* rec = (const char*)a.rec + n.at * gdr_rec_bytes<E>() + gdr_parts<E>() / 2 * gdr_part<E>() * (int)sizeof(E);
        const uint32_t to = __builtin_amdgcn_readfirstlane(1024 * w);
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (i < NA - 1 || i * 512 + t < AP) load_lds16(lds_address(sm.a) + to + i * 8192, rec + (i * 512 + t) * 16);
        const E* v = (const E*)a.v + n.c.base * a.vs[0] + (int64_t)n.c.first * a.vs[1] + n.hv * a.vs[2] + n.v0;
        const E* s = (const E*)a.hs + (n.at * a.dv + n.v0) * a.dk;
        const floatx4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 64 * TV::CPR / 512; ++i) {
            const int r = (i * 512 + t) / TV::CPR, c = ((i * 512 + t) % TV::CPR ^ TV::swz(r)) * TV::EPC;
            if (r < n.c.rows && c < n.nv) load_lds16(lds_address(sm.u) + to + i * 8192, v + r * a.vs[1] + c);
            else reinterpret_cast<floatx4*>(sm.u)[i * 512 + t] = z;
        }
#pragma unroll
        for (int i = 0; i < DV * TK::CPR / 512; ++i) {
            const int r = (i * 512 + t) / TK::CPR, c = ((i * 512 + t) % TK::CPR ^ TK::swz(r)) * TK::EPC;
            if (r < n.nv && c < a.dk) load_lds16(lds_address(sm.s) + to + i * 8192, s + r * a.dk + c);
            else reinterpret_cast<floatx4*>(sm.s)[i * 512 + t] = z;
        }
    };
    auto load1 = [&](const Next& n) {
        if (!DIRECT) ls.load((const E*)a.hs + (n.at * a.dv + n.v0) * a.dk, a.dk, n.nv, a.dk, tid);
        lx.load((const E*)a.x + n.at * GDR_C * a.dv + n.v0, a.dv, n.c.rows, n.nv, tid);
    };
    auto load2 = [&](const Next& n) {
        if (T::TWO) lx2.load((const E*)a.x2 + n.at * GDR_C * a.dv + n.v0, a.dv, n.c.rows, n.nv, tid);
        ld.load((const E*)a.dO + ((n.c.base * a.T + n.c.first) * a.Hv + n.hv) * (int64_t)a.dv + n.v0, (int64_t)a.Hv * a.dv, n.c.rows, n.nv, tid);
        if (!DIRECT) lv.load((const E*)a.v + n.c.base * a.vs[0] + (int64_t)n.c.first * a.vs[1] + n.hv * a.vs[2] + n.v0, a.vs[1], n.c.rows, n.nv, tid);
    };
    auto load3 = [&](const Next& n) {
        lk.load((const E*)a.k + n.c.base * a.ks[0] + (int64_t)n.c.first * a.ks[1] + n.hk * a.ks[2], a.ks[1], n.kr, a.dk, tid);
        lq.load((const E*)a.q + n.c.base * a.qs[0] + (int64_t)n.c.first * a.qs[1] + n.hk * a.qs[2], a.qs[1], n.kr, a.dk, tid);
        const char* record = (const char*)a.rec + n.at * gdr_rec_bytes<E>();
        const auto rec = gdr_buffer(record + gdr_parts<E>() / 2 * gdr_part<E>() * (int)sizeof(E), n.c.rows > 0 ? AP * 16 : 0);      // (A)
        if (!DIRECT)
#pragma unroll
            for (int i = 0; i < NA; ++i) la[i] = gdr_load(rec, (i * 512 + tid) * 16);
        lf = gdr_load(gdr_buffer(record + gdr_rec_bytes<E>() - GDR_VEC * 4, n.c.rows > 0 ? GDR_VEC * 4 : 0), tid * 16);
    };
    GdrChunk c, cn;
    int item = next((int)blockIdx.x - (int)gridDim.x, c), itemn;
    {
        const Next n = which(item, c, 0, 0);
        direct(n);
        load1(n);
        load2(n);
        load3(n);
    }

#pragma unroll 1
    for (; item < items; item = itemn, c = cn) {
        itemn = next(item, cn);
        const int hk = item % a.Hk, slot = item / a.Hk;
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int t = 0; t < RT; ++t) dq[y][t] = dk[y][t] = zero;
#pragma unroll 1
    for (int hg = 0; hg < G; ++hg) {
        const int hv = hk * G + hg;
        const int64_t at = (int64_t)slot * a.Hv + hv;
        floatx4 dP[2], dT[2];
        dP[0] = dP[1] = dT[0] = dT[1] = zero;
        float ss = 0.f, xs[RT], ys[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) xs[t] = ys[t] = 0.f;
#pragma unroll 1
        for (int v0 = 0; v0 < a.dv; v0 += DV) {
            GdrStage<E, DK, DV> st;
            lds_barrier();      // the head (or the values) before is done
            if (v0 == 0) {
                if (tid < GDR_VEC / 4) reinterpret_cast<floatx4*>(sm.vec)[tid] = lf;
                if (hg == 0) {
                    lk.store(sm.k, tid);
                    lq.store(sm.q, tid);
                }
            }
            ld.store(sm.d, tid);
            lx.store(sm.x, tid);
            if (T::TWO) lx2.store(sm.x2, tid);
            if (!DIRECT) {
                ls.store(sm.s, tid);
#pragma unroll
                for (int i = 0; i < NA; ++i)
                    if (i < NA - 1 || (NA - 1) * 512 + tid < AP) reinterpret_cast<floatx4*>(sm.a)[i * 512 + tid] = la[i];
                lv.store(sm.u, tid);      // (V where U will be: a wave reads and writes the same columns)
            }
            if (DIRECT) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            lds_barrier();
            st.load((const E*)a.ds + (at * a.dv + v0) * a.dk, a.dk, min(DV, a.dv - v0), a.dk, tid);
            const bool same = v0 + DV < a.dv || hg + 1 < G;
            const Next nx = which(same ? item : itemn, same ? c : cn, v0 + DV < a.dv ? hg : same ? hg + 1 : 0, v0 + DV < a.dv ? v0 + DV : 0);
            // dbeta_r = X_r.U_r / beta_r; where a beta is 0 (or next to it), from W instead
            const bool small = sm.vec[257] != 0.f;
            // W and U: 16 values a wave
            floatx4 W[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) W[t] = zero;
            if (w < DV / 16) {
                KD_LANE;
                const int col = 16 * w + l16;
#pragma unroll
                for (int p = 0; p < NK; ++p) {
                    const Frag s = T::template ld_row<DK>(sm.s, col, p, g);
#pragma unroll
                    for (int t = 0; t < 4; ++t) W[t] = T::mma(T::template ld_row<DK>(sm.k, 16 * t + l16, p, g), s, W[t]);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const floatx4 be = *reinterpret_cast<const floatx4*>(sm.vec + 16 * t + 4 * g);
                    const floatx4 bb = *reinterpret_cast<const floatx4*>(sm.vec + 64 + 16 * t + 4 * g);
                    const floatx4 v = T::template ld_acc<DV>(sm.u, t, 16 * w, lane);
                    if (small) {
                        const floatx4 b = *reinterpret_cast<const floatx4*>(sm.vec + 320 + 16 * t + 4 * g);
                        floatx4 x = T::template ld_acc<DV>(sm.x, t, 16 * w, lane);
                        if (T::TWO) x += T::template ld_acc<DV>(sm.x2, t, 16 * w, lane);
#pragma unroll
                        for (int r = 0; r < 4; ++r) x[r] = row16_sum(x[r] * (v[r] - __builtin_amdgcn_exp2f(b[r]) * W[t][r]));
                        if (l16 == 0) {
                            floatx4* to = reinterpret_cast<floatx4*>(sm.xw[w] + 16 * t + 4 * g);
                            *to = v0 == 0 ? x : *to + x;
                        }
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) W[t][r] = be[r] * v[r] - bb[r] * W[t][r];
                }
                Frag f[2], f2[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    f[j] = T::pack(W[2 * j], W[2 * j + 1]);
                    f2[j] = T::rest(W[2 * j], W[2 * j + 1], f[j]);
                    W[2 * j] = W[2 * j + 1] = zero;
                }
                const E* rec = sm.a + lane * 8;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int t = 2 * j; t < 4; ++t) {
                        const Frag A = T::ld(rec + gdr_block(t, j) * 512);
                        W[t] = gdr_mma2<E>(f[j], f2[j], A, W[t]);
                        if (T::TWO) W[t] = T::mma(f[j], T::ld(rec + gdr_part<E>() + gdr_block(t, j) * 512), W[t]);
                    }
            }
            lds_barrier();
            if (w < DV / 16) {
                KD_LANE;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const floatx4 y = W[t];
                    // lane: token, four values
                    const int to = TV::off(16 * t + l16, (16 * w + 4 * g) / TV::EPC) + 4 * g % TV::EPC;
                    const E4 hi = E4{(E)y[0], (E)y[1], (E)y[2], (E)y[3]};
                    *reinterpret_cast<E4*>(sm.u + to) = hi;
                    if (T::TWO)
                        *reinterpret_cast<E4*>(sm.u2 + (T::TWO ? to : 0)) = E4{(E)(y[0] - (float)hi[0]), (E)(y[1] - (float)hi[1]),
                                                                              (E)(y[2] - (float)hi[2]), (E)(y[3] - (float)hi[3])};
                }
            }
            // scale e^b dO S0 and -beta e^b X S0, and their products with q and k
            {
                KD_LANE;
                floatx4 dqi[2][RT], dke[2][RT];
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int t = 0; t < RT; ++t) dqi[y][t] = dke[y][t] = zero;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const Frag s[2] = {gdr_coln<DK, 8>(sm.s, j, c0, lane), gdr_coln<DK, 8>(sm.s, j, c0 + 4, lane)};
#pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        const Frag d = T::template ld_row<DV>(sm.d, 16 * (r0 + t) + l16, j, g), x = T::template ld_row<DV>(sm.x, 16 * (r0 + t) + l16, j, g);
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            dqi[y][t] = T::mma(s[y], d, dqi[y][t]);
                            dke[y][t] = T::mma(s[y], x, dke[y][t]);
                        }
                        if (T::TWO) {
                            const Frag x2 = T::template ld_row<DV>(sm.x2, 16 * (r0 + t) + l16, j, g);
#pragma unroll
                            for (int y = 0; y < 2; ++y) dke[y][t] = T::mma(s[y], x2, dke[y][t]);
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const int row = 16 * (r0 + t) + l16;
                    const float se = sm.vec[192 + row], bb = sm.vec[64 + row];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int to = TK::off(row, (c0 + 8 * g + 4 * y) / TK::EPC) + 4 * y % TK::EPC;
                        const E4 q4 = *reinterpret_cast<const E4*>(sm.q + to), k4 = *reinterpret_cast<const E4*>(sm.k + to);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = se * dqi[y][t][e], z = -bb * dke[y][t][e];
                            dq[y][t][e] += x;
                            dk[y][t][e] += z;
                            xs[t] = fmaf((float)q4[e], x, fmaf((float)k4[e], z, xs[t]));
                        }
                    }
                }
            }
            lds_barrier();
            ss += st.replace(sm.s, tid);      // dS in place of S0
            // dO U^T and X U^T
            {
                KD_LANE;
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    const int n = w + 8 * o, i = tile_i(n), j = n - i * (i + 1) / 2;
                    if (n >= 10) break;
#pragma unroll
                    for (int p = 0; p < NV; ++p) {
                        const Frag u = T::template ld_row<DV>(sm.u, 16 * j + l16, p, g);
                        const Frag d = T::template ld_row<DV>(sm.d, 16 * i + l16, p, g), x = T::template ld_row<DV>(sm.x, 16 * i + l16, p, g);
                        dP[o] = T::mma(u, d, dP[o]);
                        dT[o] = T::mma(u, x, dT[o]);
                        if (T::TWO) {
                            const Frag u2 = T::template ld_row<DV>(sm.u2, 16 * j + l16, p, g);
                            dP[o] = T::mma(u2, d, dP[o]);
                            dT[o] = T::mma(u2, x, dT[o]);
                            dT[o] = T::mma(u, T::template ld_row<DV>(sm.x2, 16 * i + l16, p, g), dT[o]);
                        }
                    }
                }
            }
            lds_barrier();
            load1(nx);
            // e^(bC - b) U dS
            {
                KD_LANE;
                floatx4 dks[2][RT];
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int t = 0; t < RT; ++t) dks[y][t] = zero;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const Frag s[2] = {gdr_coln<DK, 8>(sm.s, j, c0, lane), gdr_coln<DK, 8>(sm.s, j, c0 + 4, lane)};
#pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        const Frag u = T::template ld_row<DV>(sm.u, 16 * (r0 + t) + l16, j, g);
#pragma unroll
                        for (int y = 0; y < 2; ++y) dks[y][t] = T::mma(s[y], u, dks[y][t]);
                        if (T::TWO) {
                            const Frag u2 = T::template ld_row<DV>(sm.u2, 16 * (r0 + t) + l16, j, g);
#pragma unroll
                            for (int y = 0; y < 2; ++y) dks[y][t] = T::mma(s[y], u2, dks[y][t]);
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const int row = 16 * (r0 + t) + l16;
                    const float ec = sm.vec[128 + row];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const E4 k4 = *reinterpret_cast<const E4*>(sm.k + TK::off(row, (c0 + 8 * g + 4 * y) / TK::EPC) + 4 * y % TK::EPC);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = ec * dks[y][t][e];
                            dk[y][t][e] += x;
                            ys[t] = fmaf((float)k4[e], x, ys[t]);
                        }
                    }
                }
            }
            load2(nx);
            if (v0 + DV < a.dv) {
                if (DIRECT) lds_barrier();      // U and dS are done with
                direct(nx);
                load3(nx);
            }
        }
        const bool small = sm.vec[257] != 0.f;
        {
            KD_LANE;
            // E, F and their sums; lane: token r of block i, s = 16 j + 4 g + e
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                const int n = w + 8 * o, i = tile_i(n), j = n - i * (i + 1) / 2;
                if (n >= 10) break;
                floatx4 kk = zero, qk = zero;
#pragma unroll
                for (int p = 0; p < NK; ++p) {
                    const Frag s = T::template ld_row<DK>(sm.k, 16 * j + l16, p, g);
                    kk = T::mma(s, T::template ld_row<DK>(sm.k, 16 * i + l16, p, g), kk);
                    qk = T::mma(s, T::template ld_row<DK>(sm.q, 16 * i + l16, p, g), qk);
                }
                const int r = 16 * i + l16;
                const float *bh = sm.vec + 320, *bl = sm.vec + 384;
                const floatx4 sh = *reinterpret_cast<const floatx4*>(bh + 16 * j + 4 * g), sl = *reinterpret_cast<const floatx4*>(bl + 16 * j + 4 * g);
                const float rh = bh[r], rl = bl[r], br = sm.vec[r];
                float row = 0.f, brow = 0.f;
                floatx4 colsum;
                E4 e4, f4;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int s = 16 * j + 4 * g + e;
                    const float gam = s <= r ? __builtin_amdgcn_exp2f((rh - sh[e]) + (rl - sl[e])) : 0.f;
                    const float x = a.scale * gam * dP[o][e], y = s < r ? -gam * dT[o][e] : 0.f;
                    const float m = x * qk[e] + br * y * kk[e];
                    e4[e] = (E)x;
                    f4[e] = (E)(br * y);
                    row += m;
                    brow = fmaf(y, kk[e], brow);
                    colsum[e] = m;
                    if (s == r) sm.xu[r] = dT[o][e];
                    // F + F^T (the diagonal is 0)
                    if (s <= r) sm.f[TC::off(s, r / TC::EPC) + r % TC::EPC] = f4[e];
                }
                const int to = (16 * j + 4 * g) / TC::EPC, rest = 4 * g % TC::EPC;
                *reinterpret_cast<E4*>(sm.e + TC::off(r, to) + rest) = e4;
                if (i > j) {
                    *reinterpret_cast<E4*>(sm.f + TC::off(r, to) + rest) = f4;
                    *reinterpret_cast<E4*>(sm.e + TC::off(16 * j + l16, (16 * i + 4 * g) / TC::EPC) + rest) = E4{(E)0.f, (E)0.f, (E)0.f, (E)0.f};
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (16 * j + 4 * g + e < r) sm.f[TC::off(r, to) + rest + e] = f4[e];
                }
                row += __shfl_xor(row, 16);
                row += __shfl_xor(row, 32);
                if (small) {
                    brow += __shfl_xor(brow, 16);
                    brow += __shfl_xor(brow, 32);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) colsum[e] = row16_sum(colsum[e]);
                if (g == 0) {
                    sm.rows[j][r] = row;
                    sm.brow[j][r] = brow;
                }
                if (l16 == 0) *reinterpret_cast<floatx4*>(sm.cols[i] + 16 * j + 4 * g) = colsum;
            }
            ss = wave_sum(ss);
            if (lane == 0) sm.ss[w] = ss;
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                float x = xs[t] - ys[t], y = ys[t];
                x += __shfl_xor(x, 16);
                x += __shfl_xor(x, 32);
                y += __shfl_xor(y, 16);
                y += __shfl_xor(y, 32);
                if (g == 0) {
                    sm.dot[cg][16 * (r0 + t) + l16] = x;
                    sm.send[cg][16 * (r0 + t) + l16] = y;
                }
            }
        }
        lds_barrier();
        {
            KD_LANE;
            // E K, E^T Q and (F + F^T) K
            {
                const bool same = hg + 1 < G;
                const Next nx = which(same ? item : itemn, same ? c : cn, same ? hg + 1 : 0, 0);
                direct(nx);
                load3(nx);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                Frag k[2], q[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    k[y] = gdr_coln<DK, 8>(sm.k, j, c0 + 4 * y, lane);
                    q[y] = gdr_coln<DK, 8>(sm.q, j, c0 + 4 * y, lane);
                }
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const Frag e = T::template ld_row<64>(sm.e, 16 * (r0 + t) + l16, j, g), f = T::template ld_row<64>(sm.f, 16 * (r0 + t) + l16, j, g);
                    const Frag ec = gdr_coln<64>(sm.e, j, 16 * (r0 + t), lane);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        dq[y][t] = T::mma(k[y], e, dq[y][t]);
                        dk[y][t] = T::mma(k[y], f, dk[y][t]);
                        dk[y][t] = T::mma(q[y], ec, dk[y][t]);
                    }
                }
            }
            if (w == 7) {
                // lane: token
                const int b = lane >> 4;
                float db = 0.f, y = 0.f, dbeta = 0.f, send = 0.f;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float p = sm.rows[x][lane], m = sm.cols[x][lane];
                    db += (x <= b ? p : 0.f) - (x >= b ? m : 0.f);
                }
#pragma unroll
                for (int x = 0; x < CG; ++x) {
                    db += sm.dot[x][lane];
                    send += sm.send[x][lane];
                }
#pragma unroll
                for (int x = 0; x < 8; ++x) y += sm.ss[x];
                if (small) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) dbeta += x <= b ? sm.brow[x][lane] : 0.f;
#pragma unroll
                    for (int x = 0; x < DV / 16; ++x) dbeta += sm.xw[x][lane];
                } else {
                    dbeta = sm.xu[lane] / sm.vec[lane];
                }
                // from the chunk's end, with what e^bC multiplies
                send = wave_sum(send);
#pragma unroll
                for (int x = 1; x < 64; x *= 2) {
                    const float z = __shfl_down(db, x);
                    if (lane + x < 64) db += z;
                }
                db += send + sm.vec[256] * y;
                if (lane < c.rows) {
                    const int64_t gate = (c.base * a.T + c.first + lane) * a.Hv + hv;
                    if (a.gates32) {
                        ((float*)a.dg)[gate] = db;
                        ((float*)a.dbeta)[gate] = dbeta;
                    } else {
                        ((E*)a.dg)[gate] = (E)db;
                        ((E*)a.dbeta)[gate] = (E)dbeta;
                    }
                }
            }
        }
    }
    KD_LANE;
#undef KD_LANE
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int row = 16 * (r0 + t) + l16;
        if (row >= c.rows || c0 + 8 * g >= a.dk) continue;
        const int64_t to = ((c.base * a.T + c.first + row) * a.Hk + hk) * (int64_t)a.dk + c0 + 8 * g;
        T::st((E*)a.dq + to, T::pack(dq[0][t], dq[1][t]));
        T::st((E*)a.dk_ + to, T::pack(dk[0][t], dk[1][t]));
    }
    }
}

template <class E, int DK, int CG>
static void gdr_back(const GdrArgs& a, hipStream_t st)
{
    int run;
    const int64_t grid = gdr_pass_grid((int64_t)a.B * a.Hv * ((a.dv + 16 * CG - 1) / (16 * CG)), run);
    kd_gdr_back_kernel<E, DK, CG><<<(unsigned)grid, 128 * CG, 0, st>>>(a, run);
}

template <class E, int DK, int DV>
static hipError_t gdr_bwd(const GdrArgs& a, hipStream_t st)
{
    if constexpr (sizeof(E) == 2) {
        if (gdr_narrow(a, a.B)) gdr_back<E, DK, 2>(a, st);
        else gdr_back<E, DK, 4>(a, st);
    } else {
        gdr_back<E, DK, 2>(a, st);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.slots == 0) return e;
    const int items = a.slots * a.Hk;
    kd_gdr_grad_kernel<E, DK, DV><<<(unsigned)(items < 256 ? items : 256), 512, 0, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_gdr_bwd(int bf16, const GdrArgs& a, hipStream_t st)
{
    if (bf16) {
        if (a.dk <= 64) return a.dv <= 64 ? gdr_bwd<__bf16, 64, 64>(a, st) : gdr_bwd<__bf16, 64, 128>(a, st);
        return a.dv <= 64 ? gdr_bwd<__bf16, 128, 64>(a, st) : gdr_bwd<__bf16, 128, 128>(a, st);
    }
    return a.dk <= 64 ? gdr_bwd<float, 64, 32>(a, st) : gdr_bwd<float, 128, 32>(a, st);
}

}  // namespace kd
