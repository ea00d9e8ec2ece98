// kd_swa_decode.hip -- one decoding step of sliding-window attention with sinks
// over a rolling cache, gfx950.
//
// The cache of a sequence has `cap` slots: position s lives in slot s for
// s < S (the sinks) and in slot S + (s - S) mod (cap - S) otherwise, with
// cap >= S + W, so the keys a token at position p sees (the sinks and
// p - W + 1 .. p) are always there, however long the sequence has grown.
// The step at position p = lens[b]:
//   q, k turned to position p (when frequencies are given), k rounded to the
//   cache's type; k, v stored in p's slot; o = softmax(scale q K) V.
// The slot of p held position p - (cap - S) <= p - W, which p does not see:
// workgroups that read the cache while one of them stores the new row never
// touch that slot, and all take the new row from the inputs.
#include "kd_swa.h"
#include "kd_rope.h"
#include "kd_swa_decode.h"


namespace kd {

// slot of position s
__device__ __forceinline__ int64_t cache_slot(int s, int S, int cap) { return s < S ? s : S + (s - S) % (cap - S); }

// a pair of floats to and from the memory that every compute unit sees
__device__ __forceinline__ void swa_put(float* p, float x, float y) {
    __hip_atomic_store((unsigned long long*)p, ((unsigned long long)__float_as_uint(y) << 32) | __float_as_uint(x),
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 swa_get(const float* p) {
    const unsigned long long v = __hip_atomic_load((const unsigned long long*)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return make_float2(__uint_as_float((unsigned)v), __uint_as_float((unsigned)(v >> 32)));
}

// What a query head of one position still needs: keys seen before the new one
// are numbered 0 .. nv - 1, the sinks 0 .. ns - 1 first, then the window's.
struct Seen {
    int ns, nv, first;     // first: slot of the window's first key
};
__device__ __forceinline__ Seen swa_seen(int pos, int W, int S, int cap) {
    const int p0 = max(0, pos - W + 1);
    Seen s;
    s.ns = min(S, p0);
    s.nv = s.ns + pos - p0;
    s.first = (int)cache_slot(p0, S, cap);
    return s;
}
__device__ __forceinline__ int swa_slot(const Seen& s, int j, int S, int cap) {
    if (j < s.ns) return j;
    const int x = s.first + (j - s.ns);
    // positions below S are slots themselves, the others wrap within cap - S (once: W <= cap - S)
    return x < cap ? x : x - (cap - S);
}

// A split's maxima, sums and o in plain fp32 (rare, see its call), head by
// head, 128 keys j0 .. j1 - 1 at a time: a thread makes the score of one key,
// then sums one element over all of them.  The results go where the first
// wave's were, the second's become those of no keys.  Every thread calls it.
template <class E, int D, class Q>
__device__ __forceinline__ void swa_decode_plain(const SwaDecodeArgs& a, const Seen& se, int j0, int j1, int nh, const E* kc,
                                                 const E* vc, Q&& q, float* accs, float (*ms)[32], float (*ls)[32],
                                                 float* sc, int tid)
{
    float* const qh = accs + 32 * D;
#pragma unroll 1
    for (int h = 0; h < nh; ++h) {
        __syncthreads();
        if (tid < D) qh[tid] = q(h, tid);
        float m = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll 1
        for (int j = j0; j < j1; j += 128) {
            const int n = min(128, j1 - j);
            __syncthreads();
            if (tid < n) {
                const E* k = kc + swa_slot(se, j + tid, a.S, a.cap) * a.kcs[1];
                float s = 0.f;
#pragma unroll 4
                for (int i = 0; i < D; ++i) s = fmaf(qh[i], (float)k[i], s);
                sc[tid] = s;
            }
            __syncthreads();
            float mx = m;
#pragma unroll 1
            for (int x = 0; x < n; ++x) mx = fmaxf(mx, sc[x]);
            const float mu = mx == -INFINITY ? 0.f : mx, f = __builtin_amdgcn_exp2f(m - mu);
            m = mx;
            l *= f;
            o = o == 0.f ? 0.f : o * f;
#pragma unroll 8
            for (int x = 0; x < n; ++x) {
                const float p = __builtin_amdgcn_exp2f(sc[x] - mu);
                l += p;
                if (tid < D) o = fmaf(p, (float)vc[swa_slot(se, j + x, a.S, a.cap) * a.vcs[1] + tid], o);
            }
        }
        if (tid < D) accs[h * D + tid] = o;
        if (tid == 0) ms[0][h] = m, ls[0][h] = l, ms[1][h] = -INFINITY, ls[1][h] = 0.f;
    }
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < 32 * D; i += 128) qh[i] = 0.f;
    __syncthreads();
}

template <class E, int D, int N>
__device__ __forceinline__ void swa_join(const float* pb, int64_t pstep, int nsplit, int nh,
                                         const float (*mw)[SWA_DECODE_SPLITS + 1], const float* wl, E* o, int tid) {
    for (int i = tid; i < nh * D / 2; i += 128) {
        const int h = 2 * i / D;
        float2 v[N];
#pragma unroll
        for (int x = 0; x < N; ++x) v[x] = swa_get(pb + min(x, nsplit - 1) * pstep + 2 * i);
        float x0 = 0.f, x1 = 0.f;
#pragma unroll
        for (int x = 0; x < N; ++x) {
            if (x >= nsplit) continue;
            const float f = mw[h][x];
            x0 = fmaf(v[x].x, f, x0);
            x1 = fmaf(v[x].y, f, x1);
        }
        o[2 * i] = (E)(x0 * wl[h]);
        o[2 * i + 1] = (E)(x1 * wl[h]);
    }
}

// Workgroup (split, key head and block of up to 32 query heads, b): two waves
// share the split's keys, 32 at a time.  The heads are the columns of the same
// products that the forward pass makes with queries, St = K Qt and Ot += Vt Pt,
// so the cache is read once for all heads of a group; each wave streams its
// own tiles straight to LDS, one tile ahead, with no barrier between.  The
// matrix units have room to spare here (the step is bound by reading the
// cache), so in bf16 the queries (turned and scaled in fp32) and the weights
// go through as a rounded part and its remainder: nothing is lost to bf16 but
// the output's rounding.
//
// Bound by reading the caches: 32 sequences of up to 2052 keys, 4 key heads of
// 128, bf16 (119 MB): 34 us, 3.5 TB/s (row by row on vector units: 62 us).  One
// sequence of 1500: 14.4 us, a chain of dependent reads (length, keys, partial
// results, join).  32 keys a tile: the matrix tile's edge, and 64 KB of LDS for
// two waves with a tile ahead.
template <class E, int D>
__global__ __launch_bounds__(128, 1) void kd_swa_decode_kernel(SwaDecodeArgs a)
{
    typedef SwaT<E> T;
    typedef typename T::Frag Frag;
    typedef SwaTile<E, D> TL;
    constexpr int NK = D / T::KC, ND = D / 32, NP = 16 / T::PR;
    constexpr int ST = D * sizeof(E) > 256 ? 1 : 2;              // tiles of a wave in LDS
    constexpr int NI = 32 * TL::CPR / 64;                        // loads of one K or V tile
    constexpr bool TWO = sizeof(E) == 2;
    // K and V tiles of both waves (loads to LDS take destinations in the first 64 KB);
    // the queries pass through the second tiles' room before those are fetched
    __shared__ __align__(16) struct {
        E kv[ST][2][2][32 * D];
        float qx[ST == 2 ? 4 : 64 * D];
        float kr[D], kn[D], vn[D];      // the new key as given and as the cache holds it, the new value
        float2 cs[D / 2];
        float ms[3][32], ls[3][32], mw[32][SWA_DECODE_SPLITS + 1], wl[32];
        int last, again;
    } sm;
    auto& kv = sm.kv;
    auto& cs = sm.cs;
    float(*const ms)[32] = sm.ms;
    float(*const ls)[32] = sm.ls;
    float(*const mw)[SWA_DECODE_SPLITS + 1] = sm.mw;
    float *const kr = sm.kr, *const kn = sm.kn, *const vn = sm.vn, *const wl = sm.wl;
    int& last = sm.last;
    float* const qs = ST == 2 ? reinterpret_cast<float*>(kv[ST - 1]) : sm.qx;      // [32][D]
    float* const raw = qs + 32 * D;                                                // the queries as given
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 5;
    const int G = a.Hq / a.Hkv, nhb = (G + 31) / 32;
    const int sp = blockIdx.x, hk = blockIdx.y / nhb, hb = blockIdx.y % nhb, b = blockIdx.z;
    const int h0 = hk * G + hb * 32, nh = min(32, G - hb * 32);
    // everything that does not depend on the position loads while it does
    const E* qrow = (const E*)a.q + b * a.qb + (int64_t)h0 * D;
    const E* krow = (const E*)a.k + b * a.kb + (int64_t)hk * D;
    const E* vrow = (const E*)a.v + b * a.vb + (int64_t)hk * D;
    const int n = a.rot / 2;
    const double fr = tid < n ? a.freqs[tid] : 0.0;      // (n <= 64)
    const int pos = a.lens[b];
    for (int i = tid; i < nh * D; i += 128) raw[i] = (float)qrow[i];
    if (sp == 0)
        for (int i = tid; i < D; i += 128) {
            kr[i] = (float)krow[i];
            vn[i] = (float)vrow[i];
        }
    E* o = (E*)a.o + ((int64_t)b * a.Hq + h0) * D;
    if (pos < 0) {     // an unused row: nothing is stored, its output is zero
        if (sp == 0)
            for (int i = tid; i < nh * D; i += 128) o[i] = (E)0.f;
        return;
    }
    const Seen se = swa_seen(pos, a.W, a.S, a.cap);
    E* kc = (E*)a.kc + b * a.kcs[0] + hk * a.kcs[2];
    E* vc = (E*)a.vc + b * a.vcs[0] + hk * a.vcs[2];
    // this split's tiles of 32 keys; the wave takes every second one
    const int tiles = (se.nv + 31) / 32, per = (tiles + a.nsplit - 1) / a.nsplit;
    const int ta = min(sp * per, tiles), tb = min(ta + per, tiles);
    auto fetch = [&](int t, int st) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int at = i * 64 + lane, r = at / TL::CPR, ch = (at % TL::CPR) ^ TL::swz(r);
            // (numbers past the last key read it again; they are masked)
            const int64_t slot = swa_slot(se, min(t * 32 + r, se.nv - 1), a.S, a.cap);
            const E* ks = kc + slot * a.kcs[1] + ch * TL::EPC;
            const E* vs = vc + slot * a.vcs[1] + ch * TL::EPC;
            const uint32_t kd = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)kv[st][w][0] + 1024 * i;
            const uint32_t vd = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)kv[st][w][1] + 1024 * i;
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off\n\t"
                         "s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %3, off" ::"s"(kd),
                         "v"(ks), "s"(vd), "v"(vs)
                         : "memory", "m0");
        }
    };
    int t = ta + w;
    if (t < tb) fetch(t, 0);

    // queries (turned, times scale log2 e), and where they are needed the new key and value
    if (tid < n) cs[tid] = rope_cs((double)pos, fr, a.rope_scale, 0);
    if (tid == 0) sm.again = 0;
    __syncthreads();
    auto turned = [&](const auto* row, int i) -> float {
        const float x = (float)row[i];
        if (i >= a.rot) return x;
        const int j = a.interleaved ? i / 2 : i < n ? i : i - n;
        const bool second = a.interleaved ? (i & 1) : i >= n;
        const float y = (float)row[a.interleaved ? i ^ 1 : second ? i - n : i + n];
        return second ? fmaf(x, cs[j].x, y * cs[j].y) : fmaf(x, cs[j].x, -y * cs[j].y);
    };
    for (int i = tid; i < nh * D; i += 128) qs[i] = turned(raw + i / D * D, i % D) * a.c;
    if (sp == 0 && tid < D) {
        const E kx = (E)turned(kr, tid);
        kn[tid] = (float)kx;
        if (hb == 0) {
            const int64_t slot = cache_slot(pos, a.S, a.cap);
            kc[slot * a.kcs[1] + tid] = kx;
            vc[slot * a.vcs[1] + tid] = (E)vn[tid];
        }
    }
    __syncthreads();
    Frag q[NK], ql[TWO ? NK : 1];
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
        const float* src = qs + (lane & 31) * D + (2 * ks + g) * TL::EPC;
#pragma unroll
        for (int e = 0; e < TL::EPC; ++e) {
            const float x = (lane & 31) < nh ? src[e] : 0.f;
            q[ks][e] = (E)x;
            if (TWO) ql[TWO ? ks : 0][e] = (E)(x - (float)q[ks][e]);
        }
    }
    // the new token's score (four lanes a head)
    if (sp == 0) {
        const int h = tid / 4;
        float s = 0.f;
        if (h < nh)
            for (int i = tid % 4; i < D; i += 4) s = fmaf(qs[h * D + i], kn[i], s);
        s += __shfl_xor(s, 1);
        s += __shfl_xor(s, 2);
        if (tid % 4 == 0) {
            ms[2][h] = h < nh ? s : -INFINITY;
            ls[2][h] = 1.f;
        }
    }
    __syncthreads();

    floatx16 acc[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;
    float m = -INFINITY, l = 0.f;
    if (ST == 2 && t + 2 < tb) fetch(t + 2, 1);
    for (int st = 0; t < tb; t += 2, st ^= ST - 1) {
        if (ST == 2 && t + 2 < tb) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * NI) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        const E* kl = kv[st][w][0];
        const E* vl = kv[st][w][1];
        floatx16 sc;
#pragma unroll
        for (int r = 0; r < 16; ++r) sc[r] = 0.f;
#pragma unroll
        for (int ks = 0; ks < NK; ++ks) {
            const Frag kf = swa_ld_row<E, D>(kl, lane & 31, ks, g);
            sc = T::mma(kf, q[ks], sc);
            if (TWO) sc = T::mma(kf, ql[TWO ? ks : 0], sc);
        }
        if (t * 32 + 32 > se.nv) {
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (t * 32 + 8 * (r / 4) + 4 * g + r % 4 >= se.nv) sc[r] = -INFINITY;
        }
        float mx = sc[0];
#pragma unroll
        for (int r = 1; r < 16; ++r) mx = fmaxf(mx, sc[r]);
        mx = fmaxf(mx, swa_swap(mx));
        const float mn = fmaxf(m, mx), mu = mn == -INFINITY ? 0.f : mn;
        const float al = __builtin_amdgcn_exp2f(m - mu);
        m = mn;
        l *= al;
#pragma unroll
        for (int i = 0; i < ND; ++i) acc[i] *= al;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            sc[r] = __builtin_amdgcn_exp2f(sc[r] - mu);
            l += sc[r];
        }
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            const Frag p = T::pack(sc, j), pr = T::rest(sc, j, p);
#pragma unroll
            for (int i = 0; i < ND; ++i) {
                const Frag vf = T::template ld_col<D>(vl, (32 / NP) * j, 32 * i, lane);
                acc[i] = T::mma(vf, p, acc[i]);
                if (TWO) acc[i] = T::mma(vf, pr, acc[i]);
            }
        }
        if (t + 2 * ST < tb) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // the reads of the tile that is replaced are done
            fetch(t + 2 * ST, st);
        }
    }
    l += swa_swap(l);

    // the two waves' and the new token's results; head h of wave x at part[x][h]
    __syncthreads();
    float* const accs = reinterpret_cast<float*>(kv);      // [2][32][D]
    floatx4 zero = {0.f, 0.f, 0.f, 0.f};      // (0 times what is not finite is a NaN)
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) zero[r % 4] = fmaf(acc[i][r], 0.f, zero[r % 4]);
    if ((lane & 31) < nh) {
        if (!(zero[0] + zero[1] + (zero[2] + zero[3]) == 0.f)) sm.again = 1;
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<floatx4*>(accs + (w * 32 + (lane & 31)) * D + 32 * i + 8 * j + 4 * g) =
                    floatx4{acc[i][4 * j], acc[i][4 * j + 1], acc[i][4 * j + 2], acc[i][4 * j + 3]};
        if (g == 0) {
            ms[w][lane & 31] = m;
            ls[w][lane & 31] = l;
        }
    }
    // An infinity that is seen becomes a NaN above: a remainder's product has
    // another sign or is 0 times it, and so is a row that fills up the last
    // tile.  A split with a result that is not finite makes all of it again.
    __syncthreads();
    if (sm.again)
        swa_decode_plain<E, D>(a, se, ta * 32, min(tb * 32, se.nv), nh, kc, vc, [&](int h, int i) { return turned(qrow + h * D, i) * a.c; },
                               accs, ms, ls, reinterpret_cast<float*>(sm.mw), tid);
    const int64_t item = (int64_t)b * gridDim.y + blockIdx.y;
    const int64_t pstep = (int64_t)32 * (D + 2);
    float* part = a.part + (item * a.nsplit + sp) * pstep;
    for (int i = tid; i < nh * D / 2; i += 128) {
        const int h = 2 * i / D, e = 2 * i % D;
        const float m2 = sp == 0 ? ms[2][h] : -INFINITY;
        const float mn = fmaxf(fmaxf(ms[0][h], ms[1][h]), m2), mu = mn == -INFINITY ? 0.f : mn;
        const float f0 = __builtin_amdgcn_exp2f(ms[0][h] - mu), f1 = __builtin_amdgcn_exp2f(ms[1][h] - mu);
        const float f2 = __builtin_amdgcn_exp2f(m2 - mu);
        float x[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            x[y] = accs[h * D + e + y] * f0 + accs[(32 + h) * D + e + y] * f1;
            if (sp == 0) x[y] = fmaf(vn[e + y], f2, x[y]);
        }
        const float L = ls[0][h] * f0 + ls[1][h] * f1 + f2;
        if (a.nsplit == 1) {
            o[2 * i] = (E)(x[0] / L);
            o[2 * i + 1] = (E)(x[1] / L);
            continue;
        }
        // stores that reach the memory every compute unit sees
        swa_put(part + 2 * i, x[0], x[1]);
        if (e == 0) swa_put(part + 32 * D + 2 * h, mn, L);
    }
    if (a.nsplit == 1) return;
    // the last workgroup of (b, heads) to arrive joins the splits
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");       // the stores are done before the arrival is counted
    __syncthreads();
    if (tid == 0)
        last = __hip_atomic_fetch_add(a.count + item, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.nsplit - 1;
    __syncthreads();
    if (!last) return;
    if (tid == 0) __hip_atomic_store(a.count + item, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);   // for the next call
    const float* pb = a.part + item * a.nsplit * pstep;
    // weight of every split, 32 lanes a head
    static_assert(SWA_DECODE_SPLITS == 32, "one lane per split");
    for (int h = tid / 32; h < nh; h += 4) {
        const int x = tid % 32;
        float2 v = make_float2(-INFINITY, 0.f);
        if (x < a.nsplit) v = swa_get(pb + x * pstep + 32 * D + 2 * h);
        float mn = v.x;
#pragma unroll
        for (int y = 16; y > 0; y /= 2) mn = fmaxf(mn, __shfl_xor(mn, y));
        const float f = __builtin_amdgcn_exp2f(v.x - (mn == -INFINITY ? 0.f : mn));
        float L = f * v.y;
#pragma unroll
        for (int y = 16; y > 0; y /= 2) L += __shfl_xor(L, y);
        mw[h][x] = f;
        if (x == 0) wl[h] = 1.f / L;
    }
    __syncthreads();
    // all splits' values in flight at once
    if (a.nsplit <= 8) swa_join<E, D, 8>(pb, pstep, a.nsplit, nh, mw, wl, o, tid);
    else swa_join<E, D, SWA_DECODE_SPLITS>(pb, pstep, a.nsplit, nh, mw, wl, o, tid);
}

// Tokens of a prompt into the cache: token t of sequence b, t < lens[b], at
// position t; where two positions share a slot only the later one is stored.
// A copy, bound by memory.
template <class V>
__global__ __launch_bounds__(256) void kd_swa_store_kernel(SwaStoreArgs a)
{
    const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t per = (int64_t)a.Hkv * a.row;     // 16-byte pieces of a token
    if (idx >= (int64_t)a.T * per) return;
    const int b = blockIdx.y, t = (int)(idx / per), h = (int)(idx % per) / a.row, c = (int)(idx % a.row);
    const int n = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    if (t >= n || (t >= a.S && n - t > a.cap - a.S)) return;
    const int64_t slot = cache_slot(t, a.S, a.cap);
    const int64_t bs = a.es;
    const char* ks = (const char*)a.k + (b * a.ks[0] + t * a.ks[1] + h * a.ks[2]) * bs + 16 * c;
    const char* vs = (const char*)a.v + (b * a.vs[0] + t * a.vs[1] + h * a.vs[2]) * bs + 16 * c;
    char* kd = (char*)a.kc + (b * a.kcs[0] + slot * a.kcs[1] + h * a.kcs[2]) * bs + 16 * c;
    char* vd = (char*)a.vc + (b * a.vcs[0] + slot * a.vcs[1] + h * a.vcs[2]) * bs + 16 * c;
    *reinterpret_cast<V*>(kd) = *reinterpret_cast<const V*>(ks);
    *reinterpret_cast<V*>(vd) = *reinterpret_cast<const V*>(vs);
}

// Work items before splitting: one per sequence, key head and block of 32 of
// its query heads.
static int64_t swa_decode_items(int B, int Hq, int Hkv) { return (int64_t)B * Hkv * ((Hq / Hkv + 31) / 32); }

// Splits of a row's keys: two workgroups for each of the chip's 256 compute
// units, none below 64 keys.  Both are resident (71 KB of LDS at most of 160)
// but in fp32 with heads of 128 (103 KB), where half of them follow the others.
// Rows are split only where there are fewer than SWA_DECODE_COUNTERS items, so
// that many counters serve every call.
int swa_decode_splits(int B, int Hq, int Hkv, int seen) {
    int n = (int)(SWA_DECODE_COUNTERS / swa_decode_items(B, Hq, Hkv));
    const int most = (seen + 63) / 64;
    n = n < most ? n : most;
    n = n < SWA_DECODE_SPLITS ? n : SWA_DECODE_SPLITS;
    return n < 1 ? 1 : n;
}

// The splits' partial results (none where a row's keys are not split).
size_t swa_decode_part_bytes(int B, int Hq, int Hkv, int d, int seen) {
    const int n = swa_decode_splits(B, Hq, Hkv, seen);
    return n == 1 ? 0 : (size_t)swa_decode_items(B, Hq, Hkv) * n * 32 * (d + 2) * 4;
}

template <class E, int D>
static hipError_t swa_decode(const SwaDecodeArgs& a, hipStream_t st)
{
    const dim3 grid(a.nsplit, a.Hkv * ((a.Hq / a.Hkv + 31) / 32), a.B);
    kd_swa_decode_kernel<E, D><<<grid, 128, 0, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_swa_decode(int bf16, int d, const SwaDecodeArgs& a, hipStream_t st)
{
    if (bf16) return d == 32 ? swa_decode<__bf16, 32>(a, st) : d == 64 ? swa_decode<__bf16, 64>(a, st) : swa_decode<__bf16, 128>(a, st);
    return d == 32 ? swa_decode<float, 32>(a, st) : d == 64 ? swa_decode<float, 64>(a, st) : swa_decode<float, 128>(a, st);
}

hipError_t launch_swa_store(const SwaStoreArgs& a, int B, hipStream_t st)
{
    const int64_t n = ((int64_t)a.T * a.Hkv * a.row + 255) / 256;
    kd_swa_store_kernel<floatx4><<<dim3((unsigned)n, B), 256, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace kd
