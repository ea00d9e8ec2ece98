// kd_prefix.hip -- attention of a batch over a prefix that all its sequences
// share and over each sequence's own pages, gfx950.
//
//     o = sum_s softmax_s(scale q . k_s) v_s,   s over the prefix's P keys, then
//                                               own keys 0 .. lens[b] + r
// for row r of sequence b.  The softmax splits over any parts of its keys:
// part x gives m_x = max, l_x = sum exp(s - m_x), o_x = sum exp(s - m_x) v, and
// with M = max m_x the whole is o = sum e^(m_x - M) o_x / sum e^(m_x - M) l_x.
// So the prefix is read once for all rows of the batch together: the rows of
// all sequences and the G heads of a group stand side by side as the columns of
// the same products (T G rows per key head), and only the own keys are read per
// sequence.
//
// One launch makes all parts, a second one joins them:
//  * 128 rows a workgroup, 32 per wave, tiles of keys shared through LDS (the
//    prefix, and own keys of packed rows);
//  * own keys of single rows: 4 independent waves a workgroup, each with the
//    heads of one group as columns and its own tiles (a step's own keys: bound
//    by reading them).
// 64 rows of 16 heads over 4 key heads, 32768 shared keys, up to 1000 own ones: 51
// us, 7 of them the join, for 130 MB of keys and values (2.6 TB/s; a tile of 64
// keys takes 2 us: its scores, exponentials and sums follow each other).  2015
// such rows, 8192 shared keys: 174 us, 18 of them the join (780 TFLOP/s; a large
// product reaches 1195).
// Products, K order and tiles are those of kd_swa.h.
#include "kd_check.h"
#include "kd_paged.h"
#include "kd_swa.h"

namespace kd {

constexpr int PREFIX_ROWS = 128;          // rows of a workgroup
constexpr int PREFIX_MOST = 48;           // splits of the prefix
constexpr int PREFIX_OWN_MOST = 16;       // and of the own keys
constexpr float PREFIX_EMPTY = -1.f;      // sum of a part that has not been written

// Where keys are: a list of pages of one head.  Ids outside the cache are
// clamped into it, numbers past the last key to that key (they are masked).
template <class E>
struct PrefixKeys {
    const E *k, *v;
    int64_t kp, ks, vp, vs;       // page and slot strides
    const int* pages;
    int page, most, last;         // slots of a page, highest page id, last key

    __device__ __forceinline__ int id(int at) const { return min(max(pages[at], 0), most); }
};

// o of those of a wave's rows that ask for it (`again`; rare, see its calls),
// from the maxima they have: key by key, each for the rows that see it (key <=
// lim).
template <class E, int D>
__device__ __forceinline__ void prefix_single(floatx16* o, const typename SwaT<E>::Frag* q, const PrefixKeys<E>& K, int first,
                                              int last, int lim, float c, float mu, bool again, int lane)
{
    typedef SwaT<E> T;
    typedef E E4 __attribute__((ext_vector_type(4)));
    constexpr int NK = D / T::KC, ND = D / 32;
    const int g = lane >> 5;
    if (again)
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[i][r] = 0.f;
#pragma unroll 1
    for (int key = first; key <= last; ++key) {
        const int64_t pg = K.id(key / K.page), slot = key % K.page;
        const E* kr = K.k + pg * K.kp + slot * K.ks;
        const E* vr = K.v + pg * K.vp + slot * K.vs;
        float s = 0.f;
#pragma unroll
        for (int ks = 0; ks < NK; ++ks) s += T::dot(q[ks], swa_ld_mem<E>(kr, ks, g));
        s += swa_swap(s);
        const bool sees = key <= lim;
        const float p = sees ? __builtin_amdgcn_exp2f(fmaf(s, c, -mu)) : 0.f;
        if (again)
#pragma unroll
            for (int i = 0; i < ND; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const E4 x = *reinterpret_cast<const E4*>(vr + 32 * i + 8 * j + 4 * g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][4 * j + e] = fmaf(p, sees ? (float)x[e] : 0.f, o[i][4 * j + e]);
                }
    }
}

template <class E, int D>
__device__ __forceinline__ void prefix_part(const PrefixArgs& a, int64_t at, const floatx16* o, float m, float l, int g)
{
    float* row = a.part + at * D;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<floatx4*>(row + 32 * i + 8 * j + 4 * g) =
                floatx4{o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]};
    if (g == 0) *reinterpret_cast<float2*>(a.ml + 2 * at) = make_float2(m, l);
}

// Whether a row's o has to be made again: where it is not finite, but not where
// the row's sum is a NaN, which makes NaNs of whatever is made.
template <int ND>
__device__ __forceinline__ bool prefix_again(const floatx16* o, float l) {
    float sum = 0.f;      // (0 times what is not finite is a NaN)
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) sum = fmaf(o[i][r], 0.f, sum);
    sum += swa_swap(sum);
    return !(sum == 0.f) && l == l;
}

// Whether a sequence in use holds row t of the call (every lane asks for its
// own).  Its loads start with the object, and answers take no others while there
// are no more sequences than lanes: one's end and length a lane.
struct PrefixHeld {
    const PrefixArgs& a;
    int end, len, begin;
    bool few;
    __device__ __forceinline__ PrefixHeld(const PrefixArgs& a_, int t, int lane) : a(a_), end(0), begin(0), few(a_.B <= 64) {
        const int at = min(lane, a.B - 1);
        len = a.lens[a.cu ? at : t];
        if (a.cu) {
            end = a.cu[at + 1];
            begin = a.cu[0];
        }
    }
    __device__ __forceinline__ bool operator()(int t) const {
        if (!a.cu) return len >= 0;
        int lo = 0, hi = a.B;      // as many sequences as lo end at or before t
        while (__any(lo < hi)) {
            const int mid = min((lo + hi) / 2, a.B - 1), e = few ? __shfl(end, mid) : a.cu[mid + 1];
            const bool up = lo < hi && e <= t;
            hi = lo < hi && !up ? mid : hi;
            lo = up ? mid + 1 : lo;
        }
        const int b = min(lo, a.B - 1), n = few ? __shfl(len, b) : a.lens[b];
        return begin <= t && lo < a.B && n >= 0;
    }
};

// Tiles of BN keys, NBUF of them in LDS (all but the one in use on their way).
constexpr int PREFIX_IDS = 512;      // keys whose page ids are in LDS at once (one of two such windows)
template <class E, int D>
struct PrefixLds {
    static constexpr int KEYS = sizeof(E) == 2 ? 128 : 64;
    static constexpr int ITEMS = sizeof(E) * D > 256 ? 2 : 4; // waves with own tiles (32 keys)
    union {
        struct {
            E k[KEYS * D], v[KEYS * D];
        } tile;
        struct {
            E k[32 * D], v[32 * D];
        } own[ITEMS];
    };
    int ids[2][PREFIX_IDS + 1];
};

// 128 rows from r0 on (of nrows; row r is head r % G of row q0 + r / G) against
// keys k0 .. k1 - 1.  CAUSAL: row r sees keys up to past + r / G.
template <class E, int D, bool CAUSAL, int BN>
__device__ __forceinline__ void prefix_rows(const PrefixArgs& a, PrefixLds<E, D>& sm, const PrefixKeys<E>& K, int hk, int q0,
                                            int nrows, int r0, int64_t past, int k0, int k1, int64_t part)
{
    typedef SwaT<E> T;
    typedef typename T::Frag Frag;
    typedef SwaTile<E, D> TL;
    constexpr int NBUF = PrefixLds<E, D>::KEYS / BN, NK = D / T::KC, NS = BN / 32, ND = D / 32, NP = 16 / T::PR;
    constexpr int STEP = 256 / TL::CPR < BN ? 256 / TL::CPR : BN, NL = BN / STEP;      // rows per round of the workgroup, rounds
    constexpr int BUSY = STEP * TL::CPR;                                               // threads that load
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 5;
    const int G = a.Hq / a.Hkv, row = r0 + 32 * w + (lane & 31), rr = min(row, nrows - 1);
    const E* qrow = (const E*)a.q + (int64_t)(q0 + rr / G) * a.qs[0] + (hk * G + rr % G) * a.qs[1];
    Frag q[NK];
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) q[ks] = swa_ld_mem<E>(qrow, ks, g);
    const PrefixHeld held(a, rr / G, lane);
    // the last key that the lane's row sees, and that the wave's first and last do
    const int lim = CAUSAL ? (int)min((int64_t)k1 - 1, past + rr / G) : k1 - 1;
    const int lim0 = CAUSAL ? (int)min((int64_t)k1 - 1, past + min(r0 + 32 * w, nrows - 1) / G) : k1 - 1;
    const int lim1 = CAUSAL ? (int)min((int64_t)k1 - 1, past + min(r0 + 32 * w + 31, nrows - 1) / G) : k1 - 1;

    floatx16 o[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] = 0.f;
    float m = -INFINITY, l = 0.f;
    const int nt = (k1 - k0 + BN - 1) / BN;

    // Page ids pass through LDS, a window of PREFIX_IDS keys at a time: loads of
    // ids between the keys' would make every use of one wait for all keys before it.
    auto window = [&](int x) {
        const int key = k0 + x * PREFIX_IDS, first = key / K.page;
        const int last = key + min(PREFIX_IDS, k1 - key) - 1;      // (the window's end may lie past 31 bits)
        const int n = last / K.page - first + 1;
        for (int i = tid; i < n; i += 256) sm.ids[x & 1][i] = K.id(first + i);
        __syncthreads();
    };
    // each lane's NL rows of a tile: page number (within the window) and slot go on
    // by BN keys from tile to tile
    const int fr = tid / TL::CPR, fc = tid % TL::CPR, bq = BN / K.page, br = BN % K.page;
    int pn[NL], sl[NL];
    auto fetch = [&](int t, E* kt, E* vt) {
        constexpr int PER = PREFIX_IDS / BN;
        const int x = t / PER;
        if (t % PER == 0) window(x);
        if (t % PER == 0 || k0 + (t + 1) * BN > k1) {
            const int base = (k0 + x * PREFIX_IDS) / K.page;
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int key = min(k0 + t * BN + fr + i * STEP, k1 - 1), p = key / K.page;
                pn[i] = p - base;
                sl[i] = key - p * K.page;
            }
        } else {
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                pn[i] += bq;
                sl[i] += br;
                if (sl[i] >= K.page) {
                    sl[i] -= K.page;
                    ++pn[i];
                }
            }
        }
        const uint32_t kd = lds_address(kt) + 1024 * w, vd = lds_address(vt) + 1024 * w;
        if (BUSY == 256 || tid < BUSY) {
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int64_t id = sm.ids[x & 1][pn[i]];
                const int ch = (fc ^ TL::swz(fr + i * STEP)) * TL::EPC;
                load_lds16(kd + i * BUSY * 16, K.k + id * K.kp + sl[i] * K.ks + ch);
                load_lds16(vd + i * BUSY * 16, K.v + id * K.vp + sl[i] * K.vs + ch);
            }
        }
    };
    auto tile = [&](int i, int buf) {
        // tile i is here; the buffer of tile i - 1 is free
        if (i + NBUF - 2 < nt) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(2 * NL * (NBUF - 2)) : "memory");
        else swa_landed();
        if (i + NBUF - 1 < nt) fetch(i + NBUF - 1, sm.tile.k + (buf + NBUF - 1) % NBUF * BN * D, sm.tile.v + (buf + NBUF - 1) % NBUF * BN * D);
        const E* kl = sm.tile.k + buf * BN * D;
        const E* vl = sm.tile.v + buf * BN * D;
        const int key0 = k0 + i * BN;
        if (CAUSAL && key0 > lim1) return;      // nothing visible to the wave
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
        if (key0 + BN - 1 > lim0) {
            const int hi = lim - key0 - 4 * g;
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (32 * n + 8 * (r / 4) + r % 4 > hi) sc[n][r] = -INFINITY;
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
        // (bf16: weights are rounded here, and not in their sum: o is off by 2.2e-3,
        // where its own rounding is 1.7e-3.  Their remainder would be half as many
        // products again, which bound prompts.)
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
#pragma unroll
    for (int i = 0; i < NBUF - 1; ++i)
        if (i < nt) fetch(i, sm.tile.k + i * BN * D, sm.tile.v + i * BN * D);
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) swa_arrive(q[ks]);
    // A row that is nobody's stands among the others as zeros: what it holds would
    // reach their bits, by the rescaling that a wave's rows do together.
    if (!CAUSAL && !held(rr / G))
#pragma unroll
        for (int ks = 0; ks < NK; ++ks) q[ks] = swa_zero<E>();
    for (int i = 0; i < nt; i += NBUF) {
        tile(i, 0);
        if (i + 1 < nt) tile(i + 1, 1);
        if (NBUF > 2) {
            if (i + 2 < nt) tile(i + 2, 2 % NBUF);
            if (i + 3 < nt) tile(i + 3, 3 % NBUF);
        }
    }
    l += swa_swap(l);
    // A masked key has weight 0, and 0 times an infinity or a NaN in its values
    // would still reach the rows of its tile: rows whose outputs are not finite
    // have them made again, each from the keys that it sees.
    const bool again = prefix_again<ND>(o, l);
    if (__any(again)) prefix_single<E, D>(o, q, K, k0, lim1, lim, a.c, m == -INFINITY ? 0.f : m, again, lane);
    if (row < nrows) prefix_part<E, D>(a, part + row, o, m, l, g);
}

// Own keys k0 .. k1 - 1 of one sequence and G <= 32 of its heads from h0 on, by
// one wave.  The next tile's keys load from the products with this one's on,
// its values from the products with this one's values on.  The matrix units
// have room to spare here, so bf16 weights go through as a rounded part and its
// remainder.
template <class E, int D>
__device__ __forceinline__ void prefix_own(const PrefixArgs& a, E* kl, E* vl, const PrefixKeys<E>& K, int b, int h0, int nh,
                                           int k0, int k1, int64_t part)
{
    typedef SwaT<E> T;
    typedef typename T::Frag Frag;
    typedef SwaTile<E, D> TL;
    constexpr int NK = D / T::KC, ND = D / 32, NP = 16 / T::PR, NI = 32 * TL::CPR / 64;
    constexpr bool TWO = sizeof(E) == 2;
    const int lane = threadIdx.x & 63, g = lane >> 5, h = lane & 31;
    const E* qrow = (const E*)a.q + (int64_t)b * a.qs[0] + (h0 + min(h, nh - 1)) * a.qs[1];
    Frag q[NK];
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) q[ks] = swa_ld_mem<E>(qrow, ks, g);
    const uint32_t kd = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)kl;
    const uint32_t vd = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)vl;
    // rows of a tile: lane's row of load i is i * (64 / CPR) + lane / CPR
    int64_t id[NI], sl[NI];
    auto find = [&](int t) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int key = min(k0 + 32 * t + i * (64 / TL::CPR) + lane / TL::CPR, k1 - 1), p = key / K.page;
            id[i] = K.id(p);
            sl[i] = key - p * K.page;
        }
    };
    auto chunk = [&](int i) { return ((lane % TL::CPR) ^ TL::swz(i * (64 / TL::CPR) + lane / TL::CPR)) * TL::EPC; };
    auto keys = [&]() {
#pragma unroll
        for (int i = 0; i < NI; ++i) load_lds16(kd + 1024 * i, K.k + id[i] * K.kp + sl[i] * K.ks + chunk(i));
    };
    auto values = [&]() {
#pragma unroll
        for (int i = 0; i < NI; ++i) load_lds16(vd + 1024 * i, K.v + id[i] * K.vp + sl[i] * K.vs + chunk(i));
    };
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) swa_arrive(q[ks]);
    floatx16 o[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] = 0.f;
    float m = -INFINITY, l = 0.f;
    const int nt = (k1 - k0 + 31) / 32;
    find(0);
    keys();
    values();
    for (int t = 0; t < nt; ++t) {
        const bool more = t + 1 < nt;
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NI) : "memory");      // all but the values
        floatx16 sc;
#pragma unroll
        for (int r = 0; r < 16; ++r) sc[r] = 0.f;
#pragma unroll
        for (int ks = 0; ks < NK; ++ks) sc = T::mma(swa_ld_row<E, D>(kl, lane & 31, ks, g), q[ks], sc);
        if (more) {
            find(t + 1);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // the reads of the tile that is replaced are done
            keys();
        }
        if (k0 + 32 * t + 32 > k1) {
            const int hi = k1 - 1 - (k0 + 32 * t) - 4 * g;
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (8 * (r / 4) + r % 4 > hi) sc[r] = -INFINITY;
        }
        float mx = sc[0];
#pragma unroll
        for (int r = 1; r < 16; ++r) mx = fmaxf(mx, sc[r]);
        mx = fmaxf(mx, swa_swap(mx)) * a.c;
        const float mn = fmaxf(m, mx), mu = mn == -INFINITY ? 0.f : mn, alpha = __builtin_amdgcn_exp2f(m - mu);
        m = mn;
        l *= alpha;
#pragma unroll
        for (int i = 0; i < ND; ++i) o[i] *= alpha;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            sc[r] = __builtin_amdgcn_exp2f(fmaf(sc[r], a.c, -mu));
            l += sc[r];
        }
        if (more) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NI) : "memory");      // all but the next keys
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            const Frag p = T::pack(sc, j), pr = T::rest(sc, j, p);
#pragma unroll
            for (int i = 0; i < ND; ++i) {
                const Frag vf = T::template ld_col<D>(vl, (32 / NP) * j, 32 * i, lane);
                o[i] = T::mma(vf, p, o[i]);
                if (TWO) o[i] = T::mma(vf, pr, o[i]);
            }
        }
        if (more) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            values();
        }
    }
    l += swa_swap(l);
    // (a row that fills up the last tile, and the remainders, make NaNs of an
    // infinity that is seen)
    const bool again = prefix_again<ND>(o, l);
    if (__any(again)) prefix_single<E, D>(o, q, K, k0, k1 - 1, k1 - 1, a.c, m == -INFINITY ? 0.f : m, again, lane);
    if (h < nh) prefix_part<E, D>(a, part + h, o, m, l, g);
}

// BN: tiles of 64 keys, or of 32 with more on their way.
template <class E, int D, int BN>
__global__ __launch_bounds__(256, sizeof(E) * D > 256 ? 1 : 2) void kd_prefix_kernel(PrefixArgs a)
{
    __shared__ __align__(16) PrefixLds<E, D> sm;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int G = a.Hq / a.Hkv;
    const int64_t rows = (int64_t)a.T * G;
    PrefixKeys<E> K;
    K.kp = a.kcs[0], K.ks = a.kcs[1], K.vp = a.vcs[0], K.vs = a.vcs[1];
    K.page = a.page;
    K.most = a.pages - 1;
    if ((int)blockIdx.x < a.nprefix) {
        int64_t item;      // neighbours read the same keys
        if (!swa_item((int64_t)a.blocks * a.Hkv * a.sp, item)) return;
        const int blk = item % a.blocks;
        item /= a.blocks;
        const int hk = item % a.Hkv, sp = item / a.Hkv;
        const int tiles = (a.P + 63) / 64, per = (tiles + a.sp - 1) / a.sp;
        const int k0 = min(sp * per * 64, a.P), k1 = min(k0 + per * 64, a.P);
        K.k = (const E*)a.kc + hk * a.kcs[2];
        K.v = (const E*)a.vc + hk * a.vcs[2];
        K.pages = a.ptable;
        prefix_rows<E, D, false, BN>(a, sm, K, hk, 0, (int)rows, blk * PREFIX_ROWS, 0, k0, k1, ((int64_t)sp * a.Hkv + hk) * rows);
        return;
    }
    int64_t item = (int)blockIdx.x - a.nprefix;
    if (a.cu) {
        // slot of 128 rows: sequence s owns the slots cu[s] G / 128 + s onwards
        const int hk = item % a.Hkv;
        item /= a.Hkv;
        const int slot = item % a.nslots, so = item / a.nslots;
        const int n = wave_count(a.B, [&](int at) { return (int64_t)min(max(a.cu[at], 0), a.T) * G / PREFIX_ROWS + at <= slot; });
        if (n == 0) return;
        const int b = n - 1, q0 = min(max(a.cu[b], 0), a.T), q1 = min(max(a.cu[b + 1], q0), a.T);
        const int nrows = (q1 - q0) * G, blk = slot - (int)((int64_t)q0 * G / PREFIX_ROWS + b);
        const int len = a.lens[b];
        // (blk is negative where offsets are out of order)
        if (blk < 0 || (int64_t)blk * PREFIX_ROWS >= nrows || len < 0) return;
        const int r0 = blk * PREFIX_ROWS;
        // keys that the block's last row sees, as far as the table goes
        const int64_t all = min((int64_t)len + min(r0 + PREFIX_ROWS - 1, nrows - 1) / G + 1, (int64_t)a.width * a.page);
        const int nk = (int)min(all, (int64_t)INT32_MAX - 64), tiles = (nk + 63) / 64, per = (tiles + a.so - 1) / a.so;
        const int k0 = (int)min((int64_t)so * per * 64, (int64_t)nk), k1 = (int)min((int64_t)k0 + (int64_t)per * 64, (int64_t)nk);
        K.k = (const E*)a.kc + hk * a.kcs[2];
        K.v = (const E*)a.vc + hk * a.vcs[2];
        K.pages = a.table + b * a.ts;
        prefix_rows<E, D, true, BN>(a, sm, K, hk, q0, nrows, r0, len, k0, k1,
                                ((int64_t)(a.sp + so) * a.Hkv + hk) * rows + (int64_t)q0 * G);
        return;
    }
    constexpr int ITEMS = PrefixLds<E, D>::ITEMS;
    const int nhb = (G + 31) / 32;
    item = item * ITEMS + w;
    if (w >= ITEMS || item >= (int64_t)a.B * a.Hkv * nhb * a.so) return;
    const int so = item % a.so;
    item /= a.so;
    const int hb = item % nhb;
    item /= nhb;
    const int hk = item % a.Hkv, b = item / a.Hkv;
    const int len = a.lens[b], h0 = hk * G + hb * 32, nh = min(32, G - hb * 32);
    const int64_t part = ((int64_t)(a.sp + so) * a.Hkv + hk) * rows + (int64_t)b * G + hb * 32;
    const int64_t all = len < 0 ? 0 : min((int64_t)len + 1, (int64_t)a.width * a.page);
    const int nk = (int)min(all, (int64_t)INT32_MAX - 64), tiles = (nk + 31) / 32, per = (tiles + a.so - 1) / a.so;
    const int k0 = (int)min((int64_t)so * per * 32, (int64_t)nk), k1 = (int)min((int64_t)k0 + (int64_t)per * 32, (int64_t)nk);
    if (k0 >= k1) {      // (a split without keys: its o, which is not written, is not read)
        if (lane < nh) *reinterpret_cast<float2*>(a.ml + 2 * (part + lane)) = make_float2(-INFINITY, PREFIX_EMPTY);
        return;
    }
    K.k = (const E*)a.kc + hk * a.kcs[2];
    K.v = (const E*)a.vc + hk * a.vcs[2];
    K.pages = a.table + b * a.ts;
    prefix_own<E, D>(a, sm.own[w % ITEMS].k, sm.own[w % ITEMS].v, K, b, h0, nh, k0, k1, part);
}

// Joins the parts: R rows a workgroup, 4 / R waves each with a share of the
// splits.  A lane holds the maximum and sum of one split, then D / 64 elements
// (32: half of the lanes) of the result.
template <class E, int D, int R>
__global__ __launch_bounds__(256) void kd_prefix_join_kernel(PrefixArgs a)
{
    constexpr int N = D >= 128 ? 2 : 1, SHARE = 4 / R;
    typedef float F __attribute__((ext_vector_type(N)));
    __shared__ F part[4][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, G = a.Hq / a.Hkv, S = a.sp + a.so;
    const int64_t at = (int64_t)blockIdx.x * R + w / SHARE;
    const int t = at / a.Hq, h = at % a.Hq;
    bool held = at < (int64_t)a.T * a.Hq;
    int b = t;
    if (held && a.cu) {
        b = paged_owner(a.cu, a.B, t);
        held = b < a.B && a.cu[min(b, a.B)] <= t;      // (otherwise no sequence holds the row)
    }
    F sum;
#pragma unroll
    for (int e = 0; e < N; ++e) sum[e] = 0.f;
    float M = -INFINITY, L = 0.f;
    if (held) {
        const int64_t rows = (int64_t)a.T * G, row = (int64_t)(h / G) * rows + (int64_t)t * G + h % G;
        float2 x = make_float2(-INFINITY, PREFIX_EMPTY);
        if (lane < S && a.lens[b] >= 0) x = *reinterpret_cast<const float2*>(a.ml + 2 * (lane * (int64_t)a.Hkv * rows + row));
        M = x.x;
#pragma unroll
        for (int y = 32; y > 0; y /= 2) M = fmaxf(M, __shfl_xor(M, y));
        // (a part of no weight counts all the same: 0 times an infinity that is seen)
        const bool empty = x.y == PREFIX_EMPTY;
        const float f = empty ? PREFIX_EMPTY : x.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(x.x - M);
        L = empty ? 0.f : f * x.y;
#pragma unroll
        for (int y = 32; y > 0; y /= 2) L += __shfl_xor(L, y);
        const float* p = a.part + row * D + (lane * N < D ? lane * N : 0);
        const int64_t step = (int64_t)a.Hkv * rows * D;
#pragma unroll 1
        for (int s0 = w % SHARE; s0 < S; s0 += 8 * SHARE) {
            F v[8];
#pragma unroll
            for (int s = 0; s < 8; ++s) v[s] = *reinterpret_cast<const F*>(p + min(s0 + s * SHARE, S - 1) * step);
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int i = s0 + s * SHARE;
                const float fs = i < S ? __shfl(f, i & 63) : PREFIX_EMPTY;
                if (fs == PREFIX_EMPTY) continue;
#pragma unroll
                for (int e = 0; e < N; ++e) sum[e] = fmaf(fs, v[s][e], sum[e]);
            }
        }
    }
    if (SHARE > 1) {
        part[w][lane] = sum;
        __syncthreads();
        if (w % SHARE != 0) return;
#pragma unroll
        for (int y = 1; y < SHARE; ++y) sum += part[w + y][lane];
    }
    if (!held) return;
    // What a row sees is a matter of its keys' number: scores that are all NaN leave
    // M at -infinity too (with L a NaN), and so do scores of -infinity (0 / 0).
    const bool none = a.lens[b] < 0 || (a.P == 0 && a.width == 0);
    const float inv = none ? 0.f : 1.f / L;
    if (lane * N < D) {
        E* o = (E*)a.o + at * D + lane * N;
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] = none ? (E)0.f : (E)(sum[e] * inv);
    }
    if (a.lse && lane == 0) a.lse[(int64_t)h * a.T + t] = none ? -INFINITY : 0.6931471805599453f * (M + __log2f(L));
}

// Splits.  While every workgroup has a compute unit to itself, the prefix takes
// as long as one part's tiles of 64 keys (2 us each), and a part more costs the
// joining of its rows, little (3 rows of 16 heads over 4 key heads, 2000 keys, us
// at 8, 16 and 32 parts: 12.2, 9.1, 7.2).  Beyond that two workgroups share a
// compute unit, where a tile takes each of them 1.6 times as long as one alone,
// and a part costs its rows' traffic, as long as 8 tiles (2015 such rows, 8192
// keys, us at 1, 2, 8 and 24 parts: 241, 174, 194, 257).
static int prefix_splits(int64_t items, int P)
{
    const int tiles = (P + 63) / 64;
    int best = 1;
    double least = 1e30;
    for (int s = 1; s <= PREFIX_MOST && s <= tiles; ++s) {
        const int64_t n = items * s;
        const int part = (tiles + s - 1) / s;
        const double cost = n <= 256 ? part + 2 + s / 32.0 : 1.6 * (double)((n + 511) / 512) * (part + 8);
        if (cost < least) least = cost, best = s;
    }
    return P == 0 ? 0 : best;
}

void prefix_plan(PrefixArgs& a, bool packed)
{
    const int64_t G = a.Hq / a.Hkv, rows = a.T * G, cap = (int64_t)a.width * a.page;
    a.blocks = (int)((rows + PREFIX_ROWS - 1) / PREFIX_ROWS);
    a.sp = prefix_splits((int64_t)a.blocks * a.Hkv, a.P);
    a.nslots = (int)(rows / PREFIX_ROWS + a.B);
    // own keys: as many splits as make 2048 waves (packed: 512 workgroups), at most
    // as many as the table has room for 64 (packed: 256) keys each (64 sequences
    // of up to 1000 keys, 4 key heads, us at 1, 2, 4, 8 and 16 splits: 81, 55, 46,
    // 46, 48)
    const int64_t items = packed ? (int64_t)a.nslots * a.Hkv : (int64_t)a.B * a.Hkv * ((G + 31) / 32);
    const int64_t most = packed ? (cap + 255) / 256 : (cap + 63) / 64;
    int64_t n = (packed ? 512 : 2048) / items;
    n = n < most ? n : most;
    n = n < PREFIX_OWN_MOST ? n : PREFIX_OWN_MOST;
    a.so = n < 1 ? 1 : (int)n;
}

size_t prefix_workspace_bytes(PrefixArgs a, int d, bool packed)
{
    prefix_plan(a, packed);
    return (size_t)(a.sp + a.so) * a.T * a.Hq * (d + 2) * 4;
}

static int64_t prefix_grid(const PrefixArgs& a, bool packed, int items)
{
    const int64_t G = a.Hq / a.Hkv;
    const int64_t own = packed ? (int64_t)a.nslots * a.Hkv * a.so
                               : ((int64_t)a.B * a.Hkv * ((G + 31) / 32) * a.so + items - 1) / items;
    return swa_grid((int64_t)a.blocks * a.Hkv * a.sp) + own;
}

// Rows of o that a workgroup of the join takes: one after the other where rows
// are many, shared out to four waves where they are few (1024 rows, 40 parts: 7.8
// and 7.4 us; 48 rows, 34 parts: 6.1 and 4.8; 32240 rows, 3 parts: 20 and 69).
static int prefix_join_rows(const PrefixArgs& a) { return a.sp + a.so <= 8 || (int64_t)a.T * a.Hq > 8192 ? 4 : 1; }

bool prefix_fits(PrefixArgs a, bool packed)
{
    const int64_t G = a.Hq / a.Hkv;
    if ((int64_t)a.T * G > (1 << 30) || a.T * G / PREFIX_ROWS + a.B > (1 << 30)) return false;
    prefix_plan(a, packed);
    return grid_fits(prefix_grid(a, packed, 2), 256) && grid_fits(((int64_t)a.T * a.Hq + 3) / prefix_join_rows(a), 256);
}

template <class E, int D>
static hipError_t prefix(PrefixArgs a, hipStream_t st)
{
    prefix_plan(a, a.cu != nullptr);
    a.ml = a.part + (int64_t)(a.sp + a.so) * a.T * a.Hq * D;
    a.nprefix = (int)swa_grid((int64_t)a.blocks * a.Hkv * a.sp);
    const unsigned grid = (unsigned)prefix_grid(a, a.cu != nullptr, PrefixLds<E, D>::ITEMS);
    // few blocks of rows read the prefix from memory, many from a cache (2 blocks,
    // 32768 keys: 45.4 us with tiles of 32 keys, 46.6 with 64; 63 blocks, 8192
    // keys: 191 and 178)
    if (sizeof(E) == 4 || a.blocks <= 4) kd_prefix_kernel<E, D, 32><<<grid, 256, 0, st>>>(a);
    else kd_prefix_kernel<E, D, sizeof(E) == 4 ? 32 : 64><<<grid, 256, 0, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t rows = (int64_t)a.T * a.Hq;
    if (prefix_join_rows(a) == 4) kd_prefix_join_kernel<E, D, 4><<<(unsigned)((rows + 3) / 4), 256, 0, st>>>(a);
    else kd_prefix_join_kernel<E, D, 1><<<(unsigned)rows, 256, 0, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_prefix(int bf16, int d, const PrefixArgs& a, hipStream_t st)
{
    if (bf16) return d == 32 ? prefix<__bf16, 32>(a, st) : d == 64 ? prefix<__bf16, 64>(a, st) : prefix<__bf16, 128>(a, st);
    return d == 32 ? prefix<float, 32>(a, st) : d == 64 ? prefix<float, 64>(a, st) : prefix<float, 128>(a, st);
}

}  // namespace kd
