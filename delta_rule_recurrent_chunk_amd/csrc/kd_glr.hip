// kd_glr.hip -- element-wise gated linear recurrence and its backward pass, gfx950.
//
// Per batch element b and channel c, with the state h in fp32:
//     h_t = f_t h_{t-1} + i_t x_t          (i_t = 1 without an input gate)
// and, for L = <dh, h> + <dhT, h_T>, walking back with m = dL/dh_t from the
// tokens after t:
//     g_t = dh_t + m;  dx_t = i_t g_t;  di_t = x_t g_t;  df_t = g_t h_{t-1};  m = f_t g_t
// and dh0 = the last m.
//
// Both directions are affine in the carried value: over any run of tokens
// h_out = A h_in + Bh and m_in = A m_out + Bm with A the product of the gates.
// One workgroup takes a tile of 128 tokens by LANES * VEC channels and reads it
// once into registers; each of its GROUPS thread rows reduces its TOK tokens
// to (A, B), the rows are joined through LDS, and the tile's (A, B) joins the
// tiles of the same channels along the sequence through words in the
// workspace (a scan in one pass over the data, bound by memory).
//
// Words between tiles.  A tile publishes its (A, B) as soon as it is read, and
// its carried-out value once it knows what enters; a tile looks back at up to
// LOOK predecessors for the nearest carried-out value with all (A, B) between
// and folds them forward, c = fma(A, c, B): the very operations the tiles in
// between do themselves, so the result does not depend on how far it looked.
// Every word is one 8-byte store that carries its own validity (cleared to all
// ones by a kernel ahead of the launch), so no fence orders two of them.  The
// workgroups take their tiles from a counter, a sequence's first tiles first:
// a tile only ever waits for tiles whose workgroups started earlier and which
// wait, in turn, only for earlier ones, so every wait ends (a bound of some
// seconds, after which the results become NaN, is there all the same).
#include "kd_check.h"
#include "kd_device.h"

namespace kd {

constexpr int GLR_CHUNK = 128;   // tokens of a tile and between two kept states (KRON_DELTA_GLR_CHUNK)
constexpr int GLR_NT = 512;      // threads of a workgroup
constexpr int GLR_LOOK = 8;      // tiles one look back covers
constexpr unsigned GLR_POLLS = 1u << 20;
constexpr unsigned long long GLR_EMPTY = ~0ull;

typedef unsigned long long u64;

struct GlrArgs {
    const void *x, *f, *i, *dh;
    const float *h0, *dhT;
    const float* hs_in;
    void *h, *dx, *df, *di;
    float *hT, *hs, *dh0;
    unsigned* ticket;   // null: one tile per sequence, nothing to hand over
    u64 *agg, *inc;     // [tiles][B][D]
    int B, T, D;
};

// VEC adjacent channels of one token
template <class E, int VEC>
struct GlrVec {
    typedef E V __attribute__((ext_vector_type(VEC)));
};
template <class E>
struct GlrVec<E, 1> {
    typedef E V;
};
template <class V>
__device__ __forceinline__ float glr_at(const V& v, int e) {
    return (float)v[e];
}
template <>
__device__ __forceinline__ float glr_at<__bf16>(const __bf16& v, int) {
    return (float)v;
}
template <>
__device__ __forceinline__ float glr_at<float>(const float& v, int) {
    return v;
}
template <class E, class V>
__device__ __forceinline__ void glr_set(V& v, int e, float x) {
    v[e] = (E)x;
}
template <>
__device__ __forceinline__ void glr_set<__bf16, __bf16>(__bf16& v, int, float x) {
    v = (__bf16)x;
}
template <>
__device__ __forceinline__ void glr_set<float, float>(float& v, int, float x) {
    v = x;
}

// Makes the compiler forget what it knows of v: the second pass over a tile
// converts its bf16 values anew instead of keeping fp32 copies in registers.
template <class V>
__device__ __forceinline__ void glr_fresh(V& v) {
    if constexpr (sizeof(V) == 8) {
        typedef unsigned U2 __attribute__((ext_vector_type(2)));
        U2 r = __builtin_bit_cast(U2, v);
        asm volatile("" : "+v"(r));
        v = __builtin_bit_cast(V, r);
    }
}

// A product of gates over a run of tokens.  One that falls below fp32's range
// becomes the smallest number (a step of rounding there), so that 0 still says
// that a gate was 0: an infinite carried value survives every gate but that
// one, where it becomes a NaN, as it does token by token.
__device__ __forceinline__ float glr_least(float a) {
    return a == 0.f ? copysignf(1.401298464324817e-45f, a) : a;      // 2^-149
}
// the products A of a thread's own tokens
template <class V, int TOK, int VEC>
__device__ __forceinline__ void glr_own_gates(float (&A)[VEC], const V (&f)[TOK]) {
    bool any = false;
#pragma unroll
    for (int e = 0; e < VEC; ++e) any |= A[e] == 0.f;
    if (!any) return;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        bool zero = false;
#pragma unroll
        for (int t = 0; t < TOK; ++t) zero |= glr_at(f[t], e) == 0.f;
        if (!zero) A[e] = glr_least(A[e]);
    }
}
// pa, the product of GROUPS rows' gates, and those in front of each row, p:
// the first `rows` of them (in the order of `down`) have no 0 in them
template <int GROUPS, int CW>
__device__ __forceinline__ void glr_row_gates(float& pa, float (*p)[CW], int c, int rows, bool down) {
    if (pa != 0.f) return;
    for (int r = 0; r <= min(rows, GROUPS - 1); ++r) {
        float& x = p[down ? GROUPS - 1 - r : r][c];
        x = glr_least(x);
    }
    if (rows == GROUPS) pa = glr_least(pa);
}

__device__ __forceinline__ u64 glr_pair(float a, float b) {
    unsigned x = __float_as_uint(a);
    if (x == 0xffffffffu) x = 0x7fc00000u;      // a NaN either way; all ones means empty
    return ((u64)x << 32) | __float_as_uint(b);
}
__device__ __forceinline__ u64 glr_load(const u64* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void glr_store(u64* p, u64 v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// What enters a tile of one channel: the word of its neighbour `step` words
// away (and further ones) as described above.  `far` neighbours exist.
__device__ __forceinline__ float glr_look_back(const u64* agg, const u64* inc, int64_t step, int far) {
    for (unsigned n = 0; n < GLR_POLLS; ++n) {
        u64 iv[GLR_LOOK], av[GLR_LOOK];
        iv[0] = glr_load(inc + step);
        if (iv[0] != GLR_EMPTY) return __uint_as_float((unsigned)iv[0]);
#pragma unroll
        for (int k = 0; k < GLR_LOOK; ++k) {
            av[k] = k < far ? glr_load(agg + (k + 1) * step) : GLR_EMPTY;
            iv[k] = k < far ? glr_load(inc + (k + 1) * step) : GLR_EMPTY;
        }
        int d = -1;
        bool chain = true;
#pragma unroll
        for (int k = 0; k < GLR_LOOK; ++k)
            if (d < 0 && chain) {
                if (iv[k] != GLR_EMPTY) d = k;
                else if (av[k] == GLR_EMPTY) chain = false;
            }
        if (d >= 0) {
            float c = 0.f;
#pragma unroll
            for (int k = GLR_LOOK - 1; k >= 0; --k) {
                if (k == d) c = __uint_as_float((unsigned)iv[k]);
                else if (k < d) c = fmaf(__uint_as_float((unsigned)(av[k] >> 32)), c, __uint_as_float((unsigned)av[k]));
            }
            return c;
        }
        __builtin_amdgcn_s_sleep(1);
    }
    return __uint_as_float(0x7fc00000u);
}

// The tile of a workgroup: chunk of the sequence (counted in the direction of
// the carry), batch element and first channel.
template <int CW>
__device__ __forceinline__ void glr_tile(const GlrArgs& p, int& n, int& b, int& c0) {
    __shared__ unsigned tick;
    if (p.ticket) {
        if (threadIdx.x == 0) tick = atomicAdd(p.ticket, 1u);
        __syncthreads();
    }
    const unsigned id = p.ticket ? tick : blockIdx.x;
    const unsigned ncb = (p.D + CW - 1) / CW, row = ncb * p.B;
    n = id / row;
    b = id % row / ncb;
    c0 = id % row % ncb * CW;
}

// Forward.  Bound by memory: 8 x 2048 x 2048 bf16 with an input gate (268 MB)
// takes 64.9 us, 4.1 TB/s (a large copy: 5.1).  128 x 128 tiles: 8 tokens of 4
// channels per thread keep 48 registers of loads in flight, and the words
// handed over are 3% of the data.
template <class E, bool GATE, int VEC, int LANES>
__global__ __launch_bounds__(GLR_NT) void kd_glr_fwd_kernel(GlrArgs p)
{
    constexpr int CW = LANES * VEC, GROUPS = GLR_NT / LANES, TOK = GLR_CHUNK / GROUPS;
    typedef typename GlrVec<E, VEC>::V V;
    __shared__ __align__(16) float sA[GROUPS][CW], sB[GROUPS][CW], sh[CW];
    const int tid = threadIdx.x, g = tid / LANES, cl = tid % LANES * VEC;
    int n, b, c0;
    glr_tile<CW>(p, n, b, c0);
    const int nc = (p.T + GLR_CHUNK - 1) / GLR_CHUNK;
    if (n >= nc) return;
    const int t0 = n * GLR_CHUNK + g * TOK, left = p.T - t0;      // this row's tokens
    const bool in = c0 + cl < p.D;
    const size_t base = ((size_t)b * p.T + t0) * p.D + c0 + cl;
    V f[TOK], x[TOK], gi[TOK];
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
        const size_t at = base + (size_t)t * p.D;
        const bool ok = in && t < left;
        f[t] = ok ? *(const V*)((const E*)p.f + at) : (V)(E)1.f;      // a token past the end changes nothing
        x[t] = ok ? *(const V*)((const E*)p.x + at) : (V)(E)0.f;
        if (GATE) gi[t] = ok ? *(const V*)((const E*)p.i + at) : (V)(E)0.f;
    }
    float A[VEC], Bh[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) A[e] = 1.f, Bh[e] = 0.f;
#pragma unroll
    for (int t = 0; t < TOK; ++t)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float ff = glr_at(f[t], e), u = GATE ? glr_at(gi[t], e) * glr_at(x[t], e) : glr_at(x[t], e);
            Bh[e] = fmaf(ff, Bh[e], u);
            A[e] *= ff;
        }
    glr_own_gates(A, f);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        sA[g][cl + e] = A[e];
        sB[g][cl + e] = Bh[e];
    }
    __syncthreads();
    if (tid < CW && c0 + tid < p.D) {
        // the rows' entering (A, B), then the tile's
        float pa = 1.f, pb = 0.f;
        int rows = GROUPS;      // those in front of the first with a gate of 0
#pragma unroll
        for (int r = 0; r < GROUPS; ++r) {
            const float a = sA[r][tid], bb = sB[r][tid];
            sA[r][tid] = pa;
            sB[r][tid] = pb;
            pb = fmaf(a, pb, bb);
            pa *= a;
            rows = a == 0.f ? min(rows, r) : rows;
        }
        glr_row_gates<GROUPS>(pa, sA, tid, rows, false);
        const int64_t ch = (int64_t)b * p.D + c0 + tid, step = (int64_t)p.B * p.D, w = n * step + ch;
        float c;
        if (n == 0) {
            c = p.h0 ? p.h0[ch] : 0.f;
        } else {
            if (n < nc - 1) glr_store(p.agg + w, glr_pair(pa, pb));
            c = glr_look_back(p.agg + w, p.inc + w, -step, n);
        }
        const float out = fmaf(pa, c, pb);
        if (n < nc - 1) glr_store(p.inc + w, __float_as_uint(out));
        else if (p.hT) p.hT[ch] = out;
        if (p.hs) p.hs[((size_t)b * nc + n) * p.D + c0 + tid] = c;
        sh[tid] = c;
    }
    __syncthreads();
    if (!in) return;
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
        glr_fresh(f[t]);
        glr_fresh(x[t]);
        if (GATE) glr_fresh(gi[t]);
    }
    float s[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[e] = fmaf(sA[g][cl + e], sh[cl + e], sB[g][cl + e]);
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
        V o;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float u = GATE ? glr_at(gi[t], e) * glr_at(x[t], e) : glr_at(x[t], e);
            s[e] = fmaf(glr_at(f[t], e), s[e], u);
            glr_set<E>(o, e, s[e]);
        }
        if (t < left) *(V*)((E*)p.h + base + (size_t)t * p.D) = o;
    }
}

// Backward.  Bound by memory: 1 x 32768 x 2048 bf16 with an input gate (940 MB)
// takes 193 us, 4.9 TB/s; the forward of the same size 116 us.
// The tiles run from the sequence's end to its start.  A tile's states come
// from the kept state that entered it (fp32, so df takes no rounded state).
template <class E, bool GATE, int VEC, int LANES>
__global__ __launch_bounds__(GLR_NT) void kd_glr_bwd_kernel(GlrArgs p)
{
    constexpr int CW = LANES * VEC, GROUPS = GLR_NT / LANES, TOK = GLR_CHUNK / GROUPS;
    typedef typename GlrVec<E, VEC>::V V;
    __shared__ __align__(16) float sA[GROUPS][CW], sH[GROUPS][CW], sM[GROUPS][CW], sP[GROUPS][CW], sm[CW];
    const int tid = threadIdx.x, g = tid / LANES, cl = tid % LANES * VEC;
    int r, b, c0;
    glr_tile<CW>(p, r, b, c0);
    const int nc = (p.T + GLR_CHUNK - 1) / GLR_CHUNK;
    if (r >= nc) return;
    const int n = nc - 1 - r, t0 = n * GLR_CHUNK + g * TOK, left = p.T - t0;
    const bool in = c0 + cl < p.D;
    const size_t base = ((size_t)b * p.T + t0) * p.D + c0 + cl;
    V f[TOK], x[TOK], gi[TOK], d[TOK];
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
        const size_t at = base + (size_t)t * p.D;
        const bool ok = in && t < left;
        f[t] = ok ? *(const V*)((const E*)p.f + at) : (V)(E)1.f;
        x[t] = ok ? *(const V*)((const E*)p.x + at) : (V)(E)0.f;
        d[t] = ok ? *(const V*)((const E*)p.dh + at) : (V)(E)0.f;
        if (GATE) gi[t] = ok ? *(const V*)((const E*)p.i + at) : (V)(E)0.f;
    }
    float A[VEC], Bh[VEC], Bm[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) A[e] = 1.f, Bh[e] = Bm[e] = 0.f;
#pragma unroll
    for (int t = 0; t < TOK; ++t)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float ff = glr_at(f[t], e), u = GATE ? glr_at(gi[t], e) * glr_at(x[t], e) : glr_at(x[t], e);
            Bh[e] = fmaf(ff, Bh[e], u);
            A[e] *= ff;
        }
#pragma unroll
    for (int t = TOK - 1; t >= 0; --t)
#pragma unroll
        for (int e = 0; e < VEC; ++e) Bm[e] = glr_at(f[t], e) * (glr_at(d[t], e) + Bm[e]);
    glr_own_gates(A, f);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        sA[g][cl + e] = A[e];
        sH[g][cl + e] = Bh[e];
        sM[g][cl + e] = Bm[e];
    }
    __syncthreads();
    const int64_t step = (int64_t)p.B * p.D;
    if (tid < CW && c0 + tid < p.D) {
        float pa = 1.f, pm = 0.f;
        int rows = GROUPS;      // those behind the last with a gate of 0
#pragma unroll
        for (int q = GROUPS - 1; q >= 0; --q) {
            const float a = sA[q][tid], m = sM[q][tid];
            sP[q][tid] = pa;
            sM[q][tid] = pm;
            pm = fmaf(a, pm, m);
            pa *= a;
            rows = a == 0.f ? min(rows, GROUPS - 1 - q) : rows;
        }
        glr_row_gates<GROUPS>(pa, sP, tid, rows, true);
        const int64_t ch = (int64_t)b * p.D + c0 + tid, w = n * step + ch;
        float c;
        if (r == 0) {
            c = p.dhT ? p.dhT[ch] : 0.f;
        } else {
            if (n > 0) glr_store(p.agg + w, glr_pair(pa, pm));
            c = glr_look_back(p.agg + w, p.inc + w, step, r);
        }
        const float out = fmaf(pa, c, pm);
        if (n > 0) glr_store(p.inc + w, __float_as_uint(out));
        else if (p.dh0) p.dh0[ch] = out;
        sm[tid] = c;
    } else if (tid >= GLR_NT - CW && c0 + tid - (GLR_NT - CW) < p.D) {
        // meanwhile other threads make the state that enters each row
        const int k = tid - (GLR_NT - CW);
        float c = p.hs_in[((size_t)b * nc + n) * p.D + c0 + k];
#pragma unroll
        for (int q = 0; q < GROUPS; ++q) {
            const float o = fmaf(sA[q][k], c, sH[q][k]);
            sH[q][k] = c;
            c = o;
        }
    }
    __syncthreads();
    if (!in) return;
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
        glr_fresh(f[t]);
        glr_fresh(x[t]);
        glr_fresh(d[t]);
        if (GATE) glr_fresh(gi[t]);
    }
    float hp[TOK][VEC], s[VEC], m[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        s[e] = sH[g][cl + e];
        m[e] = fmaf(sP[g][cl + e], sm[cl + e], sM[g][cl + e]);
    }
#pragma unroll
    for (int t = 0; t < TOK; ++t)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float u = GATE ? glr_at(gi[t], e) * glr_at(x[t], e) : glr_at(x[t], e);
            hp[t][e] = s[e];
            s[e] = fmaf(glr_at(f[t], e), s[e], u);
        }
#pragma unroll
    for (int t = TOK - 1; t >= 0; --t) {
        V ox, of, oi;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float gg = glr_at(d[t], e) + m[e];
            glr_set<E>(ox, e, GATE ? glr_at(gi[t], e) * gg : gg);
            if (GATE) glr_set<E>(oi, e, glr_at(x[t], e) * gg);
            glr_set<E>(of, e, gg * hp[t][e]);
            m[e] = glr_at(f[t], e) * gg;
        }
        if (t < left) {
            const size_t at = base + (size_t)t * p.D;
            *(V*)((E*)p.dx + at) = ox;
            *(V*)((E*)p.df + at) = of;
            if (GATE) *(V*)((E*)p.di + at) = oi;
        }
    }
}

__global__ __launch_bounds__(256) void kd_glr_clear_kernel(unsigned* ticket, u64* words, int64_t n)
{
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at == 0) *ticket = 0;
    for (int64_t i = at; i < n; i += (int64_t)gridDim.x * 256) words[i] = GLR_EMPTY;
}

// One token of every row: y = h' = f h + i x, with h' kept in fp32.  A launch's
// latency: 2.3 us for 32 x 2048 bf16.
template <class E, bool GATE>
__global__ __launch_bounds__(256) void kd_glr_step_kernel(const E* __restrict__ x, const E* __restrict__ f,
                                                          const E* __restrict__ gi, const float* h_in,
                                                          E* __restrict__ y, float* h_out, int64_t n)
{
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < n; at += (int64_t)gridDim.x * 256) {
        const float u = GATE ? (float)gi[at] * (float)x[at] : (float)x[at];
        const float s = fmaf((float)f[at], h_in[at], u);
        y[at] = (E)s;
        h_out[at] = s;
    }
}

// Workgroups for n elements, which take more than one each beyond 2^30.
static unsigned glr_grid(int64_t n) { return (unsigned)min((int64_t)1 << 22, (n + 255) / 256); }


template <class E>
static hipError_t glr_step(const void* x, const void* f, const void* gi, const float* h_in, void* y, float* h_out,
                           int64_t n, hipStream_t st)
{
    const unsigned grid = glr_grid(n);
    if (gi)
        kd_glr_step_kernel<E, true><<<grid, 256, 0, st>>>((const E*)x, (const E*)f, (const E*)gi, h_in, (E*)y, h_out, n);
    else
        kd_glr_step_kernel<E, false><<<grid, 256, 0, st>>>((const E*)x, (const E*)f, nullptr, h_in, (E*)y, h_out, n);
    return hipGetLastError();
}

static int64_t glr_words(int B, int T, int D) { return ((int64_t)T + GLR_CHUNK - 1) / GLR_CHUNK * B * D; }

// The counter and two words per tile and channel; nothing where a sequence is one tile.
size_t glr_workspace_bytes(int, int B, int T, int D) {
    return T <= GLR_CHUNK ? 0 : 256 + 2 * sizeof(u64) * (size_t)glr_words(B, T, D);
}

// Four adjacent channels per thread where a row's length keeps them aligned,
// one otherwise.
static int glr_vec(int D) { return D % 4 == 0 ? 4 : 1; }
static int glr_lanes(int D) { return D % 4 == 0 ? 32 : 64; }
static int64_t glr_tiles(int B, int T, int D) {
    const int cw = glr_vec(D) * glr_lanes(D);
    return ((int64_t)D + cw - 1) / cw * B * max((int64_t)1, ((int64_t)T + GLR_CHUNK - 1) / GLR_CHUNK);
}
// (with D, T <= 2^30 and B <= 65535 their number stays below 2^63)
bool glr_fits(int B, int T, int D) { return T == 0 || grid_fits(glr_tiles(B, T, D), GLR_NT); }

template <class E, bool GATE, int VEC, int LANES>
static hipError_t glr_run(GlrArgs p, bool bwd, void* ws, hipStream_t st)
{
    const int64_t tiles = glr_tiles(p.B, p.T, p.D);
    if (p.T > GLR_CHUNK) {
        const int64_t n = glr_words(p.B, p.T, p.D);
        p.ticket = (unsigned*)ws;
        p.agg = (u64*)((char*)ws + 256);
        p.inc = p.agg + n;
        kd_glr_clear_kernel<<<(unsigned)min((int64_t)1024, (2 * n + 255) / 256), 256, 0, st>>>(p.ticket, p.agg, 2 * n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (bwd) kd_glr_bwd_kernel<E, GATE, VEC, LANES><<<(unsigned)tiles, GLR_NT, 0, st>>>(p);
    else kd_glr_fwd_kernel<E, GATE, VEC, LANES><<<(unsigned)tiles, GLR_NT, 0, st>>>(p);
    return hipGetLastError();
}

template <class E>
static hipError_t glr_any(const GlrArgs& p, bool bwd, void* ws, hipStream_t st)
{
    if (glr_vec(p.D) == 4) return p.i ? glr_run<E, true, 4, 32>(p, bwd, ws, st) : glr_run<E, false, 4, 32>(p, bwd, ws, st);
    return p.i ? glr_run<E, true, 1, 64>(p, bwd, ws, st) : glr_run<E, false, 1, 64>(p, bwd, ws, st);
}

// T = 0: the state passes through
__global__ __launch_bounds__(256) void kd_glr_pass_kernel(const float* from, float* to, int64_t n)
{
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < n; at += (int64_t)gridDim.x * 256)
        to[at] = from ? from[at] : 0.f;
}
static hipError_t glr_pass(const float* from, float* to, int B, int D, hipStream_t st)
{
    const int64_t n = (int64_t)B * D;
    kd_glr_pass_kernel<<<glr_grid(n), 256, 0, st>>>(from, to, n);
    return hipGetLastError();
}

hipError_t launch_glr_fwd(int bf16, const void* x, const void* f, const void* gi, const float* h0, void* h, float* hT,
                          float* hs, void* ws, int B, int T, int D, hipStream_t st)
{
    if (T == 0) return glr_pass(h0, hT, B, D, st);
    GlrArgs p = {};
    p.x = x;
    p.f = f;
    p.i = gi;
    p.h0 = h0;
    p.h = h;
    p.hT = hT;
    p.hs = hs;
    p.B = B;
    p.T = T;
    p.D = D;
    return bf16 ? glr_any<__bf16>(p, false, ws, st) : glr_any<float>(p, false, ws, st);
}

hipError_t launch_glr_bwd(int bf16, const void* x, const void* f, const void* gi, const float* hs, const void* dh,
                          const float* dhT, void* dx, void* df, void* di, float* dh0, void* ws, int B, int T, int D,
                          hipStream_t st)
{
    if (T == 0) return glr_pass(dhT, dh0, B, D, st);
    GlrArgs p = {};
    p.x = x;
    p.f = f;
    p.i = gi;
    p.hs_in = hs;
    p.dh = dh;
    p.dhT = dhT;
    p.dx = dx;
    p.df = df;
    p.di = di;
    p.dh0 = dh0;
    p.B = B;
    p.T = T;
    p.D = D;
    return bf16 ? glr_any<__bf16>(p, true, ws, st) : glr_any<float>(p, true, ws, st);
}

hipError_t launch_glr_step(int bf16, const void* x, const void* f, const void* gi, const float* h_in, void* y,
                           float* h_out, int64_t n, hipStream_t st)
{
    return bf16 ? glr_step<__bf16>(x, f, gi, h_in, y, h_out, n, st) : glr_step<float>(x, f, gi, h_in, y, h_out, n, st);
}

}  // namespace kd
