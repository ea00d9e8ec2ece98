// kd_gdr.h -- building blocks of the gated delta rule, gfx950.
//
// Per value head the state is S [dv x dk] and for every token
//     Sb = e^g S;  u = beta (v - Sb k);  S = Sb + u k^T;  o = scale S q.
// Over a chunk of C = 64 tokens, with b the running sum of g inside it and
// Gam_rs = e^(b_r - b_s) for s <= r (never a quotient of two decays):
//     T = tril(beta_r Gam_rs k_r.k_s, -1),  A = (I + T)^-1,  P = scale tril(Gam_rs q_r.k_s)
//     U = A (beta (V - e^b K S0^T)),   O = scale e^b Q S0^T + P U,
//     S_C = e^bC S0 + U^T (e^(bC - b) K).
// A and P do not depend on the state: a first kernel makes them for all chunks
// at once, a second one passes over the chunks with the state in registers.
// The backward pass reads the same A and P, transposed.
// The columns of S^T (values) do not mix: 16 of them are one wave's, and nothing
// goes from group to group.
//
// 16x16x32 products (kd_device.h).  bf16: what is not a rounded input goes through
// as a rounded part and its remainder, 16 bits in all (S, A), and what is added
// to a state as two remainders (U before A and after it; backwards dU, X and
// dO with its factor): with 16 bits of those the last state is off by 3.5e-6 of
// it and the first one's gradient by 2.7e-6, with 24 by 0.7e-6 and 0.6e-6 (what
// 16 bits of S and A leave), for a quarter more products (3% of the passes' time
// with two groups of columns a workgroup, up to a fifth backwards with four).
// P is rounded in o, and keeps its remainder in dU: o is off by 2.2e-3 of 64
// bits, where its own rounding is 1.7e-3, for one product a block less in a wave
// that the next chunk does not wait for but shares a SIMD with one it does.  The
// states and their gradients that the chunks' gradients start from are kept in
// the inputs' type (half the memory and traffic; dq and dk are off by 2.3e-3 to
// 2.5e-3, dg by what is left when it cancels).  fp32: the same fragments through
// eight fp32 products.
#pragma once

#include "kd_device.h"
#include "kd_swa.h"

namespace kd {

constexpr int GDR_C = 64;              // tokens of a chunk
constexpr int GDR_BLOCKS = 6;          // 16 x 32 blocks of a lower triangular 64 x 64 matrix that hold anything
constexpr int GDR_VEC = 7 * 64;        // floats of a chunk's gate factors: beta, beta e^b, e^(bC - b), scale e^b, {e^bC, whether a
                                       // beta is next to 0}, b (base 2) and what its rounding left
constexpr int GDR_MAX_STEP = 1 << 22;  // elements from one token to the next (64 of them in 32-bit offsets)

typedef float floatx8 __attribute__((ext_vector_type(8)));
typedef unsigned uintx4 __attribute__((ext_vector_type(4)));
typedef unsigned uintx2 __attribute__((ext_vector_type(2)));

struct GdrArgs {
    const void *q, *k, *v, *g, *beta;          // g, beta [B, T, Hv]
    int64_t qs[3], ks[3], vs[3];               // strides over batch, token, head
    const float* S0;                           // [B, Hv, dv, dk] or null
    void* o;                                   // [B, T, Hv, dv]
    float* ST;                                 // or null
    void* hs;                                  // states entering every chunk [slots, Hv, dv, dk], or null
    // backward
    const void* dO;
    const float* dST;
    void *dq, *dk_, *dv_, *dg, *dbeta;
    float* dS0;
    void *ds, *x, *x2;                         // dS leaving every chunk [slots, Hv, dv, dk], X [slots, Hv, 64, dv] (x2: its remainder)
    // workspace (kept from the forward for the backward)
    void* rec;                                 // the chunks' records: P and A in blocks, then gate factors
    const int* cu;
    int B, T, Hk, Hv, dk, dv;                  // packed: B sequences in T rows
    int slots, gates32;
    float scale;
    // long sequences in segments of `seg` chunks, `nseg` a sequence (packed: kd_gdr_fwd.hip), `segs` in all
    int seg, nseg, segs;
    float *SI, *M;                             // states entering segments [segs, Hv, dv, dk], their maps [segs, Hv, dk, dk]
};

// What a chunk slot holds.  Batched: chunk slot % NC of batch element slot / NC.
// Packed: sequence s owns the slots cu[s] / 64 + s onwards (kd_swa.h).
struct GdrChunk {
    int seq, n, first;        // sequence, chunks before this one, first row within batch element / packed rows
    int rows;                 // 1 .. 64
    int64_t base;             // batch element
};
__device__ __forceinline__ int gdr_chunks(int T) { return (T + GDR_C - 1) / GDR_C; }

// First row, rows and first slot of a sequence.
struct GdrSeq {
    int row0, T, slot0;
    int64_t b;
};
__device__ __forceinline__ GdrSeq gdr_seq(const GdrArgs& a, int s) {
    GdrSeq r;
    if (a.cu) {
        r.row0 = min(max(a.cu[s], 0), a.T);
        r.T = min(max(a.cu[s + 1], r.row0), a.T) - r.row0;
        r.slot0 = r.row0 / GDR_C + s;
        r.b = 0;
    } else {
        r.row0 = 0;
        r.T = a.T;
        r.slot0 = s * gdr_chunks(a.T);
        r.b = s;
    }
    return r;
}
// Segment `slot` as a sequence of its own, with its number and whether it is the
// last of its sequence.  Packed: sequence s owns the slots cu[s] / 64 / seg + s
// onwards.  False when the slot holds none (with offsets that are out of order
// also when it comes before its sequence's first).  The whole wave calls it.
struct GdrSegment {
    GdrSeq s;
    int seq, j;
    bool last;
};
__device__ __forceinline__ bool gdr_segment(const GdrArgs& a, int slot, GdrSegment& r) {
    if (!a.cu) {
        r.seq = slot / a.nseg;
        r.j = slot - r.seq * a.nseg;
    } else {
        const int n = wave_count(a.B, [&](int at) { return min(max(a.cu[at], 0), a.T) / GDR_C / a.seg + at <= slot; });
        if (n == 0) return false;
        r.seq = n - 1;
    }
    r.s = gdr_seq(a, r.seq);
    const int NC = gdr_chunks(r.s.T);
    if (a.cu) r.j = slot - (r.s.row0 / GDR_C / a.seg + r.seq);
    const int c0 = r.j * a.seg;
    if (r.j < 0 || (c0 > 0 && c0 >= NC)) return false;
    r.last = NC - c0 <= a.seg;
    r.s.row0 += c0 * GDR_C;
    r.s.T = r.last ? r.s.T - c0 * GDR_C : a.seg * GDR_C;
    r.s.slot0 += c0;
    return true;
}
// The chunk in a slot, false when it holds none (as above).  The whole wave calls it.
__device__ __forceinline__ bool gdr_slot(const GdrArgs& a, int slot, GdrChunk& c) {
    if (!a.cu) {
        const int nc = gdr_chunks(a.T);
        c.seq = slot / nc;
        c.n = slot - c.seq * nc;
    } else {
        const int n = wave_count(a.B, [&](int at) { return min(max(a.cu[at], 0), a.T) / GDR_C + at <= slot; });
        if (n == 0) return false;
        c.seq = n - 1;
    }
    const GdrSeq s = gdr_seq(a, c.seq);
    if (a.cu) c.n = slot - s.slot0;
    c.first = s.row0 + c.n * GDR_C;
    c.rows = min(s.T - c.n * GDR_C, GDR_C);
    c.base = s.b;
    return c.n >= 0 && c.rows > 0;
}

// Block (i, j) of a lower triangular matrix: rows 16 i .., columns 32 j ..;
// blocks (0,0) (1,0) (2,0) (2,1) (3,0) (3,1).  In a block lane l holds row l %
// 16 and columns 16 h + 4 (l / 16) + r at element 4 h + r: the order in which
// two accumulator tiles of 16 rows each are packed.  Its transpose has the
// blocks (0,0) (0,1) (1,0) (1,1) (2,1) (3,1).
__device__ __forceinline__ constexpr int gdr_block(int i, int j) { return i < 2 ? i : 2 * i - 2 + j; }
__device__ __forceinline__ constexpr int gdr_block_t(int i, int j) { return i < 2 ? 2 * i + j : 2 + i; }

template <class E>
struct GdrT;

template <>
struct GdrT<__bf16> {
    typedef bf16x8 Frag;
    static constexpr bool TWO = true;
    static __device__ __forceinline__ floatx4 mma(Frag a, Frag b, floatx4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    // two values in one word, and both again
    static __device__ __forceinline__ unsigned two(float x, float y) {
        return __builtin_bit_cast(unsigned, bf16x2{(__bf16)x, (__bf16)y});
    }
    static __device__ __forceinline__ Frag pack(floatx4 x, floatx4 y) {
        uintx4 u = {two(x[0], x[1]), two(x[2], x[3]), two(y[0], y[1]), two(y[2], y[3])};
        // (for rest(): the compiler would round every value once more instead of shifting it out)
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("" : "+v"(u[i]));
        return __builtin_bit_cast(Frag, u);
    }
    // what the packing rounded away
    static __device__ __forceinline__ Frag rest(floatx4 x, floatx4 y, Frag p) {
        const uintx4 u = __builtin_bit_cast(uintx4, p);
        uintx4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = i < 2 ? x[2 * i] : y[2 * i - 4], b = i < 2 ? x[2 * i + 1] : y[2 * i - 3];
            r[i] = two(a - __uint_as_float(u[i] << 16), b - __uint_as_float(u[i] & 0xffff0000u));
        }
        return __builtin_bit_cast(Frag, r);
    }
    // and what that has left (p and q were rounded from it)
    static __device__ __forceinline__ Frag rest(floatx4 x, floatx4 y, Frag p, Frag q) {
        const uintx4 u = __builtin_bit_cast(uintx4, p), v = __builtin_bit_cast(uintx4, q);
        uintx4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = i < 2 ? x[2 * i] : y[2 * i - 4], b = i < 2 ? x[2 * i + 1] : y[2 * i - 3];
            r[i] = two((a - __uint_as_float(u[i] << 16)) - __uint_as_float(v[i] << 16),
                       (b - __uint_as_float(u[i] & 0xffff0000u)) - __uint_as_float(v[i] & 0xffff0000u));
        }
        return __builtin_bit_cast(Frag, r);
    }
    static __device__ __forceinline__ Frag ld(const __bf16* p) { return *reinterpret_cast<const Frag*>(p); }
    static __device__ __forceinline__ void st(__bf16* p, Frag f) { *reinterpret_cast<Frag*>(p) = f; }
    // natural fragment of a tile's row r: columns 32 ks + 8 g ..
    template <int D>
    static __device__ __forceinline__ Frag ld_row(const __bf16* tile, int r, int ks, int g) {
        return ld(tile + SwaTile<__bf16, D>::off(r, 4 * ks + g));
    }
    // A operand with K = the tile's rows 32 j + {4g .., 16 + 4g ..} and row m =
    // column c0 + 8 (m / 4) + m % 4 (kd_device.h's transposed reads, the named
    // pieces 8 columns apart)
    template <int D>
    static __device__ __forceinline__ Frag ld_col8(const __bf16* tile, int j, int c0, int lane) {
        const int l = lane & 15, r = 32 * j + 4 * (lane >> 4) + (l >> 2), c = c0 + 8 * (l & 3);
        return tr<D>(tile, r, c);
    }
    // rows 16 t + 4 g .. + 3 of column c0 + l16, as an accumulator holds them
    template <int D>
    static __device__ __forceinline__ floatx4 ld_acc(const __bf16* tile, int t, int c0, int lane) {
        typedef SwaTile<__bf16, D> TL;
        typedef __attribute__((__vector_size__(4 * sizeof(short)))) short v4s;
        const int l = lane & 15, r = 16 * t + 4 * (lane >> 4) + (l >> 2), c = c0 + 4 * (l & 3);
        const bf16x4 x = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                        (__attribute__((address_space(3))) v4s*)(tile + TL::off(r, c / 8) + c % 8)));
        return floatx4{(float)x[0], (float)x[1], (float)x[2], (float)x[3]};
    }
    // columns 16 t + l16 of rows 4 g .. + 3 of a tile with rows of S elements
    template <int S>
    static __device__ __forceinline__ floatx4 ld_t4(const __bf16* tile, int t, int lane) {
        typedef __attribute__((__vector_size__(4 * sizeof(short)))) short v4s;
        const int l = lane & 15;
        const bf16x4 x = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                        (__attribute__((address_space(3))) v4s*)(tile + (4 * (lane >> 4) + (l >> 2)) * S + 16 * t + 4 * (l & 3))));
        return floatx4{(float)x[0], (float)x[1], (float)x[2], (float)x[3]};
    }
    // Block (i, j) of a transpose from the blocks of the matrix: lane's s = 16 i + l16, r = 32 j +
    // 16 h + 4 g + e.  Row r's four columns 4 c .. of block (r / 16, i / 2) are
    // the half i % 2 of its lane r % 16 + 16 c.
    static __device__ __forceinline__ Frag ld_at(const __bf16* rec, int i, int j, int lane) {
        typedef __attribute__((__vector_size__(4 * sizeof(short)))) short v4s;
        const int l = lane & 15, at = (4 * (lane >> 4) + (l >> 2) + 16 * (l & 3)) * 8 + 4 * (i & 1);
        s16x4 x = {0, 0, 0, 0}, y;
        if (2 * j >= i)
            x = __builtin_bit_cast(s16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                              (__attribute__((address_space(3))) v4s*)(rec + gdr_block(2 * j, i / 2) * 512 + at)));
        y = __builtin_bit_cast(s16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                          (__attribute__((address_space(3))) v4s*)(rec + gdr_block(2 * j + 1, i / 2) * 512 + at)));
        return __builtin_bit_cast(Frag, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    template <int D>
    static __device__ __forceinline__ Frag tr(const __bf16* tile, int r, int c) {
        typedef SwaTile<__bf16, D> TL;
        typedef __attribute__((__vector_size__(4 * sizeof(short)))) short v4s;
        const __bf16* lo = tile + TL::off(r, c / 8) + c % 8;
        const __bf16* hi = tile + TL::off(r + 16, c / 8) + c % 8;
        const s16x4 x = __builtin_bit_cast(s16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(lo)));
        const s16x4 y = __builtin_bit_cast(s16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(hi)));
        return __builtin_bit_cast(Frag, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

template <>
struct GdrT<float> {
    typedef floatx8 Frag;
    static constexpr bool TWO = false;
    static __device__ __forceinline__ floatx4 mma(Frag a, Frag b, floatx4 c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ Frag pack(floatx4 x, floatx4 y) {
        return Frag{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
    }
    static __device__ __forceinline__ Frag rest(floatx4, floatx4, Frag p) { return p; }
    static __device__ __forceinline__ Frag rest(floatx4, floatx4, Frag p, Frag) { return p; }
    static __device__ __forceinline__ Frag ld(const float* p) {
        const floatx4 x = *reinterpret_cast<const floatx4*>(p), y = *reinterpret_cast<const floatx4*>(p + 4);
        return pack(x, y);
    }
    static __device__ __forceinline__ void st(float* p, Frag f) {
        *reinterpret_cast<floatx4*>(p) = floatx4{f[0], f[1], f[2], f[3]};
        *reinterpret_cast<floatx4*>(p + 4) = floatx4{f[4], f[5], f[6], f[7]};
    }
    template <int D>
    static __device__ __forceinline__ Frag ld_row(const float* tile, int r, int ks, int g) {
        typedef SwaTile<float, D> TL;
        return pack(*reinterpret_cast<const floatx4*>(tile + TL::off(r, 8 * ks + 2 * g)),
                    *reinterpret_cast<const floatx4*>(tile + TL::off(r, 8 * ks + 2 * g + 1)));
    }
    template <int D>
    static __device__ __forceinline__ Frag ld_col8(const float* tile, int j, int c0, int lane) {
        const int m = lane & 15;
        return at<D>(tile, j, c0 + 8 * (m >> 2) + (m & 3), lane);
    }
    template <int D>
    static __device__ __forceinline__ floatx4 ld_acc(const float* tile, int t, int c0, int lane) {
        typedef SwaTile<float, D> TL;
        const int c = c0 + (lane & 15), r = 16 * t + 4 * (lane >> 4);
        floatx4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = tile[TL::off(r + e, c / 4) + c % 4];
        return x;
    }
    template <int S>
    static __device__ __forceinline__ floatx4 ld_t4(const float* tile, int t, int lane) {
        floatx4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = tile[(4 * (lane >> 4) + e) * S + 16 * t + (lane & 15)];
        return x;
    }
    static __device__ __forceinline__ Frag ld_at(const float* rec, int i, int j, int lane) {
        const int l = lane & 15;
        Frag f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int t = 2 * j + e / 4;      // r's tile
            f[e] = t >= i ? rec[gdr_block(t, i / 2) * 512 + (4 * (lane >> 4) + e % 4 + 16 * (l >> 2)) * 8 + 4 * (i & 1) + (l & 3)] : 0.f;
        }
        return f;
    }
    template <int D>
    static __device__ __forceinline__ Frag at(const float* tile, int j, int c, int lane) {
        typedef SwaTile<float, D> TL;
        const int r = 32 * j + 4 * (lane >> 4);
        Frag f;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = tile[TL::off(r + (e & 3) + 4 * (e & 4), c / 4) + c % 4];
        return f;
    }
};

// x y where x is a packed tile with its remainder and y exact in the type
template <class E>
__device__ __forceinline__ floatx4 gdr_mma2(typename GdrT<E>::Frag a, typename GdrT<E>::Frag a2, typename GdrT<E>::Frag b, floatx4 c) {
    c = GdrT<E>::mma(a, b, c);
    if (GdrT<E>::TWO) c = GdrT<E>::mma(a2, b, c);
    return c;
}
template <class E>
__host__ __device__ constexpr int gdr_part() { return GDR_BLOCKS * 512; }      // elements of a part
// A record: P and A, then the gate factors.  In bf16 both have a remainder, P's
// in front (only the backward pass reads it, and only its forward writes it).
// Each pass reads from its first part on: the backward pass all, the forward
// pass from P, the segments' maps from A.
template <class E>
__host__ __device__ constexpr int gdr_parts() { return sizeof(E) == 2 ? 4 : 2; }
template <class E>
__host__ __device__ constexpr int64_t gdr_rec_bytes() { return (int64_t)gdr_parts<E>() * gdr_part<E>() * (int)sizeof(E) + GDR_VEC * 4; }

// Stages 64 rows of K or Q in an LDS tile, from `row` on (past the sequence's
// last they repeat it); columns past dk keep what the tile holds (zeros).  The
// addresses are a scalar base and one 32-bit offset per lane that all chunks
// share.
template <class E, int DK, int NT>
struct GdrFetch {
    typedef SwaTile<E, DK> TL;
    static constexpr int STEP = NT / TL::CPR, NL = 64 / STEP;
    static_assert(64 % STEP == 0, "whole rounds");
    const E* base;
    int64_t rs;
    int rows, dk, r, ch;
    uint32_t lane[NL];
    bool plain;      // all columns there
    __device__ __forceinline__ GdrFetch(const E* base_, int64_t rs_, int rows_, int dk_, int tid)
        : base((const E*)swa_uniform((int64_t)base_)), rs(swa_uniform(rs_)), rows(__builtin_amdgcn_readfirstlane(rows_)), dk(dk_) {
        r = tid / TL::CPR;
        ch = tid % TL::CPR;
        plain = dk == DK;
#pragma unroll
        for (int i = 0; i < NL; ++i)
            lane[i] = (uint32_t)(((r + i * STEP) * (int)rs + (ch ^ TL::swz(r + i * STEP)) * TL::EPC) * (int)sizeof(E));
    }
    __device__ __forceinline__ void operator()(E* tile, int row, int w) const {
        const int row0 = __builtin_amdgcn_readfirstlane(row);
        const uint32_t to = lds_address(tile) + 1024 * w;
        const E* b = base + (int64_t)row0 * rs;
        if (row0 + 64 <= rows && plain) {
#pragma unroll
            for (int i = 0; i < NL; ++i)
                asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(lane[i]),
                             "s"(swa_uniform((int64_t)b)), "i"(i * NT * 16)
                             : "memory", "m0", "scc");
        } else {
            const int last = rows - 1 - row0;
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int rr = r + i * STEP, x = (ch ^ TL::swz(rr)) * TL::EPC;
                if (x < dk) load_lds16(to + i * NT * 16, b + (int64_t)min(rr, last) * rs + x);
            }
        }
    }
};

// Two groups of 16 value columns a workgroup instead of four, while that leaves
// no more workgroups than compute units: both waves of a group have a SIMD for
// themselves then (with 128 workgroups of four, sequences of 2048 tokens: heads of
// 128 x 128 87 us for 97, backwards 113 for 150; of 64 x 64 63 for 68 and 95 for
// 119).  From there on four (heads of 64 x 64, 144 of four: 71 us for 87, backwards
// 124 for 163; 192: 87 for 105 and 130 for 174; 128 x 128, 192: 101 for 139 and 162
// for 196).  For packed sequences a little later: the short ones' compute units
// come free.  Lengths are known on the device alone, so a packed call is taken to
// be ragged (8191 tokens in 13 sequences of 12 heads, 64 x 64, the longest 3.4
// times the average, 156 of four: 57 us for 67, backwards 73 for 118; eight others
// with 144 to 192, the longest 2.3 to 3.9 times the average: 8 to 19% less,
// backwards 24 to 37%).  Packed sequences of equal length lose by it what batched
// ones would (192, 64 x 64: 103 us for 88, backwards 173 for 131), nearly equal
// ones less (the longest 1.6 times the average, 128 x 128: 56 for 44 and 70 for
// 64).
__host__ __forceinline__ bool gdr_narrow(const GdrArgs& a, int segs) {
    return (int64_t)segs * a.Hv * ((a.dv + 63) / 64) <= (a.cu ? 192 : 128);
}

// What a pass reads of a chunk beside K and Q: the last PARTS parts of its record,
// the gate factors, and C columns of V (or dO).  The workgroup's NT threads load
// it to registers a chunk ahead and put it in LDS when the chunk before is done.
template <class E, int PARTS, int C>
struct GdrSide {
    static constexpr int REC = PARTS * gdr_part<E>();      // elements
    static constexpr int PIECES = (REC * (int)sizeof(E) + GDR_VEC * 4) / 16;
    static constexpr int SKIP = (gdr_parts<E>() - PARTS) * gdr_part<E>() * (int)sizeof(E);      // bytes
    E rec[REC];
    float vec[GDR_VEC];
    E v[64 * C];
};

// Rows of a matrix at a wave-uniform address as a buffer: what lies past its
// bytes reads as zero and is not written, so the ends of a sequence and of a
// head's columns need no branch.  GDR_NONE: an offset past any of them.
constexpr int GDR_NONE = 0x7ffffff0;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t gdr_buffer(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)swa_uniform((int64_t)p), 0,
                                             __builtin_amdgcn_readfirstlane((int)(bytes < 0 ? 0 : bytes)), 0x00027000);
}
__device__ __forceinline__ floatx4 gdr_load(__amdgpu_buffer_rsrc_t r, int at) {
    return __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
}
// four elements
__device__ __forceinline__ void gdr_store(__amdgpu_buffer_rsrc_t r, int at, floatx4 x, const __bf16*) {
    const bf16x4 y = {(__bf16)x[0], (__bf16)x[1], (__bf16)x[2], (__bf16)x[3]};
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(uintx2, y), r, at, 0, 0);
}
__device__ __forceinline__ void gdr_store(__amdgpu_buffer_rsrc_t r, int at, floatx4 x, const float*) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(uintx4, x), r, at, 0, 0);
}
// eight elements
__device__ __forceinline__ void gdr_store(__amdgpu_buffer_rsrc_t r, int at, bf16x8 x) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(uintx4, x), r, at, 0, 0);
}
__device__ __forceinline__ void gdr_store(__amdgpu_buffer_rsrc_t r, int at, floatx8 x) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(uintx4, floatx4{x[0], x[1], x[2], x[3]}), r, at, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(uintx4, floatx4{x[4], x[5], x[6], x[7]}), r, at + 16, 0, 0);
}

template <class E, int PARTS, int C, int NT>
struct GdrSideAhead {
    typedef SwaTile<E, C> TV;
    typedef GdrSide<E, PARTS, C> Side;
    static constexpr int N = (Side::PIECES + NT - 1) / NT, M = 64 * TV::CPR / NT, STEP = NT / TV::CPR;
    floatx4 x[N], v[M];
    const E* vb;
    int64_t vs;
    int T, cols, at;
    // rows of v: C columns from vb on, of which `cols` are there
    __device__ __forceinline__ GdrSideAhead(const E* vb_, int64_t vs_, int cols_, int T_, int tid) : vb(vb_), vs(vs_), T(T_), cols(cols_) {
        const int c = tid % TV::CPR * TV::EPC;
        at = c < cols ? (int)((tid / TV::CPR * vs + c) * (int)sizeof(E)) : GDR_NONE;
    }
    // a chunk's record from `rec` on
    __device__ __forceinline__ void load(const char* rec, int tid) {
        const auto r = gdr_buffer(rec + Side::SKIP, Side::PIECES * 16);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = gdr_load(r, (i * NT + tid) * 16);
    }
    // rows `row` .. of v
    __device__ __forceinline__ void load_v(int row) {
        const auto r = gdr_buffer(vb + row * vs, ((min(T - row, 64) - 1) * vs + min(cols, C)) * (int)sizeof(E));
#pragma unroll
        for (int i = 0; i < M; ++i) v[i] = gdr_load(r, at + (at == GDR_NONE ? 0 : (int)(i * STEP * vs * (int)sizeof(E))));
    }
    __device__ __forceinline__ void store(Side& s, int tid) const {
#pragma unroll
        for (int i = 0; i < N; ++i)      // (vec follows rec)
            if (i < N - 1 || (N - 1) * NT + tid < Side::PIECES) reinterpret_cast<floatx4*>(s.rec)[i * NT + tid] = x[i];
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const int to = i * NT + tid;
            *reinterpret_cast<floatx4*>(s.v + TV::off(to / TV::CPR, to % TV::CPR)) = v[i];
        }
    }
};

__device__ __forceinline__ float gdr_gate(const void* p, int64_t i, int gates32, const __bf16*) {
    return gates32 ? ((const float*)p)[i] : (float)((const __bf16*)p)[i];
}
__device__ __forceinline__ float gdr_gate(const void* p, int64_t i, int, const float*) { return ((const float*)p)[i]; }

// Running sum of the log decays (base 2) over the wave's 64 lanes, in 64 bits: decays
// between two tokens are exp of a difference, which far sums would spoil.  Log
// decays below -120 are e^-120 = 0 in fp32, and -infinity among them would
// make NaNs of differences.
__device__ __forceinline__ double gdr_cumsum(float g, int lane) {
    double b = (double)(g < -120.f ? -120.f : g) * 1.4426950408889634;
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
        const double x = __shfl_up(b, s);
        if (lane >= s) b += x;
    }
    return b;
}

}  // namespace kd
