// kd_swa.h -- building blocks of the sliding-window attention kernels, gfx950.
//
// A query at position p sees the keys s <= p with p - s < W (the window) or
// s < S (the sinks).  All products run on 32x32 MFMA tiles (wave64):
//   * A operand: lane l holds row l % 32, B operand: lane l holds column
//     l % 32; lane group g = l / 32 holds its share of K, one 16-byte fragment
//     (8 bf16 or 4 fp32 values) per step;
//   * C/D: lane l holds column l % 32, rows 8 (r / 4) + 4 g + r % 4, r < 16.
// The order of K in a product is free as long as A and B agree.  So a tile of
// weights that a product left as an accumulator (rows = the next product's K)
// is that product's B operand after packing, with no trip through LDS; its A
// operand is read with the same K order (ld_col).
#pragma once

#include "kd_device.h"

namespace kd {

typedef float floatx16 __attribute__((ext_vector_type(16)));

constexpr int SWA_MAX_SINKS = 64;   // KRON_DELTA_SWA_MAX_SINKS

struct SwaArgs {
    const void *q, *k, *v;
    int64_t qs[3], ks[3], vs[3];       // strides over batch, token, head (elements)
    void* o;                           // [B, Tq, Hq, d]
    float* lse;                        // [B, Hq, Tq] or null
    const void* dO;                    // [B, Tq, Hq, d]
    float2* rows;                      // [B, Hq, Tq]: lse log2(e) and delta of every query
    float* part;                       // partial dK, dV of the sinks: [B, pslots, Hq, 2, S, d]
    int pslots, chunk;                 // query chunks of the sinks' pass (0: none), their rows
    int apart;                         // packed: rows by which that pass numbers its sequences (0: one by one)
    float* shared;                     // parts of dK, dV of the workgroups that share a group's heads
    int nsp;                           // how many do
    void *dq, *dk, *dv;                // contiguous
    const int* cu;                     // packed: N + 1 offsets into the Tq == Tk rows
    int B, N, Tq, Tk, Hq, Hkv;
    int W, S;
    float scale, c;                    // c = scale log2(e)
};

// Row-major LDS tile of D columns, 16-byte chunks permuted within each row so
// that both a read of one chunk of 16 consecutive rows (ld_row) and the
// transpose read of 4 + 4 rows (ld_col) spread over all 64 banks.
template <class E, int D>
struct SwaTile {
    static constexpr int EPC = 16 / sizeof(E);    // elements per chunk
    static constexpr int CPR = D / EPC;           // chunks per row
    static __device__ __forceinline__ int swz(int r) {
        if constexpr (CPR == 4) return (r >> 2) & 3;
        if constexpr (CPR == 8) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
        if constexpr (CPR == 16) return ((r & 3) << 2) | ((r >> 2) & 3);
        return ((r & 7) << 1) | ((r >> 3) & 1);
    }
    static __device__ __forceinline__ int off(int r, int chunk) { return r * D + ((chunk ^ swz(r)) * EPC); }
};

template <class E>
struct SwaT;

template <>
struct SwaT<__bf16> {
    typedef __bf16 E;
    typedef bf16x8 Frag;
    static constexpr int KC = 16;    // K per step: one MFMA
    static constexpr int PR = 8;     // accumulator rows (registers) per packed fragment
    static __device__ __forceinline__ floatx16 mma(Frag a, Frag b, floatx16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    // registers 8j .. 8j + 7 of an accumulator: K = 16j + {4g .. 4g + 3, 8 + 4g .. 8 + 4g + 3}
    static __device__ __forceinline__ Frag pack(const floatx16& p, int j) {
        Frag r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = (__bf16)p[8 * j + e];
        return r;
    }
    // what the packing of fragment j rounded away
    static __device__ __forceinline__ Frag rest(const floatx16& p, int j, Frag x) {
        Frag r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = (__bf16)(p[8 * j + e] - (float)x[e]);
        return r;
    }
    // A operand of rows d = c0 + l % 32 with that K order, from the tile's
    // columns: two transpose reads of four rows each (ds_read_b64_tr_b16: in
    // each 16-lane block lane j names four elements of row j / 4 and receives
    // column j of the four rows)
    template <int D>
    static __device__ __forceinline__ Frag ld_col(const E* tile, int row0, int c0, int lane) {
        typedef SwaTile<E, D> TL;
        typedef __attribute__((__vector_size__(4 * sizeof(short)))) short v4s;
        const int j = lane & 15, col = c0 + 16 * ((lane >> 4) & 1) + 4 * (j & 3);
        const int r = row0 + 4 * (lane >> 5) + (j >> 2);
        const E* lo = tile + TL::off(r, col / TL::EPC) + (col % TL::EPC);
        const E* hi = tile + TL::off(r + 8, col / TL::EPC) + (col % TL::EPC);
        const s16x4 a = __builtin_bit_cast(s16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                      (__attribute__((address_space(3))) v4s*)(lo)));
        const s16x4 b = __builtin_bit_cast(s16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                      (__attribute__((address_space(3))) v4s*)(hi)));
        return __builtin_bit_cast(Frag, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    static __device__ __forceinline__ float dot(Frag a, Frag b) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf((float)a[e], (float)b[e], s);
        return s;
    }
};

template <>
struct SwaT<float> {
    typedef float E;
    typedef floatx4 Frag;
    static constexpr int KC = 8;     // K per step: four MFMAs, K = 4g + i in the i-th
    static constexpr int PR = 4;
    static __device__ __forceinline__ floatx16 mma(Frag a, Frag b, floatx16 c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ Frag pack(const floatx16& p, int j) {
        return Frag{p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]};
    }
    static __device__ __forceinline__ Frag rest(const floatx16&, int, Frag) { return Frag{0.f, 0.f, 0.f, 0.f}; }
    template <int D>
    static __device__ __forceinline__ Frag ld_col(const E* tile, int row0, int c0, int lane) {
        typedef SwaTile<E, D> TL;
        const int d = c0 + (lane & 31), r = row0 + 4 * (lane >> 5);
        Frag x;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = tile[TL::off(r + i, d / TL::EPC) + d % TL::EPC];
        return x;
    }
    static __device__ __forceinline__ float dot(Frag a, Frag b) {
        return fmaf(a[0], b[0], fmaf(a[1], b[1], fmaf(a[2], b[2], a[3] * b[3])));
    }
};

// fragment ks of row r: its chunk 2 ks + g
template <class E, int D>
__device__ __forceinline__ typename SwaT<E>::Frag swa_ld_row(const E* tile, int r, int ks, int g) {
    return *reinterpret_cast<const typename SwaT<E>::Frag*>(tile + SwaTile<E, D>::off(r, 2 * ks + g));
}
// the same from a row in memory
template <class E>
__device__ __forceinline__ typename SwaT<E>::Frag swa_ld_mem(const E* row, int ks, int g) {
    return *reinterpret_cast<const typename SwaT<E>::Frag*>(row + (2 * ks + g) * (16 / (int)sizeof(E)));
}
// and ld_col's fragment of rows row0 .. from a column in memory (row stride rs)
template <class E>
__device__ __forceinline__ typename SwaT<E>::Frag swa_ld_col_mem(const E* col, int64_t rs, int64_t row0, int g) {
    typename SwaT<E>::Frag x;
#pragma unroll
    for (int e = 0; e < SwaT<E>::PR; ++e) x[e] = col[(row0 + 4 * g + (e & 3) + 2 * (e & 4)) * rs];
    return x;
}
template <class E>
__device__ __forceinline__ typename SwaT<E>::Frag swa_zero() {
    typename SwaT<E>::Frag z;
#pragma unroll
    for (int e = 0; e < (int)(16 / sizeof(E)); ++e) z[e] = (E)0.f;
    return z;
}

// the other lane group's value of the same column
__device__ __forceinline__ float swa_swap(float x) { return __shfl_xor(x, 32); }

// Sequence and block of a workgroup.  Batched: row block `slot` of batch
// element b.  Packed: sequence s owns the slots cu[s] / R + s onwards (at
// least as many as its blocks of R rows, and no two sequences share one), so
// the grid needs T / R + N slots and no table.  Where only sequences of at
// least `apart` rows have work, cu[s] / R + cu[s] / apart serves them as well
// (one that starts after such a sequence starts at least `apart` rows later):
// T / R + T / apart slots, however many short sequences there are.  Offsets
// are clamped into [0, T].  Returns false when the slot holds no rows.
struct SwaSeq {
    int q0, nq, nk, past, blk;   // first row, rows, keys, position of row 0, block of R rows
    int slot0;                   // the sequence's first chunk of the sinks' pass
};
__device__ __forceinline__ int swa_first_slot(int row, int seq, int R, int apart) {
    return row / R + (apart > 0 ? row / apart : seq);
}
__device__ __forceinline__ bool swa_locate(const SwaArgs& a, int slot, int R, bool keys, SwaSeq& s, int apart = 0) {
    if (!a.cu) {
        s.q0 = 0;
        s.nq = a.Tq;
        s.nk = a.Tk;
        s.past = a.Tk - a.Tq;
        s.blk = slot;
        s.slot0 = 0;
        return (int64_t)slot * R < (keys ? s.nk : s.nq);
    }
    const int lane = threadIdx.x & 63;
    int n = 0;   // sequences that start at or before the slot
    for (int i = 0; i < a.N; i += 64) {
        const int at = i + lane;
        const bool in = at < a.N && swa_first_slot(min(max(a.cu[min(at, a.N)], 0), a.Tq), at, R, apart) <= slot;
        n += __popcll(__ballot(in));
    }
    if (n == 0) return false;
    const int q = n - 1;
    const int lo = min(max(a.cu[q], 0), a.Tq), hi = min(max(a.cu[q + 1], lo), a.Tq);
    s.q0 = lo;
    s.nq = s.nk = hi - lo;
    s.past = 0;
    s.blk = slot - swa_first_slot(lo, q, R, apart);
    s.slot0 = a.chunk > 0 ? swa_first_slot(lo, q, a.chunk, a.apart) : 0;
    return s.blk >= 0 && (int64_t)s.blk * R < s.nq;
}

// Whether a query at position pos sees one key or none.  The softmax of one
// score is 1 whatever the score, so nothing behind it has a gradient there:
// P (dP - delta) would be what the roundings of P and delta leave.
__device__ __forceinline__ bool swa_alone(int pos, int W, int S) { return pos <= 0 || W + S == 1; }

// Masks of a 32x32 tile whose lane holds one query at position pos and 16 of
// the keys from k0 on (key0 = k0 + 4 g; register r is key0 + 8 (r / 4) + r % 4):
// compares of constants with three numbers per lane.
__device__ __forceinline__ void swa_mask_keys(floatx16& x, int key0, int pos, int W, int S) {
    const int hi = pos - key0, lo = hi - W;
    if (key0 - (key0 & 4) >= S) {      // no sinks among the keys (one answer for the wave)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int i = 8 * (r / 4) + r % 4;
            if (!((i <= hi) & (i > lo))) x[r] = -INFINITY;
        }
    } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int i = 8 * (r / 4) + r % 4;
            if (!((i <= hi) & ((i > lo) | (i < S - key0)))) x[r] = -INFINITY;
        }
    }
}
// The same where the lane holds one key and 16 of the queries at positions p0
// on (p0 with 4 g added), of which the first `left` (less 4 g) count.
__device__ __forceinline__ void swa_mask_rows(floatx16& x, int key, int p0, int left, int W, int S) {
    const int lo = key - p0, hi = min(left, key < S ? left : lo + W);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int i = 8 * (r / 4) + r % 4;
        if (!((i >= lo) & (i < hi))) x[r] = -INFINITY;
    }
}

// Tiles of R rows of a matrix (row stride rs elements, `rows` rows) by loads
// that go straight to LDS: a wave's lane i fills the 16 bytes at its base + 16 i,
// so the chunk order within a row is set by which chunk each lane reads.  The
// addresses are a scalar base and one 32-bit offset per lane that all tiles
// share; a last tile with rows past the end repeats the last row (its keys are
// masked for every query).  The loads are in flight until swa_landed(); they
// are written out because the compiler would make every LDS read wait for a
// builtin's loads, those of the other buffer too.  Destinations lie in the
// first 64 KB of LDS.
__device__ __forceinline__ int64_t swa_uniform(int64_t x) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)x), hi = __builtin_amdgcn_readfirstlane((int)(x >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}
template <class E, int D, int R, int NT>
struct SwaFetch {
    typedef SwaTile<E, D> TL;
    static constexpr int STEP = NT / TL::CPR;              // rows per round of the workgroup
    static constexpr int NL = R / STEP;                    // loads of a tile per lane
    static_assert(R % STEP == 0, "whole instructions");
    const E* base;
    int64_t rs;
    int rows, r, ch;
    uint32_t lane[NL];
    bool far;

    __device__ __forceinline__ SwaFetch(const E* base_, int64_t rs_, int rows_, int tid)
        : base((const E*)swa_uniform((int64_t)base_)), rs(swa_uniform(rs_)), rows(__builtin_amdgcn_readfirstlane(rows_)) {
        r = tid / TL::CPR;
        ch = tid % TL::CPR;
        far = rs > (1 << 22);      // rows too far apart for 32-bit offsets
#pragma unroll
        for (int i = 0; i < NL; ++i)
            lane[i] = (uint32_t)(((r + i * STEP) * (int)rs + (ch ^ TL::swz(r + i * STEP)) * TL::EPC) * (int)sizeof(E));
    }
    // rows row0 .. into `tile`, from `ho` elements on (a head), as wave w of the workgroup
    __device__ __forceinline__ void operator()(E* tile, int64_t ho, int row, int w) const {
        const int row0 = __builtin_amdgcn_readfirstlane(row);
        const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)tile + 1024 * w;
        const E* b = base + swa_uniform(ho) + (int64_t)row0 * rs;
        if (row0 + R <= rows && !far) {
#pragma unroll
            for (int i = 0; i < NL; ++i)
                asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at), "v"(lane[i]),
                             "s"(swa_uniform((int64_t)b)), "i"(i * NT * 16)
                             : "memory", "m0", "scc");
        } else {
            // the last tile's rows; each lane's address in full
            const int last = rows - 1 - row0;
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int rr = r + i * STEP;
                const E* src = b + (int64_t)min(rr, last) * rs + (ch ^ TL::swz(rr)) * TL::EPC;
                asm volatile("s_add_u32 m0, %0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(src),
                             "i"(i * NT * 16)
                             : "memory", "m0", "scc");
            }
        }
    }
};
// all loads of this wave have landed, then all waves of the workgroup are here
__device__ __forceinline__ void swa_landed() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Work item of a workgroup: runs of 16 items go to one XCD (workgroups go
// round the 8 XCDs one by one), so that the heads of a group and neighbouring
// blocks, which read the same keys, share an L2.  False past the end.
__device__ __forceinline__ bool swa_item(int64_t n, int64_t& item) {
    const int64_t id = blockIdx.x, run = id >> 3;
    item = (run >> 4) * 128 + (id & 7) * 16 + (run & 15);
    return item < n;
}
__host__ __device__ inline int64_t swa_grid(int64_t n) { return (n + 127) / 128 * 128; }
// Slots of R rows (see swa_locate).
inline int64_t swa_slots(bool packed, int N, int T, int R) { return packed ? (int64_t)T / R + N : ((int64_t)T + R - 1) / R; }

// Waits for a loaded fragment here rather than at its first use inside a loop
// (where the wait would cover the loop's own loads).
template <class F>
__device__ __forceinline__ void swa_arrive(F& f) {
    floatx4 r = __builtin_bit_cast(floatx4, f);
    asm volatile("" : "+v"(r));
    f = __builtin_bit_cast(F, r);
}

// column q of an accumulator stack (rows = the D head elements) to a row in memory
template <class E, int D>
__device__ __forceinline__ void swa_store_row(E* row, const floatx16* acc, float f, int g) {
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            typedef E E4 __attribute__((ext_vector_type(4)));
            E4 x;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = (E)(acc[dt][4 * j + e] * f);
            *reinterpret_cast<E4*>(row + 32 * dt + 8 * j + 4 * g) = x;
        }
}

}  // namespace kd
