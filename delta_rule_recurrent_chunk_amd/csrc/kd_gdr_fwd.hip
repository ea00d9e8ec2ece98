// kd_gdr_fwd.hip -- gated delta rule: the chunks' matrices (forward and
// backward) and the forward pass over the chunks, gfx950.  The formulas are in
// kd_gdr.h.
#include "kd_check.h"
#include "kd_gdr.h"

namespace kd {

// One wave per chunk and value head: T, A = (I + T)^-1 and P of 64 tokens.
// K K^T and Q K^T take 16-row fragments straight from memory.  A by blocks of
// 16: the four diagonal blocks by substitution, one column a lane; then row by
// row of blocks A_ij = -A_ii sum_k T_ik A_kj in fp32 products, in place of T.
// SAVE (for a backward pass): P's remainder too.  Bound by memory: 8 sequences
// of 2048 tokens, 16 heads of 128, bf16: 54 us for 134 MB of keys and queries
// and 89 MB of records (4.1 TB/s; a large copy reaches 4.9).
template <class E, int DK, bool SAVE>
__global__ __launch_bounds__(64, 1) void kd_gdr_prep_kernel(GdrArgs a)
{
    typedef GdrT<E> T;
    typedef typename T::Frag Frag;
    constexpr int NK = DK / 32, LD = 68;
    constexpr int PP2 = 0, PP = T::TWO ? 1 : 0, PA = PP + 1, PA2 = PA + 1;
    __shared__ __align__(16) float M[64 * LD];
    __shared__ __align__(16) float bh[64], bl[64];
    const int lane = threadIdx.x, l16 = lane & 15, g = lane >> 4;
    const int hv = blockIdx.x % a.Hv, slot = blockIdx.x / a.Hv, hk = hv / (a.Hv / a.Hk);
    GdrChunk c;
    if (!gdr_slot(a, slot, c)) return;
    const int64_t gate = (c.base * a.T + c.first + min(lane, c.rows - 1)) * a.Hv + hv;
    const float gl = lane < c.rows ? gdr_gate(a.g, gate, a.gates32, (const E*)nullptr) : 0.f;
    const float beta = lane < c.rows ? gdr_gate(a.beta, gate, a.gates32, (const E*)nullptr) : 0.f;
    Frag k[4][NK], q[4][NK];
    const E* kb = (const E*)a.k + c.base * a.ks[0] + hk * a.ks[2];
    const E* qb = (const E*)a.q + c.base * a.qs[0] + hk * a.qs[2];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int64_t row = c.first + min(16 * t + l16, c.rows - 1);
#pragma unroll
        for (int ks = 0; ks < NK; ++ks) {
            const int col = 32 * ks + 8 * g;
#pragma unroll
            for (int e = 0; e < 8; ++e) k[t][ks][e] = (E)0.f, q[t][ks][e] = (E)0.f;
            if (col < a.dk) {
                k[t][ks] = T::ld(kb + row * a.ks[1] + col);
                q[t][ks] = T::ld(qb + row * a.qs[1] + col);
            }
        }
    }
    const double b = gdr_cumsum(gl, lane);
    const double last = __shfl(b, 63);
    bh[lane] = (float)b;
    bl[lane] = (float)(b - (double)(float)b);
    char* const record = (char*)a.rec + ((int64_t)slot * a.Hv + hv) * gdr_rec_bytes<E>();
    float* vec = (float*)(record + gdr_parts<E>() * gdr_part<E>() * (int)sizeof(E));
    const float eb = __builtin_amdgcn_exp2f((float)b);
    vec[lane] = beta;
    vec[64 + lane] = beta * eb;
    vec[128 + lane] = __builtin_amdgcn_exp2f((float)(last - b));
    vec[192 + lane] = a.scale * eb;
    const bool small = __any(lane < c.rows && fabsf(beta) < 1e-20f);
    if (lane == 0) {
        vec[256] = __builtin_amdgcn_exp2f((float)last);
        vec[257] = small ? 1.f : 0.f;
    }
    vec[320 + lane] = (float)b;
    vec[384 + lane] = (float)(b - (double)(float)b);
    __syncthreads();
    E* rec = (E*)record + lane * 8;
    const floatx4 zero = {0.f, 0.f, 0.f, 0.f};

    // lane: token r of row block i, s = 16 j + 4 g + e
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 16 * i + l16;
        const float rh = bh[r], rl = bl[r], br = __shfl(beta, r);
        floatx4 p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            p[j] = zero;
            if (j > i) continue;
            floatx4 x = zero;
#pragma unroll
            for (int ks = 0; ks < NK; ++ks) x = T::mma(k[j][ks], k[i][ks], x);
#pragma unroll
            for (int ks = 0; ks < NK; ++ks) p[j] = T::mma(k[j][ks], q[i][ks], p[j]);
            const floatx4 sh = *reinterpret_cast<const floatx4*>(bh + 16 * j + 4 * g), sl = *reinterpret_cast<const floatx4*>(bl + 16 * j + 4 * g);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int s = 16 * j + 4 * g + e;
                const float gam = __builtin_amdgcn_exp2f((rh - sh[e]) + (rl - sl[e]));
                x[e] = s < r ? br * gam * x[e] : 0.f;
                p[j][e] = s <= r ? a.scale * gam * p[j][e] : 0.f;
            }
            *reinterpret_cast<floatx4*>(M + r * LD + 16 * j + 4 * g) = x;
        }
#pragma unroll
        for (int j = 0; j <= i / 2; ++j) {
            const Frag f = T::pack(p[2 * j], p[2 * j + 1]);
            T::st(rec + PP * gdr_part<E>() + gdr_block(i, j) * 512, f);
            if (T::TWO && SAVE) T::st(rec + PP2 * gdr_part<E>() + gdr_block(i, j) * 512, T::rest(p[2 * j], p[2 * j + 1], f));
        }
    }
    __syncthreads();
    {
        // column l16 of diagonal block g
        const float* t = M + (16 * g) * LD + 16 * g;
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float sum = r == l16 ? 1.f : 0.f;
#pragma unroll
            for (int s = 0; s < r; s += 4) {
                const floatx4 y = *reinterpret_cast<const floatx4*>(t + r * LD + s);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (s + e < r) sum = fmaf(-y[e], x[s + e], sum);
            }
            x[r] = sum;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 16; ++r) M[(16 * g + r) * LD + 16 * g + l16] = x[r];
    }
    __syncthreads();
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        floatx4 y[3];
#pragma unroll
        for (int j = 0; j < i; ++j) {
            y[j] = zero;
#pragma unroll
            for (int kk = j; kk < i; ++kk) {
                const floatx4 t = *reinterpret_cast<const floatx4*>(M + (16 * i + l16) * LD + 16 * kk + 4 * g);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(t[e], M[(16 * kk + 4 * g + e) * LD + 16 * j + l16], y[j], 0, 0, 0);
            }
        }
        const floatx4 d = *reinterpret_cast<const floatx4*>(M + (16 * i + l16) * LD + 16 * i + 4 * g);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < i; ++j) {
            floatx4 x = zero;
#pragma unroll
            for (int e = 0; e < 4; ++e) x = __builtin_amdgcn_mfma_f32_16x16x4f32(-y[j][e], d[e], x, 0, 0, 0);
            *reinterpret_cast<floatx4*>(M + (16 * i + l16) * LD + 16 * j + 4 * g) = x;
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j <= i / 2; ++j) {
            const float* m = M + (16 * i + l16) * LD + 32 * j + 4 * g;
            const floatx4 x = *reinterpret_cast<const floatx4*>(m);
            const floatx4 y = 2 * j + 1 <= i ? *reinterpret_cast<const floatx4*>(m + 16) : zero;
            const Frag f = T::pack(x, y);
            T::st(rec + PA * gdr_part<E>() + gdr_block(i, j) * 512, f);
            if (T::TWO) T::st(rec + PA2 * gdr_part<E>() + gdr_block(i, j) * 512, T::rest(x, y, f));
        }
}

// The pass, two waves for every 16 value columns.  The first has the
// state in registers and makes what the next chunk waits for: K S, U, the state
// that leaves.  The second makes what nothing waits for, a chunk later, from the
// packed states and U that it finds in LDS: the outputs, all loads and stores.
// K and Q come by loads straight to LDS, two chunks' worth (fp32 with 128 key
// channels: one), A, V and the factors through its registers.
// A workgroup has CG groups of 16 columns: four, two waves to a SIMD, or two with
// a SIMD for each wave (gdr_narrow; fp32, which needs the LDS).
//
// Bound by what a chunk waits for: K S, U, A U and the state's update follow each
// other (four products, a packing of each result, two barriers), 3.0 us a chunk
// where all compute units have a workgroup of four groups: 98 us for the 32
// chunks of the sequences above (3.6 TB/s, matrix units busy in 37% of the
// cycles).  One wave for 16 columns, which made the outputs as well: 133 us; two
// waves that share every product and hand each other halves through LDS: 122 us
// (LDS has twice as much to move).
//
// Few heads and long sequences (gdr_plan): a sequence is cut into segments, all
// of which pass at once.  A segment maps the state that enters it to S M + N.
// GDR_MAPS passes over segments without their outputs, for N (from a zero
// state) and for M (dk columns, from the identity and without values); a small
// kernel chains them; then the pass runs from the states it found.  Without
// outputs there are first waves alone, which load for themselves, in two
// workgroups a compute unit (32768 tokens of 16 heads in 8 segments: 230 us;
// eight waves a workgroup that share K take a quarter longer), and the pass behind
// them 200 us.
enum { GDR_OUT, GDR_SAVE, GDR_MAPS };
template <class E, int DK, int MODE, int CG>
__global__ __launch_bounds__((MODE == GDR_MAPS ? 64 : 128) * CG, CG == 4 ? 2 : 1) void kd_gdr_pass_kernel(GdrArgs a, int run)
{
    typedef GdrT<E> T;
    typedef typename T::Frag Frag;
    constexpr int NT = 64 * CG, NC0 = 16 * CG, W = T::TWO ? 2 : 1;      // (columns of a workgroup)
    constexpr int NK = DK / 32, NBUF = sizeof(E) * DK > 256 ? 1 : 2;
    constexpr bool OUT = MODE != GDR_MAPS;
    __shared__ __align__(16) struct {
        E k[NBUF][64 * DK], q[OUT ? NBUF : 1][OUT ? 64 * DK : 8];
        GdrSide<E, W, NC0> side[OUT ? 1 : 2];
        E p[2][OUT ? gdr_part<E>() : 8];
        E s[OUT ? CG * NK * W * 512 : 8], u[OUT ? CG * 2 * W * 512 : 8];      // fragments for the second wave
    } sm;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, g = lane >> 4;
    const int cg = w % CG;
    const int vslices = (a.dv + NC0 - 1) / NC0, slices = OUT ? vslices : vslices + (a.dk + NC0 - 1) / NC0;
    const int64_t id = blockIdx.x;
    int64_t item = (id >> 3) / run * 8 * run + (id & 7) * run + (id >> 3) % run;      // neighbours, which share keys, on one XCD
    if (item >= (int64_t)a.segs * a.Hv * slices) return;
    int slice = item % slices;
    item /= slices;
    const int hv = item % a.Hv, hk = hv / (a.Hv / a.Hk), slot = item / a.Hv;
    GdrSegment sg;
    if (!gdr_segment(a, slot, sg)) return;
    const GdrSeq s = sg.s;
    const int64_t seq = sg.seq;
    const bool map = !OUT && slice >= vslices;
    if (!OUT && (sg.last || (map && sg.j == 0))) return;
    if (map) slice -= vslices;
    const int width = map ? a.dk : a.dv;
    const int dv0 = slice * NC0 + 16 * cg, col = min(dv0 + l16, width - 1);
    const bool work = dv0 < width;
    const int NC = __builtin_amdgcn_readfirstlane(gdr_chunks(s.T));
    if (a.dk < DK) {
        floatx4* z = reinterpret_cast<floatx4*>(&sm);
        for (int i = tid; i < (int)(NBUF * (OUT ? 2 : 1) * 64 * DK * sizeof(E) / 16); i += (OUT ? 2 : 1) * NT) z[i] = floatx4{0.f, 0.f, 0.f, 0.f};
        __syncthreads();
    }
    const char* rec0 = (const char*)a.rec + ((int64_t)s.slot0 * a.Hv + hv) * gdr_rec_bytes<E>();
    const int64_t recs = a.Hv * gdr_rec_bytes<E>();
    const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
    E* const xs = sm.s + cg * NK * W * 512 + lane * 8;
    E* const xu = sm.u + cg * 2 * W * 512 + lane * 8;

    const int ltid = tid % NT;
    const E* kb = (const E*)a.k + s.b * a.ks[0] + (int64_t)s.row0 * a.ks[1] + hk * a.ks[2];
    const E* vb = (const E*)a.v + s.b * a.vs[0] + (int64_t)s.row0 * a.vs[1] + hv * a.vs[2] + slice * NC0;
    const GdrFetch<E, DK, NT> kf(kb, a.ks[1], s.T, a.dk, ltid);
    GdrSideAhead<E, W, NC0, NT> ahead(vb, a.vs[1], map ? 0 : a.dv - slice * NC0, s.T, ltid);

    // Barriers of a step: one in the middle (the second wave has what it needs of
    // the chunk before, the first what it needs of A, V and the factors), one at
    // its end.
    auto end = [&](int n) __attribute__((always_inline)) {
        lds_barrier();
        if (NBUF == 1) {
            if (!OUT && n + 1 < NC) kf(sm.k[0], (n + 1) * GDR_C, cg);
            swa_landed();
        }
    };
    auto load_side = [&](int n) __attribute__((always_inline)) {
        ahead.load(rec0 + min(n, NC - 1) * recs, ltid);
        ahead.load_v(min(n, NC - 1) * GDR_C);
    };
    if (!OUT || w < CG) {
        // S^T: tile 2 p + h, register r: key channel 32 p + 8 g + 4 h + r (so that
        // two packed tiles are a fragment in natural order), column: the lane's value
        floatx4 S[2 * NK];
        const int64_t at = (int64_t)col * a.dk + 8 * g, size = (int64_t)a.dv * a.dk;
        const float* from = sg.j == 0 ? (a.S0 ? a.S0 + (seq * a.Hv + hv) * size : nullptr)
                                      : OUT ? a.SI + ((int64_t)slot * a.Hv + hv) * size : nullptr;
#pragma unroll
        for (int x = 0; x < 2 * NK; ++x) {
            S[x] = zero;
            if (map) {
#pragma unroll
                for (int r = 0; r < 4; ++r) S[x][r] = 32 * (x / 2) + 8 * g + 4 * (x & 1) + r == dv0 + l16 ? 1.f : 0.f;
            } else if (from && 32 * (x / 2) + 8 * g < a.dk) {
                S[x] = *reinterpret_cast<const floatx4*>(from + at + 32 * (x / 2) + 4 * (x & 1));
            }
        }
        auto chunk = [&](int n, int buf, int par) __attribute__((always_inline)) {
            if (!OUT) {
                if (NBUF == 2 && n + 1 < NC) kf(sm.k[buf ^ 1], (n + 1) * GDR_C, cg);
                load_side(n + 1);
            }
            if (!work) {
                if (OUT) {
                    lds_barrier();
                } else {
                    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                    ahead.store(sm.side[par ^ 1], ltid);
                }
                return end(n);
            }
            const E* kt = sm.k[buf];
            const GdrSide<E, W, NC0>& sd = sm.side[OUT ? 0 : par];
            const E* rec = sd.rec + lane * 8;
            auto factor = [&](int i, int t) { return *reinterpret_cast<const floatx4*>(sd.vec + 64 * i + 16 * t + 4 * g); };
            Frag sh[NK], sl[NK], x[4], A[6], A2[6], f[2], f2[2], f3[2], kc[2 * NK];
            floatx4 U[4], be[4], bb[4], bc[4], v[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                x[t] = T::template ld_row<DK>(kt, 16 * t + l16, 0, g);
                U[t] = zero;
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
                        v[t] = T::template ld_acc<NC0>(sd.v, t, 16 * cg, lane);
                        be[t] = factor(0, t);
                        bb[t] = factor(1, t);
                        bc[t] = factor(2, t);
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
            for (int i = 0; i < 6; ++i) {
                A[i] = T::ld(rec + i * 512);
                if (T::TWO) A2[i] = T::ld(rec + gdr_part<E>() + i * 512);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) U[t][r] = be[t][r] * v[t][r] - bb[t][r] * U[t][r];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                f[j] = T::pack(U[2 * j], U[2 * j + 1]);
                f2[j] = T::rest(U[2 * j], U[2 * j + 1], f[j]);
                f3[j] = T::rest(U[2 * j], U[2 * j + 1], f[j], f2[j]);
            }
            const float eC = sd.vec[256];
            if (OUT) {
                lds_barrier();
#pragma unroll
                for (int p = 0; p < NK; ++p) {
                    T::st(xs + p * W * 512, sh[p]);
                    if (T::TWO) T::st(xs + (p * W + W - 1) * 512, sl[p]);
                }
            }
#pragma unroll
            for (int y = 0; y < 2 * NK; ++y) kc[y] = T::template ld_col8<DK>(kt, 0, 32 * (y / 2) + 4 * (y & 1), lane);
#pragma unroll
            for (int t = 0; t < 4; ++t) U[t] = zero;
            // (every round over the four tiles: products that do not wait for each other)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int t = 2 * j; t < 4; ++t) U[t] = T::mma(A[gdr_block(t, j)], f[j], U[t]);
                if (T::TWO) {
#pragma unroll
                    for (int t = 2 * j; t < 4; ++t) U[t] = T::mma(A[gdr_block(t, j)], f2[j], U[t]);
#pragma unroll
                    for (int t = 2 * j; t < 4; ++t) U[t] = T::mma(A2[gdr_block(t, j)], f[j], U[t]);
#pragma unroll
                    for (int t = 2 * j; t < 4; ++t) U[t] = T::mma(A[gdr_block(t, j)], f3[j], U[t]);
                }
            }
#pragma unroll
            for (int y = 0; y < 2 * NK; ++y) S[y] *= eC;
            if (OUT) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    f[j] = T::pack(U[2 * j], U[2 * j + 1]);
                    T::st(xu + j * W * 512, f[j]);
                    if (T::TWO) T::st(xu + (j * W + W - 1) * 512, T::rest(U[2 * j], U[2 * j + 1], f[j]));
                }
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) U[t] *= bc[t];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                f[j] = T::pack(U[2 * j], U[2 * j + 1]);
                f2[j] = T::rest(U[2 * j], U[2 * j + 1], f[j]);
                f3[j] = T::rest(U[2 * j], U[2 * j + 1], f[j], f2[j]);
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
            if (!OUT) {
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                ahead.store(sm.side[par ^ 1], ltid);
            }
            end(n);
        };
        if (NC > 0) {
            if (!OUT) {
                load_side(0);
                kf(sm.k[0], 0, cg);
                ahead.store(sm.side[0], ltid);
            }
            swa_landed();
        }
        for (int n = 0; n < NC; n += 2) {
            chunk(n, 0, 0);
            if (n + 1 < NC) chunk(n + 1, NBUF - 1, 1);
        }
        if (OUT && NC > 0) lds_barrier();
        float* to = OUT ? (a.ST && sg.last ? a.ST + (seq * a.Hv + hv) * size : nullptr)
                    : map ? a.M + ((int64_t)slot * a.Hv + hv) * a.dk * a.dk
                          : a.SI + ((int64_t)(slot + 1) * a.Hv + hv) * size;
        if (map) {      // transposed, for the chain
#pragma unroll
            for (int x = 0; x < 2 * NK; ++x)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int c = 32 * (x / 2) + 8 * g + 4 * (x & 1) + r;
                    if (work && dv0 + l16 < width && c < a.dk) to[(int64_t)c * a.dk + dv0 + l16] = S[x][r];
                }
        } else if (to && work && dv0 + l16 < width) {
#pragma unroll
            for (int x = 0; x < 2 * NK; ++x)
                if (32 * (x / 2) + 8 * g < a.dk) *reinterpret_cast<floatx4*>(to + at + 32 * (x / 2) + 4 * (x & 1)) = S[x];
        }
        return;
    }

    const E* qb = (const E*)a.q + s.b * a.qs[0] + (int64_t)s.row0 * a.qs[1] + hk * a.qs[2];
    const E* ob = (const E*)a.o + ((s.b * a.T + s.row0) * a.Hv + hv) * (int64_t)a.dv;
    const int os = a.Hv * a.dv;
    // where the lane's four values of row 16 t + l16, and its eight of a kept state, go
    int oat[4], hat[NK];
#pragma unroll
    for (int t = 0; t < 4; ++t) oat[t] = dv0 + 4 * g < a.dv ? ((16 * t + l16) * os + dv0 + 4 * g) * (int)sizeof(E) : GDR_NONE;
#pragma unroll
    for (int p = 0; p < NK; ++p)
        hat[p] = dv0 + l16 < a.dv && 32 * p + 8 * g < a.dk ? (col * a.dk + 32 * p + 8 * g) * (int)sizeof(E) : GDR_NONE;
    const GdrFetch<E, DK, NT> qf(qb, a.qs[1], s.T, a.dk, ltid);
    // P of the chunk whose outputs come next goes through LDS like A, its pieces are
    constexpr int PP = gdr_part<E>() * (int)sizeof(E) / 16, NP = (PP + NT - 1) / NT;
    floatx4 px[NP];
    auto load = [&](int n) __attribute__((always_inline)) {
        const char* r = rec0 + min(n, NC - 1) * recs;
        load_side(n);
        const auto ps = gdr_buffer(r + (T::TWO ? PP * 16 : 0), PP * 16);
#pragma unroll
        for (int i = 0; i < NP; ++i) px[i] = gdr_load(ps, (i * NT + ltid) * 16);
    };
    auto store = [&](int par) __attribute__((always_inline)) {
        ahead.store(sm.side[0], ltid);
#pragma unroll
        for (int i = 0; i < NP; ++i)
            if (i < NP - 1 || (NP - 1) * NT + ltid < PP) reinterpret_cast<floatx4*>(sm.p[OUT ? par : 0])[OUT ? i * NT + ltid : 0] = px[i];
    };
    float se[4];
    // a step: chunk n on its way (none past the last), outputs of chunk n - 1
    auto fetch = [&](int n, int buf) __attribute__((always_inline)) {
        if (n + 1 < NC) kf(sm.k[buf ^ (NBUF - 1)], (n + 1) * GDR_C, cg);
        if (n < NC) qf(sm.q[buf], n * GDR_C, cg);
    };
    auto step = [&](int n, int buf, int par) __attribute__((always_inline)) {
        const bool out = work && n > 0;
        Frag sh[NK], sl[NK], f[2], f2[2], P[6];
        float sn[4];      // the factors of this chunk, for the next step
#pragma unroll
        for (int t = 0; t < 4; ++t) sn[t] = sm.side[0].vec[192 + 16 * t + l16];
        if (out) {
#pragma unroll
            for (int p = 0; p < NK; ++p) {
                sh[p] = T::ld(xs + p * W * 512);
                if (T::TWO) sl[p] = T::ld(xs + (p * W + W - 1) * 512);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                f[j] = T::ld(xu + j * W * 512);
                if (T::TWO) f2[j] = T::ld(xu + (j * W + W - 1) * 512);
            }
        }
        if (NBUF == 2) fetch(n, buf);
        load(n + 1);
        floatx4 O[4] = {zero, zero, zero, zero};
        const E* qt = sm.q[buf ^ (NBUF - 1)];
        auto qs = [&](int p) __attribute__((always_inline)) {
            Frag x[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) x[t] = T::template ld_row<DK>(qt, 16 * t + l16, p, g);
#pragma unroll
            for (int t = 0; t < 4; ++t) O[t] = T::mma(sh[p], x[t], O[t]);
            if (T::TWO) {
#pragma unroll
                for (int t = 0; t < 4; ++t) O[t] = T::mma(sl[p], x[t], O[t]);
            }
        };
        if (out) {
#pragma unroll
            for (int p = 0; p < NK / 2; ++p) qs(p);
#pragma unroll
            for (int i = 0; i < 6; ++i) P[i] = T::ld(sm.p[par ^ 1] + i * 512 + lane * 8);      // (its place is written again after the barrier)
        }
        lds_barrier();
        if (out) {
#pragma unroll
            for (int p = NK / 2; p < NK; ++p) qs(p);
#pragma unroll
            for (int t = 0; t < 4; ++t) O[t] *= se[t];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int t = 2 * j; t < 4; ++t) O[t] = T::mma(f[j], P[gdr_block(t, j)], O[t]);
                if (T::TWO) {
#pragma unroll
                    for (int t = 2 * j; t < 4; ++t) O[t] = T::mma(f2[j], P[gdr_block(t, j)], O[t]);
                }
            }
        }
        // the next chunk is here; the stores that follow need not have been written when it begins
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        store(par ^ 1);
        if (out) {
            const int c = n - 1;
            const auto o = gdr_buffer(ob + (int64_t)c * GDR_C * os, ((int64_t)(min(s.T - c * GDR_C, GDR_C) - 1) * os + a.dv) * (int)sizeof(E));
#pragma unroll
            for (int t = 0; t < 4; ++t) gdr_store(o, oat[t], O[t], (const E*)nullptr);
            if (MODE == GDR_SAVE) {
                const auto hs = gdr_buffer((const E*)a.hs + ((int64_t)(s.slot0 + c) * a.Hv + hv) * a.dv * a.dk, (int64_t)a.dv * a.dk * (int)sizeof(E));
#pragma unroll
                for (int p = 0; p < NK; ++p) gdr_store(hs, hat[p], sh[p]);
            }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) se[t] = sn[t];
    };
    if (NC > 0) {
        load(0);
        kf(sm.k[0], 0, cg);
        store(0);
        swa_landed();
    }
    auto turn = [&](int n, int buf, int par) __attribute__((always_inline)) {
        step(n, buf, par);
        if (n == NC) return;
        lds_barrier();
        if (NBUF == 1) {
            fetch(n, 0);
            swa_landed();
        }
    };
    for (int n = 0; n < (NC > 0 ? NC + 1 : 0); n += 2) {
        turn(n, 0, 0);
        if (n < NC) turn(n + 1, NBUF - 1, 1);
    }
}

// The states entering a sequence's segments, one after the other: SI_(j+1) =
// SI_j M_j + N_j, where SI_(j+1) holds N_j (the first one is the state itself).
// A workgroup per 16 values of a head, in fp32 products: the state's
// accumulators are the next product's B operand.  Its four waves make NT / 4
// tiles of rows each and hand them to each other through LDS; maps load a
// segment ahead (3.3 us a segment; without, 3.7 us).
template <int DK>
__global__ __launch_bounds__(256, 1) void kd_gdr_chain_kernel(GdrArgs a)
{
    constexpr int NT = DK / 16, NY = NT / 4;
    __shared__ __align__(16) floatx4 tile[2][NT][64];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, g = lane >> 4;
    const int hv = blockIdx.y, seq = blockIdx.z, v = min((int)blockIdx.x * 16 + l16, a.dv - 1);
    const GdrSeq s = gdr_seq(a, seq);
    const int n = (gdr_chunks(s.T) + a.seg - 1) / a.seg, slot = a.cu ? s.row0 / GDR_C / a.seg + seq : seq * a.nseg;
    const int64_t size = (int64_t)a.dv * a.dk;
    if (n < 3) return;
    const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
    // (tile x, register r: key channel 32 (x / 2) + 8 g + 4 (x % 2) + r, as in the pass)
    auto channel = [&](int x, int i) { return 32 * (x / 2) + 8 * i + 4 * (x & 1); };
    auto state = [&](int j, int x) {
        return a.SI + ((int64_t)(slot + j) * a.Hv + hv) * size + (int64_t)v * a.dk + channel(x, g);
    };
    floatx4 S[NT], N[2][NY], m[2][NY][NT];
    auto load = [&](int j, int b) __attribute__((always_inline)) {
        const float* M = a.M + ((int64_t)(slot + j) * a.Hv + hv) * a.dk * a.dk;
#pragma unroll
        for (int y = 0; y < NY; ++y) {
            const int own = NY * w + y, c = channel(own, l16 >> 2) + (l16 & 3);      // the operand's row, as the state's are laid out
            N[b][y] = channel(own, g) < a.dk ? *reinterpret_cast<const floatx4*>(state(j + 1, own)) : zero;
#pragma unroll
            for (int x = 0; x < NT; ++x)
                m[b][y][x] = c < a.dk && channel(x, g) < a.dk ? *reinterpret_cast<const floatx4*>(M + (int64_t)c * a.dk + channel(x, g)) : zero;
        }
    };
#pragma unroll
    for (int x = 0; x < NT; ++x) S[x] = channel(x, g) < a.dk ? *reinterpret_cast<const floatx4*>(state(1, x)) : zero;
    load(1, 0);
    auto turn = [&](int j, int b) __attribute__((always_inline)) {
        if (j + 2 < n) load(j + 1, b ^ 1);
        floatx4 R[NY];
#pragma unroll
        for (int y = 0; y < NY; ++y) R[y] = N[b][y];
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int y = 0; y < NY; ++y) R[y] = __builtin_amdgcn_mfma_f32_16x16x4f32(m[b][y][x][r], S[x][r], R[y], 0, 0, 0);
#pragma unroll
        for (int y = 0; y < NY; ++y) {
            tile[b][NY * w + y][lane] = R[y];
            if (channel(NY * w + y, g) < a.dk && blockIdx.x * 16 + l16 < a.dv) *reinterpret_cast<floatx4*>(state(j + 1, NY * w + y)) = R[y];
        }
        lds_barrier();
#pragma unroll
        for (int x = 0; x < NT; ++x) S[x] = tile[b][x][lane];
    };
    for (int j = 1; j + 1 < n; j += 2) {
        turn(j, 0);
        if (j + 2 < n) turn(j + 1, 1);
    }
}

// Workgroups of a pass (items of neighbouring slices and heads, in runs of `run`
// on one XCD, as many as leave none of the 8 XCDs idle), and their grid.
int64_t gdr_pass_grid(int64_t items, int& run)
{
    run = (int)((items + 7) / 8);
    run = run < 16 ? run : 16;
    return (items + 8 * run - 1) / (8 * run) * 8 * run;
}

template <class E, int DK>
static hipError_t gdr_prep(const GdrArgs& a, hipStream_t st)
{
    const unsigned grid = (unsigned)((int64_t)a.slots * a.Hv);
    if (grid == 0) return hipSuccess;
    if (a.hs) kd_gdr_prep_kernel<E, DK, true><<<grid, 64, 0, st>>>(a);
    else kd_gdr_prep_kernel<E, DK, false><<<grid, 64, 0, st>>>(a);
    return hipGetLastError();
}

template <class E, int DK, int MODE, int CG>
static void gdr_pass(const GdrArgs& a, hipStream_t st)
{
    constexpr int C = 16 * CG;
    int run;
    const int64_t grid = gdr_pass_grid((int64_t)a.segs * a.Hv * ((a.dv + C - 1) / C + (MODE == GDR_MAPS ? (a.dk + C - 1) / C : 0)), run);
    kd_gdr_pass_kernel<E, DK, MODE, CG><<<(unsigned)grid, (MODE == GDR_MAPS ? 64 : 128) * CG, 0, st>>>(a, run);
}
template <class E, int DK, int MODE>
static void gdr_pass(const GdrArgs& a, hipStream_t st)
{
    if constexpr (sizeof(E) == 4) {
        gdr_pass<E, DK, MODE, 2>(a, st);
    } else if constexpr (MODE == GDR_MAPS) {
        gdr_pass<E, DK, MODE, 4>(a, st);
    } else {
        if (gdr_narrow(a, a.segs)) gdr_pass<E, DK, MODE, 2>(a, st);
        else gdr_pass<E, DK, MODE, 4>(a, st);
    }
}
template <class E, int DK>
static hipError_t gdr_passes(const GdrArgs& a, hipStream_t st)
{
    const hipError_t e = gdr_prep<E, DK>(a, st);
    if (e != hipSuccess) return e;
    if (a.SI) {
        gdr_pass<E, DK, GDR_MAPS>(a, st);
        kd_gdr_chain_kernel<DK><<<dim3((a.dv + 15) / 16, a.Hv, a.B), 256, 0, st>>>(a);
    }
    if (a.hs) gdr_pass<E, DK, GDR_SAVE>(a, st);
    else gdr_pass<E, DK, GDR_OUT>(a, st);
    return hipGetLastError();
}

// Segments.  A pass takes as long as its longest sequence, a few microseconds a
// chunk, however few workgroups there are; the maps cost about as much work
// again as the pass itself.  So sequences are cut where they leave three
// quarters of the 256 compute units idle, into segments of at least 8 chunks,
// as many as make 256 workgroups (32768 tokens of 16 heads: 25 us less than with
// 512, most of it in the chain; in one piece 1.7 ms for 0.5).  Packed sequences
// are cut by what their average length would be.
void gdr_plan(GdrArgs& a, bool packed)
{
    const int64_t wgs = (int64_t)a.B * a.Hv * ((a.dv + 63) / 64);
    const int NC = packed ? (a.T / a.B + GDR_C - 1) / GDR_C : (a.T + GDR_C - 1) / GDR_C;
    int n = wgs * 4 <= 256 ? (int)(256 / wgs) : 1;
    n = n < NC / 8 ? n : NC / 8;
    if (n < 3) n = 1;
    a.seg = n > 1 ? (NC + n - 1) / n : 1 << 24;
    a.nseg = n > 1 ? (NC + a.seg - 1) / a.seg : 1;
    a.segs = packed ? (int)((int64_t)a.T / GDR_C / a.seg + a.B) : a.B * a.nseg;
}

hipError_t launch_gdr_fwd(int bf16, const GdrArgs& a, hipStream_t st)
{
    if (bf16) return a.dk <= 64 ? gdr_passes<__bf16, 64>(a, st) : gdr_passes<__bf16, 128>(a, st);
    return a.dk <= 64 ? gdr_passes<float, 64>(a, st) : gdr_passes<float, 128>(a, st);
}

// One token.  Lanes of a row's key channels, four each; both products with the
// old state in one pass: with r = S k, s = S q,
//     u = beta (v - e^g r),  S' = e^g S + u k^T,  o = scale (e^g s + u (k.q)).
// A workgroup takes `rows` rows of one head's state.  Bound by reading and
// writing the states: 32 requests, 16 heads of 128 x 128: 67 MB in 14.8 us.
template <class E, int L>
__global__ __launch_bounds__(256) void kd_gdr_step_kernel(const E* q, const E* k, const E* v, const void* gp, const void* bp,
                                                          const float* Si, float* So, E* o, int64_t qb, int64_t kb, int64_t vb,
                                                          int64_t qh, int64_t kh, int64_t vh, int Hk, int Hv, int dk, int dv,
                                                          int rows, int gates32, float scale)
{
    constexpr int PER = 256 / L, U = 4;      // rows a pass of the workgroup, passes in flight
    const int tid = threadIdx.x, c = 4 * (tid % L), part = blockIdx.x, hv = blockIdx.y, hk = hv / (Hv / Hk);
    const int64_t b = blockIdx.z;
    const bool in = c < dk;
    const int64_t head = b * Hv + hv;
    const float* Sr = Si + head * dv * dk + (in ? c : 0);
    float* Sw = So + head * dv * dk + c;
    const int r1 = min((part + 1) * rows, dv);
    floatx4 S[U];
    auto load = [&](int r0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            S[u] = *reinterpret_cast<const floatx4*>(Sr + (int64_t)min(r0 + u * PER + tid / L, dv - 1) * dk);
            if (!in) S[u] = floatx4{0.f, 0.f, 0.f, 0.f};      // (0 times an infinity of the first channels)
        }
    };
    load(part * rows);
    floatx4 kx = {0.f, 0.f, 0.f, 0.f}, qx = {0.f, 0.f, 0.f, 0.f};
    if (in) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            kx[e] = (float)k[b * kb + hk * kh + c + e];
            qx[e] = (float)q[b * qb + hk * qh + c + e];
        }
    }
    const float decay = expf(gdr_gate(gp, head, gates32, (const E*)nullptr));
    const float beta = gdr_gate(bp, head, gates32, (const E*)nullptr);
    auto sum = [&](float x) {
#pragma unroll
        for (int y = 1; y < L; y *= 2) x += __shfl_xor(x, y);
        return x;
    };
    auto dot = [](floatx4 x, floatx4 y) { return fmaf(x[0], y[0], fmaf(x[1], y[1], fmaf(x[2], y[2], x[3] * y[3]))); };
    const float kq = sum(dot(kx, qx));
    for (int r0 = part * rows; r0 < r1; r0 += U * PER) {
        if (r0 > part * rows) load(r0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = r0 + u * PER + tid / L;
            const float rk = sum(dot(S[u], kx)), rq = sum(dot(S[u], qx));
            if (row >= r1) continue;
            const float x = beta * ((float)v[b * vb + hv * vh + row] - decay * rk);
            if (in) *reinterpret_cast<floatx4*>(Sw + (int64_t)row * dk) = S[u] * decay + kx * x;
            if (tid % L == 0) o[head * dv + row] = (E)(scale * fmaf(decay, rq, x * kq));
        }
    }
}

hipError_t launch_gdr_step(int bf16, const GdrArgs& a, hipStream_t st)
{
    const int L = a.dk <= 32 ? 8 : a.dk <= 64 ? 16 : 32, per = 256 / L;
    // whole passes of four loads; more workgroups per head where heads are few
    int rows = a.dv;
    while ((int64_t)a.B * a.Hv * ((a.dv + rows - 1) / rows) < 1024 && rows > 4 * per) rows = (rows / 2 + 4 * per - 1) / (4 * per) * 4 * per;
    const dim3 grid((a.dv + rows - 1) / rows, a.Hv, a.B);
#define KD_STEP(E, L)                                                                                                        \
    kd_gdr_step_kernel<E, L><<<grid, 256, 0, st>>>((const E*)a.q, (const E*)a.k, (const E*)a.v, a.g, a.beta, a.S0, a.ST,     \
                                                   (E*)a.o, a.qs[0], a.ks[0], a.vs[0], a.qs[2], a.ks[2], a.vs[2], a.Hk, a.Hv, \
                                                   a.dk, a.dv, rows, a.gates32, a.scale)
    if (bf16) {
        if (L == 8) KD_STEP(__bf16, 8);
        else if (L == 16) KD_STEP(__bf16, 16);
        else KD_STEP(__bf16, 32);
    } else {
        if (L == 8) KD_STEP(float, 8);
        else if (L == 16) KD_STEP(float, 16);
        else KD_STEP(float, 32);
    }
#undef KD_STEP
    return hipGetLastError();
}

}  // namespace kd
