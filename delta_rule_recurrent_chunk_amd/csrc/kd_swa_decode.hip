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

#include <type_traits>

namespace kd {

// slot of position s
__device__ __forceinline__ int64_t cache_slot(int s, int S, int cap) { return s < S ? s : S + (s - S) % (cap - S); }

// sum over the LPR adjacent lanes that share a key, on every one of them
template <int LPR>
__device__ __forceinline__ float lanes_sum(float x) {
#define KD_DPP_ADD(c) x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), c, 0xf, 0xf, false))
    KD_DPP_ADD(0xB1);                               // quad_perm [1,0,3,2]
    KD_DPP_ADD(0x4E);                               // quad_perm [2,3,0,1]
    if constexpr (LPR >= 8) KD_DPP_ADD(0x141);      // row_half_mirror
    if constexpr (LPR >= 16) KD_DPP_ADD(0x140);     // row_mirror
    if constexpr (LPR >= 32) x += __shfl_xor(x, 16);
#undef KD_DPP_ADD
    return x;
}

// Workgroup (split, key head, group of GB query heads; b): four waves share the
// split's keys.  LPR lanes hold one key's row, 16 bytes each, so a wave reads
// 64 / LPR keys per instruction; every such row group keeps its own running
// maximum, sum and output, joined at the end over groups, waves and splits.
template <class E, int D, int GB>
__global__ __launch_bounds__(256) void kd_swa_decode_kernel(SwaDecodeArgs a)
{
    constexpr int EPC = 16 / sizeof(E), LPR = D / EPC, KPI = 64 / LPR, U = 4;
    typedef E Vec __attribute__((ext_vector_type(EPC)));
    __shared__ float2 cs[D / 2];
    __shared__ __align__(16) float qs[GB * D];
    __shared__ __align__(16) float accs[4][GB][D];
    __shared__ float ms[4][GB], lsum[4][GB];
    __shared__ int last;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, c = lane % LPR, kg = lane / LPR;
    const int G = a.Hq / a.Hkv, nhb = (G + GB - 1) / GB;
    const int sp = blockIdx.x, hk = blockIdx.y / nhb, hb = blockIdx.y % nhb, b = blockIdx.z;
    const int h0 = hk * G + hb * GB, nh = min(GB, G - hb * GB);
    const int pos = a.lens[b];
    E* o = (E*)a.o + ((int64_t)b * a.Hq + h0) * D;
    if (pos < 0) {     // an unused row: nothing is stored, its output is zero
        if (sp == 0)
            for (int i = tid; i < nh * D; i += 256) o[i] = (E)0.f;
        return;
    }
    // queries (turned, times scale log2 e) and, for the workgroup that stores it, the new key
    const int n = a.rot / 2;
    for (int j = tid; j < n; j += 256) cs[j] = rope_cs((double)pos, a.freqs[j], a.rope_scale, 0);
    __syncthreads();
    const E* qrow = (const E*)a.q + b * a.qb + (int64_t)h0 * D;
    auto turned = [&](const E* row, int i) -> float {
        const float x = (float)row[i];
        if (i >= a.rot) return x;
        const int j = a.interleaved ? i / 2 : i % n;
        const bool second = a.interleaved ? (i & 1) : i >= n;
        const float y = (float)row[a.interleaved ? i ^ 1 : second ? i - n : i + n];
        return second ? fmaf(x, cs[j].x, y * cs[j].y) : fmaf(x, cs[j].x, -y * cs[j].y);
    };
    for (int i = tid; i < GB * D; i += 256) qs[i] = i < nh * D ? turned(qrow + i / D * D, i % D) * a.c : 0.f;
    const E* krow = (const E*)a.k + b * a.kb + (int64_t)hk * D;
    const E* vrow = (const E*)a.v + b * a.vb + (int64_t)hk * D;
    E* kc = (E*)a.kc + b * a.kcs[0] + hk * a.kcs[2];
    E* vc = (E*)a.vc + b * a.vcs[0] + hk * a.vcs[2];
    if (sp == 0 && hb == 0 && tid < D) {
        const int64_t slot = cache_slot(pos, a.S, a.cap);
        kc[slot * a.kcs[1] + tid] = (E)turned(krow, tid);
        vc[slot * a.vcs[1] + tid] = vrow[tid];
    }
    __syncthreads();
    float q[GB][EPC], acc[GB][EPC], m[GB], l[GB];
#pragma unroll
    for (int h = 0; h < GB; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
#pragma unroll
        for (int e = 0; e < EPC; ++e) {
            q[h][e] = qs[h * D + c * EPC + e];
            acc[h][e] = 0.f;
        }
    }
    // keys seen before the new one: the sinks 0 .. ns - 1, then p0 .. pos - 1
    const int p0 = max(0, pos - a.W + 1), ns = min(a.S, p0), nv = ns + pos - p0;
    const int per = (((nv + a.nsplit - 1) / a.nsplit) + 4 * KPI - 1) / (4 * KPI) * (4 * KPI);
    const int jlo = min((int64_t)sp * per, (int64_t)nv), jhi = min(jlo + per, nv);
    auto step = [&](const Vec* kv, const Vec* vv, const bool* ok, auto un) {
        constexpr int N = decltype(un)::value;
#pragma unroll
        for (int h = 0; h < GB; ++h) {
            float s[N], mx = -INFINITY;
#pragma unroll
            for (int u = 0; u < N; ++u) {
                float d = 0.f;
#pragma unroll
                for (int e = 0; e < EPC; ++e) d = fmaf((float)kv[u][e], q[h][e], d);
                d = lanes_sum<LPR>(d);
                s[u] = ok[u] ? d : -INFINITY;
                mx = fmaxf(mx, s[u]);
            }
            const float mn = fmaxf(m[h], mx), mu = mn == -INFINITY ? 0.f : mn;
            const float al = __builtin_amdgcn_exp2f(m[h] - mu);
            m[h] = mn;
            l[h] *= al;
#pragma unroll
            for (int e = 0; e < EPC; ++e) acc[h][e] *= al;
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const float p = __builtin_amdgcn_exp2f(s[u] - mu);
                l[h] += p;
#pragma unroll
                for (int e = 0; e < EPC; ++e) acc[h][e] = fmaf(p, (float)vv[u][e], acc[h][e]);
            }
        }
    };
    for (int j0 = jlo + w * KPI; j0 < jhi; j0 += 4 * KPI * U) {
        Vec kv[U], vv[U];
        bool ok[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u * 4 * KPI + kg;
            ok[u] = j < jhi;
            if (ok[u]) {
                const int64_t slot = cache_slot(j < ns ? j : p0 + (j - ns), a.S, a.cap);
                kv[u] = *reinterpret_cast<const Vec*>(kc + slot * a.kcs[1] + c * EPC);
                vv[u] = *reinterpret_cast<const Vec*>(vc + slot * a.vcs[1] + c * EPC);
            } else {
#pragma unroll
                for (int e = 0; e < EPC; ++e) kv[u][e] = vv[u][e] = (E)0.f;
            }
        }
        step(kv, vv, ok, std::integral_constant<int, U>());
    }
    if (sp == 0 && w == 0) {     // the new token, on the wave's first row group
        Vec kv, vv;
        const bool ok = kg == 0;
#pragma unroll
        for (int e = 0; e < EPC; ++e) {
            kv[e] = (E)turned(krow, c * EPC + e);
            vv[e] = ok ? vrow[c * EPC + e] : (E)0.f;
        }
        step(&kv, &vv, &ok, std::integral_constant<int, 1>());
    }
    // row groups of the wave
#pragma unroll
    for (int h = 0; h < GB; ++h) {
#pragma unroll
        for (int x = LPR; x < 64; x *= 2) {
            const float mo = __shfl_xor(m[h], x), mn = fmaxf(m[h], mo), mu = mn == -INFINITY ? 0.f : mn;
            const float f = __builtin_amdgcn_exp2f(m[h] - mu), fo = __builtin_amdgcn_exp2f(mo - mu);
            l[h] = l[h] * f + __shfl_xor(l[h], x) * fo;
#pragma unroll
            for (int e = 0; e < EPC; ++e) acc[h][e] = acc[h][e] * f + __shfl_xor(acc[h][e], x) * fo;
            m[h] = mn;
        }
        if (kg == 0) {
#pragma unroll
            for (int e = 0; e < EPC; ++e) accs[w][h][c * EPC + e] = acc[h][e];
            if (c == 0) {
                ms[w][h] = m[h];
                lsum[w][h] = l[h];
            }
        }
    }
    __syncthreads();
    // waves, then splits: the last workgroup of (b, heads) to arrive joins them
    const int item = (b * (int)gridDim.y + blockIdx.y);
    float* part = a.part + ((int64_t)item * a.nsplit + sp) * GB * (D + 2);
    for (int i = tid; i < nh * D; i += 256) {
        const int h = i / D, e = i % D;
        const float mn = fmaxf(fmaxf(ms[0][h], ms[1][h]), fmaxf(ms[2][h], ms[3][h]));
        const float mu = mn == -INFINITY ? 0.f : mn;
        float A = 0.f, L = 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float f = __builtin_amdgcn_exp2f(ms[x][h] - mu);
            A = fmaf(accs[x][h][e], f, A);
            L = fmaf(lsum[x][h], f, L);
        }
        if (a.nsplit == 1) {
            o[i] = (E)(A / L);
            continue;
        }
        // stores that reach the memory every compute unit sees
        __hip_atomic_store(part + i, A, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (e == 0) {
            __hip_atomic_store(part + GB * D + 2 * h, mn, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(part + GB * D + 2 * h + 1, L, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    if (a.nsplit == 1) return;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_s_waitcnt(0);       // the stores are done before the arrival is counted
    __syncthreads();
    if (tid == 0)
        last = __hip_atomic_fetch_add(a.count + item, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.nsplit - 1;
    __syncthreads();
    if (!last) return;
    if (tid == 0) __hip_atomic_store(a.count + item, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);   // for the next call
    const float* pb = a.part + (int64_t)item * a.nsplit * GB * (D + 2);
    for (int i = tid; i < nh * D; i += 256) {
        const int h = i / D;
        float mn = -INFINITY, A = 0.f, L = 0.f;
        for (int x = 0; x < a.nsplit; ++x)
            mn = fmaxf(mn, __hip_atomic_load(pb + (int64_t)x * GB * (D + 2) + GB * D + 2 * h, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT));
        const float mu = mn == -INFINITY ? 0.f : mn;
        for (int x = 0; x < a.nsplit; ++x) {
            const float* px = pb + (int64_t)x * GB * (D + 2);
            const float f = __builtin_amdgcn_exp2f(
                __hip_atomic_load(px + GB * D + 2 * h, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) - mu);
            A = fmaf(__hip_atomic_load(px + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT), f, A);
            L = fmaf(__hip_atomic_load(px + GB * D + 2 * h + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT), f, L);
        }
        o[i] = (E)(A / L);
    }
}

// Tokens of a prompt into the cache: token t of sequence b, t < lens[b], at
// position t; where two positions share a slot only the later one is stored.
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

// heads of a group that one workgroup takes
static int heads_per_block(int G) { return G >= 4 ? 4 : G == 3 ? 4 : G; }

int swa_decode_items(int B, int Hq, int Hkv) {
    const int G = Hq / Hkv, gb = heads_per_block(G);
    return B * Hkv * ((G + gb - 1) / gb);
}

// Splits of a row's keys: enough workgroups to fill the chip's 256 compute
// units about four times over, none below 64 keys.  Rows are split only where
// there are fewer than SWA_DECODE_COUNTERS items, so that many counters serve
// every call.
int swa_decode_splits(int B, int Hq, int Hkv, int seen) {
    const int items = swa_decode_items(B, Hq, Hkv);
    int n = (SWA_DECODE_COUNTERS + items - 1) / items;
    const int most = (seen + 63) / 64;
    n = n < most ? n : most;
    n = n < 32 ? n : 32;
    return n < 1 ? 1 : n;
}

// The splits' partial results (none where a row's keys are not split).
size_t swa_decode_part_bytes(int B, int Hq, int Hkv, int d, int seen) {
    const int gb = heads_per_block(Hq / Hkv), n = swa_decode_splits(B, Hq, Hkv, seen);
    return n == 1 ? 0 : (size_t)swa_decode_items(B, Hq, Hkv) * n * gb * (d + 2) * 4;
}

template <class E, int D>
static hipError_t swa_decode(const SwaDecodeArgs& a, hipStream_t st)
{
    const int G = a.Hq / a.Hkv, gb = heads_per_block(G);
    const dim3 grid(a.nsplit, a.Hkv * ((G + gb - 1) / gb), a.B);
    if (gb == 1) kd_swa_decode_kernel<E, D, 1><<<grid, 256, 0, st>>>(a);
    else if (gb == 2) kd_swa_decode_kernel<E, D, 2><<<grid, 256, 0, st>>>(a);
    else kd_swa_decode_kernel<E, D, 4><<<grid, 256, 0, st>>>(a);
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
