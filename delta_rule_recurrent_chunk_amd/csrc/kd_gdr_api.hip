// kd_gdr_api.hip -- the C ABI of the gated delta rule: argument checks,
// workspace sizing and dispatch on the caller's stream.  No allocation, no
// synchronisation.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kd_check.h"
#include "kd_gdr.h"
#include "kron_delta.h"

namespace kd {
int64_t gdr_pass_grid(int64_t items, int& run);
void gdr_plan(GdrArgs& a, bool packed);
hipError_t launch_gdr_fwd(int bf16, const GdrArgs& a, hipStream_t st);
hipError_t launch_gdr_bwd(int bf16, const GdrArgs& a, hipStream_t st);
hipError_t launch_gdr_step(int bf16, const GdrArgs& a, hipStream_t st);
}  // namespace kd

namespace {

using kd::any_overlap;
using kd::grid_fits;
using kd::misaligned;
using kd::overlap;
using kd::Range;
using kd::range_of;
using kd::span;
using kd::up256;

bool known(int dtype) { return dtype == KD_F32 || dtype == KD_BF16; }
size_t es_of(int dtype) { return dtype == KD_BF16 ? 2 : 4; }
kd_status done(hipError_t e) { return e == hipSuccess ? KD_OK : KD_ERR_LAUNCH; }

struct GdrSizes {
    size_t q, k, v, o, qg, kg, gate, state, slots;      // bytes (spanned by the inputs, contiguous others), chunk slots
    size_t rec, saved;                                  // what the backward pass is given: records, then states
};

kd_status check_gdr(const kd_gdr_desc* d, bool packed, GdrSizes* s) {
    if (!d) return KD_ERR_NULL;
    if (!known(d->dtype)) return KD_ERR_DTYPE;
    if (d->B < 1 || d->T < 0 || d->T > (1 << 29) || d->Hk < 1 || d->Hv < 1 || d->Hv > 65535 || d->Hv % d->Hk != 0 ||
        d->dk < 8 || d->dk > KRON_DELTA_GDR_MAX_DK || d->dk % 8 != 0 || d->dv < 8 || d->dv > KRON_DELTA_GDR_MAX_DV ||
        d->dv % 8 != 0 || !isfinite(d->scale) || d->B > (packed ? 1 << 24 : 65535) || (int64_t)d->Hv * d->dv > kd::GDR_MAX_STEP)
        return KD_ERR_SHAPE;
    if (d->T > 1 && (d->q_stride[1] > kd::GDR_MAX_STEP || d->k_stride[1] > kd::GDR_MAX_STEP || d->v_stride[1] > kd::GDR_MAX_STEP))
        return KD_ERR_SHAPE;
    const size_t es = es_of(d->dtype);
    const int64_t nb = packed ? 1 : d->B;
    if (!span(d->q_stride, nb, d->T, d->Hk, d->dk, es, true, &s->q) || !span(d->k_stride, nb, d->T, d->Hk, d->dk, es, true, &s->k) ||
        !span(d->v_stride, nb, d->T, d->Hv, d->dv, es, true, &s->v))
        return KD_ERR_SHAPE;
    const __int128 rows = (__int128)nb * d->T;
    const __int128 slots = packed ? (__int128)d->T / 64 + d->B : (__int128)d->B * ((d->T + 63) / 64);
    if (slots > (1 << 30) || rows * d->Hv * d->dv * es > ((__int128)1 << 60) ||
        slots * d->Hv * d->dv * d->dk * es > ((__int128)1 << 60))
        return KD_ERR_SHAPE;
    s->o = (size_t)(rows * d->Hv * d->dv * es);
    s->qg = s->kg = (size_t)(rows * d->Hk * d->dk * es);
    s->gate = (size_t)(rows * d->Hv * (d->gates32 ? 4 : es));
    s->state = (size_t)d->B * d->Hv * d->dv * d->dk * 4;
    s->slots = (size_t)slots;
    s->rec = up256(s->slots * d->Hv * (d->dtype == KD_BF16 ? kd::gdr_rec_bytes<__bf16>() : kd::gdr_rec_bytes<float>()));
    s->saved = s->rec + up256(s->slots * d->Hv * d->dv * d->dk * es);
    int run;
    if (!grid_fits((int64_t)s->slots * d->Hv, 64) || !grid_fits((int64_t)s->slots * d->Hk, 512) ||
        !grid_fits(kd::gdr_pass_grid((int64_t)d->B * d->Hv * ((d->dv + 31) / 32), run), 512))
        return KD_ERR_SHAPE;
    return KD_OK;
}

kd::GdrArgs gdr_args(const kd_gdr_desc* d, const GdrSizes& s, const void* q, const void* k, const void* v, const void* g,
                     const void* beta, const int32_t* cu) {
    kd::GdrArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.beta = beta;
    for (int i = 0; i < 3; ++i) {
        a.qs[i] = d->q_stride[i];
        a.ks[i] = d->k_stride[i];
        a.vs[i] = d->v_stride[i];
    }
    a.cu = cu;
    a.B = d->B;
    a.T = d->T;
    a.Hk = d->Hk;
    a.Hv = d->Hv;
    a.dk = d->dk;
    a.dv = d->dv;
    a.slots = (int)s.slots;
    a.gates32 = d->gates32 != 0;
    a.scale = d->scale;
    return a;
}

// Offsets of the workspace's parts.  Forward: records (their room is asked for
// also where they are saved, and not used then), the segments' states and maps
// (equal where a sequence is not cut).  Backward: dS, X and (bf16) its remainder.
struct GdrSpace {
    size_t ds, x, x2, si, m, bytes;
};
GdrSpace gdr_space(const kd_gdr_desc* d, const GdrSizes& s, bool packed, bool bwd) {
    const size_t n = s.slots * d->Hv, es = es_of(d->dtype);
    GdrSpace w = {};
    if (bwd) {
        w.x = up256(n * d->dv * d->dk * es);
        w.x2 = w.x + up256(n * kd::GDR_C * d->dv * es);
        w.bytes = w.x2 + (es == 2 ? up256(n * kd::GDR_C * d->dv * es) : 0);
        return w;
    }
    kd::GdrArgs a = gdr_args(d, s, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
    kd::gdr_plan(a, packed);
    w.si = s.rec;
    w.m = w.si + (a.nseg > 1 ? up256((size_t)a.segs * d->Hv * d->dv * d->dk * 4) : 0);
    w.bytes = w.m + (a.nseg > 1 ? up256((size_t)a.segs * d->Hv * d->dk * d->dk * 4) : 0);
    return w;
}

}  // namespace

extern "C" {

size_t kron_delta_gdr_saved_bytes(const kd_gdr_desc* d, int packed) {
    GdrSizes s;
    return check_gdr(d, packed != 0, &s) == KD_OK ? s.saved : 0;
}

size_t kron_delta_gdr_workspace_bytes(const kd_gdr_desc* d, int packed, int backward) {
    GdrSizes s;
    if (check_gdr(d, packed != 0, &s) != KD_OK) return 0;
    return gdr_space(d, s, packed != 0, backward != 0).bytes;
}

kd_status kron_delta_gdr_fwd(const kd_gdr_desc* d, const int32_t* cu, const void* q, const void* k, const void* v,
                             const void* g, const void* beta, const float* S0, void* o, float* ST, void* saved, void* ws,
                             size_t ws_bytes, void* stream) {
    GdrSizes s;
    const kd_status st = check_gdr(d, cu != nullptr, &s);
    if (st != KD_OK) return st;
    if (d->T > 0 && (!q || !k || !v || !g || !beta || !o)) return KD_ERR_NULL;
    const void* ptrs[] = {q, k, v, g, beta, S0, o, ST, saved, ws};
    for (const void* p : ptrs)
        if (misaligned(p)) return KD_ERR_ALIGN;
    if (((uintptr_t)cu & 3u) != 0) return KD_ERR_ALIGN;
    const GdrSpace w = gdr_space(d, s, cu != nullptr, false);
    const Range ins[] = {range_of(q, s.q),         range_of(k, s.k),       range_of(v, s.v),
                         range_of(g, s.gate),      range_of(beta, s.gate), range_of(S0, S0 ? s.state : 0),
                         range_of(cu, cu ? (size_t)(d->B + 1) * 4 : 0)};
    const Range outs[] = {range_of(o, s.o), range_of(ST, ST ? s.state : 0), range_of(saved, saved ? s.saved : 0), range_of(ws, ws ? w.bytes : 0)};
    if (any_overlap(outs, 4, ins, 7)) return KD_ERR_ALIAS;
    if (w.bytes > 0 && (!ws || ws_bytes < w.bytes)) return KD_ERR_WORKSPACE;
    if (d->T == 0 && !ST) return KD_OK;
    kd::GdrArgs a = gdr_args(d, s, q, k, v, g, beta, cu);
    a.S0 = S0;
    a.o = o;
    a.ST = ST;
    a.rec = saved ? saved : ws;
    a.hs = saved ? (char*)saved + s.rec : nullptr;
    kd::gdr_plan(a, cu != nullptr);
    if (w.m > w.si) {
        a.SI = (float*)((char*)ws + w.si);
        a.M = (float*)((char*)ws + w.m);
    }
    return done(kd::launch_gdr_fwd(d->dtype == KD_BF16, a, (hipStream_t)stream));
}

kd_status kron_delta_gdr_bwd(const kd_gdr_desc* d, const int32_t* cu, const void* q, const void* k, const void* v,
                             const void* g, const void* beta, const void* saved, const void* dO, const float* dST, void* dq,
                             void* dk, void* dv, void* dg, void* dbeta, float* dS0, void* ws, size_t ws_bytes,
                             void* stream) {
    GdrSizes s;
    const kd_status st = check_gdr(d, cu != nullptr, &s);
    if (st != KD_OK) return st;
    if (d->T > 0 && (!q || !k || !v || !g || !beta || !saved || !dO || !dq || !dk || !dv || !dg || !dbeta)) return KD_ERR_NULL;
    const void* ptrs[] = {q, k, v, g, beta, saved, dO, dST, dq, dk, dv, dg, dbeta, dS0, ws};
    for (const void* p : ptrs)
        if (misaligned(p)) return KD_ERR_ALIGN;
    if (((uintptr_t)cu & 3u) != 0) return KD_ERR_ALIGN;
    const GdrSpace w = gdr_space(d, s, cu != nullptr, true);
    const Range ins[] = {range_of(q, s.q),    range_of(k, s.k),       range_of(v, s.v),
                         range_of(g, s.gate), range_of(beta, s.gate), range_of(saved, saved ? s.saved : 0),
                         range_of(dO, s.o),   range_of(dST, dST ? s.state : 0), range_of(cu, cu ? (size_t)(d->B + 1) * 4 : 0)};
    const Range outs[] = {range_of(dq, s.qg),   range_of(dk, s.kg),      range_of(dv, s.o),
                          range_of(dg, s.gate), range_of(dbeta, s.gate), range_of(dS0, dS0 ? s.state : 0),
                          range_of(ws, ws ? w.bytes : 0)};
    if (any_overlap(outs, 7, ins, 9)) return KD_ERR_ALIAS;
    if (w.bytes > 0 && (!ws || ws_bytes < w.bytes)) return KD_ERR_WORKSPACE;
    if (d->T == 0 && !dS0) return KD_OK;
    kd::GdrArgs a = gdr_args(d, s, q, k, v, g, beta, cu);
    a.rec = const_cast<void*>(saved);
    a.hs = (char*)const_cast<void*>(saved) + s.rec;
    a.dO = dO;
    a.dST = dST;
    a.dq = dq;
    a.dk_ = dk;
    a.dv_ = dv;
    a.dg = dg;
    a.dbeta = dbeta;
    a.dS0 = dS0;
    a.ds = (char*)ws + w.ds;
    a.x = (char*)ws + w.x;
    a.x2 = (char*)ws + w.x2;
    return done(kd::launch_gdr_bwd(d->dtype == KD_BF16, a, (hipStream_t)stream));
}

kd_status kron_delta_gdr_step(const kd_gdr_desc* d, const void* q, const void* k, const void* v, const void* g,
                              const void* beta, const float* S_in, void* o, float* S_out, void* stream) {
    GdrSizes s;
    const kd_status st = check_gdr(d, false, &s);
    if (st != KD_OK) return st;
    if (d->T != 1) return KD_ERR_SHAPE;
    if (!q || !k || !v || !g || !beta || !S_in || !o || !S_out) return KD_ERR_NULL;
    const void* ptrs[] = {q, k, v, g, beta, S_in, o, S_out};
    for (const void* p : ptrs)
        if (misaligned(p)) return KD_ERR_ALIGN;
    const Range ins[] = {range_of(q, s.q),    range_of(k, s.k),       range_of(v, s.v),
                         range_of(g, s.gate), range_of(beta, s.gate), range_of(S_in == S_out ? nullptr : S_in, s.state)};
    const Range outs[] = {range_of(o, s.o), range_of(S_out, s.state)};
    if (any_overlap(outs, 2, ins, 6)) return KD_ERR_ALIAS;
    kd::GdrArgs a = gdr_args(d, s, q, k, v, g, beta, nullptr);
    a.S0 = S_in;
    a.o = o;
    a.ST = S_out;
    return done(kd::launch_gdr_step(d->dtype == KD_BF16, a, (hipStream_t)stream));
}

}  // extern "C"
