// kd_layers_api.hip -- the C ABI of the layers beside the mixer (gated linear
// recurrence, rotary positions, sliding-window attention): argument checks,
// workspace sizing and dispatch on the caller's stream.  No allocation, no
// synchronisation.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <utility>

#include "kd_check.h"
#include "kd_rope.h"
#include "kd_swa.h"
#include "kd_swa_decode.h"
#include "kron_delta.h"

namespace kd {
size_t glr_workspace_bytes(int bf16, int B, int T, int D);
bool glr_fits(int B, int T, int D);
hipError_t launch_glr_fwd(int bf16, const void* x, const void* f, const void* gi, const float* h0, void* h, float* hT,
                          float* hs, void* ws, int B, int T, int D, hipStream_t st);
hipError_t launch_glr_bwd(int bf16, const void* x, const void* f, const void* gi, const float* hs, const void* dh,
                          const float* dhT, void* dx, void* df, void* di, float* dh0, void* ws, int B, int T, int D,
                          hipStream_t st);
hipError_t launch_glr_step(int bf16, const void* x, const void* f, const void* gi, const float* h_in, void* y,
                           float* h_out, int64_t n, hipStream_t st);
bool rope_fits(int bf16, RopeArgs a);
hipError_t launch_rope(int bf16, const RopeArgs& a, hipStream_t st);
bool swa_fwd_fits(const SwaArgs& a);
hipError_t launch_swa_fwd(int bf16, int d, const SwaArgs& a, hipStream_t st);
bool swa_bwd_fits(bool packed, int N, int B, int Tq, int Tk, int Hq, int Hkv, int d, int W, int S);
hipError_t launch_swa_bwd(int bf16, int d, const SwaArgs& a, void* ws, hipStream_t st);
size_t swa_bwd_workspace_bytes(bool packed, int B, int Tq, int Tk, int Hq, int Hkv, int d, int W, int S);
hipError_t launch_swa_decode(int bf16, int d, const SwaDecodeArgs& a, hipStream_t st);
hipError_t launch_swa_store(const SwaStoreArgs& a, int B, hipStream_t st);
int swa_decode_splits(int B, int Hq, int Hkv, int seen);
size_t swa_decode_part_bytes(int B, int Hq, int Hkv, int d, int seen);
}  // namespace kd

namespace {

using kd::grid_fits;
using kd::misaligned;
using kd::overlap;
using kd::Range;
using kd::range_of;
using kd::up256;

bool known(int dtype) { return dtype == KD_F32 || dtype == KD_BF16; }
size_t es_of(int dtype) { return dtype == KD_BF16 ? 2 : 4; }

// Bytes a strided [n0, n1, n2, d] tensor spans from its first element; false
// for a negative stride or one that does not keep 16-byte pieces aligned
// (align16), or an extent beyond 2^62.
bool span(const int64_t st[3], int64_t n0, int64_t n1, int64_t n2, int64_t d, size_t es, bool align16, size_t* bytes) {
    const int64_t n[3] = {n0, n1, n2};
    if (n0 == 0 || n1 == 0 || n2 == 0) {
        *bytes = 0;
        return true;
    }
    __int128 last = d;
    for (int i = 0; i < 3; ++i) {
        if (st[i] < 0) return false;
        if (align16 && n[i] > 1 && (st[i] * (int64_t)es) % 16 != 0) return false;
        last += (__int128)st[i] * (n[i] - 1);
    }
    if (last * es > ((__int128)1 << 62)) return false;
    *bytes = (size_t)(last * es);
    return true;
}

// Whether no two elements of a strided [n0, n1, n2, d] tensor share an address
// (an output that is written as such): in the order of their strides, every
// dimension steps over all that the smaller ones span.
bool distinct(const int64_t st[3], int64_t n0, int64_t n1, int64_t n2, int64_t d) {
    int64_t n[3] = {n0, n1, n2}, s[3] = {st[0], st[1], st[2]};
    if (n0 == 0 || n1 == 0 || n2 == 0) return true;
    __int128 ext = d;
    for (int k = 0; k < 3; ++k) {
        int at = -1;
        for (int i = 0; i < 3; ++i)
            if (n[i] > 1 && (at < 0 || s[i] < s[at])) at = i;
        if (at < 0) return true;
        if (s[at] < ext) return false;
        ext += (__int128)s[at] * (n[at] - 1);
        n[at] = 1;
    }
    return true;
}

// Whether two tensors of one shape and the same strides, `delta` elements
// apart, share no address although their spans interleave: the shift falls in
// the gap that one dimension's stride leaves behind the smaller dimensions.
bool interleaved_apart(const int64_t st[3], int64_t n0, int64_t n1, int64_t n2, int64_t d, int64_t delta) {
    const int64_t n[3] = {n0, n1, n2};
    if (delta < 0) delta = -delta;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        __int128 ext = d;      // what the dimensions of smaller stride span
        for (int j = 0; j < 3; ++j)
            if (j != i && n[j] > 1 && st[j] < st[i]) ext += (__int128)st[j] * (n[j] - 1);
        if (delta >= ext && delta + ext <= st[i]) return true;
    }
    return false;
}

bool any_overlap(const Range* outs, int no, const Range* ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlap(outs[i], ins[j])) return true;
        for (int j = i + 1; j < no; ++j)
            if (overlap(outs[i], outs[j])) return true;
    }
    return false;
}

kd_status done(hipError_t e) { return e == hipSuccess ? KD_OK : KD_ERR_LAUNCH; }

// ------------------------------------------------- gated linear recurrence
kd_status check_glr(const kd_glr_desc* d) {
    if (!d) return KD_ERR_NULL;
    if (!known(d->dtype)) return KD_ERR_DTYPE;
    if (d->B < 1 || d->B > 65535 || d->D < 1 || d->T < 0 || d->T > (1 << 30) || d->D > (1 << 30)) return KD_ERR_SHAPE;
    return KD_OK;
}

size_t glr_chunks(const kd_glr_desc* d) {
    return ((size_t)d->T + KRON_DELTA_GLR_CHUNK - 1) / KRON_DELTA_GLR_CHUNK;
}

}  // namespace

extern "C" {

size_t kron_delta_glr_workspace_bytes(const kd_glr_desc* d) {
    if (check_glr(d) != KD_OK || !kd::glr_fits(d->B, d->T, d->D)) return 0;
    return kd::glr_workspace_bytes(d->dtype == KD_BF16, d->B, d->T, d->D);
}

kd_status kron_delta_glr_fwd(const kd_glr_desc* d, const void* x, const void* f, const void* i, const float* h0,
                             void* h, float* hT, float* hs, void* ws, size_t ws_bytes, void* stream) {
    const kd_status st = check_glr(d);
    if (st != KD_OK) return st;
    if (!kd::glr_fits(d->B, d->T, d->D)) return KD_ERR_SHAPE;
    const size_t n = (size_t)d->B * d->T * d->D, xb = n * es_of(d->dtype), sb = (size_t)d->B * d->D * 4;
    if (n > 0 && (!x || !f || !h)) return KD_ERR_NULL;
    const size_t need = kd::glr_workspace_bytes(d->dtype == KD_BF16, d->B, d->T, d->D);
    const void* ptrs[] = {x, f, i, h0, h, hT, hs, ws};
    for (const void* p : ptrs)
        if (misaligned(p)) return KD_ERR_ALIGN;
    const Range ins[] = {range_of(x, xb), range_of(f, xb), range_of(i, i ? xb : 0), range_of(h0, h0 ? sb : 0)};
    const Range outs[] = {range_of(h, xb), range_of(hT, hT ? sb : 0), range_of(hs, hs ? sb * glr_chunks(d) : 0),
                          range_of(ws, ws ? need : 0)};
    if (any_overlap(outs, 4, ins, 4)) return KD_ERR_ALIAS;
    if (need > 0 && (!ws || ws_bytes < need)) return KD_ERR_WORKSPACE;
    if (n == 0 && !hT) return KD_OK;
    return done(kd::launch_glr_fwd(d->dtype == KD_BF16, x, f, i, h0, h, hT, hs, ws, d->B, d->T, d->D,
                                   (hipStream_t)stream));
}

kd_status kron_delta_glr_bwd(const kd_glr_desc* d, const void* x, const void* f, const void* i, const float* hs,
                             const void* dh, const float* dhT, void* dx, void* df, void* di, float* dh0, void* ws,
                             size_t ws_bytes, void* stream) {
    const kd_status st = check_glr(d);
    if (st != KD_OK) return st;
    if (!kd::glr_fits(d->B, d->T, d->D)) return KD_ERR_SHAPE;
    const size_t n = (size_t)d->B * d->T * d->D, xb = n * es_of(d->dtype), sb = (size_t)d->B * d->D * 4;
    if (n > 0 && (!x || !f || !hs || !dh || !dx || !df || (i && !di))) return KD_ERR_NULL;
    const size_t need = kd::glr_workspace_bytes(d->dtype == KD_BF16, d->B, d->T, d->D);
    const void* ptrs[] = {x, f, i, hs, dh, dhT, dx, df, di, dh0, ws};
    for (const void* p : ptrs)
        if (misaligned(p)) return KD_ERR_ALIGN;
    const Range ins[] = {range_of(x, xb),  range_of(f, xb), range_of(i, i ? xb : 0), range_of(hs, sb * glr_chunks(d)),
                         range_of(dh, xb), range_of(dhT, dhT ? sb : 0)};
    const Range outs[] = {range_of(dx, xb), range_of(df, xb), range_of(di, i ? xb : 0), range_of(dh0, dh0 ? sb : 0),
                          range_of(ws, ws ? need : 0)};
    if (any_overlap(outs, 5, ins, 6)) return KD_ERR_ALIAS;
    if (need > 0 && (!ws || ws_bytes < need)) return KD_ERR_WORKSPACE;
    if (n == 0 && !dh0) return KD_OK;
    return done(kd::launch_glr_bwd(d->dtype == KD_BF16, x, f, i, hs, dh, dhT, dx, df, di, dh0, ws, d->B, d->T, d->D,
                                   (hipStream_t)stream));
}

kd_status kron_delta_glr_step(const kd_glr_desc* d, const void* x, const void* f, const void* i, const float* h_in,
                              void* y, float* h_out, void* stream) {
    const kd_status st = check_glr(d);
    if (st != KD_OK) return st;
    if (d->T != 1) return KD_ERR_SHAPE;
    const size_t n = (size_t)d->B * d->D, xb = n * es_of(d->dtype), sb = n * 4;
    if (!x || !f || !h_in || !y || !h_out) return KD_ERR_NULL;
    const void* ptrs[] = {x, f, i, h_in, y, h_out};
    for (const void* p : ptrs)
        if (misaligned(p)) return KD_ERR_ALIGN;
    const Range ins[] = {range_of(x, xb), range_of(f, xb), range_of(i, i ? xb : 0),
                         range_of(h_in == h_out ? nullptr : h_in, sb)};
    const Range outs[] = {range_of(y, xb), range_of(h_out, sb)};
    if (any_overlap(outs, 2, ins, 4)) return KD_ERR_ALIAS;
    return done(kd::launch_glr_step(d->dtype == KD_BF16, x, f, i, h_in, y, h_out, (int64_t)n, (hipStream_t)stream));
}

// ---------------------------------------------------------- rotary positions
// One of the tensors of a rotation, as its address, strides, heads and span.
struct RopeHeads {
    const void* p;
    const int64_t* st;
    int heads;
    size_t bytes;
};

// Whether two of them share no address: apart in memory, or different heads of
// one tensor with the batch and token strides of both, in any order.  The
// heads of both then lie in one block per token, or go on from one to the
// other in steps of the head stride.
static bool rope_apart(const kd_rope_desc* d, RopeHeads a, RopeHeads b, int64_t es) {
    if (a.heads == 0 || b.heads == 0 || !overlap(range_of(a.p, a.bytes), range_of(b.p, b.bytes))) return true;
    if ((d->B > 1 && a.st[0] != b.st[0]) || (d->T > 1 && a.st[1] != b.st[1])) return false;
    if ((const char*)a.p > (const char*)b.p) std::swap(a, b);
    const int64_t bytes = (const char*)b.p - (const char*)a.p, gap = bytes / es;
    if (bytes % es != 0) return false;
    const int64_t block[3] = {a.st[0], a.st[1], 0};
    const __int128 ea = (__int128)a.st[2] * (a.heads - 1) + d->d, eb = (__int128)b.st[2] * (b.heads - 1) + d->d;
    if (gap >= ea && gap + eb < INT64_MAX && distinct(block, d->B, d->T, 1, (int64_t)(gap + eb))) return true;
    const int64_t step = a.heads > 1 ? a.st[2] : b.heads > 1 ? b.st[2] : gap;
    if (step <= 0 || gap % step != 0 || gap / step < a.heads || (a.heads > 1 && b.heads > 1 && a.st[2] != b.st[2])) return false;
    const int64_t all[3] = {a.st[0], a.st[1], step};
    return distinct(all, d->B, d->T, gap / step + b.heads, d->d);
}

kd_status kron_delta_rope(const kd_rope_desc* d, const void* q, const void* k, const void* pos, const double* freqs,
                          void* q_out, void* k_out, void* stream) {
    if (!d) return KD_ERR_NULL;
    if (!known(d->dtype)) return KD_ERR_DTYPE;
    if (d->B < 1 || d->T < 0 || d->Hq < 1 || d->Hk < 0 || d->d < 1 || d->d > kd::ROPE_MAX_D || d->rot < 2 ||
        d->rot > d->d || d->rot % 2 != 0 || d->layout < 0 || d->layout > 1 || !isfinite(d->scale))
        return KD_ERR_SHAPE;
    if (d->Hq > kd::ROPE_MAX_H || d->Hk > kd::ROPE_MAX_H || (int64_t)d->B * d->T > INT32_MAX) return KD_ERR_SHAPE;
    const size_t es = es_of(d->dtype);
    size_t qi, ki, qo, ko;
    if (!span(d->q_stride, d->B, d->T, d->Hq, d->d, es, false, &qi) ||
        !span(d->k_stride, d->B, d->T, d->Hk, d->d, es, false, &ki) ||
        !span(d->q_out_stride, d->B, d->T, d->Hq, d->d, es, false, &qo) ||
        !span(d->k_out_stride, d->B, d->T, d->Hk, d->d, es, false, &ko))
        return KD_ERR_SHAPE;
    if (!distinct(d->q_out_stride, d->B, d->T, d->Hq, d->d) || !distinct(d->k_out_stride, d->B, d->T, d->Hk, d->d))
        return KD_ERR_ALIAS;
    const int64_t ntok = (int64_t)d->B * d->T;
    if (ntok == 0) return KD_OK;
    if (!q || !q_out || !pos || !freqs || (d->Hk > 0 && (!k || !k_out))) return KD_ERR_NULL;
    if (((uintptr_t)pos % (d->pos64 ? 8 : 4)) != 0 || ((uintptr_t)freqs & 7u) != 0) return KD_ERR_ALIGN;
    const void* ptrs[] = {q, k, q_out, k_out};
    for (const void* p : ptrs)
        if (((uintptr_t)p % es) != 0) return KD_ERR_ALIGN;
    // in place: the same tensor, strides included
    const bool sq = q == q_out && d->q_stride[0] == d->q_out_stride[0] && d->q_stride[1] == d->q_out_stride[1] &&
                    d->q_stride[2] == d->q_out_stride[2];
    const bool sk = k == k_out && d->k_stride[0] == d->k_out_stride[0] && d->k_stride[1] == d->k_out_stride[1] &&
                    d->k_stride[2] == d->k_out_stride[2];
    const Range rp = range_of(pos, (size_t)(d->pos_batched ? ntok : d->T) * (d->pos64 ? 8 : 4));
    const Range rf = range_of(freqs, (size_t)(d->rot / 2) * 8);
    // q and k (in or out) may be the heads of one tensor
    const RopeHeads hq = {q, d->q_stride, d->Hq, qi}, hk = {k, d->k_stride, d->Hk, ki};
    const RopeHeads gq = {q_out, d->q_out_stride, d->Hq, qo}, gk = {k_out, d->k_out_stride, d->Hk, ko};
    if (!rope_apart(d, gq, gk, es) || !rope_apart(d, gq, hk, es) || !rope_apart(d, gk, hq, es) ||
        (!sq && !rope_apart(d, gq, hq, es)) || (!sk && !rope_apart(d, gk, hk, es)))
        return KD_ERR_ALIAS;
    const Range oq = range_of(q_out, qo), ok = range_of(k_out, ko);
    if (overlap(oq, rp) || overlap(oq, rf) || overlap(ok, rp) || overlap(ok, rf)) return KD_ERR_ALIAS;
    kd::RopeArgs a;
    a.side[0] = {q, q_out, {d->q_stride[0], d->q_stride[1], d->q_stride[2]},
                 {d->q_out_stride[0], d->q_out_stride[1], d->q_out_stride[2]}, d->Hq};
    a.side[1] = {k, k_out, {d->k_stride[0], d->k_stride[1], d->k_stride[2]},
                 {d->k_out_stride[0], d->k_out_stride[1], d->k_out_stride[2]}, d->Hk};
    a.pos = pos;
    a.freqs = freqs;
    a.B = d->B;
    a.T = d->T;
    a.d = d->d;
    a.rot = d->rot;
    a.pos64 = d->pos64 != 0;
    a.pos_batched = d->pos_batched != 0;
    a.interleaved = d->layout == KD_ROPE_INTERLEAVED;
    a.inverse = d->inverse != 0;
    a.scale = d->scale;
    if (!kd::rope_fits(d->dtype == KD_BF16, a)) return KD_ERR_SHAPE;
    return done(kd::launch_rope(d->dtype == KD_BF16, a, (hipStream_t)stream));
}

// ------------------------------------------------- sliding-window attention
namespace {

struct SwaSpans {
    size_t q, k, v, o, kg;   // bytes spanned by q, k, v and by contiguous o and dk
};

kd_status check_swa(const kd_swa_desc* d, bool packed, SwaSpans* s) {
    if (!d) return KD_ERR_NULL;
    if (!known(d->dtype)) return KD_ERR_DTYPE;
    if (d->B < 1 || d->Tq < 0 || d->Tk < 0 || d->Tq > (1 << 29) || d->Tk > (1 << 29) || d->Hq < 1 || d->Hkv < 1 ||
        d->Hq > 65535 || d->Hq % d->Hkv != 0 || (d->d != 32 && d->d != 64 && d->d != 128) || d->window < 1 ||
        d->sinks < 0 || d->sinks > kd::SWA_MAX_SINKS || !(d->scale > 0.f) || !isfinite(d->scale))
        return KD_ERR_SHAPE;
    if (packed) {
        // one packed batch element of Tq == Tk rows, B sequences
        if (d->Tq != d->Tk || d->B > (1 << 24)) return KD_ERR_SHAPE;
    } else if (d->B > 65535) {
        return KD_ERR_SHAPE;
    }
    const size_t es = es_of(d->dtype);
    const int64_t nb = packed ? 1 : d->B;
    if (!span(d->q_stride, nb, d->Tq, d->Hq, d->d, es, true, &s->q) ||
        !span(d->k_stride, nb, d->Tk, d->Hkv, d->d, es, true, &s->k) ||
        !span(d->v_stride, nb, d->Tk, d->Hkv, d->d, es, true, &s->v))
        return KD_ERR_SHAPE;
    s->o = (size_t)nb * d->Tq * d->Hq * d->d * es;
    s->kg = (size_t)nb * d->Tk * d->Hkv * d->d * es;
    return KD_OK;
}

bool swa_bwd_fits(const kd_swa_desc* d, bool packed) {
    return kd::swa_bwd_fits(packed, d->B, packed ? 1 : d->B, d->Tq, d->Tk, d->Hq, d->Hkv, d->d, d->window, d->sinks);
}

kd::SwaArgs swa_args(const kd_swa_desc* d, const int32_t* cu, const void* q, const void* k, const void* v) {
    kd::SwaArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    for (int i = 0; i < 3; ++i) {
        a.qs[i] = d->q_stride[i];
        a.ks[i] = d->k_stride[i];
        a.vs[i] = d->v_stride[i];
    }
    a.cu = cu;
    a.N = cu ? d->B : 0;
    a.B = cu ? 1 : d->B;
    a.Tq = d->Tq;
    a.Tk = d->Tk;
    a.Hq = d->Hq;
    a.Hkv = d->Hkv;
    a.W = d->window < d->Tk ? d->window : (d->Tk > 0 ? d->Tk : 1);   // a wider window sees no more
    a.S = d->sinks;
    a.scale = d->scale;
    a.c = d->scale * 1.4426950408889634f;
    return a;
}

}  // namespace

size_t kron_delta_swa_workspace_bytes(const kd_swa_desc* d, int packed) {
    SwaSpans s;
    if (check_swa(d, packed != 0, &s) != KD_OK || !swa_bwd_fits(d, packed != 0)) return 0;
    return kd::swa_bwd_workspace_bytes(packed != 0, d->B, d->Tq, d->Tk, d->Hq, d->Hkv, d->d, d->window, d->sinks);
}

kd_status kron_delta_swa_fwd(const kd_swa_desc* d, const int32_t* cu, const void* q, const void* k, const void* v,
                             void* o, float* lse, void* stream) {
    SwaSpans s;
    const kd_status st = check_swa(d, cu != nullptr, &s);
    if (st != KD_OK) return st;
    if (d->Tq == 0) return KD_OK;
    if (!q || !o || (d->Tk > 0 && (!k || !v))) return KD_ERR_NULL;
    const void* ptrs[] = {q, k, v, o};
    for (const void* p : ptrs)
        if (misaligned(p)) return KD_ERR_ALIGN;
    if (((uintptr_t)lse & 3u) != 0 || ((uintptr_t)cu & 3u) != 0) return KD_ERR_ALIGN;
    const size_t lb = s.o / es_of(d->dtype) / d->d * 4;
    const Range ins[] = {range_of(q, s.q), range_of(k, s.k), range_of(v, s.v),
                         range_of(cu, cu ? ((size_t)d->B + 1) * 4 : 0)};
    const Range outs[] = {range_of(o, s.o), range_of(lse, lse ? lb : 0)};
    if (any_overlap(outs, 2, ins, 4)) return KD_ERR_ALIAS;
    kd::SwaArgs a = swa_args(d, cu, q, k, v);
    a.o = o;
    a.lse = lse;
    if (!kd::swa_fwd_fits(a)) return KD_ERR_SHAPE;
    return done(kd::launch_swa_fwd(d->dtype == KD_BF16, d->d, a, (hipStream_t)stream));
}

kd_status kron_delta_swa_bwd(const kd_swa_desc* d, const int32_t* cu, const void* q, const void* k, const void* v,
                             const void* o, const float* lse, const void* dO, void* dq, void* dk, void* dv, void* ws,
                             size_t ws_bytes, void* stream) {
    SwaSpans s;
    const kd_status st = check_swa(d, cu != nullptr, &s);
    if (st != KD_OK) return st;
    if (!swa_bwd_fits(d, cu != nullptr)) return KD_ERR_SHAPE;
    if (d->Tk == 0 && d->Tq == 0) return KD_OK;
    if (d->Tq > 0 && (!q || !o || !lse || !dO || !dq)) return KD_ERR_NULL;
    if (d->Tk > 0 && (!k || !v || !dk || !dv)) return KD_ERR_NULL;
    const void* ptrs[] = {q, k, v, o, dO, dq, dk, dv, ws};
    for (const void* p : ptrs)
        if (misaligned(p)) return KD_ERR_ALIGN;
    if (((uintptr_t)lse & 3u) != 0 || ((uintptr_t)cu & 3u) != 0) return KD_ERR_ALIGN;
    const size_t lb = s.o / es_of(d->dtype) / d->d * 4;
    const size_t need = kron_delta_swa_workspace_bytes(d, cu != nullptr);
    const Range ins[] = {range_of(q, s.q),   range_of(k, s.k),  range_of(v, s.v), range_of(o, s.o),
                         range_of(lse, lb), range_of(dO, s.o), range_of(cu, cu ? ((size_t)d->B + 1) * 4 : 0)};
    const Range outs[] = {range_of(dq, s.o), range_of(dk, s.kg), range_of(dv, s.kg), range_of(ws, ws ? need : 0)};
    if (any_overlap(outs, 4, ins, 7)) return KD_ERR_ALIAS;
    if (need > 0 && (!ws || ws_bytes < need)) return KD_ERR_WORKSPACE;
    kd::SwaArgs a = swa_args(d, cu, q, k, v);
    a.o = const_cast<void*>(o);
    a.lse = const_cast<float*>(lse);
    a.dO = dO;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    return done(kd::launch_swa_bwd(d->dtype == KD_BF16, d->d, a, ws, (hipStream_t)stream));
}

namespace {

kd_status check_cache(const kd_swa_cache_desc* d, size_t* kc, size_t* vc) {
    if (!d) return KD_ERR_NULL;
    if (!known(d->dtype)) return KD_ERR_DTYPE;
    if (d->B < 1 || d->B > 65535 || d->Hq < 1 || d->Hkv < 1 || d->Hq > 65535 || d->Hq % d->Hkv != 0 ||
        (d->d != 32 && d->d != 64 && d->d != 128) || d->window < 1 || d->sinks < 0 || d->sinks > kd::SWA_MAX_SINKS ||
        (int64_t)d->cap < (int64_t)d->sinks + d->window || d->cap > (1 << 30) || !(d->scale > 0.f) ||
        !isfinite(d->scale))
        return KD_ERR_SHAPE;
    const size_t es = es_of(d->dtype);
    if (!span(d->k_stride, d->B, d->cap, d->Hkv, d->d, es, true, kc) ||
        !span(d->v_stride, d->B, d->cap, d->Hkv, d->d, es, true, vc))
        return KD_ERR_SHAPE;
    if (!distinct(d->k_stride, d->B, d->cap, d->Hkv, d->d) || !distinct(d->v_stride, d->B, d->cap, d->Hkv, d->d))
        return KD_ERR_ALIAS;
    return KD_OK;
}

// Whether the two caches share an address.  Views of one allocation, such as
// [B, cap, 2, Hkv, d], interleave without doing so.
bool caches_overlap(const kd_swa_cache_desc* d, const void* k, size_t kb, const void* v, size_t vb) {
    if (!overlap(range_of(k, kb), range_of(v, vb))) return false;
    for (int i = 0; i < 3; ++i)
        if (d->k_stride[i] != d->v_stride[i]) return true;
    const int64_t es = (int64_t)es_of(d->dtype), delta = (const char*)v - (const char*)k;
    return !interleaved_apart(d->k_stride, d->B, d->cap, d->Hkv, d->d, delta / es);
}

}  // namespace

size_t kron_delta_swa_decode_workspace_bytes(const kd_swa_cache_desc* d) {
    size_t kc, vc;
    if (check_cache(d, &kc, &vc) != KD_OK) return 0;
    return kd::SWA_DECODE_COUNTERS * sizeof(int) +
           up256(kd::swa_decode_part_bytes(d->B, d->Hq, d->Hkv, d->d, d->window + d->sinks));
}

kd_status kron_delta_swa_decode(const kd_swa_cache_desc* d, const void* q, const void* k, const void* v,
                                const int64_t in_stride[3], void* k_cache, void* v_cache, const int32_t* lens,
                                const double* freqs, void* o, void* ws, size_t ws_bytes, void* stream) {
    size_t kcb, vcb;
    const kd_status st = check_cache(d, &kcb, &vcb);
    if (st != KD_OK) return st;
    if (d->rot < 0 || d->rot > d->d || d->rot % 2 != 0 || d->layout < 0 || d->layout > 1 || !isfinite(d->rope_scale))
        return KD_ERR_SHAPE;
    if (!q || !k || !v || !in_stride || !k_cache || !v_cache || !lens || !o || (d->rot > 0 && !freqs))
        return KD_ERR_NULL;
    const size_t es = es_of(d->dtype);
    const int64_t qs[3] = {in_stride[0], 0, d->d}, ks[3] = {in_stride[1], 0, d->d}, vs[3] = {in_stride[2], 0, d->d};
    size_t qb, kb, vb;
    if (!span(qs, d->B, 1, d->Hq, d->d, es, false, &qb) || !span(ks, d->B, 1, d->Hkv, d->d, es, false, &kb) ||
        !span(vs, d->B, 1, d->Hkv, d->d, es, false, &vb))
        return KD_ERR_SHAPE;
    const void* ptrs[] = {k_cache, v_cache, o, ws};
    for (const void* p : ptrs)
        if (misaligned(p)) return KD_ERR_ALIGN;
    const void* small[] = {q, k, v};
    for (const void* p : small)
        if (((uintptr_t)p % es) != 0) return KD_ERR_ALIGN;
    if (((uintptr_t)lens & 3u) != 0 || ((uintptr_t)freqs & 7u) != 0) return KD_ERR_ALIGN;
    const size_t need = kron_delta_swa_decode_workspace_bytes(d);
    const Range ins[] = {range_of(q, qb), range_of(k, kb), range_of(v, vb), range_of(lens, (size_t)d->B * 4),
                         range_of(freqs, freqs ? (size_t)(d->rot / 2) * 8 : 0)};
    const Range outs[] = {range_of(k_cache, kcb), range_of(v_cache, vcb),
                          range_of(o, (size_t)d->B * d->Hq * d->d * es), range_of(ws, ws ? need : 0)};
    for (const Range& a : outs)
        for (const Range& b : ins)
            if (overlap(a, b)) return KD_ERR_ALIAS;
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 4; ++j)
            if (i == 0 && j == 1 ? caches_overlap(d, k_cache, kcb, v_cache, vcb) : overlap(outs[i], outs[j]))
                return KD_ERR_ALIAS;
    if (!ws || ws_bytes < need) return KD_ERR_WORKSPACE;
    kd::SwaDecodeArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.qb = in_stride[0];
    a.kb = in_stride[1];
    a.vb = in_stride[2];
    a.kc = k_cache;
    a.vc = v_cache;
    for (int i = 0; i < 3; ++i) {
        a.kcs[i] = d->k_stride[i];
        a.vcs[i] = d->v_stride[i];
    }
    a.lens = lens;
    a.freqs = freqs;
    a.o = o;
    a.count = (int*)ws;
    a.part = (float*)((int*)ws + kd::SWA_DECODE_COUNTERS);
    a.B = d->B;
    a.Hq = d->Hq;
    a.Hkv = d->Hkv;
    a.cap = d->cap;
    a.W = d->window;
    a.S = d->sinks;
    a.rot = d->rot;
    a.interleaved = d->layout == KD_ROPE_INTERLEAVED;
    a.nsplit = kd::swa_decode_splits(d->B, d->Hq, d->Hkv, d->window + d->sinks);
    a.c = d->scale * 1.4426950408889634f;
    a.rope_scale = d->rope_scale;
    return done(kd::launch_swa_decode(d->dtype == KD_BF16, d->d, a, (hipStream_t)stream));
}

kd_status kron_delta_swa_cache_store(const kd_swa_cache_desc* d, int32_t T, const void* k, const void* v,
                                     const int64_t k_stride[3], const int64_t v_stride[3], const int32_t* lens,
                                     void* k_cache, void* v_cache, void* stream) {
    size_t kcb, vcb, kb, vb;
    const kd_status st = check_cache(d, &kcb, &vcb);
    if (st != KD_OK) return st;
    if (T < 0 || T > (1 << 30)) return KD_ERR_SHAPE;
    if (T == 0) return KD_OK;
    if (!k || !v || !k_stride || !v_stride || !k_cache || !v_cache) return KD_ERR_NULL;
    const size_t es = es_of(d->dtype);
    if (!span(k_stride, d->B, T, d->Hkv, d->d, es, true, &kb) || !span(v_stride, d->B, T, d->Hkv, d->d, es, true, &vb))
        return KD_ERR_SHAPE;
    kd::SwaStoreArgs a = {};
    a.row = (int)(d->d * es / 16);
    if (!grid_fits(((int64_t)T * d->Hkv * a.row + 255) / 256, 256)) return KD_ERR_SHAPE;
    const void* ptrs[] = {k, v, k_cache, v_cache};
    for (const void* p : ptrs)
        if (misaligned(p)) return KD_ERR_ALIGN;
    if (((uintptr_t)lens & 3u) != 0) return KD_ERR_ALIGN;
    const Range ins[] = {range_of(k, kb), range_of(v, vb), range_of(lens, lens ? (size_t)d->B * 4 : 0)};
    const Range outs[] = {range_of(k_cache, kcb), range_of(v_cache, vcb)};
    for (const Range& o : outs)
        for (const Range& i : ins)
            if (overlap(o, i)) return KD_ERR_ALIAS;
    if (caches_overlap(d, k_cache, kcb, v_cache, vcb)) return KD_ERR_ALIAS;
    a.k = k;
    a.v = v;
    for (int i = 0; i < 3; ++i) {
        a.ks[i] = k_stride[i];
        a.vs[i] = v_stride[i];
        a.kcs[i] = d->k_stride[i];
        a.vcs[i] = d->v_stride[i];
    }
    a.kc = k_cache;
    a.vc = v_cache;
    a.lens = lens;
    a.T = T;
    a.Hkv = d->Hkv;
    a.es = (int)es;
    a.cap = d->cap;
    a.S = d->sinks;
    return done(kd::launch_swa_store(a, d->B, (hipStream_t)stream));
}

}  // extern "C"
