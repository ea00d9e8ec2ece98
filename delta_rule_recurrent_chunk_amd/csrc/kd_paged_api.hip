// kd_paged_api.hip -- the C ABI of the paged cache and of the attention over a
// shared prefix: argument checks, workspace sizing and dispatch on the caller's
// stream.  No allocation, no synchronisation.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kd_check.h"
#include "kd_paged.h"
#include "kd_rope.h"
#include "kron_delta.h"

namespace kd {
bool append_fits(int bf16, AppendArgs a);
hipError_t launch_append(int bf16, const AppendArgs& a, hipStream_t st);
bool prefix_fits(PrefixArgs a, bool packed);
size_t prefix_workspace_bytes(PrefixArgs a, int d, bool packed);
hipError_t launch_prefix(int bf16, int d, const PrefixArgs& a, hipStream_t st);
}  // namespace kd

namespace {

using kd::any_overlap;
using kd::distinct;
using kd::interleaved_apart;
using kd::misaligned;
using kd::overlap;
using kd::Range;
using kd::range_of;
using kd::span;
using kd::up256;

bool known(int dtype) { return dtype == KD_F32 || dtype == KD_BF16; }
size_t es_of(int dtype) { return dtype == KD_BF16 ? 2 : 4; }
kd_status done(hipError_t e) { return e == hipSuccess ? KD_OK : KD_ERR_LAUNCH; }

// What both operators ask of a batch and its cache; the bytes the pages span.
kd_status check_paged(const kd_paged_desc* d, size_t* kc, size_t* vc) {
    if (!d) return KD_ERR_NULL;
    if (!known(d->dtype)) return KD_ERR_DTYPE;
    if (d->B < 1 || d->B > (1 << 24) || d->T < 0 || d->T > (1 << 29) || d->Hq < 0 || d->Hq > kd::ROPE_MAX_H || d->Hkv < 1 ||
        d->Hkv > kd::ROPE_MAX_H || d->d < 1 || d->page < 1 || d->pages < 1 || d->width < 0 || d->table_stride < 0)
        return KD_ERR_SHAPE;
    const size_t es = es_of(d->dtype);
    if (d->d * es % 16 != 0) return KD_ERR_SHAPE;
    if (!span(d->k_stride, d->pages, d->page, d->Hkv, d->d, es, true, kc) ||
        !span(d->v_stride, d->pages, d->page, d->Hkv, d->d, es, true, vc))
        return KD_ERR_SHAPE;
    return KD_OK;
}

// Bytes of a [T, H, d] tensor with strides over token and head.
bool rows_span(const int64_t st[2], int64_t T, int64_t H, int64_t d, size_t es, size_t* bytes) {
    const int64_t s[3] = {0, st[0], st[1]};
    return span(s, 1, T, H, d, es, true, bytes);
}

size_t table_bytes(const kd_paged_desc* d) {
    return d->width == 0 ? 0 : ((size_t)d->table_stride * (d->B - 1) + d->width) * 4;
}

kd::PrefixArgs prefix_args(const kd_paged_desc* d) {
    kd::PrefixArgs a = {};
    for (int i = 0; i < 3; ++i) {
        a.kcs[i] = d->k_stride[i];
        a.vcs[i] = d->v_stride[i];
    }
    a.ts = d->table_stride;
    a.B = d->B;
    a.T = d->T;
    a.Hq = d->Hq;
    a.Hkv = d->Hkv;
    a.page = d->page;
    a.pages = d->pages;
    a.width = d->width;
    a.P = d->prefix;
    a.scale = d->scale;
    a.c = d->scale * 1.4426950408889634f;
    return a;
}

kd_status check_prefix(const kd_paged_desc* d, bool packed, size_t* kc, size_t* vc) {
    const kd_status st = check_paged(d, kc, vc);
    if (st != KD_OK) return st;
    if (d->Hq < 1 || d->Hq % d->Hkv != 0 || (d->d != 32 && d->d != 64 && d->d != 128) || d->prefix < 0 ||
        d->prefix > (1 << 30) || d->prefix_width < 0 || (int64_t)d->prefix > (int64_t)d->prefix_width * d->page ||
        !(d->scale > 0.f) || !isfinite(d->scale) || (!packed && d->T != d->B))
        return KD_ERR_SHAPE;
    return d->T == 0 || kd::prefix_fits(prefix_args(d), packed) ? KD_OK : KD_ERR_SHAPE;
}

}  // namespace

extern "C" {

kd_status kron_delta_paged_append(const kd_paged_desc* d, const void* q, const void* k, const void* v,
                                  const int64_t in_stride[6], void* k_pages, void* v_pages, const int32_t* table,
                                  const int32_t* lens, const int32_t* cu, const double* freqs, void* q_out, void* stream) {
    size_t kcb, vcb;
    const kd_status st = check_paged(d, &kcb, &vcb);
    if (st != KD_OK) return st;
    if (d->d > kd::APPEND_MAX_D || d->rot < 0 || d->rot > d->d || d->rot % 2 != 0 || d->layout < 0 || d->layout > 1 ||
        !isfinite(d->rope_scale) || d->offset < -((int64_t)1 << 40) || d->offset > ((int64_t)1 << 40) || (!cu && d->T != d->B))
        return KD_ERR_SHAPE;
    if (!distinct(d->k_stride, d->pages, d->page, d->Hkv, d->d) || !distinct(d->v_stride, d->pages, d->page, d->Hkv, d->d))
        return KD_ERR_ALIAS;
    if (d->T == 0) return KD_OK;
    if (!k || !v || !in_stride || !k_pages || !v_pages || (d->width > 0 && !table) || !lens || (d->rot > 0 && !freqs) ||
        (d->Hq > 0 && (!q || !q_out)))
        return KD_ERR_NULL;
    const size_t es = es_of(d->dtype);
    size_t qb, kb, vb;
    if (!rows_span(in_stride, d->T, d->Hq, d->d, es, &qb) || !rows_span(in_stride + 2, d->T, d->Hkv, d->d, es, &kb) ||
        !rows_span(in_stride + 4, d->T, d->Hkv, d->d, es, &vb))
        return KD_ERR_SHAPE;
    const void* ptrs[] = {q, k, v, k_pages, v_pages, q_out};
    for (const void* p : ptrs)
        if (misaligned(p)) return KD_ERR_ALIGN;
    if ((((uintptr_t)table | (uintptr_t)lens | (uintptr_t)cu) & 3u) != 0 || ((uintptr_t)freqs & 7u) != 0) return KD_ERR_ALIGN;
    const Range ins[] = {range_of(q, qb),
                         range_of(k, kb),
                         range_of(v, vb),
                         range_of(table, table_bytes(d)),
                         range_of(lens, (size_t)d->B * 4),
                         range_of(cu, cu ? (size_t)(d->B + 1) * 4 : 0),
                         range_of(freqs, d->rot > 0 ? (size_t)(d->rot / 2) * 8 : 0)};
    const Range outs[] = {range_of(k_pages, kcb), range_of(v_pages, vcb),
                          range_of(q_out, (size_t)d->T * d->Hq * d->d * es)};
    for (const Range& o : outs)
        for (const Range& i : ins)
            if (overlap(o, i)) return KD_ERR_ALIAS;
    if (overlap(outs[0], outs[2]) || overlap(outs[1], outs[2])) return KD_ERR_ALIAS;
    if (overlap(outs[0], outs[1])) {      // the two may be views of one allocation that interleave
        for (int i = 0; i < 3; ++i)
            if (d->k_stride[i] != d->v_stride[i]) return KD_ERR_ALIAS;
        const int64_t delta = (const char*)v_pages - (const char*)k_pages;
        if (!interleaved_apart(d->k_stride, d->pages, d->page, d->Hkv, d->d, delta / (int64_t)es)) return KD_ERR_ALIAS;
    }
    kd::AppendArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    for (int i = 0; i < 2; ++i) {
        a.qs[i] = in_stride[i];
        a.ks[i] = in_stride[2 + i];
        a.vs[i] = in_stride[4 + i];
    }
    a.qo = q_out;
    a.kc = k_pages;
    a.vc = v_pages;
    for (int i = 0; i < 3; ++i) {
        a.kcs[i] = d->k_stride[i];
        a.vcs[i] = d->v_stride[i];
    }
    a.table = table;
    a.lens = lens;
    a.cu = cu;
    a.ts = d->table_stride;
    a.freqs = freqs;
    a.offset = d->offset;
    a.B = d->B;
    a.T = d->T;
    a.Hq = d->Hq;
    a.Hkv = d->Hkv;
    a.d = d->d;
    a.rot = d->rot;
    a.page = d->page;
    a.pages = d->pages;
    a.width = d->width;
    a.interleaved = d->layout == KD_ROPE_INTERLEAVED;
    a.scale = d->rope_scale;
    if (!kd::append_fits(d->dtype == KD_BF16, a)) return KD_ERR_SHAPE;
    return done(kd::launch_append(d->dtype == KD_BF16, a, (hipStream_t)stream));
}

size_t kron_delta_prefix_attn_workspace_bytes(const kd_paged_desc* d, int packed) {
    size_t kc, vc;
    if (check_prefix(d, packed != 0, &kc, &vc) != KD_OK || d->T == 0) return 0;
    return up256(kd::prefix_workspace_bytes(prefix_args(d), d->d, packed != 0));
}

kd_status kron_delta_prefix_attn(const kd_paged_desc* d, const void* q, const int64_t q_stride[2], const void* k_pages,
                                 const void* v_pages, const int32_t* prefix_table, const int32_t* table,
                                 const int32_t* lens, const int32_t* cu, void* o, float* lse, void* ws, size_t ws_bytes,
                                 void* stream) {
    size_t kcb, vcb, qb;
    const kd_status st = check_prefix(d, cu != nullptr, &kcb, &vcb);
    if (st != KD_OK) return st;
    if (d->T == 0) return KD_OK;
    if (!q || !q_stride || !k_pages || !v_pages || (d->prefix > 0 && !prefix_table) || (d->width > 0 && !table) || !lens || !o)
        return KD_ERR_NULL;
    const size_t es = es_of(d->dtype);
    if (!rows_span(q_stride, d->T, d->Hq, d->d, es, &qb)) return KD_ERR_SHAPE;
    const void* ptrs[] = {q, k_pages, v_pages, o, ws};
    for (const void* p : ptrs)
        if (misaligned(p)) return KD_ERR_ALIGN;
    if ((((uintptr_t)prefix_table | (uintptr_t)table | (uintptr_t)lens | (uintptr_t)cu | (uintptr_t)lse) & 3u) != 0)
        return KD_ERR_ALIGN;
    const size_t need = kron_delta_prefix_attn_workspace_bytes(d, cu != nullptr);
    const Range ins[] = {range_of(q, qb),
                         range_of(k_pages, kcb),
                         range_of(v_pages, vcb),
                         range_of(prefix_table, d->prefix > 0 ? (size_t)d->prefix_width * 4 : 0),
                         range_of(table, table_bytes(d)),
                         range_of(lens, (size_t)d->B * 4),
                         range_of(cu, cu ? (size_t)(d->B + 1) * 4 : 0)};
    const Range outs[] = {range_of(o, (size_t)d->T * d->Hq * d->d * es), range_of(lse, lse ? (size_t)d->T * d->Hq * 4 : 0),
                          range_of(ws, ws ? need : 0)};
    if (any_overlap(outs, 3, ins, 7)) return KD_ERR_ALIAS;
    if (!ws || ws_bytes < need) return KD_ERR_WORKSPACE;
    kd::PrefixArgs a = prefix_args(d);
    a.q = q;
    a.qs[0] = q_stride[0];
    a.qs[1] = q_stride[1];
    a.kc = k_pages;
    a.vc = v_pages;
    a.ptable = prefix_table;
    a.table = table;
    a.lens = lens;
    a.cu = cu;
    a.o = o;
    a.lse = lse;
    a.part = (float*)ws;
    return done(kd::launch_prefix(d->dtype == KD_BF16, d->d, a, (hipStream_t)stream));
}

}  // extern "C"
