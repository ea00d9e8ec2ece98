"""A paged cache and attention over a shared prefix -- binding of their part of the C ABI.

    q = paged_append(k, v, k_pages, v_pages, page_table, lens, q=q, freqs=freqs)      tokens into the cache
    o = prefix_attn(q, k_pages, v_pages, prefix_table, prefix_len, page_table, lens)  attention over it

Argument marshalling only, as in the package's module; ``include/kron_delta.h`` defines both operators.
"""
from __future__ import annotations

import ctypes
import math

from . import layers as _la
from .layers import _call, _check, _code, _fits, _freqs, _int32, _layout, _need_cuda, _ptr, _ready, _same_device, _workspace

EXPORTED = ("kron_delta_paged_append", "kron_delta_prefix_attn_workspace_bytes", "kron_delta_prefix_attn")

_i32, _i64, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_s2, _s3, _s6 = _i64 * 2, _i64 * 3, _i64 * 6


class KdPagedDesc(ctypes.Structure):
    _fields_ = [("B", _i32), ("T", _i32), ("Hq", _i32), ("Hkv", _i32), ("d", _i32), ("dtype", _i32), ("page", _i32),
                ("pages", _i32), ("width", _i32), ("rot", _i32), ("layout", _i32), ("rope_scale", _f32),
                ("offset", _i64), ("prefix", _i32), ("prefix_width", _i32), ("scale", _f32), ("k_stride", _s3),
                ("v_stride", _s3), ("table_stride", _i64)]


def declare(L):
    """Argument types of this part of the library."""
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    P = ctypes.POINTER
    L.kron_delta_paged_append.restype = i32
    L.kron_delta_paged_append.argtypes = [P(KdPagedDesc)] + [vp] * 3 + [P(_i64)] + [vp] * 7 + [vp]
    L.kron_delta_prefix_attn_workspace_bytes.restype = sz
    L.kron_delta_prefix_attn_workspace_bytes.argtypes = [P(KdPagedDesc), i32]
    L.kron_delta_prefix_attn.restype = i32
    L.kron_delta_prefix_attn.argtypes = [P(KdPagedDesc), vp, P(_i64)] + [vp] * 8 + [vp, sz, vp]


def _packed_rows(t):
    """[T, H, d] as the kernels read it: contiguous last dimension, strides and
    address in whole 16-byte pieces (a copy where it is not so)."""
    (n, h, d), (s0, s1, s2), es = t.shape, t.stride(), t.element_size()
    if t.data_ptr() % 16 == 0 and (d == 1 or s2 == 1) and (n <= 1 or s0 * es % 16 == 0) and (h <= 1 or s1 * es % 16 == 0):
        return t
    return t.clone() if t.is_contiguous() else t.contiguous()


def _batch(dev, k_pages, v_pages, page_table, lens, cu_seqlens, T):
    """Checks of the cache, the table and the batch; B and cu_seqlens."""
    torch = _la._torch
    if k_pages.dim() != 4 or k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype:
        raise ValueError("k_pages and v_pages must be [pages, page, Hkv, d] of one dtype")
    _fits("k_pages", k_pages.shape)
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError("%s must have a contiguous last dimension" % name)
    if page_table.dim() != 2 or page_table.dtype != torch.int32:
        raise ValueError("page_table must be int32 [B, width]")
    if page_table.shape[1] > 1 and page_table.stride(1) != 1:
        raise ValueError("page_table must have contiguous rows")
    _fits("page_table", page_table.shape)
    B = page_table.shape[0]
    _check("lens", lens, (B,), torch.int32)
    if B > 1 and lens.stride(0) != 1:
        lens = lens.contiguous()
    if cu_seqlens is not None:
        _check("cu_seqlens", cu_seqlens, (B + 1,), torch.int32)
        cu_seqlens = cu_seqlens.contiguous()
    elif T != B:
        raise ValueError("without cu_seqlens every sequence has one row: %d rows for %d sequences" % (T, B))
    _same_device(dev, k_pages=k_pages, v_pages=v_pages, page_table=page_table, lens=lens, cu_seqlens=cu_seqlens)
    return B, lens, cu_seqlens


def _desc(k_pages, v_pages, page_table, B, T, Hq, **fields):
    pages, page, Hkv, d = k_pages.shape
    return KdPagedDesc(B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, dtype=_code(k_pages.dtype), page=page, pages=pages,
                       width=page_table.shape[1], k_stride=k_pages.stride()[:3], v_stride=v_pages.stride()[:3],
                       table_stride=page_table.stride(0) if B > 1 else 0, **fields)


def paged_append(k, v, k_pages, v_pages, page_table, lens, *, q=None, cu_seqlens=None, freqs=None, layout="half",
                 rope_scale=1.0, offset=0):
    """New keys and values [T, Hkv, d] into k_pages, v_pages [pages, page, Hkv,
    d] through page_table int32 [B, width]: one row per sequence (T = B), or
    packed ones with cu_seqlens int32 [B + 1].  lens int32 [B]: own tokens
    before these (not changed; negative: an unused sequence).  freqs: turn k,
    and q [T, Hq, d] when given, to positions offset + lens[b], ... first.
    Tokens without a page are not stored.  Returns the turned q, or None."""
    torch, L = _ready()
    dev = _need_cuda(k, "k")
    if k.dim() != 3 or (q is not None and q.dim() != 3):
        raise ValueError("k and v must be [T, Hkv, d], q [T, Hq, d]")
    T = k.shape[0]
    B, lens, cu_seqlens = _batch(dev, k_pages, v_pages, page_table, lens, cu_seqlens, T)
    Hkv, d = k_pages.shape[2:]
    _fits("k", k.shape)
    _check("k", k, (T, Hkv, d), k_pages.dtype)
    _check("v", v, (T, Hkv, d), k_pages.dtype)
    Hq = 0
    if q is not None:
        Hq = q.shape[1]
        _fits("q", q.shape)
        _check("q", q, (T, Hq, d), k_pages.dtype)
        q = _packed_rows(q)
    _same_device(dev, v=v, q=q)
    k, v = _packed_rows(k), _packed_rows(v)
    rot = 0
    if freqs is not None:
        freqs = _freqs(freqs, dev)
        rot = _int32(2 * freqs.numel())
    desc = _desc(k_pages, v_pages, page_table, B, T, Hq, rot=rot, layout=_layout(layout), rope_scale=rope_scale,
                 offset=min(max(int(offset), -(1 << 62)), 1 << 62))
    out = None if q is None else torch.empty((T, Hq, d), dtype=q.dtype, device=dev)
    strides = _s6(*((0, 0) if q is None else q.stride()[:2]), *k.stride()[:2], *v.stride()[:2])
    _call("kron_delta_paged_append", dev, L.kron_delta_paged_append, ctypes.byref(desc), _ptr(q), k.data_ptr(),
          v.data_ptr(), strides, k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), lens.data_ptr(),
          _ptr(cu_seqlens), _ptr(freqs), _ptr(out))
    return out


def prefix_attn_workspace(q, k_pages, prefix_len, page_table):
    """A workspace for prefix_attn calls with these shapes, packed or not.  One
    per stream."""
    torch, L = _ready()
    need = 0
    for packed in (0, 1):
        if packed or q.shape[0] == page_table.shape[0]:
            desc = _desc(k_pages, k_pages, page_table, page_table.shape[0], q.shape[0], q.shape[1], scale=1.0,
                         prefix=_int32(prefix_len), prefix_width=1 << 30)
            need = max(need, int(L.kron_delta_prefix_attn_workspace_bytes(ctypes.byref(desc), packed)))
    return torch.empty(max(need, 16), dtype=torch.uint8, device=k_pages.device)


def prefix_attn(q, k_pages, v_pages, prefix_table, prefix_len, page_table, lens, *, scale=None, cu_seqlens=None,
                return_lse=False, workspace=None):
    """Attention of rows q [T, Hq, d] over the first prefix_len keys of the
    pages prefix_table (int32 vector; shared by all sequences) and over their
    sequence's own keys: row r of sequence b sees own keys 0 .. lens[b] + r
    through page_table int32 [B, width].  One row per sequence (T = B), or
    packed ones with cu_seqlens int32 [B + 1].  scale None: 1 / sqrt(d).
    Returns o, with return_lse (o, lse [Hq, T] float32).  Packed rows that no
    sequence holds are not written: those of a new tensor hold anything."""
    torch, L = _ready()
    dev = _need_cuda(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [T, Hq, d]")
    T, Hq, d = q.shape
    B, lens, cu_seqlens = _batch(dev, k_pages, v_pages, page_table, lens, cu_seqlens, T)
    _fits("q", q.shape)
    _check("q", q, (T, Hq, k_pages.shape[3]), k_pages.dtype)
    if prefix_table.dim() != 1 or prefix_table.dtype != torch.int32:
        raise ValueError("prefix_table must be an int32 vector")
    _fits("prefix_table", prefix_table.shape)
    _same_device(dev, prefix_table=prefix_table)
    prefix_table, q = prefix_table.contiguous(), _packed_rows(q)
    desc = _desc(k_pages, v_pages, page_table, B, T, Hq, scale=1.0 / math.sqrt(d) if scale is None else scale,
                 prefix=_int32(prefix_len), prefix_width=prefix_table.numel())
    need = int(L.kron_delta_prefix_attn_workspace_bytes(ctypes.byref(desc), int(cu_seqlens is not None)))
    ws, wsb = _workspace(workspace, need, dev)
    o = torch.empty((T, Hq, d), dtype=q.dtype, device=dev)
    lse = torch.empty((Hq, T), dtype=torch.float32, device=dev) if return_lse else None
    _call("kron_delta_prefix_attn", dev, L.kron_delta_prefix_attn, ctypes.byref(desc), q.data_ptr(), _s2(*q.stride()[:2]),
          k_pages.data_ptr(), v_pages.data_ptr(), prefix_table.data_ptr(), page_table.data_ptr(), lens.data_ptr(),
          _ptr(cu_seqlens), o.data_ptr(), _ptr(lse), _ptr(ws), wsb)
    return (o, lse) if return_lse else o
