"""A paged cache and attention over a shared prefix -- binding of their part of the C ABI.

    q = paged_append(k, v, k_pages, v_pages, page_table, lens, q=q, freqs=freqs)      tokens into the cache
    o = prefix_attn(q, k_pages, v_pages, prefix_table, prefix_len, page_table, lens)  attention over it

Argument marshalling only, as in the package's module; ``include/kron_delta.h`` defines both operators.
"""
from __future__ import annotations

import ctypes
import math
import struct

from . import layers as _la
from .gdr import _heads
from .layers import _call, _check, _code, _fits, _freqs, _int32, _layout, _need_cuda, _ready

EXPORTED = ("kron_delta_paged_append", "kron_delta_prefix_attn_workspace_bytes", "kron_delta_prefix_attn")

_i32, _i64, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_s2, _s3, _s6 = _i64 * 2, _i64 * 3, _i64 * 6


class KdPagedDesc(ctypes.Structure):
    _fields_ = [("B", _i32), ("T", _i32), ("Hq", _i32), ("Hkv", _i32), ("d", _i32), ("dtype", _i32), ("page", _i32),
                ("pages", _i32), ("width", _i32), ("rot", _i32), ("layout", _i32), ("rope_scale", _f32),
                ("offset", _i64), ("prefix", _i32), ("prefix_width", _i32), ("scale", _f32), ("k_stride", _s3),
                ("v_stride", _s3), ("table_stride", _i64)]


# the descriptor and the rows' strides as bytes: a step's calls are short, and
# ctypes takes a third of their host time to build the same structure
_DESC = struct.Struct("@11ifqiif7q").pack
_S2, _S6 = struct.Struct("@2q").pack, struct.Struct("@6q").pack


def declare(L):
    """Argument types of this part of the library."""
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    L.kron_delta_paged_append.restype = i32
    L.kron_delta_paged_append.argtypes = [vp] * 13
    L.kron_delta_prefix_attn_workspace_bytes.restype = sz
    L.kron_delta_prefix_attn_workspace_bytes.argtypes = [vp, i32]
    L.kron_delta_prefix_attn.restype = i32
    L.kron_delta_prefix_attn.argtypes = [vp] * 12 + [sz, vp]


def _batch(dev, k_pages, v_pages, page_table, lens, cu_seqlens, T):
    """Checks of the cache, the table and the batch.  Returns B, lens, cu_seqlens."""
    torch = _la._torch
    shape, i32 = k_pages.shape, torch.int32
    if len(shape) != 4 or v_pages.shape != shape or v_pages.dtype != k_pages.dtype:
        raise ValueError("k_pages and v_pages must be [pages, page, Hkv, d] of one dtype")
    if page_table.dim() != 2 or page_table.dtype != i32:
        raise ValueError("page_table must be int32 [B, width]")
    B, width = page_table.shape
    _fits("the cache or its table", (*shape, B, width, T))
    if shape[3] > 1 and (k_pages.stride(3) != 1 or v_pages.stride(3) != 1):
        raise ValueError("k_pages and v_pages must have a contiguous last dimension")
    if width > 1 and page_table.stride(1) != 1:
        raise ValueError("page_table must have contiguous rows")
    if cu_seqlens is not None:
        _check("cu_seqlens", cu_seqlens, (B + 1,), i32)
        cu_seqlens = cu_seqlens.contiguous()
        if cu_seqlens.device != dev:
            raise ValueError("cu_seqlens is on %s, not on %s" % (cu_seqlens.device, dev))
    elif T != B:
        raise ValueError("without cu_seqlens every sequence has one row: %d rows for %d sequences" % (T, B))
    if lens.shape != (B,) or lens.dtype != i32:
        _check("lens", lens, (B,), i32)
    if k_pages.device != dev or v_pages.device != dev or page_table.device != dev or lens.device != dev:
        raise ValueError("the cache, its table and lens must be on %s" % dev)
    return B, lens if lens.is_contiguous() else lens.contiguous(), cu_seqlens


def _row_check(name, t, shape, dt, dev):
    if t.shape != shape or t.dtype != dt or t.device != dev:
        _check(name, t, shape, dt)
        raise ValueError("%s is on %s, not on %s" % (name, t.device, dev))


def _desc(k_pages, v_pages, page_table, B, T, Hq, rot=0, layout=0, rope_scale=1.0, offset=0, prefix=0, prefix_width=0,
          scale=1.0):
    pages, page, Hkv, d = k_pages.shape
    a, b, c, _ = k_pages.stride()
    e, f, g, _ = v_pages.stride()
    return _DESC(B, T, Hq, Hkv, d, _code(k_pages.dtype), page, pages, page_table.shape[1], rot, layout, rope_scale, offset,
                 prefix, prefix_width, scale, a, b, c, e, f, g, page_table.stride(0) if B > 1 else 0)


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
    (_, _, Hkv, d), dt = k_pages.shape, k_pages.dtype
    _row_check("k", k, (T, Hkv, d), dt, dev)
    _row_check("v", v, (T, Hkv, d), dt, dev)
    k, v = _heads(k), _heads(v)
    if q is None:
        Hq, out, qp, op, q0, q1 = 0, None, None, None, 0, 0
    else:
        Hq = q.shape[1]
        _fits("q", (T, Hq))
        _row_check("q", q, (T, Hq, d), dt, dev)
        q = _heads(q)
        out = torch.empty((T, Hq, d), dtype=dt, device=dev)
        (q0, q1, _), qp, op = q.stride(), q.data_ptr(), out.data_ptr()
    rot = fp = 0
    if freqs is not None:
        freqs = _freqs(freqs, dev)
        rot, fp = _int32(2 * freqs.numel()), freqs.data_ptr()
    desc = _desc(k_pages, v_pages, page_table, B, T, Hq, rot, _layout(layout), rope_scale,
                 min(max(int(offset), -(1 << 62)), 1 << 62))
    (k0, k1, _), (v0, v1, _) = k.stride(), v.stride()
    _call("kron_delta_paged_append", dev, L.kron_delta_paged_append, desc, qp, k.data_ptr(), v.data_ptr(),
          _S6(q0, q1, k0, k1, v0, v1), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), lens.data_ptr(),
          None if cu_seqlens is None else cu_seqlens.data_ptr(), fp, op)
    return out


def prefix_attn_workspace(q, k_pages, prefix_len, page_table):
    """A workspace for prefix_attn calls with these shapes, packed or not.  One
    per stream."""
    torch, L = _ready()
    need = 0
    for packed in (0, 1):
        if packed or q.shape[0] == page_table.shape[0]:
            _fits("the batch", q.shape + k_pages.shape + page_table.shape)
            desc = _desc(k_pages, k_pages, page_table, page_table.shape[0], q.shape[0], q.shape[1], scale=1.0,
                         prefix=_int32(prefix_len), prefix_width=1 << 30)
            need = max(need, int(L.kron_delta_prefix_attn_workspace_bytes(desc, packed)))
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
    _fits("q", (T, Hq))
    _row_check("q", q, (T, Hq, k_pages.shape[3]), k_pages.dtype, dev)
    if prefix_table.dim() != 1 or prefix_table.dtype != torch.int32 or prefix_table.device != dev:
        raise ValueError("prefix_table must be an int32 vector on %s" % dev)
    width = prefix_table.numel()
    _fits("prefix_table", (width, 0))
    prefix_table, q = prefix_table.contiguous(), _heads(q)
    desc = _desc(k_pages, v_pages, page_table, B, T, Hq, 0, 0, 1.0, 0, _int32(prefix_len), width,
                 1.0 / math.sqrt(d) if scale is None else scale)
    if workspace is None:
        need = int(L.kron_delta_prefix_attn_workspace_bytes(desc, int(cu_seqlens is not None)))
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    elif not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError("workspace must be contiguous and on %s" % dev)
    o = torch.empty((T, Hq, d), dtype=q.dtype, device=dev)
    lse = torch.empty((Hq, T), dtype=torch.float32, device=dev) if return_lse else None
    q0, q1, _ = q.stride()
    _call("kron_delta_prefix_attn", dev, L.kron_delta_prefix_attn, desc, q.data_ptr(), _S2(q0, q1), k_pages.data_ptr(),
          v_pages.data_ptr(), prefix_table.data_ptr(), page_table.data_ptr(), lens.data_ptr(),
          None if cu_seqlens is None else cu_seqlens.data_ptr(), o.data_ptr(), None if lse is None else lse.data_ptr(),
          workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return (o, lse) if return_lse else o
