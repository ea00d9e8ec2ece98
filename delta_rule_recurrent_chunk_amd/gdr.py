"""The gated delta rule -- binding of its part of the C ABI.

    o, ST        = gdr_fwd(q, k, v, g, beta, S0=None)                     chunked, batched or packed
    o, ST, saved = gdr_fwd(..., save_states=True)
    grads        = gdr_bwd(q, k, v, g, beta, saved, dO, dST=None)
    o            = gdr_step(q, k, v, g, beta, S)                          one token, the state updated in place

Argument marshalling only, as in the package's module; ``include/kron_delta.h`` defines the operator.
"""
from __future__ import annotations

import ctypes
import math
import struct

from . import layers as _la
from .layers import _call, _check, _code, _fits, _flat, _need_cuda, _ptr, _ready, _rows, _same_device, _workspace

GDR_MAX_DK, GDR_MAX_DV = 128, 256
GDR_MAX_STEP = 1 << 22

EXPORTED = ("kron_delta_gdr_workspace_bytes", "kron_delta_gdr_saved_bytes", "kron_delta_gdr_fwd", "kron_delta_gdr_bwd", "kron_delta_gdr_step")

_i32, _i64, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_s3 = _i64 * 3


class KdGdrDesc(ctypes.Structure):
    _fields_ = [("B", _i32), ("T", _i32), ("Hk", _i32), ("Hv", _i32), ("dk", _i32), ("dv", _i32), ("dtype", _i32),
                ("gates32", _i32), ("scale", _f32), ("q_stride", _s3), ("k_stride", _s3), ("v_stride", _s3)]


_DESC = struct.Struct("@8if9q").pack      # the same as bytes (a step's calls are short)


def declare(L):
    """Argument types of this part of the library."""
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    P = ctypes.POINTER
    L.kron_delta_gdr_workspace_bytes.restype = sz
    L.kron_delta_gdr_workspace_bytes.argtypes = [P(KdGdrDesc), i32, i32]
    L.kron_delta_gdr_saved_bytes.restype = sz
    L.kron_delta_gdr_saved_bytes.argtypes = [P(KdGdrDesc), i32]
    L.kron_delta_gdr_fwd.restype = i32
    L.kron_delta_gdr_fwd.argtypes = [P(KdGdrDesc)] + [vp] * 10 + [vp, sz, vp]
    L.kron_delta_gdr_bwd.restype = i32
    L.kron_delta_gdr_bwd.argtypes = [P(KdGdrDesc)] + [vp] * 15 + [vp, sz, vp]
    L.kron_delta_gdr_step.restype = i32
    L.kron_delta_gdr_step.argtypes = [vp] * 10


def _gdr(q, k, v, g, beta, scale, cu):
    """Checks of the inputs: device, descriptor, inputs as the kernels read them, the states' batch."""
    torch = _la._torch
    dev = _need_cuda(q, "q")
    dims = 3 if cu is not None else 4
    if q.dim() != dims or k.dim() != dims or v.dim() != dims:
        raise ValueError("q, k, v must be [B, T, H, d], or [T, H, d] with cu_seqlens")
    for name, t in (("k", k), ("v", v)):
        if t.dtype != q.dtype:
            raise TypeError("%s has dtype %s, q has %s" % (name, t.dtype, q.dtype))
    if k.shape != q.shape or v.shape[:-2] != q.shape[:-2]:
        raise ValueError("q and k must be one shape, v theirs but for its heads and their size")
    if g.dtype != beta.dtype or g.dtype not in (q.dtype, torch.float32):
        raise TypeError("g and beta must both be %s or float32, got %s and %s" % (q.dtype, g.dtype, beta.dtype))
    for name, t in (("q", q), ("v", v)):
        _fits(name, t.shape)
    _check("g", g, v.shape[:-1], g.dtype)
    _check("beta", beta, v.shape[:-1], g.dtype)
    _same_device(dev, k=k, v=v, g=g, beta=beta, cu_seqlens=cu)
    # (tokens too far apart for the kernels' offsets are copied as well)
    q, k, v = (t.contiguous() if t.stride(-3) > GDR_MAX_STEP and t.shape[-3] > 1 else t for t in map(_rows, (q, k, v)))
    g, beta = _flat(g), _flat(beta)
    (T, Hk, dk), (Hv, dv) = q.shape[-3:], v.shape[-2:]
    if cu is not None:
        if cu.dtype != torch.int32 or cu.dim() != 1 or cu.numel() < 2:
            raise ValueError("cu_seqlens must be an int32 device vector [N + 1]")
        _fits("cu_seqlens", cu.shape)
        cu = cu.contiguous()
        B, strides = cu.numel() - 1, [(0,) + t.stride()[:2] for t in (q, k, v)]
    else:
        B, strides = q.shape[0], [t.stride()[:3] for t in (q, k, v)]
    desc = KdGdrDesc(B, T, Hk, Hv, dk, dv, _code(q.dtype), int(g.dtype == torch.float32 and q.dtype != torch.float32),
                     1.0 / math.sqrt(dk) if scale is None else scale, *strides)
    return dev, desc, q, k, v, g, beta, cu


def _heads(t):
    """[n, H, d] as the kernels read it: contiguous last dimension, strides and
    address in whole 16-byte pieces (a copy where it is not so)."""
    s0, s1, s2 = t.stride()
    if s2 == 1 and not ((s0 | s1) * t.element_size() | t.data_ptr()) & 15:
        return t
    return t.clone() if t.is_contiguous() else t.contiguous()


def _state(name, S, desc, dev):
    if S is not None:
        _check(name, S, (desc.B, desc.Hv, desc.dv, desc.dk), _la._torch.float32)
        _same_device(dev, **{name: S})
        S = _flat(S)
    return S


def gdr_fwd(q, k, v, g, beta, S0=None, *, scale=None, cu_seqlens=None, return_state=True, save_states=False,
            workspace=None):
    """S <- e^g S, S <- S + beta (v - S k) k^T, o = scale S q over q, k [B, T,
    Hk, dk], v [B, T, Hv, dv] and g, beta [B, T, Hv] (q's type or both float32)
    from S0 [B, Hv, dv, dk] float32 (None: 0); or packed [T, H, d] with
    cu_seqlens int32 [N + 1].  scale None: 1 / sqrt(dk).  Returns (o, ST), with
    save_states also what gdr_bwd starts from; ST is None if return_state=False.
    Packed rows that no sequence holds are not written: those of a new tensor
    hold anything."""
    torch, L = _ready()
    dev, desc, q, k, v, g, beta, cu = _gdr(q, k, v, g, beta, scale, cu_seqlens)
    S0 = _state("S0", S0, desc, dev)
    o = torch.empty(v.shape, dtype=q.dtype, device=dev)
    shape = (desc.B, desc.Hv, desc.dv, desc.dk)
    ST = torch.empty(shape, dtype=torch.float32, device=dev) if return_state else None
    saved = None
    if save_states:
        saved = torch.empty(int(L.kron_delta_gdr_saved_bytes(ctypes.byref(desc), int(cu is not None))), dtype=torch.uint8,
                            device=dev)
    need = int(L.kron_delta_gdr_workspace_bytes(ctypes.byref(desc), int(cu is not None), 0))
    ws, wsb = _workspace(workspace, need, dev)
    _call("kron_delta_gdr_fwd", dev, L.kron_delta_gdr_fwd, ctypes.byref(desc), _ptr(cu), _ptr(q), _ptr(k), _ptr(v),
          _ptr(g), _ptr(beta), _ptr(S0), _ptr(o), _ptr(ST), _ptr(saved), _ptr(ws), wsb)
    return (o, ST, saved) if save_states else (o, ST)


def gdr_bwd(q, k, v, g, beta, saved, dO, dST=None, *, scale=None, cu_seqlens=None, return_dS0=True, workspace=None):
    """Gradients of <dO, o> + <dST, ST> from gdr_fwd's inputs and what it
    saved: a dict with dq, dk, dv, dg, dbeta (in their tensors' types) and dS0
    [B, Hv, dv, dk] float32 (None if return_dS0=False).  Packed rows that no
    sequence holds are not written, as in gdr_fwd."""
    torch, L = _ready()
    dev, desc, q, k, v, g, beta, cu = _gdr(q, k, v, g, beta, scale, cu_seqlens)
    shape = (desc.B, desc.Hv, desc.dv, desc.dk)
    _check("saved", saved, (int(L.kron_delta_gdr_saved_bytes(ctypes.byref(desc), int(cu is not None))),), torch.uint8)
    _check("dO", dO, v.shape, q.dtype)
    _same_device(dev, saved=saved, dO=dO)
    saved, dO, dST = _flat(saved), _flat(dO), _state("dST", dST, desc, dev)
    out = dict(dq=torch.empty(q.shape, dtype=q.dtype, device=dev), dk=torch.empty(k.shape, dtype=q.dtype, device=dev),
               dv=torch.empty(v.shape, dtype=q.dtype, device=dev), dg=torch.empty_like(g), dbeta=torch.empty_like(beta),
               dS0=torch.empty(shape, dtype=torch.float32, device=dev) if return_dS0 else None)
    need = int(L.kron_delta_gdr_workspace_bytes(ctypes.byref(desc), int(cu is not None), 1))
    ws, wsb = _workspace(workspace, need, dev)
    _call("kron_delta_gdr_bwd", dev, L.kron_delta_gdr_bwd, ctypes.byref(desc), _ptr(cu), _ptr(q), _ptr(k), _ptr(v),
          _ptr(g), _ptr(beta), _ptr(saved), _ptr(dO), _ptr(dST), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
          _ptr(out["dg"]), _ptr(out["dbeta"]), _ptr(out["dS0"]), _ptr(ws), wsb)
    return out


def gdr_step(q, k, v, g, beta, S, *, scale=None, S_out=None):
    """One token of every sequence: q, k [B, Hk, dk], v [B, Hv, dv], g, beta [B,
    Hv], the state S [B, Hv, dv, dk] float32.  Returns o [B, Hv, dv]; the new
    state goes to S_out, or into S itself when it is None."""
    torch, L = _ready()
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3 or g.dim() != 2 or beta.dim() != 2:
        raise ValueError("q, k must be [B, Hk, dk], v [B, Hv, dv], g, beta [B, Hv]")
    dev, dt, (B, Hk, dk), (_, Hv, dv), gt = _need_cuda(q, "q"), q.dtype, q.shape, v.shape, g.dtype
    if gt != dt and gt != torch.float32:
        raise TypeError("g and beta must both be %s or float32, got %s" % (dt, gt))
    out = S if S_out is None else S_out
    state, f32 = (B, Hv, dv, dk), torch.float32
    for name, t, shape, ty in (("k", k, (B, Hk, dk), dt), ("v", v, (B, Hv, dv), dt), ("g", g, (B, Hv), gt),
                               ("beta", beta, (B, Hv), gt), ("S", S, state, f32), ("S_out", out, state, f32)):
        if t.shape != shape or t.dtype != ty or t.device != dev:
            _check(name, t, shape, ty)
            raise ValueError("%s is on %s, not on %s" % (name, t.device, dev))
    if not S.is_contiguous() or not out.is_contiguous():
        raise ValueError("S and S_out must be contiguous")
    _fits("the state", state)
    q, k, v = _heads(q), _heads(k), _heads(v)
    g, beta = _flat(g), _flat(beta)
    (q0, q1, _), (k0, k1, _), (v0, v1, _) = q.stride(), k.stride(), v.stride()
    desc = _DESC(B, 1, Hk, Hv, dk, dv, _code(dt), gt != dt, 1.0 / math.sqrt(dk) if scale is None else scale, q0, 0, q1, k0,
                 0, k1, v0, 0, v1)
    o = torch.empty((B, Hv, dv), dtype=dt, device=dev)
    _call("kron_delta_gdr_step", dev, L.kron_delta_gdr_step, desc, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          g.data_ptr(), beta.data_ptr(), S.data_ptr(), o.data_ptr(), out.data_ptr())
    return o
