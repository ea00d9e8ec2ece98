"""The layers beside the mixer -- binding of their part of the C ABI.

    h, hT = glr_fwd(x, f, i=None, h0=None)                        gated linear recurrence
    grads = glr_bwd(x, f, i, hs, dh, dhT=None)                    (hs: glr_fwd(..., save_states=True))
    y     = glr_step(x, f, i, h)                                  one token, the state updated in place
    q, k  = rope(q, k, positions, freqs)                          rotary positions; rope_bwd for gradients
    o     = swa_fwd(q, k, v, window, sinks)                       sliding-window attention with sinks
    grads = swa_bwd(q, k, v, o, lse, dO, window, sinks)
    o     = swa_decode(q, k, v, k_cache, v_cache, lens, window, sinks)   one token over a rolling cache
    swa_cache_store(k, v, k_cache, v_cache, window, sinks)        a prompt into that cache

Argument marshalling only, as in the package's module; ``include/kron_delta.h`` defines every operator.
"""
from __future__ import annotations

import ctypes
import math

KD_ROPE_HALF, KD_ROPE_INTERLEAVED = 0, 1
GLR_CHUNK = 128
SWA_MAX_SINKS = 64

EXPORTED = ("kron_delta_glr_workspace_bytes", "kron_delta_glr_fwd", "kron_delta_glr_bwd", "kron_delta_glr_step",
            "kron_delta_rope", "kron_delta_swa_workspace_bytes", "kron_delta_swa_fwd", "kron_delta_swa_bwd",
            "kron_delta_swa_decode_workspace_bytes", "kron_delta_swa_decode", "kron_delta_swa_cache_store")

_i32, _i64, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_s3 = _i64 * 3


class KdGlrDesc(ctypes.Structure):
    _fields_ = [("B", _i32), ("T", _i32), ("D", _i32), ("dtype", _i32)]


class KdRopeDesc(ctypes.Structure):
    _fields_ = [("B", _i32), ("T", _i32), ("Hq", _i32), ("Hk", _i32), ("d", _i32), ("rot", _i32), ("layout", _i32),
                ("dtype", _i32), ("pos64", _i32), ("pos_batched", _i32), ("inverse", _i32), ("scale", _f32),
                ("q_stride", _s3), ("k_stride", _s3), ("q_out_stride", _s3), ("k_out_stride", _s3)]


class KdSwaDesc(ctypes.Structure):
    _fields_ = [("B", _i32), ("Tq", _i32), ("Tk", _i32), ("Hq", _i32), ("Hkv", _i32), ("d", _i32), ("dtype", _i32),
                ("window", _i32), ("sinks", _i32), ("scale", _f32), ("q_stride", _s3), ("k_stride", _s3),
                ("v_stride", _s3)]


class KdSwaCacheDesc(ctypes.Structure):
    _fields_ = [("B", _i32), ("Hq", _i32), ("Hkv", _i32), ("d", _i32), ("cap", _i32), ("dtype", _i32),
                ("window", _i32), ("sinks", _i32), ("scale", _f32), ("rot", _i32), ("layout", _i32),
                ("rope_scale", _f32), ("k_stride", _s3), ("v_stride", _s3)]


def declare(L):
    """Argument types of this part of the library."""
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    P = ctypes.POINTER
    L.kron_delta_glr_workspace_bytes.restype = sz
    L.kron_delta_glr_workspace_bytes.argtypes = [P(KdGlrDesc)]
    L.kron_delta_glr_fwd.restype = i32
    L.kron_delta_glr_fwd.argtypes = [P(KdGlrDesc)] + [vp] * 7 + [vp, sz, vp]
    L.kron_delta_glr_bwd.restype = i32
    L.kron_delta_glr_bwd.argtypes = [P(KdGlrDesc)] + [vp] * 10 + [vp, sz, vp]
    L.kron_delta_glr_step.restype = i32
    L.kron_delta_glr_step.argtypes = [P(KdGlrDesc)] + [vp] * 6 + [vp]
    L.kron_delta_rope.restype = i32
    L.kron_delta_rope.argtypes = [P(KdRopeDesc)] + [vp] * 6 + [vp]
    L.kron_delta_swa_workspace_bytes.restype = sz
    L.kron_delta_swa_workspace_bytes.argtypes = [P(KdSwaDesc), i32]
    L.kron_delta_swa_fwd.restype = i32
    L.kron_delta_swa_fwd.argtypes = [P(KdSwaDesc)] + [vp] * 6 + [vp]
    L.kron_delta_swa_bwd.restype = i32
    L.kron_delta_swa_bwd.argtypes = [P(KdSwaDesc)] + [vp] * 10 + [vp, sz, vp]
    L.kron_delta_swa_decode_workspace_bytes.restype = sz
    L.kron_delta_swa_decode_workspace_bytes.argtypes = [P(KdSwaCacheDesc)]
    L.kron_delta_swa_decode.restype = i32
    L.kron_delta_swa_decode.argtypes = [P(KdSwaCacheDesc)] + [vp] * 3 + [P(_i64)] + [vp] * 5 + [vp, sz, vp]
    L.kron_delta_swa_cache_store.restype = i32
    L.kron_delta_swa_cache_store.argtypes = [P(KdSwaCacheDesc), _i32, vp, vp, P(_i64), P(_i64), vp, vp, vp, vp]


_torch = None
_lib = None
_done = None
_stream = None        # device index -> its current stream
_device = None        # the current device's index


def _load():
    """torch and the library, imported on the first call."""
    global _torch, _lib, _done, _stream, _device
    import torch

    import delta_rule_recurrent_chunk_amd as kd
    _lib, _done = kd.lib(), kd._done
    # (torch's own functions behind the public calls take a tenth of their time)
    _stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda i: torch.cuda.current_stream(i).cuda_stream)
    _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _torch = torch
    return torch, _lib


def _ready():
    return (_torch, _lib) if _torch is not None else _load()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _call(what, dev, fn, *args):
    """Runs a library call on the current stream of the tensors' device."""
    i = dev.index
    if _device() == i:
        r = fn(*args, _stream(i))
    else:
        with _torch.cuda.device(i):
            r = fn(*args, _stream(i))
    _done(r, what, dev)


def _same_device(dev, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError("%s is on %s, not on %s" % (name, t.device, dev))


def _need_cuda(t, name):
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    return t.device


def _check(name, t, shape, dtype):
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))


def _code(dt):
    if dt == _torch.bfloat16:
        return 1
    if dt == _torch.float32:
        return 0
    raise TypeError("tensors must be bfloat16 or float32, got %s" % dt)


def _int32(x):
    """An integer for an int32 field: a value outside its range becomes the nearest one in it."""
    return min(max(int(x), -(1 << 31)), (1 << 31) - 1)


def _fits(name, shape):
    """Refuses a dimension that an int32 field of a descriptor would wrap."""
    if max(shape) > 0x7fffffff:
        raise ValueError("%s has a dimension past 32 bits: %s" % (name, list(shape)))


def _flat(t):
    """The tensor, contiguous and at a 16-byte address (a copy where it is not)."""
    if t is None or (t.is_contiguous() and t.data_ptr() % 16 == 0):
        return t
    return t.clone(memory_format=_torch.contiguous_format)


def _workspace(workspace, need, dev):
    """The caller's workspace, or a new one when there is none."""
    if need == 0 and workspace is None:
        return None, 0
    if workspace is None:
        workspace = _torch.empty(need, dtype=_torch.uint8, device=dev)
    elif not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError("workspace must be contiguous and on %s" % dev)
    return workspace, workspace.numel() * workspace.element_size()


# ------------------------------------------------- gated linear recurrence
def _glr(x, f, i):
    dev = _need_cuda(x, "x")
    shape, dt = x.shape, x.dtype
    _fits("x", shape)
    for name, t in (("f", f), ("i", i)):
        if t is not None and (t.shape != shape or t.dtype != dt or t.device != dev):
            _check(name, t, shape, dt)
            raise ValueError("%s is on %s, not on %s" % (name, t.device, dev))
    return dev, _flat(x), _flat(f), _flat(i)


def glr_workspace_bytes(B, T, D, dtype_code) -> int:
    _fits("the layer", (B, T, D))
    return int(_ready()[1].kron_delta_glr_workspace_bytes(ctypes.byref(KdGlrDesc(B, T, D, dtype_code))))


def glr_fwd(x, f, i=None, h0=None, *, save_states=False, workspace=None):
    """h_t = f_t h_{t-1} + i_t x_t over x, f, i [B, T, D] (i None: 1) from h0
    [B, D] float32 (None: 0).  Returns (h, hT), with save_states also the
    states that glr_bwd starts from."""
    torch, L = _ready()
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    dev, x, f, i = _glr(x, f, i)
    B, T, D = x.shape
    if h0 is not None:
        _check("h0", h0, (B, D), torch.float32)
        _same_device(dev, h0=h0)
        h0 = _flat(h0)
    desc = KdGlrDesc(B, T, D, _code(x.dtype))
    h = torch.empty_like(x)
    hT = torch.empty((B, D), dtype=torch.float32, device=dev)
    hs = torch.empty((B, (T + GLR_CHUNK - 1) // GLR_CHUNK, D), dtype=torch.float32, device=dev) if save_states else None
    ws, wsb = _workspace(workspace, int(L.kron_delta_glr_workspace_bytes(ctypes.byref(desc))), dev)
    _call("kron_delta_glr_fwd", dev, L.kron_delta_glr_fwd, ctypes.byref(desc), _ptr(x), _ptr(f), _ptr(i), _ptr(h0),
          _ptr(h), _ptr(hT), _ptr(hs), _ptr(ws), wsb)
    return (h, hT, hs) if save_states else (h, hT)


def glr_bwd(x, f, i, hs, dh, dhT=None, *, workspace=None):
    """Gradients of <dh, h> + <dhT, hT>: a dict with dx, df, di (None without
    i) and dh0 [B, D] float32."""
    torch, L = _ready()
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    dev, x, f, i = _glr(x, f, i)
    B, T, D = x.shape
    _check("hs", hs, (B, (T + GLR_CHUNK - 1) // GLR_CHUNK, D), torch.float32)
    _check("dh", dh, x.shape, x.dtype)
    _same_device(dev, hs=hs, dh=dh, dhT=dhT)
    hs, dh = _flat(hs), _flat(dh)
    if dhT is not None:
        _check("dhT", dhT, (B, D), torch.float32)
        dhT = _flat(dhT)
    desc = KdGlrDesc(B, T, D, _code(x.dtype))
    out = dict(dx=torch.empty_like(x), df=torch.empty_like(x), di=None if i is None else torch.empty_like(x),
               dh0=torch.empty((B, D), dtype=torch.float32, device=dev))
    ws, wsb = _workspace(workspace, int(L.kron_delta_glr_workspace_bytes(ctypes.byref(desc))), dev)
    _call("kron_delta_glr_bwd", dev, L.kron_delta_glr_bwd, ctypes.byref(desc), _ptr(x), _ptr(f), _ptr(i), _ptr(hs),
          _ptr(dh), _ptr(dhT), _ptr(out["dx"]), _ptr(out["df"]), _ptr(out["di"]), _ptr(out["dh0"]), _ptr(ws), wsb)
    return out


def glr_step(x, f, i, h, *, h_out=None):
    """One token: x, f, i [B, D], the state h [B, D] float32.  Returns y in
    x's dtype; the new state goes to h_out, or into h itself when it is None."""
    torch, L = _ready()
    if x.dim() != 2:
        raise ValueError("x must be [B, D]")
    dev, x, f, i = _glr(x, f, i)
    out = h if h_out is None else h_out
    shape = x.shape
    for name, t in (("h", h), ("h_out", out)):
        if t.shape != shape or t.dtype != torch.float32 or t.device != dev or not t.is_contiguous():
            _check(name, t, shape, torch.float32)
            raise ValueError("%s must be contiguous and on %s" % (name, dev))
    y = torch.empty_like(x)
    desc = KdGlrDesc(shape[0], 1, shape[1], _code(x.dtype))
    _call("kron_delta_glr_step", dev, L.kron_delta_glr_step, ctypes.byref(desc), x.data_ptr(), f.data_ptr(), _ptr(i),
          h.data_ptr(), y.data_ptr(), out.data_ptr())
    return y


# ---------------------------------------------------------- rotary positions
def rope_frequencies(rot, base=10000.0, *, scaling=None, factor=1.0, original_length=None, low_turns=1.0,
                     high_turns=32.0, device=None):
    """Angles per position of the rot / 2 pairs (float64) and the factor the
    rotated part is multiplied by.

    scaling None: base^(-2j / rot).  "linear": positions stretched by factor.
    "ntk": the base raised so that the slowest pair is stretched by factor and
    the fastest keeps its angle.  "byparts": pairs that make more than
    high_turns turns within original_length positions keep their angle, those
    with fewer than low_turns are stretched by factor, the ones between are
    blended; the rotated part is multiplied by 0.1 log(factor) + 1."""
    import torch
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2")
    if not (math.isfinite(factor) and factor >= 1.0):
        raise ValueError("factor must be at least 1")
    n, mscale = rot // 2, 1.0
    if scaling == "ntk":
        if rot > 2:
            base = base * factor ** (rot / (rot - 2.0))
    w = [base ** (-2.0 * j / rot) for j in range(n)]
    if scaling == "linear":
        w = [a / factor for a in w]
    elif scaling == "byparts":
        if not original_length or high_turns <= low_turns:
            raise ValueError("byparts needs original_length and high_turns > low_turns")
        keep = [min(max((original_length * a / (2 * math.pi) - low_turns) / (high_turns - low_turns), 0.0), 1.0)
                for a in w]
        w = [a * t + a / factor * (1.0 - t) for a, t in zip(w, keep)]
        mscale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'byparts'")
    return torch.tensor(w, dtype=torch.float64, device=device), mscale


def _layout(layout):
    if layout == "half":
        return KD_ROPE_HALF
    if layout == "interleaved":
        return KD_ROPE_INTERLEAVED
    raise ValueError("layout must be 'half' or 'interleaved'")


def _freqs(freqs, dev):
    if freqs.dtype != _torch.float64 or freqs.dim() != 1 or freqs.numel() < 1:
        raise TypeError("freqs must be a float64 vector (rope_frequencies)")
    if freqs.device != dev:
        raise ValueError("freqs is on %s, not on %s" % (freqs.device, dev))
    return freqs.contiguous()


def rope(q, k, positions, freqs, *, layout="half", scale=1.0, inverse=False, out=None):
    """Rotary positions on q [B, T, Hq, d] and k [B, T, Hk, d] (or packed
    [T, H, d]; k may be None) at positions [T] or [B, T] (int32 or int64).
    Pairs past len(freqs) stay as they are.  Returns (q, k) rotated: new
    tensors, or those of `out` (which may be the inputs themselves)."""
    torch, L = _ready()
    dev = _need_cuda(q, "q")
    nd = q.dim()
    if nd not in (3, 4):
        raise ValueError("q must be [B, T, H, d] or [T, H, d]")
    qs = q.shape
    _fits("q", qs)
    if nd == 4:
        B, T, Hq, d = qs
    else:
        B, (T, Hq, d) = 1, qs
    Hk = 0
    if k is not None:
        ks = k.shape
        if k.dtype != q.dtype:
            raise TypeError("k has dtype %s, q has %s" % (k.dtype, q.dtype))
        if len(ks) != nd or ks[:-2] != qs[:-2] or ks[-1] != d:
            raise ValueError("k must be shaped like q but for its heads")
        if k.device != dev:
            raise ValueError("k is on %s, not on %s" % (k.device, dev))
        _fits("k", ks)
        Hk = ks[-2]
        if k.stride(-1) != 1 and d > 1:
            k = k.contiguous()
    if q.stride(-1) != 1 and d > 1:
        q = q.contiguous()
    if out is None:
        oq = torch.empty(qs, dtype=q.dtype, device=dev)
        ok = None if k is None else torch.empty(ks, dtype=q.dtype, device=dev)
    else:
        oq, ok = out
        if (ok is None) != (k is None):
            raise ValueError("out must hold a tensor for each of q and k")
        for name, o, x in (("out[0]", oq, q), ("out[1]", ok, k)):
            if x is None:
                continue
            _check(name, o, x.shape, x.dtype)
            if o.device != dev:
                raise ValueError("%s is on %s, not on %s" % (name, o.device, dev))
            if o.stride(-1) != 1 and d > 1:
                raise ValueError("out must have a contiguous last dimension")
    pdt, pdim = positions.dtype, positions.dim()
    if pdt != torch.int64 and pdt != torch.int32:
        raise TypeError("positions must be int32 or int64")
    if not (positions.shape == (T,) or (nd == 4 and positions.shape == (B, T))):
        raise ValueError("positions must be [T] or [B, T]")
    if positions.device != dev:
        raise ValueError("positions is on %s, not on %s" % (positions.device, dev))
    positions, freqs = positions.contiguous(), _freqs(freqs, dev)

    def strides(t):
        return (0, 0, 0) if t is None else t.stride()[:3] if nd == 4 else (0,) + t.stride()[:2]

    desc = KdRopeDesc(B, T, Hq, Hk, d, 2 * freqs.numel(), _layout(layout), _code(q.dtype), pdt == torch.int64,
                      pdim == 2, bool(inverse), scale, strides(q), strides(k), strides(oq), strides(ok))
    _call("kron_delta_rope", dev, L.kron_delta_rope, ctypes.byref(desc), q.data_ptr(), _ptr(k), positions.data_ptr(),
          freqs.data_ptr(), oq.data_ptr(), _ptr(ok))
    return oq, ok


def rope_bwd(dq, dk, positions, freqs, *, layout="half", scale=1.0, out=None):
    """Gradients of rope's inputs from those of its outputs: the inverse turn."""
    return rope(dq, dk, positions, freqs, layout=layout, scale=scale, inverse=True, out=out)


# ------------------------------------------------- sliding-window attention
def _rows(t):
    """The tensor as the kernels read it: contiguous last dimension, strides
    and address in whole 16-byte pieces (a copy where it is not so)."""
    es = t.element_size()
    ok = t.data_ptr() % 16 == 0 and (t.shape[-1] == 1 or t.stride(-1) == 1) and all(
        n <= 1 or (s >= 0 and s * es % 16 == 0) for n, s in zip(t.shape[:-1], t.stride()[:-1]))
    return t if ok else t.clone() if t.is_contiguous() else t.contiguous()


def _swa(q, k, v, window, sinks, scale, cu):
    torch = _torch
    dev = _need_cuda(q, "q")
    dims = 3 if cu is not None else 4
    if q.dim() != dims or k.dim() != dims or v.dim() != dims:
        raise ValueError("q, k, v must be [B, T, H, d], or [T, H, d] with cu_seqlens")
    for name, t in (("k", k), ("v", v)):
        if t.dtype != q.dtype:
            raise TypeError("%s has dtype %s, q has %s" % (name, t.dtype, q.dtype))
    if k.shape != v.shape or k.shape[-1] != q.shape[-1] or (dims == 4 and k.shape[0] != q.shape[0]):
        raise ValueError("k and v must be one shape and match q's batch and head size")
    _fits("q", q.shape)
    _fits("k", k.shape)
    _same_device(dev, k=k, v=v, cu_seqlens=cu)
    q, k, v = _rows(q), _rows(k), _rows(v)
    if cu is not None:
        if cu.dtype != torch.int32 or cu.dim() != 1 or cu.numel() < 2:
            raise ValueError("cu_seqlens must be an int32 device vector [N + 1]")
        _fits("cu_seqlens", cu.shape)
        cu = cu.contiguous()
        B, q4, k4, v4 = cu.numel() - 1, q[None], k[None], v[None]
    else:
        B, q4, k4, v4 = q.shape[0], q, k, v
    d = q.shape[-1]
    desc = KdSwaDesc(B, q4.shape[1], k4.shape[1], q4.shape[2], k4.shape[2], d, _code(q.dtype), _int32(window), _int32(sinks),
                     float(1.0 / math.sqrt(d) if scale is None else scale), _s3(*q4.stride()[:3]),
                     _s3(*k4.stride()[:3]), _s3(*v4.stride()[:3]))
    return dev, desc, q, k, v, cu


def swa_fwd(q, k, v, window, sinks=0, *, scale=None, cu_seqlens=None, return_lse=False, out=None):
    """Attention over the last `window` keys and the first `sinks` ones.  q
    [B, Tq, Hq, d], k, v [B, Tk, Hkv, d], the queries at the end of the keys; or
    packed [T, H, d] with cu_seqlens int32 [N + 1].  scale None: 1 / sqrt(d).
    Returns o, with return_lse (o, lse [B, Hq, Tq] or [Hq, T] float32).  Packed
    rows that no sequence holds are not written: those of a new tensor hold
    anything."""
    torch, L = _ready()
    dev, desc, q, k, v, cu = _swa(q, k, v, window, sinks, scale, cu_seqlens)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    else:
        _check("out", out, q.shape, q.dtype)
        _same_device(dev, out=out)
        if not out.is_contiguous():
            raise ValueError("out must be contiguous")
    lse = None
    if return_lse:
        shape = (desc.Hq, desc.Tq) if cu is not None else (desc.B, desc.Hq, desc.Tq)
        lse = torch.empty(shape, dtype=torch.float32, device=dev)
    _call("kron_delta_swa_fwd", dev, L.kron_delta_swa_fwd, ctypes.byref(desc), _ptr(cu), _ptr(q), _ptr(k), _ptr(v),
          _ptr(out), _ptr(lse))
    return (out, lse) if return_lse else out


def swa_bwd(q, k, v, o, lse, dO, window, sinks=0, *, scale=None, cu_seqlens=None, workspace=None):
    """Gradients of <dO, o> from swa_fwd's o and lse: a dict with dq, dk, dv
    (packed rows that no sequence holds are not written, as in swa_fwd)."""
    torch, L = _ready()
    dev, desc, q, k, v, cu = _swa(q, k, v, window, sinks, scale, cu_seqlens)
    _check("o", o, q.shape, q.dtype)
    _check("dO", dO, q.shape, q.dtype)
    _check("lse", lse, (desc.Hq, desc.Tq) if cu is not None else (desc.B, desc.Hq, desc.Tq), torch.float32)
    _same_device(dev, o=o, dO=dO, lse=lse)
    o, dO, lse = _flat(o), _flat(dO), lse.contiguous()
    out = dict(dq=torch.empty(q.shape, dtype=q.dtype, device=dev), dk=torch.empty(k.shape, dtype=k.dtype, device=dev),
               dv=torch.empty(v.shape, dtype=v.dtype, device=dev))
    need = int(L.kron_delta_swa_workspace_bytes(ctypes.byref(desc), int(cu is not None)))
    ws, wsb = _workspace(workspace, need, dev)
    _call("kron_delta_swa_bwd", dev, L.kron_delta_swa_bwd, ctypes.byref(desc), _ptr(cu), _ptr(q), _ptr(k), _ptr(v),
          _ptr(o), _ptr(lse), _ptr(dO), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(ws), wsb)
    return out


def _cache_desc(q_heads, k_cache, v_cache, window, sinks, scale=1.0, rot=0, layout=0, rope_scale=1.0):
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype:
        raise ValueError("k_cache and v_cache must be [B, cap, Hkv, d] of one dtype")
    B, cap, Hkv, d = k_cache.shape
    _fits("k_cache", (B, cap, Hkv, d, q_heads))
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError("%s must have a contiguous last dimension" % name)
    return KdSwaCacheDesc(B, q_heads, Hkv, d, cap, _code(k_cache.dtype), _int32(window), _int32(sinks), scale,
                          rot, layout, rope_scale, k_cache.stride()[:3], v_cache.stride()[:3])


def swa_decode_workspace(q, k_cache):
    """A workspace for swa_decode calls with these shapes and any window (zero
    filled; every call leaves it ready for the next).  One per stream."""
    torch, L = _ready()
    cap = k_cache.shape[1]
    # the splits grow with the number of visible keys: the widest window needs most
    desc = _cache_desc(q.shape[1], k_cache, k_cache, cap, 0)
    need = int(L.kron_delta_swa_decode_workspace_bytes(ctypes.byref(desc)))
    if need == 0:
        raise ValueError("unsupported cache for q [B, Hq, d]: %s, %s" % (list(q.shape), list(k_cache.shape)))
    return torch.zeros(need, dtype=torch.uint8, device=k_cache.device)


def swa_decode(q, k, v, k_cache, v_cache, lens, window, sinks=0, *, scale=None, freqs=None, layout="half",
               rope_scale=1.0, workspace=None):
    """One token of every sequence: q [B, Hq, d], k, v [B, Hkv, d]; the caches
    [B, cap, Hkv, d] (cap >= sinks + window) hold lens[b] tokens (int32 [B])
    and receive the new one; lens is not changed.  freqs: turn q and k to their
    position first.  Rows with a negative length are skipped (their o is 0).
    Returns o [B, Hq, d]."""
    torch, L = _ready()
    dev = _need_cuda(q, "q")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [B, Hq, d], k and v [B, Hkv, d]")
    if k_cache.dim() != 4:
        raise ValueError("k_cache and v_cache must be [B, cap, Hkv, d] of one dtype")
    (B, _, Hkv, d), dt, Hq = k_cache.shape, k_cache.dtype, q.shape[1]
    one = (B, Hkv, d)
    for name, t, shape, ty in (("q", q, (B, Hq, d), dt), ("k", k, one, dt), ("v", v, one, dt),
                               ("lens", lens, (B,), torch.int32)):
        if t.shape != shape or t.dtype != ty or t.device != dev:
            _check(name, t, shape, ty)
            raise ValueError("%s is on %s, not on %s" % (name, t.device, dev))
    if k_cache.device != dev or v_cache.device != dev:
        raise ValueError("the caches must be on %s" % dev)

    def heads(t):      # heads and elements contiguous, any batch stride
        b, h, e = t.stride()
        return t if e == 1 and (h == d or t.shape[1] == 1) else t.contiguous()

    q, k, v, lens = heads(q), heads(k), heads(v), lens.contiguous()
    rot = 0
    if freqs is not None:
        freqs = _freqs(freqs, dev)
        rot = 2 * freqs.numel()
    desc = _cache_desc(Hq, k_cache, v_cache, window, sinks, 1.0 / math.sqrt(d) if scale is None else scale, rot,
                       _layout(layout), rope_scale)
    if workspace is None:
        need = int(L.kron_delta_swa_decode_workspace_bytes(ctypes.byref(desc)))
        workspace = torch.zeros(max(need, 16), dtype=torch.uint8, device=dev)
    elif not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError("workspace must be contiguous and on %s" % dev)
    o = torch.empty((B, Hq, d), dtype=dt, device=dev)
    _call("kron_delta_swa_decode", dev, L.kron_delta_swa_decode, ctypes.byref(desc), q.data_ptr(), k.data_ptr(),
          v.data_ptr(), _s3(q.stride(0), k.stride(0), v.stride(0)), k_cache.data_ptr(), v_cache.data_ptr(),
          lens.data_ptr(), _ptr(freqs), o.data_ptr(), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return o


def swa_cache_store(k, v, k_cache, v_cache, window, sinks=0, *, lens=None):
    """A prompt's (turned) keys and values [B, T, Hkv, d] into the caches of
    swa_decode: token t at position t for t < lens[b] (int32 [B]; None: all)."""
    torch, L = _ready()
    dev = _need_cuda(k, "k")
    B, _, Hkv, d = k_cache.shape
    if k.dim() != 4:
        raise ValueError("k and v must be [B, T, Hkv, d]")
    T = k.shape[1]
    _fits("k", k.shape)
    _check("k", k, (B, T, Hkv, d), k_cache.dtype)
    _check("v", v, (B, T, Hkv, d), k_cache.dtype)
    if lens is not None:
        _check("lens", lens, (B,), torch.int32)
        lens = lens.contiguous()
    _same_device(dev, v=v, k_cache=k_cache, v_cache=v_cache, lens=lens)
    k, v = _rows(k), _rows(v)
    desc = _cache_desc(Hkv, k_cache, v_cache, window, sinks)
    _call("kron_delta_swa_cache_store", dev, L.kron_delta_swa_cache_store, ctypes.byref(desc), T, _ptr(k), _ptr(v),
          _s3(*k.stride()[:3]), _s3(*v.stride()[:3]), _ptr(lens), _ptr(k_cache), _ptr(v_cache))
