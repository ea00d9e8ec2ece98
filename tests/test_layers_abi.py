"""Refusals of the layers' entry points: every call below fails its checks (or has nothing to do) before any launch,
so the addresses are never used (CPU)."""
import ctypes
import os

import pytest

import delta_rule_recurrent_chunk_amd as kd
from delta_rule_recurrent_chunk_amd import layers as la

OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, ALIAS = 0, -1, -2, -3, -4, -5, -7
S3 = ctypes.c_int64 * 3


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(kd.LIB_PATH):
        from delta_rule_recurrent_chunk_amd import build
        build.build()
    return kd.lib()


def P(i, off=0):
    return ctypes.c_void_p(0x7F0000000000 + (i << 40) + off)


def test_limits_match_the_header():
    text = open(os.path.join(os.path.dirname(kd.__file__), "..", "include", "kron_delta.h")).read()
    assert "#define KRON_DELTA_GLR_CHUNK %d" % la.GLR_CHUNK in text
    assert "#define KRON_DELTA_SWA_MAX_SINKS %d" % la.SWA_MAX_SINKS in text


def test_glr_checks(L):
    def desc(B=2, T=300, D=64, dtype=1):
        return la.KdGlrDesc(B, T, D, dtype)

    def fwd(d, wsb=1 << 40, **o):
        p = dict(x=P(0), f=P(1), i=P(2), h0=P(3), h=P(4), hT=P(5), hs=P(6), ws=P(7))
        p.update(o)
        return L.kron_delta_glr_fwd(ctypes.byref(d) if d else None, *p.values(), wsb, None)

    assert fwd(None) == NULL
    assert fwd(desc(dtype=2)) == DTYPE
    for bad in (dict(B=0), dict(D=0), dict(T=-1), dict(B=65536), dict(T=(1 << 30) + 1), dict(D=(1 << 30) + 1)):
        assert fwd(desc(**bad)) == SHAPE, bad
    assert fwd(desc(), x=None) == NULL and fwd(desc(), f=None) == NULL and fwd(desc(), h=None) == NULL
    assert fwd(desc(), x=P(0, 8)) == ALIGN and fwd(desc(), hs=P(6, 4)) == ALIGN and fwd(desc(), ws=P(7, 8)) == ALIGN
    assert fwd(desc(), h=P(0)) == ALIAS and fwd(desc(), hT=P(3)) == ALIAS and fwd(desc(), hs=P(4)) == ALIAS
    assert fwd(desc(), h=P(1, 32)) == ALIAS
    assert fwd(desc(T=0), x=None, f=None, i=None, h=None, hT=None, ws=None, wsb=0) == OK
    need = L.kron_delta_glr_workspace_bytes(ctypes.byref(desc(T=70000)))
    assert L.kron_delta_glr_workspace_bytes(ctypes.byref(desc(B=0))) == 0
    if need:
        assert fwd(desc(T=70000), ws=None) == WORKSPACE and fwd(desc(T=70000), wsb=need - 1) == WORKSPACE
        assert fwd(desc(T=70000), ws=P(0)) == ALIAS

    def bwd(d, wsb=1 << 40, **o):
        p = dict(x=P(0), f=P(1), i=P(2), hs=P(3), dh=P(4), dhT=P(5), dx=P(6), df=P(7), di=P(8), dh0=P(9), ws=P(10))
        p.update(o)
        return L.kron_delta_glr_bwd(ctypes.byref(d) if d else None, *p.values(), wsb, None)

    assert bwd(None) == NULL and bwd(desc(), hs=None) == NULL and bwd(desc(), di=None) == NULL
    assert bwd(desc(), dh=None) == NULL and bwd(desc(), dx=P(6, 2)) == ALIGN
    assert bwd(desc(), dx=P(0)) == ALIAS and bwd(desc(), dh0=P(5)) == ALIAS and bwd(desc(), df=P(6)) == ALIAS
    assert bwd(desc(T=0), x=None, f=None, i=None, hs=None, dh=None, dx=None, df=None, dh0=None, ws=None) == OK

    def step(d, **o):
        p = dict(x=P(0), f=P(1), i=None, h=P(3), y=P(4), ho=P(5))
        p.update(o)
        return L.kron_delta_glr_step(ctypes.byref(d), *p.values(), None)

    assert step(desc()) == SHAPE and step(desc(T=1), h=None) == NULL and step(desc(T=1), ho=None) == NULL
    assert step(desc(T=1), y=P(3)) == ALIAS and step(desc(T=1), ho=P(0)) == ALIAS and step(desc(T=1), y=P(4, 4)) == ALIGN


def test_rope_checks(L):
    def desc(B=2, T=5, Hq=4, Hk=2, d=64, rot=32, layout=0, dtype=1, pos64=0, pb=0, scale=1.0, **st):
        c = lambda H: S3(T * H * d, H * d, d)
        s = dict(q=c(Hq), k=c(Hk), qo=c(Hq), ko=c(Hk))
        s.update({n: S3(*v) for n, v in st.items()})
        return la.KdRopeDesc(B, T, Hq, Hk, d, rot, layout, dtype, pos64, pb, 0, scale, s["q"], s["k"], s["qo"], s["ko"])

    def call(d, **o):
        p = dict(q=P(0), k=P(1), pos=P(2), fr=P(3), qo=P(4), ko=P(5))
        p.update(o)
        return L.kron_delta_rope(ctypes.byref(d) if d else None, *p.values(), None)

    assert call(None) == NULL and call(desc(dtype=5)) == DTYPE
    for bad in (dict(B=0), dict(T=-1), dict(Hq=0), dict(d=257), dict(rot=0), dict(rot=33), dict(rot=66), dict(layout=2),
                dict(scale=float("nan")), dict(q=(-1, 1, 1)), dict(B=1 << 20, T=1 << 20)):
        assert call(desc(**bad)) == SHAPE, bad
    assert call(desc(qo=(0, 256, 64))) == ALIAS and call(desc(ko=(640, 128, 0))) == ALIAS
    for n in ("q", "pos", "fr", "qo", "k", "ko"):
        assert call(desc(), **{n: None}) == NULL, n
    assert call(desc(Hk=0), k=None, ko=None, q=None) == NULL
    assert call(desc(), q=P(0, 1)) == ALIGN and call(desc(), fr=P(3, 4)) == ALIGN and call(desc(), pos=P(2, 2)) == ALIGN
    assert call(desc(pos64=1), pos=P(2, 4)) == ALIGN
    assert call(desc(), qo=P(0, 2)) == ALIAS and call(desc(), ko=P(0)) == ALIAS and call(desc(), qo=P(5)) == ALIAS
    assert call(desc(), qo=P(2)) == ALIAS and call(desc(), ko=P(3)) == ALIAS
    assert call(desc(), ko=P(1), qo=P(1)) == ALIAS
    assert call(desc(T=0)) == OK


def _swa(B=2, Tq=100, Tk=100, Hq=4, Hkv=2, d=64, dtype=1, window=16, sinks=4, scale=0.125, **st):
    s = dict(q=S3(Tq * Hq * d, Hq * d, d), k=S3(Tk * Hkv * d, Hkv * d, d), v=S3(Tk * Hkv * d, Hkv * d, d))
    s.update({n: S3(*v) for n, v in st.items()})
    return la.KdSwaDesc(B, Tq, Tk, Hq, Hkv, d, dtype, window, sinks, scale, s["q"], s["k"], s["v"])


def test_swa_checks(L):
    def fwd(d, **o):
        p = dict(cu=None, q=P(0), k=P(1), v=P(2), o=P(3), lse=P(4))
        p.update(o)
        return L.kron_delta_swa_fwd(ctypes.byref(d) if d else None, *p.values(), None)

    def bwd(d, wsb=1 << 40, **o):
        p = dict(cu=None, q=P(0), k=P(1), v=P(2), o=P(3), lse=P(4), dO=P(5), dq=P(6), dk=P(7), dv=P(8), ws=P(9))
        p.update(o)
        return L.kron_delta_swa_bwd(ctypes.byref(d) if d else None, *p.values(), wsb, None)

    for f in (fwd, bwd):
        assert f(None) == NULL and f(_swa(dtype=9)) == DTYPE
        for bad in (dict(B=0), dict(Tq=-1), dict(Hq=3), dict(Hkv=0), dict(d=96), dict(window=0), dict(sinks=-1),
                    dict(sinks=65), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(B=65536),
                    dict(q=(25600, 252, 64)), dict(k=(-1, 128, 64)), dict(Tk=(1 << 30) + 1)):
            assert f(_swa(**bad)) == SHAPE, bad
        assert f(_swa(Tk=101), cu=P(20)) == SHAPE            # packed queries and keys are the same rows
        assert f(_swa(), cu=P(20, 2)) == ALIGN
        for n in ("q", "k", "v", "o"):
            assert f(_swa(), **{n: None}) == NULL, n
        assert f(_swa(), q=P(0, 8)) == ALIGN and f(_swa(), lse=P(4, 2)) == ALIGN
    assert fwd(_swa(), o=P(1)) == ALIAS and fwd(_swa(), lse=P(3)) == ALIAS and fwd(_swa(), cu=P(20), o=P(20)) == ALIAS
    assert fwd(_swa(Tq=0), q=None, o=None) == OK
    assert bwd(_swa(), dq=P(0)) == ALIAS and bwd(_swa(), dk=P(8)) == ALIAS and bwd(_swa(), dv=P(5)) == ALIAS
    assert bwd(_swa(), lse=None) == NULL and bwd(_swa(), dO=None) == NULL and bwd(_swa(), dv=None) == NULL
    need = L.kron_delta_swa_workspace_bytes(ctypes.byref(_swa()), 0)
    assert need >= 2 * 4 * 100 * 4 and L.kron_delta_swa_workspace_bytes(ctypes.byref(_swa(d=48)), 0) == 0
    assert L.kron_delta_swa_workspace_bytes(ctypes.byref(_swa()), 1) <= need
    assert bwd(_swa(), ws=None) == WORKSPACE and bwd(_swa(), wsb=need - 1) == WORKSPACE and bwd(_swa(), ws=P(3)) == ALIAS
    assert bwd(_swa(Tq=0, Tk=0)) == OK


def test_decode_and_store_checks(L):
    def desc(B=2, Hq=4, Hkv=2, d=64, cap=40, dtype=1, window=32, sinks=4, scale=0.125, rot=32, layout=0, rs=1.0, **st):
        s = dict(k=S3(cap * Hkv * d, Hkv * d, d), v=S3(cap * Hkv * d, Hkv * d, d))
        s.update({n: S3(*v) for n, v in st.items()})
        return la.KdSwaCacheDesc(B, Hq, Hkv, d, cap, dtype, window, sinks, scale, rot, layout, rs, s["k"], s["v"])

    def dec(d, wsb=1 << 40, st=(256, 128, 128), **o):
        p = dict(q=P(0), k=P(1), v=P(2), kc=P(3), vc=P(4), lens=P(5), fr=P(6), o=P(7), ws=P(8))
        p.update(o)
        return L.kron_delta_swa_decode(ctypes.byref(d) if d else None, p["q"], p["k"], p["v"], S3(*st) if st else None,
                                       p["kc"], p["vc"], p["lens"], p["fr"], p["o"], p["ws"], wsb, None)

    def store(d, T=10, ks=(1280, 128, 64), vs=(1280, 128, 64), **o):
        p = dict(k=P(0), v=P(1), lens=P(2), kc=P(3), vc=P(4))
        p.update(o)
        return L.kron_delta_swa_cache_store(ctypes.byref(d) if d else None, T, p["k"], p["v"], S3(*ks), S3(*vs),
                                            p["lens"], p["kc"], p["vc"], None)

    for f in (dec, store):
        assert f(None) == NULL and f(desc(dtype=4)) == DTYPE
        for bad in (dict(B=0), dict(B=65536), dict(Hq=3), dict(d=80), dict(window=0), dict(sinks=65), dict(cap=35),
                    dict(scale=-1.0), dict(k=(5120, 124, 64))):
            assert f(desc(**bad)) == SHAPE, bad
        assert f(desc(k=(5120, 0, 64))) == ALIAS and f(desc(v=(64, 128, 64))) == ALIAS   # slots on each other
        for n in ("k", "v", "kc", "vc"):
            assert f(desc(), **{n: None}) == NULL, n
        assert f(desc(), vc=P(3)) == ALIAS and f(desc(), kc=P(3, 8)) == ALIGN and f(desc(), lens=P(5, 2)) == ALIGN
        assert f(desc(), vc=P(3, 128)) == ALIAS          # the values one head behind the keys
    for bad in (dict(rot=33), dict(rot=66), dict(rot=-2), dict(layout=3), dict(rs=float("inf"))):
        assert dec(desc(**bad)) == SHAPE, bad
    assert dec(desc(), fr=None) == NULL and dec(desc(), lens=None) == NULL and dec(desc(), o=None) == NULL
    assert dec(desc(), st=None) == NULL and dec(desc(), st=(-256, 128, 128)) == SHAPE
    assert dec(desc(), o=P(0)) == ALIAS and dec(desc(), kc=P(7)) == ALIAS and dec(desc(), ws=P(4)) == ALIAS
    assert dec(desc(), q=P(3)) == ALIAS and dec(desc(), fr=P(6, 4)) == ALIGN and dec(desc(), q=P(0, 1)) == ALIGN
    need = L.kron_delta_swa_decode_workspace_bytes(ctypes.byref(desc()))
    assert need > 0 and L.kron_delta_swa_decode_workspace_bytes(ctypes.byref(desc(cap=35))) == 0
    assert dec(desc(), ws=None) == WORKSPACE and dec(desc(), wsb=need - 1) == WORKSPACE
    # interleaved caches pass the overlap check (and fail the next one)
    two = dict(k=(10240, 256, 64), v=(10240, 256, 64))
    assert dec(desc(**two), vc=P(3, 256), wsb=0) == WORKSPACE
    assert dec(desc(**two), vc=P(3, 128), wsb=0) == ALIAS
    assert store(desc(), T=-1) == SHAPE and store(desc(), ks=(1280, 100, 64)) == SHAPE
    assert store(desc(), k=P(3)) == ALIAS and store(desc(), T=0) == OK


def test_binding_refuses_host_tensors_and_bad_arguments():
    import torch
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError):
        kd.glr_fwd(x, x)
    with pytest.raises(ValueError):
        kd.rope(x[None], None, torch.arange(1), torch.ones(2, dtype=torch.float64))
    with pytest.raises(ValueError):
        kd.swa_fwd(x[None], x[None], x[None], 4)
    for kw in (dict(rot=3), dict(rot=4, scaling="cubic"), dict(rot=4, scaling="byparts", factor=2.0),
               dict(rot=4, factor=0.5)):
        with pytest.raises(ValueError):
            kd.rope_frequencies(**kw)
    assert la._int32(10 ** 12) == 2 ** 31 - 1 and la._int32(-10 ** 12) == -2 ** 31 and la._int32(5) == 5   # (no wrap)
    w, m = kd.rope_frequencies(8, scaling="linear", factor=4.0)
    assert m == 1.0 and torch.allclose(w * 4, kd.rope_frequencies(8)[0])
    w, m = kd.rope_frequencies(64, scaling="byparts", factor=8.0, original_length=4096)
    b = kd.rope_frequencies(64)[0]
    assert w[0] == b[0] and torch.isclose(w[-1], b[-1] / 8) and m > 1.2 and (w <= b).all() and (w >= b / 8 * (1 - 1e-12)).all()
    w, _ = kd.rope_frequencies(64, scaling="ntk", factor=8.0)
    assert w[0] == b[0] and torch.isclose(w[-1], b[-1] / 8)
