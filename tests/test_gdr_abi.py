"""Refusals of the gated delta rule's entry points: every call below fails its checks (or has nothing to do) before any
launch, so the addresses are never used (CPU)."""
import ctypes
import os

import pytest

import delta_rule_recurrent_chunk_amd as kd
from delta_rule_recurrent_chunk_amd import gdr

OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, ALIAS = 0, -1, -2, -3, -4, -5, -7


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(kd.LIB_PATH):
        from delta_rule_recurrent_chunk_amd import build
        build.build()
    return kd.lib()


def P(i, off=0):
    return ctypes.c_void_p(0x7F0000000000 + (i << 40) + off)


def desc(**o):
    f = dict(B=2, T=100, Hk=2, Hv=4, dk=64, dv=128, dtype=1, gates32=0, scale=0.125, q_stride=(12800, 128, 64),
             k_stride=(12800, 128, 64), v_stride=(51200, 512, 128))
    f.update(o)
    return gdr.KdGdrDesc(**f)


BAD = [dict(B=0), dict(B=65536), dict(T=-1), dict(T=(1 << 29) + 1), dict(Hk=0), dict(Hv=3), dict(dk=4), dict(dk=60),
       dict(dk=136), dict(dv=0), dict(dv=132), dict(dv=264), dict(scale=float("nan")), dict(q_stride=(12800, 128, -64)),
       dict(v_stride=(51200, 500, 128)), dict(k_stride=(12800, 128, 4))]


def test_limits_match_the_header():
    text = open(os.path.join(os.path.dirname(kd.__file__), "..", "include", "kron_delta.h")).read()
    assert "#define KRON_DELTA_GDR_MAX_DK %d" % gdr.GDR_MAX_DK in text
    assert "#define KRON_DELTA_GDR_MAX_DV %d" % gdr.GDR_MAX_DV in text


def test_forward_and_backward_checks(L):
    def fwd(d, wsb=1 << 40, **o):
        p = dict(cu=None, q=P(0), k=P(1), v=P(2), g=P(3), beta=P(4), S0=P(5), o=P(6), ST=P(7), saved=P(8), ws=P(9))
        p.update(o)
        return L.kron_delta_gdr_fwd(ctypes.byref(d) if d else None, *p.values(), wsb, None)

    def bwd(d, wsb=1 << 40, **o):
        p = dict(cu=None, q=P(0), k=P(1), v=P(2), g=P(3), beta=P(4), saved=P(5), dO=P(6), dST=P(7), dq=P(8), dk=P(9), dv=P(10),
                 dg=P(11), dbeta=P(12), dS0=P(13), ws=P(14))
        p.update(o)
        return L.kron_delta_gdr_bwd(ctypes.byref(d) if d else None, *p.values(), wsb, None)

    need = L.kron_delta_gdr_workspace_bytes
    for f in (fwd, bwd):
        assert f(None) == NULL and f(desc(dtype=7)) == DTYPE
        for bad in BAD:
            assert f(desc(**bad)) == SHAPE and need(ctypes.byref(desc(**bad)), 0, 1) == 0, bad
        for name in ("q", "k", "v", "g", "beta"):
            assert f(desc(), **{name: None}) == NULL and f(desc(), **{name: P(20, 8)}) == ALIGN, name
        assert f(desc(), cu=P(20, 2)) == ALIGN
        assert f(desc(), ws=None) == WORKSPACE
        assert f(desc(), ws=P(2, 256)) == ALIAS
        assert f(desc(B=1, T=1 << 29, Hv=65535, Hk=65535)) == SHAPE      # launches past 32 bits of threads
    for name in ("S0", "o", "ST", "saved", "ws"):
        assert fwd(desc(), **{name: P(20, 8)}) == ALIGN, name
    for name in ("saved", "dO", "dST", "dq", "dk", "dv", "dg", "dbeta", "dS0", "ws"):
        assert bwd(desc(), **{name: P(20, 8)}) == ALIGN, name
    for name in ("saved", "dO", "dq", "dk", "dv", "dg", "dbeta"):
        assert bwd(desc(), **{name: None}) == NULL, name
    assert fwd(desc(), o=None) == NULL
    assert fwd(desc(), o=P(2)) == ALIAS and fwd(desc(), ST=P(5)) == ALIAS and fwd(desc(), saved=P(6)) == ALIAS
    assert bwd(desc(), dv=P(6)) == ALIAS and bwd(desc(), dq=P(0)) == ALIAS and bwd(desc(), dg=P(12)) == ALIAS
    for back, f in ((0, fwd), (1, bwd)):
        size = need(ctypes.byref(desc()), 0, back)
        assert size > 0 and f(desc(), wsb=size - 1) == WORKSPACE
    assert need(ctypes.byref(desc()), 0, 1) > need(ctypes.byref(desc()), 0, 0)
    assert fwd(desc(T=0), q=None, k=None, v=None, g=None, beta=None, o=None, ST=None, ws=None, wsb=0) == OK
    assert bwd(desc(T=0), q=None, k=None, v=None, g=None, beta=None, saved=None, dO=None, dq=None, dk=None, dv=None, dg=None,
               dbeta=None, dS0=None, ws=None, wsb=0) == OK


def test_descriptors_as_bytes_are_the_structure():
    d = desc()
    assert bytes(d) == gdr._DESC(*(x for n, _ in d._fields_ for x in (
        lambda v: v if hasattr(v, "__len__") else (v,))(getattr(d, n))))


def test_step_checks(L):
    def step(d, **o):
        p = dict(q=P(0), k=P(1), v=P(2), g=P(3), beta=P(4), Si=P(5), o=P(6), So=P(5))
        p.update(o)
        return L.kron_delta_gdr_step(ctypes.byref(d) if d else None, *p.values(), None)

    assert step(None) == NULL and step(desc()) == SHAPE and step(desc(T=1, dtype=3)) == DTYPE
    for name in ("q", "k", "v", "g", "beta", "Si", "o", "So"):
        assert step(desc(T=1), **{name: None}) == NULL and step(desc(T=1), **{name: P(20, 4)}) == ALIGN, name
    assert step(desc(T=1), So=P(5, 256)) == ALIAS
    assert step(desc(T=1), o=P(2)) == ALIAS and step(desc(T=1), o=P(5)) == ALIAS


def test_binding_refuses_bad_arguments():
    import torch
    q, g = torch.zeros(1, 4, 2, 64), torch.zeros(1, 4, 2)
    with pytest.raises(ValueError, match="device tensor"):
        kd.gdr_fwd(q, q, q, g, g)
    with pytest.raises(ValueError, match="must be"):
        kd.gdr_step(q, q, q, g, g, q)
