"""Refusals of the paged cache's entry points: every call below fails its checks (or has nothing to do) before any
launch, so the addresses are never used (CPU)."""
import ctypes
import os

import pytest

import delta_rule_recurrent_chunk_amd as kd
from delta_rule_recurrent_chunk_amd import paged as pg

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
    f = dict(B=3, T=3, Hq=4, Hkv=2, d=64, dtype=1, page=16, pages=10, width=3, rot=64, layout=0, rope_scale=1.0,
             offset=0, prefix=40, prefix_width=3, scale=0.125, k_stride=(2048, 128, 64), v_stride=(2048, 128, 64),
             table_stride=3)
    f.update(o)
    return pg.KdPagedDesc(**f)


BAD = [dict(B=0), dict(T=-1), dict(Hkv=0), dict(d=4), dict(page=0), dict(pages=0), dict(width=-1), dict(table_stride=-1),
       dict(k_stride=(2048, 128, -64)), dict(v_stride=(2048, 100, 64)), dict(T=4), dict(Hq=1 << 20), dict(B=(1 << 24) + 1)]


def test_descriptors_as_bytes_are_the_structure():
    d = desc(offset=-5, k_stride=(7, 6, 5), v_stride=(4, 3, 2))
    assert bytes(d) == pg._DESC(*(x for n, _ in d._fields_ for x in (
        lambda v: v if hasattr(v, "__len__") else (v,))(getattr(d, n)))).ljust(ctypes.sizeof(d), b"\0")


def test_append_checks(L):
    def call(d, stride=(256, 64, 128, 64, 128, 64), **o):
        p = dict(q=P(0), k=P(1), v=P(2), stride=pg._S6(*stride), kp=P(3), vp=P(4), table=P(5), lens=P(6), cu=None,
                 freqs=P(8), out=P(9))
        p.update(o)
        return L.kron_delta_paged_append(ctypes.byref(d) if d else None, *p.values(), None)

    assert call(None) == NULL
    assert call(desc(dtype=2)) == DTYPE
    for bad in BAD + [dict(rot=3), dict(rot=66), dict(rot=-2), dict(layout=2), dict(rope_scale=float("nan")),
                      dict(offset=1 << 41), dict(d=512, k_stride=(16384, 1024, 512), v_stride=(16384, 1024, 512))]:
        assert call(desc(**bad)) == SHAPE, bad
    for name in ("q", "k", "v", "kp", "vp", "table", "lens", "freqs", "out"):
        assert call(desc(), **{name: None}) == NULL, name
    for name in ("q", "k", "v", "kp", "vp", "out"):
        assert call(desc(), **{name: P(11, 8)}) == ALIGN, name
    for name in ("table", "lens", "cu"):
        assert call(desc(), **{name: P(11, 2)}) == ALIGN, name
    assert call(desc(), freqs=P(11, 4)) == ALIGN
    assert call(desc(), stride=(256, 64, 128, 60, 128, 64)) == SHAPE and call(desc(), stride=(-256, 64) * 3) == SHAPE
    assert call(desc(k_stride=(2048, 64, 64))) == ALIAS                  # slots that overlap
    assert call(desc(), out=P(0)) == ALIAS and call(desc(), kp=P(1)) == ALIAS and call(desc(), vp=P(3)) == ALIAS
    assert call(desc(), vp=P(3, 128)) == ALIAS and call(desc(), out=P(4, 64)) == ALIAS and call(desc(), lens=P(3, 64)) == ALIAS
    wide = desc(k_stride=(4096, 256, 64), v_stride=(4096, 256, 64))
    assert call(wide, vp=P(3, 128), lens=None) == NULL                    # (interleaved caches get past their overlap)
    assert call(wide, vp=P(3, 320)) == ALIAS
    assert call(desc(T=0, B=3), cu=P(7), k=None, v=None, q=None) == OK


def test_prefix_checks(L):
    def call(d, wsb=1 << 40, stride=(256, 64), **o):
        p = dict(q=P(0), stride=pg._S2(*stride), kp=P(1), vp=P(2), pt=P(3), table=P(4), lens=P(5), cu=None, o=P(6),
                 lse=P(7), ws=P(8))
        p.update(o)
        return L.kron_delta_prefix_attn(ctypes.byref(d) if d else None, *p.values(), wsb, None)

    need = L.kron_delta_prefix_attn_workspace_bytes
    assert call(None) == NULL and need(None, 0) == 0
    assert call(desc(dtype=2)) == DTYPE
    for bad in BAD + [dict(Hq=0), dict(Hq=3), dict(d=96, k_stride=(4096, 192, 96), v_stride=(4096, 192, 96)), dict(prefix=-1),
                      dict(prefix=49), dict(prefix_width=-1), dict(scale=0.0), dict(scale=float("inf"))]:
        assert call(desc(**bad)) == SHAPE and need(ctypes.byref(desc(**bad)), 0) == 0, bad
    assert need(ctypes.byref(desc(T=0)), 1) == 0 and need(ctypes.byref(desc()), 0) > 0
    for name in ("q", "kp", "vp", "pt", "table", "lens", "o"):
        assert call(desc(), **{name: None}) == NULL, name
    for name in ("q", "kp", "vp", "o", "ws"):
        assert call(desc(), **{name: P(11, 8)}) == ALIGN, name
    for name in ("pt", "table", "lens", "cu", "lse"):
        assert call(desc(), **{name: P(11, 2)}) == ALIGN, name
    assert call(desc(), stride=(256, 60)) == SHAPE
    assert call(desc(), o=P(0)) == ALIAS and call(desc(), lse=P(6)) == ALIAS and call(desc(), ws=P(1)) == ALIAS
    size = need(ctypes.byref(desc()), 0)
    assert call(desc(), ws=None) == WORKSPACE and call(desc(), wsb=size - 1) == WORKSPACE
    # launches past 32 bits of threads
    huge = desc(T=1 << 29, B=3, Hq=64, Hkv=1)
    assert call(huge, cu=P(9), stride=(4096, 64)) == SHAPE
    assert call(desc(T=0, B=3), cu=P(9), q=None, o=None, ws=None) == OK


def test_binding_refuses_bad_arguments():
    import torch
    q, kp, t, n = torch.zeros(2, 4, 64), torch.zeros(3, 16, 2, 64), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        kd.prefix_attn(q, kp, kp, n, 4, t, n)
    with pytest.raises(ValueError, match="device tensor"):
        kd.paged_append(q[:, :2], q[:, :2], kp, kp, t, n)
