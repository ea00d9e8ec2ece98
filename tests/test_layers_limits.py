"""Sizes of the layers beside the mixer: workspaces and refusals (CPU; no call here reaches a launch)."""
import ctypes

import pytest

import delta_rule_recurrent_chunk_amd as kd
from delta_rule_recurrent_chunk_amd import layers as la
from tests.test_layers_abi import ALIAS, SHAPE, L, P, S3  # noqa: F401  (L is a fixture)


def swa(B, T, Hq, Hkv, d, window, sinks, dtype=1):
    s = [S3(T * H * d, H * d, d) for H in (Hq, Hkv, Hkv)]
    return la.KdSwaDesc(B, T, T, Hq, Hkv, d, dtype, window, sinks, 0.125, *s)


@pytest.mark.parametrize("N,T,window,sinks", [(512, 65536, 1024, 4), (2048, 65536, 1024, 4), (1024, 32768, 512, 64), (1, 65536, 1024, 4),
                                              (13, 8191, 512, 1), (30000, 30000, 100, 1)])
def test_packed_workspace_does_not_grow_with_short_sequences(L, N, T, window, sinks):
    """Rows' statistics (8 bytes) and, per 256 to 4096 rows and per sequence that is long enough to have queries beyond
    the window, 2 fp32 rows of each sink and head."""
    Hq, d = 32, 128
    need = L.kron_delta_swa_workspace_bytes(ctypes.byref(swa(N, T, Hq, 8, d, window, sinks)), 1)
    long = min(N, T // (128 + window))
    assert 8 * T * Hq <= need <= 8 * T * Hq + 256 + (T // 256 + long) * Hq * 2 * sinks * d * 4
    if sinks == 4:
        assert need < 100 << 20


@pytest.mark.parametrize("strides,gap", [((110, 100, 10), 10), ((200, 100, 10), 95), ((100, 200, 10), -95), ((110, 100, 10), -10)])
def test_rope_outputs_that_meet_in_other_tokens_are_refused(L, strides, gap):
    """q_out and k_out of one head each in rows that interleave: apart in every token, but not from the next one."""
    s = S3(*strides)
    d = la.KdRopeDesc(2, 2, 1, 1, 10, 4, 0, 0, 0, 0, 0, 1.0, s, s, s, s)
    assert L.kron_delta_rope(ctypes.byref(d), P(0), P(1), P(2), P(3), P(4, 4000), P(4, 4000 + 4 * gap), None) == ALIAS


def test_launches_past_32_bits_of_threads_are_refused(L):
    """Within the bounds of the single sizes; the launch itself would fail."""
    g = la.KdGlrDesc(65535, 1 << 20, 1, 1)
    assert L.kron_delta_glr_workspace_bytes(ctypes.byref(g)) == 0
    assert L.kron_delta_glr_fwd(ctypes.byref(g), *[P(i) for i in range(8)], 1 << 40, None) == SHAPE
    assert L.kron_delta_glr_bwd(ctypes.byref(g), *[P(i) for i in range(11)], 1 << 40, None) == SHAPE
    s = S3(2 << 30, 2, 2)
    r = la.KdRopeDesc(1, 1 << 30, 1, 0, 2, 2, 0, 1, 0, 0, 0, 1.0, s, s, s, s)
    assert L.kron_delta_rope(ctypes.byref(r), P(0), None, P(2), P(3), P(4), None, None) == SHAPE
    a = swa(65535, 1, 512, 1, 32, 8, 0)
    assert L.kron_delta_swa_fwd(ctypes.byref(a), None, *[P(i) for i in range(5)], None) == SHAPE
    assert L.kron_delta_swa_workspace_bytes(ctypes.byref(a), 0) == 0
    assert L.kron_delta_swa_bwd(ctypes.byref(a), None, *[P(i) for i in range(10)], 1 << 40, None) == SHAPE
    c = S3(16 * 16 * 128, 16 * 128, 128)
    c = la.KdSwaCacheDesc(1, 16, 16, 128, 16, 1, 8, 0, 1.0, 0, 0, 1.0, c, c)
    k = S3(1 << 39, 16 * 128, 128)
    assert L.kron_delta_swa_cache_store(ctypes.byref(c), 1 << 27, P(0), P(1), k, k, None, P(3), P(4), None) == SHAPE
