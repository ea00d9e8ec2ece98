"""Sizes of the layers beside the mixer: workspaces and refusals (CPU; no call here reaches a launch)."""
import ctypes

import pytest

import delta_rule_recurrent_chunk_amd as kd
from delta_rule_recurrent_chunk_amd import layers as la
from tests.test_layers_abi import ALIAS, L, P, S3  # noqa: F401  (L is a fixture)


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
