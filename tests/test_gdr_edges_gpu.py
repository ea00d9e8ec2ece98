"""Edges of the gated delta rule on the GPU."""
import numpy as np
import pytest

import gdr_ref as R
from test_gdr_gpu import NAMES, _torch, check, f64, inputs

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ one token
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dk", [8, 24, 40, 64, 72, 128])
def test_an_infinity_in_a_steps_state_stays_one(dk, dtype):
    """Element 0 of a row infinite: S k is infinite, and with it the row's other elements, whatever the lanes past dk hold."""
    import delta_rule_recurrent_chunk_amd as kd
    t = inputs((2, 1), 1, 2, dk, 16, dtype, dk)
    a = {n: f64(x) for n, x in t.items()}
    S = t["S0"].clone()
    S[0, 1, 3, 0] = float("inf")
    kd.gdr_step(*(t[n][:, 0] for n in NAMES), S)
    got, before = f64(S), a["S0"]
    for b in range(2):
        for h in range(2):
            _, st = R.tokens(*(a[n][b, :1, h // 2 if n in ("q", "k") else h] for n in NAMES), before[b, h], dk ** -0.5)
            rows = [r for r in range(16) if (b, h, r) != (0, 1, 3)]
            mag = np.abs(before[b, h]).sum(1, keepdims=True) + np.abs(a["v"][b, 0, h])[:, None] + np.abs(st[1])
            check("S", S[b, h][rows], st[1][rows], ((dk + 8) * R.W * mag)[rows])
    k = a["k"][0, 0, 0]
    assert np.isnan(got[0, 1, 3, 0]) and np.array_equal(got[0, 1, 3, 1:], -np.inf * np.sign(k[0]) * np.sign(k[1:]))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("g", [float("-inf"), -1e30, -200.0, -110.0, -95.0, -30.0, 0.0])
def test_steps_with_resets_and_strong_decays(g, dtype):
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    dk, dv, u = 40, 72, 2.0 ** -8 if dtype == "bf16" else R.W
    t = inputs((3, 2), 1, 2, dk, dv, dtype, 90)
    t["g"][:2] = g
    t["beta"][1, :, 1] = 0.0
    a = {n: f64(x) for n, x in t.items()}
    S = t["S0"].clone()
    o = torch.stack([kd.gdr_step(*(t[n][:, s] for n in NAMES), S) for s in range(2)], 1)
    for b in range(3):
        for h in range(2):
            with np.errstate(under="ignore"):
                ro, st = R.tokens(*(a[n][b, :, h // 2 if n in ("q", "k") else h] for n in NAMES), a["S0"][b, h], dk ** -0.5)
            # two tokens of dk + 8 operations on what is there, written or decayed (none of them lengthens it)
            mag = sum(np.abs(x).sum(1, keepdims=True) for x in st) + np.abs(a["v"][b, :, h]).sum(0)[:, None]
            check("S", S[b, h], st[2], 2 * (dk + 8) * R.W * mag + 1e-37)
            check("o", o[b, :, h], ro, 1.01 * u * np.abs(ro) +
                  2 * (dk + 8) * R.W * (mag[:, 0] * np.abs(a["q"][b]).max() * dk ** 0.5) + 1e-37)
