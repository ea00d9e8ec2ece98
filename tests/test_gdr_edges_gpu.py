"""Edges of the gated delta rule on the GPU."""
import numpy as np
import pytest

import gdr_ref as R
from test_gdr_gpu import NAMES, _torch, check, compare, f64, inputs, run

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


# ------------------------------------- packed calls around the widths' borders
@pytest.mark.parametrize("lens,H,d", [([70] * 9, 16, 64), ([1, 200, 0, 64, 129, 3, 90, 65, 2, 150], 16, 64), ([65] * 12, 16, 64),
                                      ([66] * 13, 16, 64), ([100, 1, 63, 130, 5, 64], 16, 128), ([70] * 7, 16, 128)])
def test_packed_calls_of_many_heads(lens, H, d):
    """128 to 224 workgroups of four groups of value columns: each sequence has the bits of a call for itself, and some
    heads of it the results."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    print("case", lens, H, d, flush=True)
    cu = np.concatenate([[0], np.cumsum(lens)])
    t = inputs((int(cu[-1]),), H // 4, H, d, d, "bf16", sum(lens), n=len(lens))
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    got = run(t, 0.2, c)
    for i, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        one = {n: x[i:i + 1] if n in ("S0", "dST") else x[None, a:b] for n, x in t.items()}
        alone = run(one, 0.2)
        assert all(torch.equal(alone[n][0], got[n][i] if n in ("ST", "dS0") else got[n][a:b]) for n in got), i
    i = int(np.argmax(lens))
    few = {n: (x[i:i + 1, :4] if n in ("S0", "dST") else x[None, cu[i]:cu[i + 1], :1 if n in ("q", "k") else 4]) for n, x in t.items()}
    part = {n: (x[i:i + 1, :4] if n in ("ST", "dS0") else x[None, cu[i]:cu[i + 1], :1 if n in ("dq", "dk") else 4]) for n, x in got.items()}
    compare(few, part, 0.2, "bf16")
