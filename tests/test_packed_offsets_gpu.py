"""Offsets of packed sequences that are out of order: rows without meaning, but none outside the tensors."""
import ctypes

import pytest

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "g", "beta")
# (sequence 0 starts late: the slots before its own, which lie behind sequence 1's, are nobody's)
OFFSETS = [[640, 0, 700], [1000, 0, 1000, 10], [900, 300, 100, 0], [64, 1000, 0, 1000], [1000, 0, 0, 0]]


def _torch():
    import torch
    return torch


class Guard:
    """A tensor between two stretches that hold what nothing may change (inputs: that nothing may use)."""

    def __init__(self, shape, dtype, fill, pad=1 << 16):
        torch = _torch()
        n = 1
        for s in shape:
            n *= s
        self.all = torch.full((pad + n + pad,), fill, dtype=dtype, device="cuda")
        self.t, self.fill, self.pad, self.n = self.all[pad:pad + n].view(shape), fill, pad, n

    def intact(self):
        return bool((self.all[:self.pad] == self.fill).all() and (self.all[self.pad + self.n:] == self.fill).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cu", OFFSETS + [[8 * x for x in cu] for cu in OFFSETS])
def test_delta_rule(cu, dtype):
    """(The long ones are cut into segments.)"""
    import delta_rule_recurrent_chunk_amd as kd
    from delta_rule_recurrent_chunk_amd import gdr, layers
    torch = _torch()
    print("offsets", cu, dtype, flush=True)
    L, dt, T, N = kd.lib(), torch.bfloat16 if dtype == "bf16" else torch.float32, 8000 if max(cu) > 1000 else 1000, len(cu) - 1
    G = torch.Generator(device="cuda").manual_seed(T)
    t = {n: Guard((T, 1, 64), dt, 3.0) for n in "qkv"}
    t.update({n: Guard((T, 1), dt, 3.0) for n in ("g", "beta")})
    for n in NAMES:
        t[n].t.normal_(generator=G).mul_(0.1)
    t["g"].t.abs_().neg_()
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    layers._ready()
    dev, desc, *_ = gdr._gdr(*(t[n].t for n in NAMES), 0.2, c)
    d, s = ctypes.byref(desc), torch.cuda.current_stream().cuda_stream
    u8 = torch.uint8
    out = {n: Guard((T, 1, 64), dt, 7.0) for n in ("o", "dq", "dk", "dv")}
    out.update({n: Guard((T, 1), dt, 7.0) for n in ("dg", "dbeta")})
    out.update({n: Guard((N, 1, 64, 64), torch.float32, 7.0) for n in ("ST", "dS0")})
    out["saved"] = Guard((L.kron_delta_gdr_saved_bytes(d, 1),), u8, 7)
    for back in (0, 1):
        out["ws%d" % back] = Guard((L.kron_delta_gdr_workspace_bytes(d, 1, back),), u8, 7)
    p = {n: x.t.data_ptr() for n, x in {**t, **out}.items()}
    args = [c.data_ptr()] + [p[n] for n in NAMES]
    assert L.kron_delta_gdr_fwd(d, *args, None, p["o"], p["ST"], p["saved"], p["ws0"], out["ws0"].n, s) == 0
    torch.cuda.synchronize()
    assert L.kron_delta_gdr_bwd(d, *args, p["saved"], p["o"], None, p["dq"], p["dk"], p["dv"], p["dg"], p["dbeta"], p["dS0"],
                                p["ws1"], out["ws1"].n, s) == 0
    torch.cuda.synchronize()
    assert all(x.intact() for x in {**t, **out}.values()), [n for n, x in out.items() if not x.intact()]


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cu", OFFSETS)
def test_paged_cache(cu, dtype, heads_first):
    """(Heads first: a row before the first one would lie a head's rows before the tensor.)"""
    import delta_rule_recurrent_chunk_amd as kd
    from delta_rule_recurrent_chunk_amd import paged
    torch = _torch()
    print("offsets", cu, dtype, heads_first, flush=True)
    L, dt, T, N = kd.lib(), torch.bfloat16 if dtype == "bf16" else torch.float32, 1000, len(cu) - 1
    G = torch.Generator(device="cuda").manual_seed(T)
    q, k, v = Guard((T, 4, 64), dt, 3.0), Guard((T, 2, 64), dt, 3.0), Guard((T, 2, 64), dt, 3.0)
    kp, vp = Guard((8, 16, 2, 64), dt, 7.0), Guard((8, 16, 2, 64), dt, 7.0)
    o, lse = Guard((T, 4, 64), dt, 7.0), Guard((4, T), torch.float32, 7.0)
    for x in (q, k, v, kp, vp):
        x.t.normal_(generator=G)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    c, lens, table, ptable = i32(cu), i32([5] * N), i32([[0, 1, 2]] * N), i32([6, 7])
    kd.paged_append(k.t, v.t, kp.t, vp.t, table, lens, cu_seqlens=c)
    desc = paged._desc(kp.t, vp.t, table, N, T, 4, scale=0.125, prefix=30, prefix_width=2)
    ws = Guard((L.kron_delta_prefix_attn_workspace_bytes(desc, 1),), torch.uint8, 7)
    st = L.kron_delta_prefix_attn(desc, q.t.data_ptr(), paged._S2(*(64, 64 * T) if heads_first else (256, 64)), kp.t.data_ptr(), vp.t.data_ptr(),
                                  ptable.data_ptr(), table.data_ptr(), lens.data_ptr(), c.data_ptr(), o.t.data_ptr(),
                                  lse.t.data_ptr(), ws.t.data_ptr(), ws.n, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and all(x.intact() for x in (q, k, v, kp, vp, o, lse, ws))
