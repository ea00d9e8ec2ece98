"""What the gated delta rule's results are off by, against 64 bits, in the root of the sum of squares: the roundings
that its kernels keep to (gdr_rounded) and fp32 sums, and no more.  The tolerances tell each of the remainders, and
each part of the segments' maps, from a kernel without it (CPU); the kernels are held to them (GPU)."""
import functools

import numpy as np
import pytest

import gdr_ref as R
import gdr_rounded as C

NAMES = ("q", "k", "v", "g", "beta")


@functools.lru_cache(None)
def solved(T, dk, dv, gates, seed, dtype="bf16"):
    """A head's inputs and its results in 64 bits."""
    x, S0, dO, dST = C.problem(T, dk, dv, gates, seed, C.bf16 if dtype == "bf16" else lambda y: np.float32(y).astype(np.float64))
    a = [x[n] for n in NAMES]
    o, st = R.tokens(*a, S0, dk ** -0.5)
    g = R.tokens_bwd(*a, st, dO, dST, dk ** -0.5)
    ref = dict(o=o, ST=st[-1], dq=g[0], dk=g[1], dv=g[2], dg=g[3], dbeta=g[4], dS0=g[5][0])
    return x, S0, dO, dST, ref


@functools.lru_cache(None)
def rounded(T, dk, dv, gates, seed, **keep):
    """How far the roundings alone put the results off."""
    x, S0, dO, dST, ref = solved(T, dk, dv, gates, seed)
    ch = C.Chunks(*(x[n] for n in NAMES), dk ** -0.5, C.Keep(**keep))
    o, states = ch.forward(S0)
    got = dict(o=o, ST=states[-1], **ch.backward(states, dO, dST))
    for n in ("o", "dq", "dk", "dv"):
        got[n] = C.bf16(got[n])
    return {n: C.off(got[n], ref[n]) for n in ref}


def tolerance(T, dk, dv, gates, seed, dtype="bf16"):
    """fp32: the terms of a sum are dk + dv + 128 at most, its error W times their number's root, relative to them; what
    a chunk adds to a state stays until it is forgotten, at once or ("slow") to the end: as many such errors as chunks,
    independent of each other.  dg is a sum of such sums over a chunk that cancel to a tenth of them or less ("slow":
    hundredth), dbeta a row's.  bf16: the roundings as well (the same ones but where fp32 moves a value across a border)."""
    w = R.W * (dk + dv + 128) ** 0.5 * (1.0 if gates == "fast" else (T / 64 + 1) ** 0.5)
    w = dict(o=w, ST=w, dq=2 * w, dk=2 * w, dv=2 * w, dbeta=4 * w, dg=(20 if gates == "fast" else 200) * w, dS0=w)
    if dtype == "fp32":
        return {n: 2 * x for n, x in w.items()}
    e = rounded(T, dk, dv, gates, seed)
    return {n: (1.5 if n in ("ST", "dS0") else 1.1) * e[n] + w[n] for n in w}


SHAPES = [(1024, 128, 128, "fast"), (700, 64, 72, "fast"), (700, 64, 72, "slow"), (130, 40, 64, "slow")]
PLANTED = [(dict(added=2), ("ST", "dS0")), (dict(P_bwd=1), ("dS0", "dbeta")), (dict(state=1), ("ST", "dS0", "dv", "dbeta")),
           (dict(A=1), ("ST", "dS0")), (dict(X=1), ("dbeta",)), (dict(U=1), ("dbeta", "dq"))]


@pytest.mark.parametrize("shape", SHAPES[:2])
@pytest.mark.parametrize("keep,names", PLANTED)
def test_the_tolerances_tell_a_dropped_remainder(keep, names, shape):
    tol, e = tolerance(*shape, 1), rounded(*shape, 1, **keep)
    assert all(e[n] > tol[n] for n in names), {n: (e[n], tol[n]) for n in names}
    assert all(x <= tol[n] for n, x in rounded(*shape, 1).items())


LONG = (2100, 64, 72, "slow")


@pytest.mark.parametrize("plant", ["zero", "transposed", "order"])
def test_the_tolerances_tell_a_wrong_map(plant):
    tol = tolerance(*LONG, 2)
    e = rounded(*LONG, 2, segment=9, plant=plant)
    assert e["ST"] > 20 * tol["ST"] and e["o"] > 1.2 * tol["o"], (e, tol)
    assert all(x <= tol[n] for n, x in rounded(*LONG, 2, segment=9).items())


# ---------------------------------------------------------------------- GPU
def run(problems, dk, cu=None, lead=None):
    """Results of heads (or of packed sequences of one head each) side by side."""
    import torch

    import delta_rule_recurrent_chunk_amd as kd
    dt, f32 = (torch.bfloat16 if problems[0][1] == "bf16" else torch.float32), torch.float32
    heads = [p[0] for p in problems]
    dev = lambda x, d: torch.tensor(np.ascontiguousarray(x), dtype=f32, device="cuda").to(d)  # noqa: E731
    if cu is None:
        t = {n: dev(np.stack([h[0][n] for h in heads], 1)[None], f32 if n in ("g", "beta") else dt) for n in NAMES}
        S0, dST = (dev(np.stack([h[i] for h in heads])[None], f32) for i in (1, 3))
        dO = dev(np.stack([h[2] for h in heads], 1)[None], dt)
    else:
        t = {n: dev(np.concatenate([h[0][n] for h in heads])[:, None], f32 if n in ("g", "beta") else dt) for n in NAMES}
        S0, dST = (dev(np.stack([h[i] for h in heads])[:, None], f32) for i in (1, 3))
        dO = dev(np.concatenate([h[2] for h in heads])[:, None], dt)
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    a = [t[n] for n in NAMES]
    o, ST, saved = kd.gdr_fwd(*a, S0, cu_seqlens=cu, save_states=True)
    out = dict(o=o, ST=ST, **kd.gdr_bwd(*a, saved, dO, dST, cu_seqlens=cu))
    o2, ST2 = kd.gdr_fwd(*a, S0, cu_seqlens=cu)
    assert torch.equal(o, o2) and torch.equal(ST, ST2)
    return {n: x.double().cpu().numpy() for n, x in out.items()}


def hold(got, head, ref, tol, cut=None):
    off = {}
    for n in ref:
        y = got[n][head, 0] if cut is not None and n in ("ST", "dS0") else got[n][0, head] if n in ("ST", "dS0") else \
            got[n][cut, 0] if cut is not None else got[n][0, :, head]
        off[n] = C.off(y, ref[n])
    print(" ".join("%s %.2e/%.2e" % (n, off[n], tol[n]) for n in off), flush=True)
    assert all(off[n] <= tol[n] for n in off)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_results_are_off_by_their_roundings(shape, dtype):
    heads = [solved(*shape, s, dtype) for s in (1, 2)]
    got = run([(h, dtype) for h in heads], shape[1])
    for i, h in enumerate(heads):
        hold(got, i, h[4], tolerance(*shape, i + 1, dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("shape,H", [((200, 64, 64, "fast"), 160), ((200, 128, 128, "fast"), 80)])
def test_results_of_many_heads_are_off_by_their_roundings(shape, H):
    """Four groups of value columns a workgroup."""
    heads = [solved(*shape, s % 5) for s in range(H)]
    got = run([(h, "bf16") for h in heads], shape[1])
    for i in (0, 1, 2, H - 2, H - 1):
        hold(got, i, heads[i][4], tolerance(*shape, i % 5))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [LONG, (2100, 40, 24, "slow"), (2100, 72, 128, "slow"), (4200, 128, 64, "slow")])
def test_segments_carry_their_states(shape, dtype):
    """At least four segments; the first state still matters behind the last."""
    heads = [solved(*shape, s, dtype) for s in (2, 3)]
    got = run([(h, dtype) for h in heads], shape[1])
    for i, h in enumerate(heads):
        hold(got, i, h[4], tolerance(*shape, i + 2, dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 40)])
def test_packed_segments_carry_their_states(dk, dv, dtype):
    shapes = [(3000, dk, dv, "slow"), (5, dk, dv, "slow"), (2300, dk, dv, "slow")]
    seqs = [solved(*s, 4 + i, dtype) for i, s in enumerate(shapes)]
    cu = np.concatenate([[0], np.cumsum([s[0] for s in shapes])])
    got = run([(h, dtype) for h in seqs], dk, cu)
    for i, h in enumerate(seqs):
        hold(got, i, h[4], tolerance(*shapes[i], 4 + i, dtype), slice(int(cu[i]), int(cu[i + 1])))
