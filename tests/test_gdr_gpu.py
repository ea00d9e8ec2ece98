"""The gated delta rule against its reference in 64 bits."""
import numpy as np
import pytest

import gdr_ref as R

pytestmark = pytest.mark.gpu
NAMES = ("q", "k", "v", "g", "beta")


def _torch():
    import torch
    return torch


def f64(t):
    return t.detach().double().cpu().numpy()


def check(name, got, ref, tol):
    g = f64(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), "%s: %d of %d beyond the bound, first at %s: %r for %r, bound %r" % (
        name, bad.sum(), bad.size, tuple(np.argwhere(bad)[0]), g[bad][0], ref[bad][0], np.broadcast_to(tol, g.shape)[bad][0])


def inputs(lead, Hk, Hv, dk, dv, dtype, seed, gates32=False, n=None, state=True, strong=False):
    torch = _torch()
    G = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    mk = lambda *s: torch.randn(*s, generator=G, device="cuda")  # noqa: E731
    k = mk(*lead, Hk, dk)
    t = dict(q=mk(*lead, Hk, dk) / dk ** 0.5, k=0.99 * k / k.norm(dim=-1, keepdim=True), v=mk(*lead, Hv, dv))
    t = {x: y.to(dt) for x, y in t.items()}
    gt = torch.float32 if gates32 else dt
    g = torch.nn.functional.logsigmoid(mk(*lead, Hv) * (3 if strong else 1) + (0 if strong else 3))
    if strong:      # resets, decays past fp32's range, and tokens that write nothing
        r = torch.rand(*lead, Hv, generator=G, device="cuda")
        g = torch.where(r < 0.1, torch.full_like(g, float("-inf")), torch.where(r < 0.2, torch.full_like(g, -100.0), g))
        t["beta"] = torch.where(r > 0.9, 0.0, torch.sigmoid(mk(*lead, Hv))).to(gt)
    else:
        t["beta"] = torch.sigmoid(mk(*lead, Hv)).to(gt)
    t["g"] = g.to(gt)
    n = lead[0] if n is None else n
    t["S0"] = mk(n, Hv, dv, dk) if state else None
    t["dO"] = mk(*lead, Hv, dv).to(dt)
    t["dST"] = mk(n, Hv, dv, dk) if state else None
    return t


def reference(t, scale, dtype, spans=None):
    """Results and bounds of every output for sequences (batch, first row, end row); the final rounding included."""
    a = {n: None if x is None else f64(x) for n, x in t.items()}
    packed = spans is not None
    if packed:
        a = {n: x[None] if n in NAMES + ("dO",) else x for n, x in a.items()}
    else:
        spans = [(b, 0, a["q"].shape[1]) for b in range(a["q"].shape[0])]
    Hk, Hv = a["q"].shape[2], a["v"].shape[2]
    u = 2.0 ** -8 if dtype == "bf16" else R.W
    ug = u if t["g"].dtype == t["q"].dtype else R.W
    val = dict(o=np.zeros(a["v"].shape), dq=np.zeros(a["q"].shape), dk=np.zeros(a["q"].shape), dv=np.zeros(a["v"].shape),
               dg=np.zeros(a["g"].shape), dbeta=np.zeros(a["g"].shape))
    err = {n: np.zeros(x.shape) for n, x in val.items()}
    ST, eST, dS0, edS0 = [], [], [], []
    zero = np.zeros((Hv, a["v"].shape[-1], a["q"].shape[-1]))
    for i, (b, r0, r1) in enumerate(spans):
        S0 = zero if a["S0"] is None else a["S0"][i]
        dST = zero if a["dST"] is None else a["dST"][i]
        out = []
        for h in range(Hv):
            x = [a[n][b, r0:r1, h // (Hv // Hk) if n in ("q", "k") else h] for n in NAMES]
            dO = a["dO"][b, r0:r1, h]
            with np.errstate(under="ignore"):
                o, st = R.tokens(*x, S0[h], scale)
                gr = R.tokens_bwd(*x, st, dO, dST[h], scale)
                e, es, ed = R.bounds(*x, st, scale, u, dO, gr[5]) if r1 > r0 else ({}, 0.0 * zero[0] + R.W, 0.0 * zero[0] + R.W)
            for n, y in zip(("o", "dq", "dk", "dv", "dg", "dbeta"), (o,) + gr[:5]):
                at = (b, slice(r0, r1), h // (Hv // Hk) if n in ("dq", "dk") else h)
                val[n][at] += y
                if e:
                    err[n][at] += e[n]
            out.append((st[-1], es, gr[5][0], ed))
        for lst, y in zip((ST, eST, dS0, edS0), zip(*out)):
            lst.append(np.stack(y))
    for n in val:
        err[n] = 1.01 * (err[n] + (ug if n in ("dg", "dbeta") else u) * np.abs(val[n])) + 1e-30
        if packed:
            val[n], err[n] = val[n][0], err[n][0]
    for n, y, e in (("ST", ST, eST), ("dS0", dS0, edS0)):
        val[n], err[n] = np.stack(y), np.stack(e)
    return val, err


def run(t, scale=None, cu=None, **kw):
    import delta_rule_recurrent_chunk_amd as kd
    o, ST, saved = kd.gdr_fwd(*(t[n] for n in NAMES), t["S0"], scale=scale, cu_seqlens=cu, save_states=True, **kw)
    g = kd.gdr_bwd(*(t[n] for n in NAMES), saved, t["dO"], t["dST"], scale=scale, cu_seqlens=cu)
    return dict(o=o, ST=ST, **g)


def compare(t, got, scale, dtype, spans=None, rows=None):
    val, err = reference(t, scale, dtype, spans)
    for n in ("o", "ST", "dv", "dS0", "dq", "dk", "dbeta", "dg"):
        if rows is not None and n not in ("ST", "dS0"):
            check(n, got[n][rows], val[n][rows], err[n][rows])
        else:
            check(n, got[n], val[n], err[n])


# B, T, Hk, Hv, dk, dv
SHAPES = [(1, 1, 1, 1, 64, 64), (2, 5, 1, 2, 8, 8), (1, 63, 2, 2, 128, 128), (2, 64, 1, 1, 64, 128), (1, 65, 1, 3, 48, 80),
          (2, 130, 2, 4, 128, 64), (1, 200, 1, 1, 72, 136), (1, 150, 1, 2, 128, 256), (3, 128, 1, 1, 24, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, dtype):
    B, T, Hk, Hv, dk, dv = shape
    torch = _torch()
    print("case", shape, dtype, flush=True)
    t = inputs((B, T), Hk, Hv, dk, dv, dtype, T + dk, gates32=T % 2 == 1)
    got = run(t, 0.2)
    compare(t, got, 0.2, dtype)
    again = run(t, 0.2)
    assert all(torch.equal(got[n], again[n]) for n in got)
    # without states
    t["S0"] = t["dST"] = None
    compare(t, run(t, 0.2), 0.2, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_resets_strong_decays_and_no_writes(dtype):
    t = inputs((2, 150), 1, 2, 64, 64, dtype, 5, strong=True)
    compare(t, run(t, 0.2), 0.2, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [[3], [64, 1, 0, 70], [0, 130, 65, 1, 1], [200, 0]])
def test_packed_sequences(lens, dtype):
    torch = _torch()
    cu = np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1]) + 3                     # rows that no sequence holds
    t = inputs((T,), 1, 2, 64, 72, dtype, sum(lens), n=len(lens))
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    got = run(t, 0.2, c)
    compare(t, got, 0.2, dtype, [(0, int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])], slice(0, T - 3))
    # each alone gives the same bits
    import delta_rule_recurrent_chunk_amd as kd
    for i, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        o, ST = kd.gdr_fwd(*(t[n][None, a:b] for n in NAMES), t["S0"][i:i + 1], scale=0.2)
        assert torch.equal(o[0], got["o"][a:b]) and torch.equal(ST[0], got["ST"][i])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,Hk,Hv,dk,dv,state", [([1700], 1, 1, 64, 64, True), ([2051], 1, 2, 128, 72, False),
                                                    ([1600, 1600], 1, 1, 40, 16, True)])
def test_long_sequences_of_few_heads(lens, Hk, Hv, dk, dv, state, dtype):
    """Cut into segments that pass at once."""
    torch = _torch()
    t = inputs((len(lens), lens[0]), Hk, Hv, dk, dv, dtype, lens[0], state=state)
    got = run(t, 0.2)
    compare(t, got, 0.2, dtype)
    assert all(torch.equal(x, run(t, 0.2)[n]) for n, x in got.items())


@pytest.mark.parametrize("B,T,H,d", [(3, 70, 48, 128), (1, 1600, 32, 128), (9, 65, 16, 72)])
def test_forward_of_many_heads(B, T, H, d):
    """Four groups of value columns a workgroup, in the maps of segments too."""
    import delta_rule_recurrent_chunk_amd as kd
    t = inputs((B, T), H // 4, H, d, d, "bf16", T)
    o, ST = kd.gdr_fwd(*(t[n] for n in NAMES), t["S0"])
    o2, ST2, _ = kd.gdr_fwd(*(t[n] for n in NAMES), t["S0"], save_states=True)
    assert _torch().equal(o, o2) and _torch().equal(ST, ST2)
    a = {n: f64(x) for n, x in t.items()}
    for b in range(B):
        for h in range(b, H, 5 if T < 100 else 16):
            x = [a[n][b, :, h // 4 if n in ("q", "k") else h] for n in NAMES]
            ro, st = R.tokens(*x, a["S0"][b, h], d ** -0.5)
            e, es, _ = R.bounds(*x, st, d ** -0.5, 2.0 ** -8)
            check("o", o[b, :, h], ro, 1.01 * (e["o"] + 2.0 ** -8 * np.abs(ro)))
            check("ST", ST[b, h], st[-1], es)


def test_long_packed_sequences_of_few_heads():
    torch = _torch()
    lens = [2000, 1, 0, 700, 5000]
    cu = np.concatenate([[0], np.cumsum(lens)])
    t = inputs((int(cu[-1]),), 1, 1, 64, 64, "fp32", 77, n=len(lens))
    got = run(t, 0.2, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    compare(t, got, 0.2, "fp32", [(0, int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])])


def test_rows_behind_the_last_sequence_are_left_and_bad_offsets_stay_inside():
    import ctypes

    import delta_rule_recurrent_chunk_amd as kd
    from delta_rule_recurrent_chunk_amd import gdr
    torch = _torch()
    t = inputs((70,), 1, 1, 64, 64, "bf16", 9, n=2)
    L = kd.lib()
    for cu, held in (([0, 30, 66], 66), ([5, 1000, 3], None), ([70, -4, 1 << 30], None), ([0, 0, 0], 0)):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        dev, desc, *_ = gdr._gdr(*(t[n] for n in NAMES), 0.2, c)
        o = torch.full_like(t["v"], 7.0)
        ST = torch.empty_like(t["S0"])
        need = L.kron_delta_gdr_workspace_bytes(ctypes.byref(desc), 1, 0)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        st = L.kron_delta_gdr_fwd(ctypes.byref(desc), c.data_ptr(), *(t[n].data_ptr() for n in NAMES), t["S0"].data_ptr(),
                                  o.data_ptr(), ST.data_ptr(), None, ws.data_ptr(), need,
                                  torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert st == 0
        if held is not None:
            assert (o[held:] == 7).all() and not (o[:held] == 7).all(-1).any()
        if cu == [0, 0, 0]:
            assert torch.equal(ST, t["S0"])
        run(t, 0.2, c)
    torch.cuda.synchronize()


def test_empty_sequences_and_strided_inputs():
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    t = inputs((2, 0), 1, 2, 64, 64, "bf16", 3, n=2)
    got = run(t, 0.2)
    assert got["o"].shape == (2, 0, 2, 64) and torch.equal(got["ST"], t["S0"]) and torch.equal(got["dS0"], t["dST"])
    t = inputs((2, 90), 2, 2, 64, 64, "bf16", 4)
    ref = run(t, 0.2)
    fused = torch.stack([t["q"], t["k"], t["v"]], 2)                    # heads of one projection
    head_first = {n: t[n].transpose(1, 2).contiguous().transpose(1, 2) for n in ("q", "k", "v")}
    odd = {n: torch.nn.functional.pad(t[n], (0, 1))[..., :64] for n in ("q", "k", "v")}
    for q, k, v in ((fused[:, :, 0], fused[:, :, 1], fused[:, :, 2]), head_first.values(), odd.values()):
        got = run({**t, "q": q, "k": k, "v": v, "beta": t["beta"].transpose(1, 2).contiguous().transpose(1, 2)}, 0.2)
        assert all(torch.equal(ref[n], got[n]) for n in ref)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,Hk,Hv,dk,dv", [(1, 1, 1, 64, 64), (3, 1, 2, 8, 16), (2, 2, 2, 128, 128), (1, 1, 3, 40, 200),
                                           (5, 4, 4, 24, 8), (1, 2, 4, 128, 256)])
def test_step(B, Hk, Hv, dk, dv, dtype):
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    t = inputs((B, 4), Hk, Hv, dk, dv, dtype, dk + dv, gates32=B == 1)
    a = {n: f64(x) for n, x in t.items()}
    S = t["S0"].clone()
    u = 2.0 ** -8 if dtype == "bf16" else R.W
    ref = [R.tokens(*(a[n][b, :, h // (Hv // Hk) if n in ("q", "k") else h] for n in NAMES), a["S0"][b, h], dk ** -0.5)
           for b in range(B) for h in range(Hv)]
    for s in range(4):
        before = S.clone()
        o = kd.gdr_step(*(t[n][:, s] for n in NAMES), S)
        # a token's products of dk terms, five more operations; four tokens, none lengthens what is there
        for i, (ro, rs) in enumerate(ref):
            b, h = divmod(i, Hv)
            w = (s + 1) * (dk + 8) * R.W
            mag = np.abs(rs[s]).sum(1, keepdims=True) + np.abs(a["v"][b, s, h])[:, None] + np.abs(rs[s + 1])
            check("S", S[b, h], rs[s + 1], w * mag)
            check("o", o[b, h], ro[s], 1.01 * u * np.abs(ro[s]) + w * (mag.max(1) * np.abs(a["q"][b, s]).max() * dk ** 0.5))
        other = torch.empty_like(S)
        assert torch.equal(kd.gdr_step(*(t[n][:, s] for n in NAMES), before, S_out=other), o) and torch.equal(other, S)


def test_prefill_then_steps_equal_one_pass():
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    t = inputs((2, 90), 1, 2, 64, 64, "bf16", 6)
    o, ST = kd.gdr_fwd(*(t[n] for n in NAMES), t["S0"])
    o1, S = kd.gdr_fwd(*(t[n][:, :75] for n in NAMES), t["S0"])
    outs = [o1] + [kd.gdr_step(*(t[n][:, s] for n in NAMES), S)[:, None] for s in range(75, 90)]
    val, err = reference(t, 64 ** -0.5, "bf16")
    check("o", torch.cat(outs, 1), val["o"], err["o"])
    check("S", S, val["ST"], err["ST"])
    check("ST", ST, val["ST"], err["ST"])


def test_gradients_against_differences():
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    t = inputs((1, 70), 1, 2, 64, 64, "fp32", 8)
    gr = run(t, 0.2)
    G = torch.Generator(device="cuda").manual_seed(1)

    def loss(x):
        o, ST = kd.gdr_fwd(*(x[n] for n in NAMES), x["S0"], scale=0.2)
        return (o.double() * t["dO"]).sum().item() + (ST.double() * t["dST"]).sum().item()

    for n in NAMES + ("S0",):
        d = torch.randn(t[n].shape, generator=G, device="cuda") * (0.05 if n in ("g", "beta") else 1.0)
        # a step h: the third derivatives of a smooth loss leave h^2, fp32 results of 3e-6 over h
        h = 2e-3
        num = (loss({**t, n: t[n] + h * d}) - loss({**t, n: t[n] - h * d})) / (2 * h)
        got = (gr["d" + n].double() * d).sum().item()
        size = (gr["d" + n].double().norm() * d.double().norm()).item()
        assert abs(num - got) <= 5e-3 * size, (n, num, got, size)


def test_streams_and_graphs():
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    t = inputs((2, 150), 1, 2, 64, 64, "bf16", 12)
    ref = run(t, 0.2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run(t, 0.2)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(ref[n], other[n]) for n in ref)
    S = t["S0"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(t, 0.2)
        o = kd.gdr_step(*(t[n][:, 0] for n in NAMES), S, S_out=t["S0"].new_empty(t["S0"].shape))
    step = kd.gdr_step(*(t[n][:, 0] for n in NAMES), S.clone())
    for _ in range(3):
        for x in out.values():
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(ref[n], out[n]) for n in ref) and torch.equal(o, step)
        assert all(torch.equal(ref[n], x) for n, x in run(t, 0.2).items())


@pytest.mark.parametrize("B,T,Hk,Hv,dk,dv", [(9, 70, 8, 16, 128, 64), (17, 65, 2, 8, 64, 72), (5, 130, 4, 16, 128, 136)])
def test_backward_of_many_heads(B, T, Hk, Hv, dk, dv):
    """Four groups of value columns a workgroup."""
    t = inputs((B, T), Hk, Hv, dk, dv, "bf16", T + dv)
    compare(t, run(t, 0.2), 0.2, "bf16")


def test_backward_of_many_packed_sequences():
    torch = _torch()
    lens = [(37 * i) % 71 for i in range(110)]
    cu = np.concatenate([[0], np.cumsum(lens)])
    t = inputs((int(cu[-1]),), 1, 2, 64, 64, "bf16", 31, n=len(lens))
    got = run(t, 0.2, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    compare(t, got, 0.2, "bf16", [(0, int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])])


@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 64, 72), ("bf16", 128, 200), ("fp32", 40, 40)])
def test_what_is_not_finite_stays_in_its_head(dtype, dk, dv):
    """More chunks than workgroups: what one leaves in LDS does not reach the next."""
    torch = _torch()
    t = inputs((3, 1600), 4, 4, dk, dv, dtype, 21)
    ref = run(t, 0.2)
    bad = {n: None if x is None else x.clone() for n, x in t.items()}
    bad["v"][0, 3, 0] = float("inf")
    bad["dO"][1, 1500, 2] = float("nan")
    got = run(bad, 0.2)
    for n, x in ref.items():
        for b in range(3):
            for h in range(4):
                if (b, h) in ((0, 0), (1, 2)):
                    continue
                at = (b, h) if n in ("ST", "dS0") else (b, slice(None), h)
                assert torch.equal(got[n][at], x[at]), (n, b, h)
    assert not torch.isfinite(got["o"][0, 3:, 0]).any() and torch.equal(got["o"][1], ref["o"][1])


def test_calls_that_run_at_once():
    torch = _torch()
    ts = [inputs((2, 700), 2, 4, 64, 64, "bf16", 40 + i) for i in range(2)]
    refs = [run(t, 0.2) for t in ts]
    streams = [torch.cuda.Stream() for _ in ts]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(run(ts[i], 0.2))
    torch.cuda.synchronize()
    for ref, rs in zip(refs, outs):
        assert all(torch.equal(ref[n], r[n]) for r in rs for n in ref)
