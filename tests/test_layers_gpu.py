"""The layers beside the mixer on the GPU against their references in 64 bits (tests/layers_ref.py, which also gives
the bound that each result's arithmetic may be off by)."""
import numpy as np
import pytest

from tests import layers_ref as R

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def dev(a, dtype):
    """The array on the device in the type, and the values it holds there."""
    torch = _torch()
    t = torch.tensor(a, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    return t, t.double().cpu().numpy()


def host(t):
    return t.double().cpu().numpy()


def check(name, got, ref, tol):
    got = host(got) if not isinstance(got, np.ndarray) else got
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    same = got == ref          # infinities among them
    with np.errstate(invalid="ignore"):
        bad = ~same & ~(np.abs(got - ref) <= tol)
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        raise AssertionError("%s: %d of %d off, first at %s: %r against %r, allowed %.3g" %
                             (name, bad.sum(), bad.size, at, got[at], ref[at], np.broadcast_to(tol, ref.shape)[at]))


# ------------------------------------------------- gated linear recurrence
def glr_case(B, T, D, dtype, gate, h0, seed, plain=False):
    torch = _torch()
    r = np.random.default_rng(seed)
    f = 1 / (1 + np.exp(-(r.standard_normal((B, T, D)) * 2 + 2)))
    f[r.random(f.shape) < 0.02] = 0.0        # resets
    f[r.random(f.shape) < 0.02] = 1.0
    c = dict(x=r.standard_normal((B, T, D)), f=f, i=r.random((B, T, D)) if gate else None,
             dh=r.standard_normal((B, T, D)))
    t, v = {}, {}
    for n, a in c.items():
        t[n], v[n] = (None, None) if a is None else dev(a, dtype)
    for n in ("h0", "dhT"):
        t[n], v[n] = dev(r.standard_normal((B, D)), "fp32") if h0 else (None, None)
    return t, v


GLR = [(1, 1, 1), (2, 1, 64), (1, 7, 5), (3, 64, 96), (2, 127, 33), (2, 128, 128), (1, 129, 130), (2, 300, 256),
       (1, 1000, 67), (2, 2049, 36), (1, 9000, 18), (17, 130, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,D", GLR)
def test_glr_forward_and_backward(B, T, D, dtype):
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    for gate, h0 in ((True, True), (False, False)):
        t, v = glr_case(B, T, D, dtype, gate, h0, 10 * T + D)
        print("case", (B, T, D), dtype, gate, h0, flush=True)
        h, hT, hs = kd.glr_fwd(t["x"], t["f"], t["i"], t["h0"], save_states=True)
        g = kd.glr_bwd(t["x"], t["f"], t["i"], hs, t["dh"], t["dhT"])
        torch.cuda.synchronize()
        u = R.unit(dtype)
        ref = R.glr(v["x"], v["f"], v["i"], v["h0"])
        eh, eg, H, G = R.glr_bounds(v["x"], v["f"], v["i"], v["h0"], v["dh"], v["dhT"])
        check("h", h, ref[:, 1:], eh[:, 1:] + u * np.abs(ref[:, 1:]) * 1.01)
        check("hT", hT, ref[:, -1], eh[:, -1])
        check("hs", hs, ref[:, :-1][:, ::128], eh[:, :-1][:, ::128])
        gr, dx, df, di, dh0 = R.glr_bwd(v["x"], v["f"], v["i"], ref, v["dh"], v["dhT"])
        a = np.abs
        i = 1.0 if v["i"] is None else a(v["i"])
        check("dx", g["dx"], dx, 1.01 * (i * eg + (u + R.W) * a(dx)))
        # (g + eg)(h + eh) - g h
        check("df", g["df"], df, 1.01 * (G * eh[:, :-1] + (H[:, :-1] + eh[:, :-1]) * eg + (u + R.W) * a(df)))
        if gate:
            check("di", g["di"], di, 1.01 * (a(v["x"]) * eg + (u + R.W) * a(di)))
        # one more product behind the first g
        check("dh0", g["dh0"], dh0, 1.01 * (a(v["f"][:, 0]) * eg[:, 0] + 140 * R.W * a(v["f"][:, 0]) * G[:, 0]))
        # no schedule in the results
        h2, hT2, hs2 = kd.glr_fwd(t["x"], t["f"], t["i"], t["h0"], save_states=True)
        g2 = kd.glr_bwd(t["x"], t["f"], t["i"], hs2, t["dh"], t["dhT"])
        assert torch.equal(h, h2) and torch.equal(hT, hT2) and torch.equal(hs, hs2)
        assert all(torch.equal(g[n], g2[n]) for n in g if g[n] is not None)


def test_glr_empty_sequence_and_strided_inputs():
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    h0 = torch.randn(3, 8, device="cuda")
    e = torch.empty(3, 0, 8, dtype=torch.bfloat16, device="cuda")
    h, hT, hs = kd.glr_fwd(e, e, e, h0, save_states=True)
    assert h.shape == (3, 0, 8) and torch.equal(hT, h0) and hs.shape == (3, 0, 8)
    g = kd.glr_bwd(e, e, e, hs, e, h0)
    assert torch.equal(g["dh0"], h0) and g["dx"].shape == (3, 0, 8)
    assert torch.equal(kd.glr_bwd(e, e, None, hs, e)["dh0"], torch.zeros_like(h0))
    x = torch.randn(2, 70, 3, 40, device="cuda").to(torch.bfloat16)
    f = torch.sigmoid(torch.randn(2, 70, 40, device="cuda")).to(torch.bfloat16)
    a, _ = kd.glr_fwd(x[:, :, 1], f[:, :1].expand_as(f), None)
    b, _ = kd.glr_fwd(x[:, :, 1].contiguous(), f[:, :1].repeat(1, 70, 1), None)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,D", [(1, 1), (3, 7), (32, 2048), (5, 1003)])
def test_glr_step_continues_the_forward(B, D, dtype):
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    t, v = glr_case(B, 6, D, dtype, True, True, 77 + D)
    ref = R.glr(v["x"], v["f"], v["i"], v["h0"])
    eh = R.glr_bounds(v["x"], v["f"], v["i"], v["h0"])
    h = t["h0"].clone()
    for s in range(6):
        y = kd.glr_step(t["x"][:, s], t["f"][:, s], t["i"][:, s], h)
        check("h", h, ref[:, s + 1], eh[:, s + 1])
        assert torch.equal(y, h.to(y.dtype))
    other = torch.empty_like(h)
    keep = h.clone()
    kd.glr_step(t["x"][:, 0], t["f"][:, 0], None, h, h_out=other)
    assert torch.equal(h, keep) and not torch.equal(other, h)


def test_glr_split_sequence_continues_from_its_state():
    import delta_rule_recurrent_chunk_amd as kd
    t, v = glr_case(2, 500, 48, "fp32", True, True, 5)
    ref = R.glr(v["x"], v["f"], v["i"], v["h0"])
    eh = R.glr_bounds(v["x"], v["f"], v["i"], v["h0"])
    h = t["h0"]
    for a, b in ((0, 1), (1, 200), (200, 500)):
        y, h = kd.glr_fwd(t["x"][:, a:b], t["f"][:, a:b], t["i"][:, a:b], h)
        check("h", y, ref[:, a + 1:b + 1], eh[:, a + 1:b + 1] + R.W * np.abs(ref[:, a + 1:b + 1]))


# ---------------------------------------------------------- rotary positions
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (64, 36), (32, 2), (256, 256), (80, 80), (7, 6), (64, 48), (16, 16), (24, 10)])
def test_rope(d, rot, layout, dtype):
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    r = np.random.default_rng(d + rot)
    B, T, Hq, Hk = 2, 9, 5, 2
    (q, qv), (k, kv) = dev(r.standard_normal((B, T, Hq, d)), dtype), dev(r.standard_normal((B, T, Hk, d)), dtype)
    freqs, _ = kd.rope_frequencies(rot, device="cuda")
    fr = freqs.cpu().numpy()
    pos = r.integers(0, 1 << 20, (B, T))
    pos[0, :3] = (0, 1, -5)
    u = R.unit(dtype)
    for p, pv in ((torch.tensor(pos, device="cuda"), pos),
                  (torch.tensor(pos[0], dtype=torch.int32, device="cuda"), np.broadcast_to(pos[0], pos.shape))):
        for inverse in (False, True):
            f = kd.rope_bwd if inverse else kd.rope
            qo, ko = f(q, k, p, freqs, layout=layout, scale=1.25)
            for n, got, x in (("q", qo, qv), ("k", ko, kv)):
                ref, e = R.rope(x, pv, fr, layout, 1.25, inverse)
                check(n, got, ref, 1.01 * (e + u * np.abs(ref)))
                assert np.array_equal(host(got)[..., rot:], x[..., rot:])
    # in place, without k, packed
    a = q.clone()
    kd.rope(a, None, torch.tensor(pos, device="cuda"), freqs, layout=layout, out=(a, None))
    b, none = kd.rope(q, None, torch.tensor(pos, device="cuda"), freqs, layout=layout)
    assert none is None and torch.equal(a, b)
    c, _ = kd.rope(q[1], None, torch.tensor(pos[1], device="cuda"), freqs, layout=layout)
    assert torch.equal(c, b[1])


@pytest.mark.parametrize("B,T,Hq,Hk,d,rot", [(1, 1, 1, 0, 16, 16), (3, 77, 5, 1, 64, 36), (2, 1000, 1, 0, 16, 16),
                                             (1, 3, 700, 300, 128, 128), (5, 130, 16, 4, 128, 64), (1, 9, 1, 1, 2, 2)])
def test_rope_sizes(B, T, Hq, Hk, d, rot):
    """Sizes that fill a workgroup's tokens in different ways, against the reference."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    r = np.random.default_rng(B * T)
    freqs, _ = kd.rope_frequencies(rot, device="cuda")
    pos = torch.arange(7, 7 + T, dtype=torch.int32, device="cuda")
    for layout in ("half", "interleaved"):
        for dtype in ("bf16", "fp32"):
            q, qv = dev(r.standard_normal((B, T, Hq, d)), dtype)
            k, kv = dev(r.standard_normal((B, T, Hk, d)), dtype) if Hk else (None, None)
            qo, ko = kd.rope(q, k, pos, freqs, layout=layout)
            for got, x in ((qo, qv), (ko, kv)):
                if x is not None:
                    ref, e = R.rope(x, np.broadcast_to(np.arange(7, 7 + T), (B, T)), freqs.cpu().numpy(), layout, 1.0)
                    check("rope", got, ref, 1.01 * (e + R.unit(dtype) * np.abs(ref)))


def test_rope_far_positions_and_gradient_by_differences():
    """At 2^27 an fp32 angle would be lost; and the backward is the transpose of the forward."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    r = np.random.default_rng(0)
    q, qv = dev(r.standard_normal((1, 4, 1, 64)), "fp32")
    pos = np.array([[1 << 27, (1 << 27) + 1, 10 ** 8, 12345678]])
    freqs, _ = kd.rope_frequencies(64, device="cuda")
    p = torch.tensor(pos[0], device="cuda")
    out, _ = kd.rope(q, None, p, freqs)
    ref, e = R.rope(qv, pos, freqs.cpu().numpy(), "half", 1.0)
    check("q", out, ref, 1.01 * (e + R.W * np.abs(ref)))
    g, gv = dev(r.standard_normal((1, 4, 1, 64)), "fp32")
    dx = host(kd.rope_bwd(g, None, p, freqs)[0])
    # <g, rope(x + t y) - rope(x)> / t for a linear map is <rope_bwd(g), y>
    y, yv = dev(r.standard_normal((1, 4, 1, 64)), "fp32")
    lhs = (gv * (host(kd.rope(q + y, None, p, freqs)[0]) - host(out))).sum()
    assert abs(lhs - (dx * (host(q + y) - qv)).sum()) < 1e-4


def test_rope_on_views_of_a_fused_projection():
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    for dtype in (torch.bfloat16, torch.float32):
        qkv = torch.randn(2, 6, 8, 64, device="cuda").to(dtype)
        freqs, _ = kd.rope_frequencies(32, device="cuda")
        pos = torch.arange(6, device="cuda")
        ref_q, ref_k = kd.rope(qkv[:, :, :4].contiguous(), qkv[:, :, 4:6].contiguous(), pos, freqs)
        new = torch.zeros_like(qkv)
        kd.rope(qkv[:, :, :4], qkv[:, :, 4:6], pos, freqs, out=(new[:, :, :4], new[:, :, 4:6]))
        assert torch.equal(new[:, :, :4], ref_q) and torch.equal(new[:, :, 4:6], ref_k) and not new[:, :, 6:].any()
        v = qkv[:, :, 6:].clone()
        kd.rope(qkv[:, :, :4], qkv[:, :, 4:6], pos, freqs, out=(qkv[:, :, :4], qkv[:, :, 4:6]))
        assert torch.equal(qkv[:, :, :4], ref_q) and torch.equal(qkv[:, :, 6:], v)
        t = qkv.transpose(1, 2).contiguous().transpose(1, 2)      # [B, H, T, d] in memory
        a, _ = kd.rope(t[:, :, :4], None, pos, freqs, inverse=True)
        b, _ = kd.rope(qkv[:, :, :4].contiguous(), None, pos, freqs, inverse=True)
        assert torch.equal(a, b)


# ------------------------------------------------- sliding-window attention
def swa_inputs(B, Tq, Tk, Hq, Hkv, d, dtype, seed):
    r = np.random.default_rng(seed)
    return [dev(r.standard_normal((B, n, H, d)), dtype) for n, H in ((Tq, Hq), (Tk, Hkv), (Tk, Hkv), (Tq, Hq))]


SWA = [  # Tq, Tk, Hq, Hkv, window, sinks
    (1, 1, 1, 1, 1, 0), (1, 300, 4, 1, 64, 4), (5, 5, 2, 2, 2, 1), (64, 64, 2, 1, 64, 0), (130, 130, 3, 1, 33, 4),
    (200, 200, 4, 2, 1, 0), (200, 200, 2, 2, 1, 64), (257, 257, 2, 1, 1000, 3), (129, 320, 2, 1, 100, 7),
    (300, 170, 2, 1, 50, 2), (7, 0, 2, 1, 4, 1), (0, 9, 2, 1, 4, 1), (333, 333, 8, 1, 65, 64), (600, 600, 1, 1, 129, 4),
    (2300, 2300, 2, 1, 100, 40), (1500, 1700, 2, 2, 700, 5)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("Tq,Tk,Hq,Hkv,window,sinks", SWA)
def test_swa_forward_and_backward(Tq, Tk, Hq, Hkv, window, sinks, d, dtype):
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    print("case", (Tq, Tk, Hq, Hkv, window, sinks, d), dtype, flush=True)
    (q, qv), (k, kv), (v, vv), (dO, ov) = swa_inputs(2, Tq, Tk, Hq, Hkv, d, dtype, Tq + Tk + d)
    o, lse = kd.swa_fwd(q, k, v, window, sinks, return_lse=True)
    g = kd.swa_bwd(q, k, v, o, lse, dO, window, sinks)
    torch.cuda.synchronize()
    for b in range(2):
        val, err = R.attention_heads(qv[b], kv[b], vv[b], window, sinks, 1 / np.sqrt(d), ov[b], R.unit(dtype))
        check("o", o[b], val["o"], err["o"])
        check("lse", lse[b], val["lse"], err["lse"])
        for n in ("dq", "dk", "dv"):
            check(n, g[n][b], val[n], err[n])
    assert torch.equal(kd.swa_fwd(q, k, v, window, sinks), o)
    g2 = kd.swa_bwd(q, k, v, o, lse, dO, window, sinks)
    assert all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("Tq,Tk,Hq,Hkv,window,sinks", [(300, 300, 8, 1, 1000, 3), (800, 800, 24, 8, 100, 5),
                                                       (260, 700, 16, 2, 300, 64), (600, 200, 8, 2, 300, 0), (513, 513, 5, 1, 1, 1)])
def test_swa_gradients_with_few_blocks_of_keys(Tq, Tk, Hq, Hkv, window, sinks, d, dtype):
    """Few key blocks and long groups: workgroups share the heads of a group (evenly or not)."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    print("case", (Tq, Tk, Hq, Hkv, window, sinks, d), dtype, flush=True)
    (q, qv), (k, kv), (v, vv), (dO, ov) = swa_inputs(2, Tq, Tk, Hq, Hkv, d, dtype, Tq + 3 * Tk + d)
    o, lse = kd.swa_fwd(q, k, v, window, sinks, return_lse=True)
    ws = torch.full((1 << 27,), 255, dtype=torch.uint8, device="cuda")      # (NaNs: nothing is read that was not written)
    g = kd.swa_bwd(q, k, v, o, lse, dO, window, sinks, workspace=ws)
    g2 = kd.swa_bwd(q, k, v, o, lse, dO, window, sinks)
    torch.cuda.synchronize()
    assert all(torch.equal(g[n], g2[n]) for n in g)
    for b in range(2):
        val, err = R.attention_heads(qv[b], kv[b], vv[b], window, sinks, 1 / np.sqrt(d), ov[b], R.unit(dtype))
        for n in ("dq", "dk", "dv"):
            check(n, g[n][b], val[n], err[n])


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("Tq,Tk,Hq,Hkv,window,sinks", [
    (2, 2, 1, 1, 7, 0), (6, 6, 1, 1, 17, 9), (5, 5, 4, 2, 551, 4), (9, 9, 2, 1, 1121, 9), (20, 20, 3, 1, 3, 2),
    (31, 50, 2, 1, 4, 0), (30, 100, 2, 2, 20, 5), (10, 300, 1, 1, 30, 2)])
def test_swa_gradients_that_few_keys_make_up_lose_the_rounding_of_the_result_alone(Tq, Tk, Hq, Hkv, window, sinks, d):
    """Where a sum has few terms its weights' roundings to bf16 do not average out, nor does the one in delta: there
    the weights carry their remainders (two bf16 numbers: 2^-16 of each term; 2^-14 is allowed) and delta is summed
    in fp32, which leaves the rounding of the result, 2^-8 of it."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    print("case", (Tq, Tk, Hq, Hkv, window, sinks, d), flush=True)
    (q, qv), (k, kv), (v, vv), (dO, ov) = swa_inputs(2, Tq, Tk, Hq, Hkv, d, "bf16", 7 * Tq + Tk + d)
    o, lse = kd.swa_fwd(q, k, v, window, sinks, return_lse=True)
    g = kd.swa_bwd(q, k, v, o, lse, dO, window, sinks)
    torch.cuda.synchronize()
    for b in range(2):
        val, err = R.attention_heads(qv[b], kv[b], vv[b], window, sinks, 1 / np.sqrt(d), ov[b], 2.0 ** -14)
        for n in ("dq", "dk", "dv"):
            check(n, g[n][b], val[n], err[n] + 2.0 ** -8 * np.abs(val[n]))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [[1], [0, 5, 0], [128, 128, 1, 127], [300, 1, 1, 0, 77, 129, 256],
                                  [3] * 70 + [200], [1500, 1, 2100, 90]])
def test_swa_packed_equals_each_sequence_alone(lens, dtype):
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    print("case", lens[:8], dtype, flush=True)
    T, tail = sum(lens), 3          # rows behind the last sequence
    (q, _), (k, _), (v, _), (dO, _) = swa_inputs(1, T + tail, T + tail, 4, 2, 64, dtype, T)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    out = torch.full((T + tail, 4, 64), 7.0, dtype=q.dtype, device="cuda")
    o, lse = kd.swa_fwd(q[0], k[0], v[0], 40, 2, cu_seqlens=cu, return_lse=True, out=out)
    g = kd.swa_bwd(q[0], k[0], v[0], o, lse, dO[0], 40, 2, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert (out[T:] == 7.0).all()
    a = 0
    for n in lens:
        s = slice(a, a + n)
        a += n
        if n == 0:
            continue
        oo, ll = kd.swa_fwd(q[:, s], k[:, s], v[:, s], 40, 2, return_lse=True)
        gg = kd.swa_bwd(q[:, s], k[:, s], v[:, s], oo, ll, dO[:, s], 40, 2)
        assert torch.equal(o[s], oo[0]) and torch.equal(lse[:, s], ll[0])
        assert all(torch.equal(g[m][s], gg[m][0]) for m in g)


def test_swa_packed_with_bad_offsets_stays_inside():
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    (q, _), (k, _), (v, _), (dO, _) = swa_inputs(1, 200, 200, 2, 1, 64, "bf16", 1)
    for cu in ([-50, 100, 900], [0, 300, 100], [5, 5, 5], [200, 0, 200], [1000, 2000, 3000]):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        o, lse = kd.swa_fwd(q[0], k[0], v[0], 40, 2, cu_seqlens=cu, return_lse=True)
        kd.swa_bwd(q[0], k[0], v[0], o.zero_(), lse.zero_(), dO[0], 40, 2, cu_seqlens=cu)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_swa_hidden_infinities_and_nans_stay_hidden(d, dtype):
    """Keys and values that are not finite reach the queries that see them and no others (a padded batch's tail, a
    bad token outside the window)."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    T, W, S = 300, 70, 3
    (q, qv), (k, kv), (v, vv), _ = swa_inputs(1, T, T, 2, 1, d, dtype, d)
    val, err = R.attention_heads(qv[0], kv[0], vv[0], W, S, 1 / np.sqrt(d), None, R.unit(dtype))
    pos = np.arange(T)
    inf, nan = float("inf"), float("nan")
    for at, value in ((1, nan), (100, inf), (129, nan), (130, -inf), (250, nan), (T - 1, inf)):
        sees = (pos >= at) & ((pos - at < W) | (at < S))
        bad = v.clone()
        bad[0, at, 0, ::5] = value
        o, l = kd.swa_fwd(q, k, bad, W, S, return_lse=True)
        o = host(o[0])
        check("hidden from", o[~sees], val["o"][~sees], err["o"][~sees])
        check("lse", l[0], val["lse"], err["lse"])
        # (a weight can be zero in fp32; none is here: scores are a few units apart)
        got = o[sees][..., ::5]
        assert np.isnan(got).all() if value != value else (got == value).all(), at
        rest = [i for i in range(d) if i % 5]
        check("other elements", o[sees][..., rest], val["o"][sees][..., rest], err["o"][sees][..., rest])
        bad = k.clone()
        bad[0, at] = value
        check("key", host(kd.swa_fwd(q, bad, v, W, S)[0])[~sees], val["o"][~sees], err["o"][~sees])
    # everything behind token 200 is garbage: the first 200 rows do not see it
    kk, vv2, qq = k.clone(), v.clone(), q.clone()
    kk[:, 200:], vv2[:, 200:], qq[:, 200:] = nan, nan, nan
    check("padded", host(kd.swa_fwd(qq, kk, vv2, W, S)[0, :200]), val["o"][:200], err["o"][:200])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("W,S", [(37, 0), (50, 3), (400, 5)])
@pytest.mark.parametrize("what,at", [("k", 131), ("v", 131), ("kv", slice(200, None)), ("kvqg", slice(200, None)),
                                     ("kvqg", slice(0, 70)), ("q", 140), ("g", 140), ("v", 299)])
def test_swa_gradients_of_what_does_not_see_infinities_and_nans(what, at, W, S, d, dtype):
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    T = 300
    print("case", what, at, W, S, d, dtype, flush=True)
    (q, qv), (k, kv), (v, vv), (dO, ov) = swa_inputs(1, T, T, 2, 1, d, dtype, 11 + d)
    val, err = R.attention_heads(qv[0], kv[0], vv[0], W, S, 1 / np.sqrt(d), ov[0], R.unit(dtype))
    vis = R.visible(T, T, W, S)
    row = np.zeros(T, bool)
    row[at] = True
    queries = row & (("q" in what) or ("g" in what))
    if "k" in what or "v" in what:
        queries = queries | vis[:, row].any(1)
    keys = vis[queries].any(0) | (row & (("k" in what) or ("v" in what)))
    for value in (float("nan"), float("inf")):
        kk, v2, qq, gg = k.clone(), v.clone(), q.clone(), dO.clone()
        for n, t in (("k", kk), ("v", v2), ("q", qq), ("g", gg)):
            if n in what:
                t[:, at] = value
        o, lse = kd.swa_fwd(qq, kk, v2, W, S, return_lse=True)
        g = kd.swa_bwd(qq, kk, v2, o, lse, gg, W, S)
        check("dq", host(g["dq"][0])[~queries], val["dq"][~queries], err["dq"][~queries])
        for n in ("dk", "dv"):
            check(n, host(g[n][0])[~keys], val[n][~keys], err[n][~keys])


def test_swa_on_views_and_pieces():
    """Views of a fused projection, [B, H, T, d] memory, a broadcast batch; a prompt in pieces."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    qkv = torch.randn(2, 150, 8, 64, device="cuda").to(torch.bfloat16)
    q, k, v = qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:]
    ref, lse = kd.swa_fwd(q.contiguous(), k.contiguous(), v.contiguous(), 50, 4, return_lse=True)
    assert torch.equal(kd.swa_fwd(q, k, v, 50, 4), ref)
    th = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v)]
    assert torch.equal(kd.swa_fwd(*th, 50, 4), ref)
    dO = torch.randn_like(ref)
    a, b = kd.swa_bwd(q, k, v, ref, lse, dO, 50, 4), kd.swa_bwd(*th, ref, lse, dO, 50, 4)
    assert all(torch.equal(a[n], b[n]) for n in a)
    e = [t[:1].expand(2, -1, -1, -1) for t in (q, k, v)]
    assert torch.equal(kd.swa_fwd(*e, 50, 4)[1], ref[0])
    odd = torch.randn(2, 150, 4, 65, device="cuda").to(torch.bfloat16)[..., 1:]     # rows at odd addresses
    assert torch.equal(kd.swa_fwd(odd, k, v, 50, 4), kd.swa_fwd(odd.contiguous(), k, v, 50, 4))
    (qf, qv), (kf, kv), (vf, vv), _ = swa_inputs(1, 150, 150, 4, 2, 64, "bf16", 3)
    val, err = R.attention_heads(qv[0], kv[0], vv[0], 50, 4, 1 / 8, None, R.unit("bf16"))
    for s, t in ((0, 100), (100, 101), (101, 150)):
        o = kd.swa_fwd(qf[:, s:t], kf[:, :t], vf[:, :t], 50, 4)
        check("o", o[0], val["o"][s:t], err["o"][s:t])


def test_swa_long_sequence_sampled_rows():
    """The hybrid's window over the long-context length, rows sampled across it."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    T, W, S, d = 32768, 2048, 4, 128
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randn(1, T, h, d, generator=g, device="cuda").to(torch.bfloat16) for h in (4, 2, 2))
    o, lse = kd.swa_fwd(q, k, v, W, S, return_lse=True)
    kv, vv = host(k[0]), host(v[0])
    for t in (0, 3, 4, 127, 128, 2047, 2048, 2051, 2052, 10000, 20011, 32767):
        seen = R.seen(t, W, S)
        qv = host(q[0, t])
        for h in range(4):
            kk, vs = kv[seen, h // 2], vv[seen, h // 2]
            val, err = R.attention(qv[None, h], kk, vs, T, 0, 1 / np.sqrt(d), None, R.unit("bf16"))
            check("o", o[0, t, h][None], val["o"], err["o"])
            check("lse", lse[0, h, t][None], val["lse"], err["lse"])


# ---------------------------------------------------------------- decoding
class Cache:
    """The rolling cache as lists of positions, in 64 bits."""

    def __init__(self, B, cap, Hkv, d, sinks):
        self.k, self.v = np.zeros((B, cap, Hkv, d)), np.zeros((B, cap, Hkv, d))
        self.sinks, self.cap = sinks, cap

    def step(self, b, p, q, k, v, window, scale, u):
        s = R.slot(p, self.sinks, self.cap)
        self.k[b, s], self.v[b, s] = k, v
        at = [R.slot(j, self.sinks, self.cap) for j in R.seen(p, window, self.sinks)]
        return R.attention_heads(q[None], self.k[b, at], self.v[b, at], len(at), 0, scale, None, u)


DEC = [  # Hq, Hkv, d, window, sinks, cap
    (1, 1, 32, 1, 0, 1), (4, 4, 64, 5, 2, 7), (8, 2, 128, 64, 4, 68), (6, 2, 64, 100, 0, 131), (16, 1, 128, 33, 64, 97),
    (10, 2, 32, 300, 1, 400), (4, 1, 128, 2048, 4, 2052), (40, 1, 64, 70, 3, 90), (66, 2, 128, 40, 4, 44),
    (2, 2, 128, 500, 30, 700)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("Hq,Hkv,d,window,sinks,cap", DEC)
def test_swa_decode_over_a_rolling_cache(Hq, Hkv, d, window, sinks, cap, dtype):
    """Prompts of different lengths into the caches, then steps that roll them over; one row unused; slots that no
    token has reached hold NaN."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    r = np.random.default_rng(cap)
    B, T0 = 4, min(2 * cap + 3, 2500)
    lens = np.array([0, min(3, T0), -1, T0], dtype=np.int32)
    kc = torch.full((B, cap, Hkv, d), float("nan"), dtype=torch.bfloat16 if dtype == "bf16" else torch.float32,
                    device="cuda")
    vc = kc.clone()
    (k0, k0v), (v0, v0v) = dev(r.standard_normal((B, T0, Hkv, d)), dtype), dev(r.standard_normal((B, T0, Hkv, d)), dtype)
    ln = torch.tensor(lens, device="cuda")
    kd.swa_cache_store(k0, v0, kc, vc, window, sinks, lens=ln)
    ref = Cache(B, cap, Hkv, d, sinks)
    for b in range(B):
        for t in range(max(lens[b], 0)):
            s = R.slot(t, sinks, cap)
            ref.k[b, s], ref.v[b, s] = k0v[b, t], v0v[b, t]
    u = R.unit(dtype)
    ws = kd.swa_decode_workspace(torch.empty(B, Hq, d, device="cuda"), kc)
    for step in range(6):
        (q, qv), (k, kv), (v, vv) = (dev(r.standard_normal((B, h, d)), dtype) for h in (Hq, Hkv, Hkv))
        print("case", (Hq, Hkv, d, window, sinks, cap), dtype, "step", step, flush=True)
        o = kd.swa_decode(q, k, v, kc, vc, ln, window, sinks, workspace=ws if step % 2 else None)
        torch.cuda.synchronize()
        for b in range(B):
            if lens[b] < 0:
                assert not o[b].any() and torch.isnan(kc[b]).all() and torch.isnan(vc[b]).all()
                continue
            val, err = ref.step(b, int(lens[b]), qv[b], kv[b], vv[b], window, 1 / np.sqrt(d), u)
            check("o", o[b][None], val["o"], err["o"])
            used = [R.slot(s, sinks, cap) for s in range(lens[b] + 1)]
            assert np.array_equal(host(kc[b])[used], ref.k[b][used]) and np.array_equal(host(vc[b])[used], ref.v[b][used])
            lens[b] += 1
        ln += (ln >= 0).int()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_swa_decode_turns_queries_and_keys(dtype, layout):
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    r = np.random.default_rng(8)
    B, Hq, Hkv, d, window, sinks, cap, rot = 3, 4, 2, 64, 20, 2, 30, 36
    lens = torch.tensor([0, 17, 100000], dtype=torch.int32, device="cuda")
    (kc, kcv), (vc, vcv) = dev(r.standard_normal((B, cap, Hkv, d)), dtype), dev(r.standard_normal((B, cap, Hkv, d)), dtype)
    (q, qv), (k, kv), (v, vv) = (dev(r.standard_normal((B, h, d)), dtype) for h in (Hq, Hkv, Hkv))
    freqs, _ = kd.rope_frequencies(rot, device="cuda")
    o = kd.swa_decode(q, k, v, kc, vc, lens, window, sinks, freqs=freqs, layout=layout, rope_scale=1.1)
    kr = kd.rope(k[:, None], None, lens[:, None], freqs, layout=layout, scale=1.1)[0][:, 0]
    qr, e = R.rope(qv[:, None], host(lens)[:, None], freqs.cpu().numpy(), layout, 1.1)
    u = R.unit(dtype)
    for b, p in enumerate(host(lens).astype(int)):
        s = R.slot(p, sinks, cap)
        assert torch.equal(kc[b, s], kr[b]) and torch.equal(vc[b, s], v[b])
        kcv[b, s], vcv[b, s] = host(kr[b]), vv[b]
        assert np.array_equal(host(kc[b]), kcv[b]) and np.array_equal(host(vc[b]), vcv[b])
        at = [R.slot(j, sinks, cap) for j in R.seen(p, window, sinks)]
        val, err = R.attention_heads(qr[b], kcv[b, at], vcv[b, at], len(at), 0, 1 / 8, None, u)
        # the turned query's own error, at most e, through the scores: relative 2 |dq . k| of every weight
        more = 2 * np.einsum("hd,khd->hk", np.broadcast_to(e[b, 0], (Hq, d)), np.abs(np.repeat(kcv[b, at], 2, 1))).max() / 8
        check("o", o[b][None], val["o"], err["o"] + 2 * more * np.abs(vcv[b, at]).max())


def test_swa_decode_interleaved_caches_and_strided_inputs():
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    both = torch.randn(2, 40, 2, 2, 64, device="cuda").to(torch.bfloat16)
    a, b = both[:, :, 0], both[:, :, 1]
    kc, vc = a.clone(), b.clone()
    qkv = torch.randn(2, 8, 64, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([10, 200], dtype=torch.int32, device="cuda")
    o = kd.swa_decode(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], a, b, lens, 32, 4)
    r = kd.swa_decode(qkv[:, :4].contiguous(), qkv[:, 4:6].contiguous(), qkv[:, 6:].contiguous(), kc, vc, lens, 32, 4)
    assert torch.equal(o, r) and torch.equal(a, kc) and torch.equal(b, vc)
    bh = torch.randn(2, 2, 40, 64, device="cuda").to(torch.bfloat16)       # [B, H, cap, d] in memory
    x, y = bh.transpose(1, 2), bh.clone().transpose(1, 2)
    o = kd.swa_decode(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], x, y, lens, 32, 4)
    r = kd.swa_decode(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], bh.transpose(1, 2).contiguous(), y.contiguous(), lens, 32, 4)
    # (the contiguous copies were made after the step above, which stored the same rows)
    assert torch.equal(o, r)


def test_swa_decode_workspace_serves_different_calls():
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    ws = kd.swa_decode_workspace(torch.empty(8, 32, 128, device="cuda"),
                                 torch.empty(8, 1100, 4, 128, dtype=torch.bfloat16, device="cuda"))
    for B, Hq, Hkv, d, cap, window in ((8, 32, 4, 128, 1100, 1000), (1, 4, 4, 64, 500, 400), (8, 32, 4, 128, 1100, 1100),
                                       (3, 6, 1, 32, 90, 64), (8, 32, 4, 128, 1100, 300)):
        kc, vc = (torch.randn(B, cap, Hkv, d, device="cuda").to(torch.bfloat16) for _ in range(2))
        q, k, v = (torch.randn(B, h, d, device="cuda").to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
        lens = torch.arange(cap - B, cap, dtype=torch.int32, device="cuda")
        a = kd.swa_decode(q, k, v, kc, vc, lens, window, 0, workspace=ws)
        b = kd.swa_decode(q, k, v, kc, vc, lens, window, 0)
        assert torch.equal(a, b)


# -------------------------------------------------------------- used together
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_prompt_then_decoding_equals_one_forward(layout):
    """A local layer as it is served: rope and attention over the prompt, its keys into rolling caches, then tokens one
    by one; against one pass over the whole text."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    r = np.random.default_rng(11)
    B, T, T0, Hq, Hkv, d, window, sinks = 2, 90, 70, 4, 2, 64, 24, 3
    (q, qv), (k, kv), (v, vv) = (dev(r.standard_normal((B, T, h, d)), "bf16") for h in (Hq, Hkv, Hkv))
    freqs, m = kd.rope_frequencies(48, scaling="byparts", factor=4.0, original_length=64, device="cuda")
    pos = torch.arange(T, device="cuda")
    qr, kr = kd.rope(q, k, pos, freqs, layout=layout, scale=m)
    whole = kd.swa_fwd(qr, kr, v, window, sinks)
    cap = window + sinks
    kc = torch.full((B, cap, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    kd.swa_cache_store(kr[:, :T0], v[:, :T0], kc, vc, window, sinks)
    lens = torch.full((B,), T0, dtype=torch.int32, device="cuda")
    fr = freqs.cpu().numpy()
    qx, e = R.rope(qv, np.broadcast_to(np.arange(T), (B, T)), fr, layout, m)
    for t in range(T0, T):
        o = kd.swa_decode(q[:, t], k[:, t], v[:, t], kc, vc, lens, window, sinks, freqs=freqs, layout=layout, rope_scale=m)
        lens += 1
        for b in range(B):
            val, err = R.attention_heads(qx[b, t:t + 1], host(kr[b, :t + 1]), vv[b, :t + 1], window, sinks, 1 / 8, None,
                                         R.unit("bf16"))
            kk = np.abs(np.repeat(host(kr[b, :t + 1]), 2, 1))
            sc = lambda x: 2 * np.einsum("hd,khd->hk", x, kk).max() / 8 * np.abs(vv[b]).max()
            check("o", o[b][None], val["o"], err["o"] + 2 * sc(e[b, t]))
            # the prompt pass turned its query to bf16: half a step of every element more
            check("whole", whole[b, t][None], val["o"], err["o"] + 2 * sc(e[b, t] + R.unit("bf16") * np.abs(qx[b, t])))


def test_a_layer_trains_through_rope_and_attention():
    """Gradients of rope, then attention, chained by hand, against differences of the chained forward in 64 bits."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    r = np.random.default_rng(12)
    B, T, Hq, Hkv, d, window, sinks = 1, 40, 2, 1, 32, 9, 2
    (q, qv), (k, kv), (v, vv), (dO, ov) = swa_inputs(B, T, T, Hq, Hkv, d, "fp32", 4)
    freqs, _ = kd.rope_frequencies(d, device="cuda")
    pos = torch.arange(T, device="cuda")
    qr, kr = kd.rope(q, k, pos, freqs)
    o, lse = kd.swa_fwd(qr, kr, v, window, sinks, return_lse=True)
    g = kd.swa_bwd(qr, kr, v, o, lse, dO, window, sinks)
    dq, dk = kd.rope_bwd(g["dq"], g["dk"], pos, freqs)
    fr, p = freqs.cpu().numpy(), np.arange(T)[None]

    def loss(q, k, v):
        a, b = R.rope(q, p, fr, "half", 1.0)[0], R.rope(k, p, fr, "half", 1.0)[0]
        return (R.attention_heads(a[0], b[0], v[0], window, sinks, 1 / np.sqrt(d))[0]["o"] * ov[0]).sum()

    for x, got in ((0, dq), (1, dk), (2, g["dv"])):
        y = [qv, kv, vv]
        step = r.standard_normal(y[x].shape)
        up, lo = list(y), list(y)
        up[x], lo[x] = y[x] + 1e-5 * step, y[x] - 1e-5 * step
        num = (loss(*up) - loss(*lo)) / 2e-5
        # the sum over n products of gradients that fp32 leaves off by some 1e-5 of their size
        assert abs(num - (host(got) * step).sum()) < 1e-4 * np.abs(host(got) * step).sum() + 1e-6


def test_dimensions_past_32_bits_are_refused():
    """Views of one element: a count that wrapped would leave 128 tokens, a call that succeeds."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    n = (1 << 32) + 128
    one = torch.zeros(1, dtype=torch.bfloat16, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    freqs, _ = kd.rope_frequencies(16, device="cuda")
    row, x = one.expand(1, n), one.expand(1, n, 1)
    heads = one.expand(1, n, 1, 32)
    for call in (lambda: kd.glr_fwd(x, x), lambda: kd.glr_step(row, row, None, torch.zeros(1, 1, device="cuda").expand(1, n)),
                 lambda: kd.rope(heads, None, lens.expand(n), freqs), lambda: kd.swa_fwd(heads, heads, heads, 8, 0),
                 lambda: kd.swa_decode(heads[:, 0], heads[:, 0], heads[:, 0], heads, heads, lens, 8, 0),
                 lambda: kd.swa_cache_store(heads, heads, heads[:, :128], heads[:, :128], 8, 0)):
        with pytest.raises(ValueError, match="past 32 bits"):
            call()


def test_streams_and_graphs():
    """Another stream than the current one of the allocation, and captured calls replayed between eager ones."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    x, f, i, dh = (torch.rand(2, 700, 96, device="cuda").to(torch.bfloat16) for _ in range(4))
    q, k, v, dO = (torch.randn(2, 300, h, 64, device="cuda").to(torch.bfloat16) for h in (4, 2, 2, 4))
    kc, vc = (torch.randn(2, 600, 2, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    lens = torch.tensor([520, 100], dtype=torch.int32, device="cuda")
    freqs, _ = kd.rope_frequencies(64, device="cuda")
    pos = torch.arange(300, device="cuda")
    ws = kd.swa_decode_workspace(q[:, 0], kc)

    def run():
        h, hT, hs = kd.glr_fwd(x, f, i, None, save_states=True)
        g = kd.glr_bwd(x, f, i, hs, dh)
        qr, kr = kd.rope(q, k, pos, freqs)
        o, lse = kd.swa_fwd(qr, kr, v, 100, 4, return_lse=True)
        s = kd.swa_bwd(qr, kr, v, o, lse, dO, 100, 4)
        dq, dk = kd.rope_bwd(s["dq"], s["dk"], pos, freqs)
        y = kd.swa_decode(q[:, 0], k[:, 0], v[:, 0], kc, vc, lens, 500, 4, freqs=freqs, workspace=ws)
        z = kd.glr_step(x[:, 0], f[:, 0], i[:, 0], hT, h_out=torch.empty_like(hT))
        return [h, hT, hs, g["dx"], g["df"], g["di"], g["dh0"], o, lse, dq, dk, s["dv"], y, z]

    first = [t.clone() for t in run()]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = run()
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for n in range(4):
        for t in (x, q, v, dh, dO):      # new inputs
            t.copy_(torch.rand_like(t))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), n
