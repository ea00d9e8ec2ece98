"""The layers beside the mixer where offsets pass 32 bits: against the same calls on parts, whose offsets do not."""
import pytest

from tests.test_layers_gpu import _torch

pytestmark = pytest.mark.gpu


def bf(torch, *shape):
    return torch.randn(*shape, dtype=torch.bfloat16, device="cuda")


def test_glr_past_32_bits():
    """Channels are independent: the last ones alone give the same bits."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    B, T, D = 1, (1 << 20) + 3, 2100
    x, dh = bf(torch, B, T, D), bf(torch, B, T, D)
    f = torch.rand(B, T, D, dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 1 << 31
    h, hT, hs = kd.glr_fwd(x, f, None, save_states=True)
    g = kd.glr_bwd(x, f, None, hs, dh)
    c = slice(D - 8, D)
    h1, hT1, hs1 = kd.glr_fwd(x[:, :, c], f[:, :, c], None, save_states=True)
    g1 = kd.glr_bwd(x[:, :, c].contiguous(), f[:, :, c], None, hs1, dh[:, :, c])
    assert torch.equal(h[:, :, c], h1) and torch.equal(hT[:, c], hT1) and torch.equal(hs[:, :, c], hs1)
    assert all(torch.equal(g[n][..., c], g1[n]) for n in ("dx", "df", "dh0"))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_past_32_bits(layout):
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    T, H, d = 1 << 18, 66, 128
    q, k = bf(torch, 1, T, H, d), bf(torch, 1, T, 2, d)
    assert q.numel() > 1 << 31
    freqs, _ = kd.rope_frequencies(96, device="cuda")
    pos = torch.arange(T, device="cuda")
    a, b = kd.rope(q, k, pos, freqs, layout=layout)
    for s in (slice(0, 5), slice(T - 11, T)):
        x, y = kd.rope(q[:, s].contiguous(), k[:, s].contiguous(), pos[s], freqs, layout=layout)
        assert torch.equal(a[:, s], x) and torch.equal(b[:, s], y)


@pytest.mark.parametrize("packed", [False, True])
def test_swa_past_32_bits(packed):
    """The second sequence alone gives the same bits (enough rows that neither call shares heads, and chunks of the
    sinks' pass of the same length)."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    T, Hq, Hkv, d, W, S = (1 << 17) + 5, 64, 8, 128, 70, 3
    q, k, v, dO = (bf(torch, 2, T, h, d) for h in (Hq, Hkv, Hkv, Hq))
    assert q.numel() > 1 << 31
    o1, l1 = kd.swa_fwd(q[1:], k[1:], v[1:], W, S, return_lse=True)
    g1 = kd.swa_bwd(q[1:], k[1:], v[1:], o1, l1, dO[1:], W, S)
    if packed:
        cu = torch.tensor([0, T, 2 * T], dtype=torch.int32, device="cuda")
        q, k, v, dO = (t.flatten(0, 1) for t in (q, k, v, dO))
        o, lse = kd.swa_fwd(q, k, v, W, S, cu_seqlens=cu, return_lse=True)
        g = kd.swa_bwd(q, k, v, o, lse, dO, W, S, cu_seqlens=cu)
        o, lse, g = o[T:], lse[:, T:], {n: t[T:] for n, t in g.items()}
    else:
        o, lse = kd.swa_fwd(q, k, v, W, S, return_lse=True)
        g = kd.swa_bwd(q, k, v, o, lse, dO, W, S)
        o, lse, g = o[1], lse[1], {n: t[1] for n, t in g.items()}
    assert torch.equal(o, o1[0]) and torch.equal(lse, l1[0])
    assert all(torch.equal(g[n], g1[n][0]) for n in g)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_swa_rows_far_apart(dtype):
    """Rows more than 2^22 elements apart do not fit the kernels' short offsets."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    T, d, W, S = 270, 64, 100, 3
    for stride in ((1 << 22) - 64, 1 << 22, (1 << 22) + 64):
        far = [torch.empty_strided((1, T, 1, d), (0, stride, d, 1), dtype=dt, device="cuda") for _ in range(2)]
        for t in far:
            t.copy_(torch.randn(1, T, 1, d, device="cuda"))
        k, v = far
        q, dO = (torch.randn(1, T, 2, d, device="cuda").to(dt) for _ in range(2))
        o, lse = kd.swa_fwd(q, k, v, W, S, return_lse=True)
        g = kd.swa_bwd(q, k, v, o, lse, dO, W, S)
        kc, vc = k.contiguous(), v.contiguous()
        assert torch.equal(o, kd.swa_fwd(q, kc, vc, W, S))
        c = kd.swa_bwd(q, kc, vc, o, lse, dO, W, S)
        assert all(torch.equal(g[n], c[n]) for n in g)
        g2 = kd.swa_bwd(k, q[:, :, :1], v, *kd.swa_fwd(k, q[:, :, :1], v, W, S, return_lse=True), dO[:, :, :1], W, S)
        c2 = kd.swa_bwd(kc, q[:, :, :1], vc, *kd.swa_fwd(kc, q[:, :, :1], vc, W, S, return_lse=True), dO[:, :, :1], W, S)
        assert all(torch.equal(g2[n], c2[n]) for n in g2)


@pytest.mark.parametrize("layout", ["bthd", "bhtd"])
def test_decoding_and_store_past_32_bits(layout):
    """Caches of 2^30 elements per sequence against rolling ones as long as the window."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    B, cap, Hkv, Hq, d, W, S = 3, 1 << 20, 8, 16, 128, 300, 4
    shape = (B, cap, Hkv, d) if layout == "bthd" else (B, Hkv, cap, d)
    kc, vc = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    if layout == "bhtd":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    assert kc.numel() > 1 << 31
    T = cap - 2
    k, v = bf(torch, B, T, Hkv, d), bf(torch, B, T, Hkv, d)
    lens = torch.tensor([T, 500, T - 7], dtype=torch.int32, device="cuda")
    kd.swa_cache_store(k, v, kc, vc, W, S, lens=lens)
    kr, vr = (torch.zeros(B, W + S, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kd.swa_cache_store(k, v, kr, vr, W, S, lens=lens)
    for b, n in enumerate(lens.tolist()):
        assert torch.equal(kc[b, n - 400:n], k[b, n - 400:n]) and torch.equal(vc[b, :9], v[b, :9])
    del k, v
    ws = kd.swa_decode_workspace(torch.empty(B, Hq, d, device="cuda"), kc)
    for step in range(4):        # the last ones roll the long caches over, too
        q, kn, vn = (bf(torch, B, h, d) for h in (Hq, Hkv, Hkv))
        a = kd.swa_decode(q, kn, vn, kc, vc, lens, W, S, workspace=ws)
        b = kd.swa_decode(q, kn, vn, kr, vr, lens, W, S)
        assert torch.equal(a, b), step
        lens += 1
