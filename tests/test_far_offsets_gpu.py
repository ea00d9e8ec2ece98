"""Offsets past 32 bits: caches, prompts and states of more than 2^31 elements."""
import pytest

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _room(gib):
    torch = _torch()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip("needs %d GiB of device memory" % gib)


def test_pages_past_32_bits():
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    _room(16)
    G = torch.Generator(device="cuda").manual_seed(1)
    page, Hkv, d, few = 64, 4, 128, 40
    pages = (1 << 31) // (page * Hkv * d) + few + 5
    big = [torch.empty(pages, page, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    small = [torch.randn(few, page, Hkv, d, generator=G, device="cuda").bfloat16() for _ in range(2)]
    far = pages - few
    for b, s in zip(big, small):
        b[far:].copy_(s)
    B = 5
    ids = torch.randperm(few, generator=G, device="cuda").int()
    prefix, table = ids[:16], ids[16:36].view(B, 4).contiguous()
    lens = torch.tensor([0, 70, 200, 63, 64], dtype=torch.int32, device="cuda")
    q = torch.randn(B, 16, d, generator=G, device="cuda").bfloat16()
    k, v = (torch.randn(B, Hkv, d, generator=G, device="cuda").bfloat16() for _ in range(2))
    freqs = torch.rand(d // 2, generator=G, device="cuda", dtype=torch.float64)
    out = []
    for (kp, vp), at in ((small, 0), (big, far)):
        turned = kd.paged_append(k, v, kp, vp, table + at, lens, q=q, freqs=freqs, offset=1000)
        out.append((turned, *kd.prefix_attn(turned, kp, vp, prefix + at, 1000, table + at, lens, return_lse=True)))
    assert all(torch.equal(x, y) for x, y in zip(*out))
    assert all(torch.equal(s, b[far:]) for s, b in zip(small, big))


def test_packed_prompts_and_results_past_32_bits():
    """More than 2^31 elements of q and o, one sequence behind another."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    _room(40)
    G = torch.Generator(device="cuda").manual_seed(2)
    Hq, Hkv, d, page = 32, 1, 128, 64
    n = (1 << 31) // (Hq * d) + 100
    q = torch.empty(n, Hq, d, dtype=torch.bfloat16, device="cuda")
    q[-100:].normal_(generator=G)
    k, v = (torch.randn(n, Hkv, d, generator=G, device="cuda").bfloat16() for _ in range(2))
    kp, vp = (torch.zeros(4, page, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    freqs = torch.rand(d // 2, generator=G, device="cuda", dtype=torch.float64)
    lens = torch.tensor([-1, 3], dtype=torch.int32, device="cuda")      # the first sequence is not in use
    table = torch.tensor([[0, 1], [2, 1]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n - 100, n], dtype=torch.int32, device="cuda")
    got = kd.paged_append(k, v, kp, vp, table, lens, q=q, cu_seqlens=cu, freqs=freqs)[-100:].clone()
    kp2, vp2 = torch.zeros_like(kp), torch.zeros_like(vp)
    want = kd.paged_append(k[-100:].clone(), v[-100:].clone(), kp2, vp2, table[1:], lens[1:], q=q[-100:].clone(),
                           cu_seqlens=torch.tensor([0, 100], dtype=torch.int32, device="cuda"), freqs=freqs)
    assert torch.equal(got, want) and torch.equal(kp, kp2) and torch.equal(vp, vp2)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_delta_rule_with_far_batches(dtype):
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    _room(48)
    G = torch.Generator(device="cuda").manual_seed(3)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    T, Hk, Hv, dk, dv = 130, 1, 2, 64, 72
    buf = torch.empty((1 << 31) + (T + 4) * 4096, dtype=dt, device="cuda")
    near = [torch.randn(2, T, h, d, generator=G, device="cuda").mul_(0.3).to(dt) for h, d in ((Hk, dk), (Hk, dk), (Hv, dv))]
    # tokens 4096 elements apart, the second batch 2^31 behind the first
    far = [buf.as_strided((2, T, *x.shape[2:]), (1 << 31, 4096, x.shape[3], 1), 512 * i) for i, x in enumerate(near)]
    for f, x in zip(far, near):
        f.copy_(x)
    g = torch.nn.functional.logsigmoid(torch.randn(2, T, Hv, generator=G, device="cuda")).to(dt)
    beta = torch.rand(2, T, Hv, generator=G, device="cuda").to(dt)
    dO = torch.randn(2, T, Hv, dv, generator=G, device="cuda").to(dt)
    out = []
    for q, k, v in (near, far):
        o, ST, saved = kd.gdr_fwd(q, k, v, g, beta, save_states=True)
        out.append(dict(o=o, ST=ST, **kd.gdr_bwd(q, k, v, g, beta, saved, dO)))
    assert all(torch.equal(out[0][n], out[1][n]) for n in out[0])


def test_own_keys_up_to_31_bits():
    """The last of 2^31 - 65 own keys, in a page of its own, takes nearly all the weight."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    page, d, n = 256, 32, 2 ** 31 - 65
    kp, vp = (torch.zeros(2, page, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kp[1], vp[1] = 4.0, 1.0                       # scores of 128 there, of 0 elsewhere
    table = torch.zeros(1, 1 << 23, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    q = torch.ones(1, 1, d, dtype=torch.bfloat16, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    o, lse = kd.prefix_attn(q, kp, vp, i32([]), 0, table, i32([n - 1]), scale=1.0, cu_seqlens=i32([0, 1]), return_lse=True)
    # 191 keys of weight 1 in the last page; e^-128 of 2^31 others adds nothing
    assert torch.equal(o, torch.ones_like(o)) and abs(lse.item() - 128 - torch.tensor(191.0).log().item()) < 1e-4


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_delta_rule_with_far_states(dtype):
    """More than 2^31 elements of states, of those that are kept per chunk and of their gradients: the last sequences
    against a call for themselves."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    _room(100)
    G = torch.Generator(device="cuda").manual_seed(4)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    Hk, Hv, dk, dv, few = 2, 16, 128, 256, 6
    N = (1 << 31) // (Hv * dv * dk) + few
    lens = torch.ones(N, dtype=torch.int64)
    lens[-few:] = torch.tensor([1, 70, 0, 3, 130, 2])
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])
    T, first = int(cu[-1]), int(cu[-few - 1])
    mk = lambda *s: torch.randn(*s, generator=G, device="cuda")  # noqa: E731
    q, k, v, dO = (mk(T, h, d).mul_(0.1).to(dt) for h, d in ((Hk, dk), (Hk, dk), (Hv, dv), (Hv, dv)))
    g, beta = -torch.rand(T, Hv, generator=G, device="cuda"), torch.rand(T, Hv, generator=G, device="cuda")
    S0 = torch.zeros(N, Hv, dv, dk, device="cuda")
    S0[-few:].normal_(generator=G)
    dST = torch.zeros(few, Hv, dv, dk, device="cuda").normal_(generator=G)
    small = {}
    for part in (slice(first, T), slice(0, T)):
        alone = part.start > 0
        c = (cu[-few - 1:] - first if alone else cu).to("cuda", torch.int32)
        x = [t[part] for t in (q, k, v, g, beta)]
        o, ST, saved = kd.gdr_fwd(*x, S0[-few:] if alone else S0, cu_seqlens=c, save_states=True)
        if not alone:
            S0.zero_()
            S0[-few:] = dST           # (the states' place for their gradients)
        r = kd.gdr_bwd(*x, saved, dO[part], dST if alone else S0, cu_seqlens=c)
        n = T - first
        out = dict(o=o[-n:], ST=ST[-few:], dS0=r.pop("dS0")[-few:], **{m: t[-n:] for m, t in r.items()})
        if alone:
            small = {m: t.clone() for m, t in out.items()}
        else:
            assert saved.numel() > (1 << 31) * q.element_size()
            assert all(torch.equal(small[m], out[m]) for m in out)


def test_results_behind_a_prefix_past_32_bits():
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    _room(60)
    G = torch.Generator(device="cuda").manual_seed(5)
    Hq, Hkv, d, page, few = 32, 1, 128, 64, 100
    n = (1 << 31) // (Hq * d) + few
    q = torch.zeros(n, Hq, d, dtype=torch.bfloat16, device="cuda")
    q[-few:].normal_(generator=G)
    kp, vp = (torch.randn(4, page, Hkv, d, generator=G, device="cuda").bfloat16() for _ in range(2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, table, prefix = i32([-1, 3]), i32([[0, 1], [2, 1]]), i32([3])
    o, lse = kd.prefix_attn(q, kp, vp, prefix, 60, table, lens, cu_seqlens=i32([0, n - few, n]), return_lse=True)
    want, wl = kd.prefix_attn(q[-few:].clone(), kp, vp, prefix, 60, table[1:], lens[1:], cu_seqlens=i32([0, few]),
                              return_lse=True)
    assert torch.equal(o[-few:], want) and torch.equal(lse[:, -few:], wl) and not o[:n - few].any()
