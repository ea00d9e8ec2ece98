"""Many packed sequences, most of them empty: the same bits as the others alone."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "g", "beta")


def _torch():
    import torch
    return torch


def offsets(N, held, seed):
    """Offsets of N sequences of which `held` have rows (every second of them one), those alone, and which they are."""
    r = np.random.default_rng(seed)
    at = np.sort(r.choice(N, held, replace=False))
    n = r.integers(1, 90, held)
    n[::2] = 1
    lens = np.zeros(N, np.int64)
    lens[at] = n
    full, few = (np.concatenate([[0], np.cumsum(x)]) for x in (lens, n))
    return [_torch().tensor(x, dtype=_torch().int32, device="cuda") for x in (full, few, at)]


@pytest.mark.parametrize("N,held", [(64, 64), (65, 60), (66, 5), (4096, 290), (4097, 290), (70001, 290)])
def test_delta_rule(N, held):
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    full, few, at = offsets(N, held, N)
    T, H = int(few[-1]), 2
    G = torch.Generator(device="cuda").manual_seed(N)
    t = {n: torch.randn(T, H, 64, generator=G, device="cuda").mul_(0.125).bfloat16() for n in "qkv"}
    t["g"], t["beta"] = -torch.rand(T, H, generator=G, device="cuda"), torch.rand(T, H, generator=G, device="cuda")
    S0 = torch.randn(held, H, 64, 64, generator=G, device="cuda")
    dO = torch.randn(T, H, 64, generator=G, device="cuda").bfloat16()
    S0s = torch.zeros(N, H, 64, 64, device="cuda")
    S0s[at.long()] = S0
    out = []
    for cu, S in ((few, S0), (full, S0s)):
        o, ST, saved = kd.gdr_fwd(*(t[n] for n in NAMES), S, cu_seqlens=cu, save_states=True)
        out.append(dict(o=o, ST=ST, **kd.gdr_bwd(*(t[n] for n in NAMES), saved, dO, cu_seqlens=cu)))
    for n in ("ST", "dS0"):
        out[1][n] = out[1][n][at.long()]
    assert all(torch.equal(out[0][n], out[1][n]) for n in out[0])


@pytest.mark.parametrize("N,held", [(64, 64), (65, 60), (4096, 600), (4097, 600), (70001, 600)])
def test_paged_cache(N, held):
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    full, few, at = offsets(N, held, N + 1)
    T = int(few[-1])
    G = torch.Generator(device="cuda").manual_seed(N)
    q, k, v = (torch.randn(T, h, 64, generator=G, device="cuda").bfloat16() for h in (4, 2, 2))
    kp0, vp0 = (torch.randn(held * 6 + 8, 16, 2, 64, generator=G, device="cuda").bfloat16() for _ in range(2))
    tables = torch.full((N, 6), -1, dtype=torch.int32, device="cuda")
    tables[at.long()] = torch.arange(held * 6, dtype=torch.int32, device="cuda").view(held, 6)
    lens = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    lens[at.long()] = 3
    prefix = torch.arange(held * 6, held * 6 + 8, dtype=torch.int32, device="cuda")
    out = []
    for cu, table, ln in ((few, tables[at.long()].contiguous(), lens[at.long()]), (full, tables, lens)):
        kp, vp = kp0.clone(), vp0.clone()
        kd.paged_append(k, v, kp, vp, table, ln, cu_seqlens=cu)
        out.append((kp, vp, *kd.prefix_attn(q, kp, vp, prefix, 120, table, ln, cu_seqlens=cu, return_lse=True)))
    assert all(torch.equal(x, y) for x, y in zip(*out))
