"""The paged cache and the attention over a shared prefix against plain references in 64 bits."""
import math

import numpy as np
import pytest

import layers_ref as LR
import paged_ref as R

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def dtype_of(name):
    return getattr(_torch(), "bfloat16" if name == "bf16" else "float32")


def f64(t):
    return t.detach().double().cpu().numpy()


def check(name, got, ref, tol):
    g = f64(got) if hasattr(got, "detach") else got
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    same = (g == ref) | (np.isnan(g) & np.isnan(ref))
    with np.errstate(invalid="ignore"):
        bad = ~same & ~(np.abs(g - ref) <= tol)
    assert not bad.any(), "%s: %d of %d beyond the bound, first at %s: %r for %r, bound %r" % (
        name, bad.sum(), bad.size, tuple(np.argwhere(bad)[0]), g[bad][0], ref[bad][0],
        np.broadcast_to(tol, g.shape)[bad][0])


class Case:
    """A batch with its cache: every slot that no sequence and no prefix reaches holds NaN."""

    def __init__(self, lens, new, P, page, Hq, Hkv, d, dtype, seed=0, packed=None, spare=3, gap=0):
        torch = _torch()
        rng = np.random.default_rng(seed)
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.B, self.page, self.P = list(lens), len(lens), page, P
        self.packed = any(n != 1 for n in new) if packed is None else packed
        self.cu = np.concatenate([[0], np.cumsum(new)]) if self.packed else None
        self.T = (int(self.cu[-1]) if self.packed else self.B) + gap
        self.dt, self.Hq, self.Hkv, self.d = dtype_of(dtype), Hq, Hkv, d
        own = [max(0, -(-(max(n, 0) + m) // page)) for n, m in zip(lens, new)]
        np_ = -(-P // page)
        self.pages = sum(own) + np_ + spare
        ids = rng.permutation(self.pages)
        self.ptable = ids[:np_].astype(np.int32)
        self.width = max(own + [1])
        self.table = np.full((self.B, self.width), -1, np.int32)
        at = np_
        for b, n in enumerate(own):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.kp, self.vp = (torch.full((self.pages, page, Hkv, d), float("nan"), device="cuda", dtype=self.dt)
                            for _ in range(2))
        live = np.zeros((self.pages, page), bool)
        for i in range(P):
            live[self.ptable[i // page], i % page] = True
        for b, (n, m) in enumerate(zip(lens, new)):
            for i in range(max(n, 0) + m):
                live[self.table[b, i // page], i % page] = True
        mask = torch.tensor(live, device="cuda")
        for t in (self.kp, self.vp):
            t[mask] = self.normal(int(live.sum()), Hkv, d)
        self.q = self.normal(self.T, Hq, d)

    def normal(self, *shape):
        return _torch().randn(*shape, generator=self.g, device="cuda").to(self.dt)

    def dev(self, x, dtype="int32"):
        return None if x is None else _torch().tensor(np.asarray(x), dtype=getattr(_torch(), dtype), device="cuda")

    def args(self):
        return (self.q, self.kp, self.vp, self.dev(self.ptable), self.P, self.dev(self.table), self.dev(self.lens))

    def run(self, **kw):
        import delta_rule_recurrent_chunk_amd as kd
        return kd.prefix_attn(*self.args(), cu_seqlens=self.dev(self.cu), **kw)

    def check(self, o, lse=None, scale=None, rows=None, u=None):
        scale = 1.0 / math.sqrt(self.d) if scale is None else scale
        q, k, v = f64(self.q), f64(self.kp), f64(self.vp)
        u = (2.0 ** -8 if self.dt == _torch().bfloat16 else R.W) if u is None else u
        owner = R.rows_of(self.lens, self.cu, self.T)
        for r in range(self.T) if rows is None else rows:
            if owner[r] is None:
                continue
            if owner[r][1] is None:
                assert not f64(o[r]).any()
                if lse is not None:
                    assert np.isneginf(f64(lse[:, r])).all()
                continue
            at = R.keys_of(owner[r], self.lens, self.cu, self.ptable, self.P, self.table, self.page, self.pages)
            pg, sl = (np.array([x[i] for x in at], int) for i in (0, 1))
            for h in range(self.Hq):
                hk = h // (self.Hq // self.Hkv)
                ro, eo, rl, el = R.attend(q[r, h], k[pg, sl, hk], v[pg, sl, hk], scale, u)
                check("o of row %d, head %d" % (r, h), o[r, h], ro, eo)
                if lse is not None:
                    check("lse", np.float64(lse[h, r].item()), np.float64(rl), el)


# lens, new rows, prefix, page, Hq, Hkv
DECODE = [([0], [1], 0, 16, 1, 1), ([0, 5, 63, 64, 200], [1] * 5, 0, 16, 8, 2), ([3, 0, 17], [1] * 3, 1, 1, 4, 4),
          ([31, 32, 33, 1, -1, 0], [1] * 6, 63, 24, 6, 2), ([400, 7], [1] * 2, 1000, 64, 16, 4),
          ([10] * 33, [1] * 33, 64, 32, 4, 1), ([70, 3], [1] * 2, 65, 128, 33, 1), ([5, 900], [1] * 2, 300, 7, 80, 2)]
PACKED = [([0], [1], 0, 16, 1, 1), ([0, 0, 4], [5, 0, 1], 70, 16, 4, 2), ([60, 0, -1, 2], [9, 130, 3, 1], 129, 24, 6, 2),
          ([0, 300], [200, 33], 64, 64, 16, 4), ([0], [129], 0, 1, 2, 1), ([0, 1, 2, 3], [0, 0, 0, 0], 5, 16, 4, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("i", range(len(DECODE)))
def test_one_row_per_sequence(i, d, dtype):
    lens, new, P, page, Hq, Hkv = DECODE[i]
    print("case", DECODE[i], d, dtype, flush=True)
    c = Case(lens, new, P, page, Hq, Hkv, d, dtype, seed=i, packed=False)
    o, lse = c.run(return_lse=True)
    c.check(o, lse)
    again, lse2 = c.run(return_lse=True)
    assert _torch().equal(o, again) and _torch().equal(lse, lse2)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("i", range(len(PACKED)))
def test_packed_rows(i, d, dtype):
    lens, new, P, page, Hq, Hkv = PACKED[i]
    print("case", PACKED[i], d, dtype, flush=True)
    c = Case(lens, new, P, page, Hq, Hkv, d, dtype, seed=50 + i, packed=True, gap=2)
    o, lse = c.run(return_lse=True)
    c.check(o, lse)
    assert _torch().equal(o[:c.T - 2], c.run()[:c.T - 2])


def test_many_splits_and_a_long_prefix():
    c = Case([1500, 0, 700], [1] * 3, 20000, 48, 8, 2, 128, "bf16", seed=7)
    c.check(c.run(scale=0.05), scale=0.05)
    c = Case([0, 0], [150, 40], 9000, 64, 8, 2, 64, "bf16", seed=8)
    c.check(c.run(), rows=list(range(0, 190, 17)) + [149, 150, 189])


def test_a_steep_softmax_keeps_its_maxima():
    torch = _torch()
    for new in ([1, 1], [40, 3]):
        c = Case([100, 9], new, 500, 16, 4, 2, 64, "bf16", seed=9)
        c.q *= 30
        # the largest scores at the end of the prefix, in its middle, and in the own keys
        c.kp[int(c.ptable[499 // 16]), 499 % 16, 0] = c.q[0, 0]
        c.kp[int(c.ptable[17 // 16]), 1, 1] = c.q[0, 2]
        torch.cuda.synchronize()
        o, lse = c.run(return_lse=True)
        c.check(o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
def test_what_a_row_does_not_see_stays_hidden(value, dtype):
    c = Case([3, 0], [20, 40], 70, 16, 4, 2, 64, dtype, seed=11)
    x = float(value)
    # row 30 of the second sequence has a key and a value that are not finite: rows before it do not see them
    pg, sl = int(c.table[1, 30 // 16]), 30 % 16
    c.kp[pg, sl, :, 3], c.vp[pg, sl] = x, x
    o = c.run()
    c.check(o, rows=range(50))
    # the rows that see the value of infinite weight or none at all: as IEEE arithmetic has it
    c.kp[pg, sl] = 0
    c.check(c.run())


def test_infinities_that_are_seen_show():
    for packed in (False, True):
        c = Case([40, 7], [1, 1], 100, 16, 4, 2, 64, "bf16", seed=12, packed=packed)
        c.vp[int(c.table[0, 40 // 16]), 40 % 16, 0, 5] = float("inf")       # the last own key fills up its tile
        c.vp[int(c.ptable[99 // 16]), 99 % 16, 1, 6] = float("-inf")        # and the last of the prefix
        c.check(c.run())


def test_bad_tables_stay_inside_the_cache():
    torch = _torch()
    c = Case([40, 7, 2], [1] * 3, 100, 16, 4, 2, 64, "bf16", seed=13)
    c.kp.nan_to_num_(0.25)
    c.vp.nan_to_num_(0.5)
    c.table[0, 1], c.table[1, 0], c.ptable[2] = 1 << 30, -7, -(1 << 31)
    c.check(c.run())
    # lengths past the table end with it
    c.lens = [10 ** 9, 2 ** 31 - 1, 2]
    c.table[:] = np.maximum(c.table, 0)
    c.check(c.run())
    # offsets that are out of order or out of range: nothing outside is touched, and nothing hangs
    import delta_rule_recurrent_chunk_amd as kd
    c = Case([3, 0, 5], [20, 40, 4], 70, 16, 4, 2, 64, "bf16", seed=14)
    for cu in ([0, 1000, 5, 64], [-5, 20, 10, 64], [64, 3, 2, 1], [0, 0, 0, 1 << 30]):
        kd.prefix_attn(*c.args(), cu_seqlens=c.dev(cu))
        kd.paged_append(c.normal(c.T, 2, 64), c.normal(c.T, 2, 64), c.kp, c.vp, c.dev(c.table), c.dev(c.lens),
                        cu_seqlens=c.dev(cu))
    torch.cuda.synchronize()


def test_rows_behind_the_last_sequence_are_left():
    import delta_rule_recurrent_chunk_amd as kd
    from delta_rule_recurrent_chunk_amd import paged
    torch = _torch()
    c = Case([3, 0], [2, 3], 20, 16, 4, 2, 64, "bf16", seed=15, gap=3)
    ref = c.run()
    o, lse = torch.full_like(c.q, 7.0), torch.full((4, c.T), 7.0, device="cuda")
    ws = kd.prefix_attn_workspace(c.q, c.kp, c.P, c.dev(c.table))
    cu, pt, tb, ln = c.dev(c.cu), c.dev(c.ptable), c.dev(c.table), c.dev(c.lens)
    desc = paged._desc(c.kp, c.vp, tb, c.B, c.T, 4, scale=0.125, prefix=c.P, prefix_width=len(c.ptable))
    st = kd.lib().kron_delta_prefix_attn(
        desc, c.q.data_ptr(), paged._S2(*c.q.stride()[:2]), c.kp.data_ptr(), c.vp.data_ptr(),
        pt.data_ptr(), tb.data_ptr(), ln.data_ptr(), cu.data_ptr(), o.data_ptr(), lse.data_ptr(), ws.data_ptr(),
        ws.numel(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(o[:5], ref[:5]) and (o[5:] == 7).all() and (lse[:, 5:] == 7).all()


def test_views_strides_and_workspaces():
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    c = Case([40, 7, 12], [1] * 3, 100, 16, 4, 2, 64, "bf16", seed=16)
    ref = c.run()
    both = torch.stack([c.kp, c.vp], 2)                       # [pages, page, 2, Hkv, d]
    heads_first = torch.stack([c.kp, c.vp], 0).transpose(2, 3).contiguous().transpose(2, 3)
    wide = torch.zeros(3, 8, 64, device="cuda", dtype=torch.bfloat16)
    wide[:, 2:6] = c.q
    table = torch.zeros(3, c.width + 5, dtype=torch.int32, device="cuda")
    table[:, :c.width] = c.dev(c.table)
    big = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
    for k, v in ((both[:, :, 0], both[:, :, 1]), (heads_first[0], heads_first[1])):
        o = kd.prefix_attn(wide[:, 2:6], k, v, c.dev(c.ptable), c.P, table[:, :c.width], c.dev(c.lens), workspace=big)
        assert torch.equal(o, ref)
    odd = torch.zeros(3 * 4 * 65 + 1, device="cuda", dtype=torch.bfloat16)[1:].view(3, 4, 65)[..., :64]
    odd.copy_(c.q)
    assert torch.equal(kd.prefix_attn(odd, *c.args()[1:]), ref)


# ------------------------------------------------------------------ appending
def append_ref(c, k, v, q, rot, layout, offset, scale=1.0):
    """kp, vp, q (with bounds) from the definitions."""
    owner = R.rows_of(c.lens, c.cu, c.T)
    freqs = [10000.0 ** (-2.0 * j / rot) for j in range(rot // 2)] if rot else []
    kp, vp = f64(c.kp), f64(c.vp)
    ek = np.zeros_like(kp)
    qo, eq = (f64(q), np.zeros(q.shape)) if q is not None else (None, None)
    u = 2.0 ** -8 if c.dt == _torch().bfloat16 else R.W
    for r, o in enumerate(owner):
        if o is None:
            continue
        b, p = o
        if p is None:
            if q is not None:
                qo[r] = 0
            continue

        def turn(x):
            if not rot:
                return x, np.zeros_like(x)
            y, e = LR.rope(x[None, None], np.array([[p + offset]]), freqs, layout, scale)
            m = np.ones_like(y)
            m[..., rot:] = 0         # elements behind the turned part are copied
            return y[0, 0], ((e + 1.01 * u * np.abs(y)) * m)[0, 0]

        if q is not None:
            qo[r], eq[r] = turn(f64(q[r]))
        at = R.slot(c.table[b], c.page, c.pages, p)
        if at is not None:
            kp[at], ek[at] = turn(f64(k[r]))
            vp[at] = f64(v[r])
    return kp, ek, vp, qo, eq


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("lens,new,page,Hq,Hkv,d,rot", [
    ([0], [1], 16, 1, 1, 64, 64), ([0, 5, -1, 40], [1] * 4, 16, 4, 2, 128, 128), ([3, 0, 17], [1] * 3, 1, 0, 4, 32, 0),
    ([0, 0, 7, -3, 20], [50, 0, 1, 4, 33], 24, 6, 2, 64, 36), ([0, 2], [130, 9], 64, 16, 4, 128, 64),
    ([9, 1], [3, 2], 5, 3, 3, 96, 34), ([0], [300], 7, 2, 1, 256, 256), ([4, 0], [2, 5], 16, 5, 1, 8, 2),
    ([0, 1], [6, 7], 16, 40, 8, 128, 128), ([0, 0, 9], [3100, 1, 2050], 64, 2, 1, 64, 64), ([5], [8500], 128, 1, 1, 8, 8),
    ([0, 3], [2030, 1100], 48, 20, 4, 128, 64)])
def test_append(lens, new, page, Hq, Hkv, d, rot, layout, dtype):
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    if dtype == "fp32" and d == 256 and layout == "interleaved":
        rot = 254
    c = Case(lens, new, 0, page, Hkv, Hkv, d, dtype, seed=d + rot, gap=2 if any(n != 1 for n in new) else 0)
    k, v = c.normal(c.T, Hkv, d), c.normal(c.T, Hkv, d)
    q = c.normal(c.T, Hq, d) if Hq else None
    c.table[0, -1] = -1 if c.table[0, -1] < 0 else c.table[0, -1]
    freqs = c.dev([10000.0 ** (-2.0 * j / rot) for j in range(rot // 2)], "float64") if rot else None
    offset = 100000
    kp, ek, vp, qo, eq = append_ref(c, k, v, q, rot, layout, offset)
    got = kd.paged_append(k, v, c.kp, c.vp, c.dev(c.table), c.dev(c.lens), q=q, cu_seqlens=c.dev(c.cu), freqs=freqs,
                          layout=layout, offset=offset)
    torch.cuda.synchronize()
    check("k_pages", c.kp, kp, ek)
    check("v_pages", c.vp, vp, 0.0)
    if Hq:
        held = np.array([o is not None for o in R.rows_of(c.lens, c.cu, c.T)])
        check("q", f64(got)[held], qo[held], eq[held])
    else:
        assert got is None



def test_append_to_bad_pages_leaves_the_cache():
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    c = Case([0, 30, 5, 12], [1] * 4, 0, 16, 2, 2, 64, "bf16", seed=21)
    c.table[0, 0], c.table[1, 1], c.table[2, 0] = -1, c.pages, 1 << 30
    c.lens = [0, 30, 5, 16 * c.width]           # the last one past the table
    before = c.kp.clone(), c.vp.clone()
    q = c.normal(4, 2, 64)
    freqs = c.dev([1.0, 0.1], "float64")
    got = kd.paged_append(c.normal(4, 2, 64), c.normal(4, 2, 64), c.kp, c.vp, c.dev(c.table), c.dev(c.lens), q=q,
                          freqs=freqs)
    torch.cuda.synchronize()
    for a, b in zip(before, (c.kp, c.vp)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    want, _ = kd.rope(q[:, None], None, c.dev(np.array(c.lens)[:, None]), freqs)
    assert torch.equal(got, want[:, 0])


def test_append_agrees_with_rope_and_strided_tensors():
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    c = Case([0, 9, 33], [20, 1, 7], 0, 16, 4, 4, 64, "bf16", seed=22)
    fused = c.normal(c.T, 4 + 2 * 4, 64)                       # one projection's heads
    q, k, v = fused[:, :4], fused[:, 4:8], fused[:, 8:]
    both = torch.zeros(c.pages, 16, 2, 4, 64, device="cuda", dtype=c.dt)
    freqs, _ = kd.rope_frequencies(64, device="cuda")
    got = kd.paged_append(k, v, both[:, :, 0], both[:, :, 1], c.dev(c.table), c.dev(c.lens), q=q,
                          cu_seqlens=c.dev(c.cu), freqs=freqs, offset=77)
    owner = R.rows_of(c.lens, c.cu, c.T)
    pos = c.dev([p + 77 for _, p in owner], "int64")
    rq, rk = kd.rope(q, k, pos, freqs)
    assert torch.equal(got, rq)
    for r, (b, p) in enumerate(owner):
        at = R.slot(c.table[b], 16, c.pages, p)
        assert torch.equal(both[at[0], at[1], 0], rk[r]) and torch.equal(both[at[0], at[1], 1], v[r])


# ------------------------------------------------------------ used together
def test_prompts_then_steps_behind_a_shared_prompt():
    """A shared prompt into its pages, each request's own prompt behind it, then decoding steps, against one plain
    attention over each request's whole text (sliding-window attention with a window that holds all of it)."""
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(3)
    P, own, steps, page, Hq, Hkv, d = 150, [33, 1, 64], 4, 16, 8, 2, 64
    freqs, _ = kd.rope_frequencies(d, device="cuda")
    mk = lambda n, h: torch.randn(n, h, d, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    prefix = [mk(P, h) for h in (Hq, Hkv, Hkv)]
    text = [[mk(n + steps, h) for h in (Hq, Hkv, Hkv)] for n in own]
    npp, nown = -(-P // page), -(-(max(own) + steps) // page)
    ids = torch.randperm(npp + 3 * nown, generator=g, device="cuda").int()
    ptable, table = ids[:npp], ids[npp:].view(3, nown)
    kp = torch.full((len(ids), page, Hkv, d), float("nan"), device="cuda", dtype=torch.bfloat16)
    vp = kp.clone()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kd.paged_append(prefix[1], prefix[2], kp, vp, ptable[None], i32([0]), cu_seqlens=i32([0, P]), freqs=freqs)
    cu = i32([0, 33, 34, 98])
    q, k, v = (torch.cat([t[i][:n] for t, n in zip(text, own)]) for i in range(3))
    q = kd.paged_append(k, v, kp, vp, table, i32([0, 0, 0]), q=q, cu_seqlens=cu, freqs=freqs, offset=P)
    first = kd.prefix_attn(q, kp, vp, ptable, P, table, i32([0, 0, 0]), cu_seqlens=cu)
    lens = i32(own)
    ws = kd.prefix_attn_workspace(q[:3], kp, P, table)
    outs = []
    for s in range(steps):
        q, k, v = (torch.stack([t[i][n + s] for t, n in zip(text, own)]) for i in range(3))
        q = kd.paged_append(k, v, kp, vp, table, lens, q=q, freqs=freqs, offset=P)
        outs.append(kd.prefix_attn(q, kp, vp, ptable, P, table, lens, workspace=ws))
        lens += 1
    at = 0
    for b, n in enumerate(own):
        x = [torch.cat([prefix[i], text[b][i]])[None] for i in range(3)]
        fq, fk = kd.rope(x[0], x[1], torch.arange(P + n + steps, device="cuda"), freqs)
        ref = kd.swa_fwd(fq.contiguous(), fk, x[2], P + n + steps)[0, P:].float()
        got = torch.cat([first[at:at + n], torch.stack([o[b] for o in outs])]).float()
        at += n
        # both results: weights rounded (2^-8, values of about 1: a sum of |v| weights below 5) and rounded again
        assert (got - ref).abs().max().item() <= 2 * 2.0 ** -8 * (5.0 + ref.abs().max().item())


def test_streams_and_graphs():
    import delta_rule_recurrent_chunk_amd as kd
    torch = _torch()
    c = Case([40, 7, 12], [1] * 3, 300, 16, 4, 2, 64, "bf16", seed=31)
    k, v, q0 = c.normal(3, 2, 64), c.normal(3, 2, 64), c.q.clone()
    freqs, _ = kd.rope_frequencies(64, device="cuda")
    table, lens, ptable = c.dev(c.table), c.dev(c.lens), c.dev(c.ptable)
    kp0, vp0 = c.kp.clone(), c.vp.clone()

    def step():
        q = kd.paged_append(k, v, c.kp, c.vp, table, lens, q=q0, freqs=freqs, offset=300)
        return kd.prefix_attn(q, c.kp, c.vp, ptable, 300, table, lens)

    ref = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        c.kp.copy_(kp0)
        c.vp.copy_(vp0)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
        assert torch.equal(step(), ref)
