"""The layers a hybrid model puts beside the Kronecker delta rule mixer, as cases to measure.

Three operators, each in the forms that training and serving call:

* the element-wise gated linear recurrence  h_t = f_t h_{t-1} + i_t x_t  (``glr_fwd``, ``glr_bwd``,
  ``glr_step``);
* attention over a sliding window with a few first tokens that stay visible (``swa_fwd``, ``swa_bwd``,
  ``swa_decode`` over a rolling cache);
* rotary positions on queries and keys (``rope``, ``rope_bwd``).

``run`` computes a case in elementary torch operations (32 bits, rounded once at the end; angles in 64) when
``own`` is false and through the library's entry points when it is true.  ``exact`` computes the same from the
definitions in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"


def _kd():
    import delta_rule_recurrent_chunk_amd as kd
    return kd


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _es(case):
    return 2 if case["dtype"] == "bf16" else 4


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the recurrence in one layer's prefill: the token count and width of the mixer's train_step
        dict(name="glr_fwd_layer", op="glr_fwd", B=8, T=2048, D=2048, dtype="bf16", gate=True, h0=False),
        # a training step over one long sequence (few channels, a long scan): the long-context length
        dict(name="glr_train_long", op="glr_train", B=1, T=32768, D=2048, dtype="bf16", gate=True, h0=False),
        # a training step at odd sizes in fp32, carried on from a state, without an input gate
        dict(name="glr_train_odd", op="glr_train", B=3, T=1111, D=1003, dtype="fp32", gate=False, h0=True),
        # one decoding step of 32 requests: latency
        dict(name="glr_step", op="glr_step", B=32, D=2048, dtype="bf16", gate=True),
        # prefill of one long prompt by a local layer (the hybrid's window of 2048), grouped heads
        dict(name="swa_fwd_long", op="swa_fwd", B=1, T=32768, past=0, Hq=16, Hkv=4, d=128, W=2048, S=4, N=0,
             dtype="bf16"),
        # a training step of a local layer
        dict(name="swa_train", op="swa_train", B=4, T=4096, past=0, Hq=16, Hkv=4, d=128, W=1024, S=4, N=0,
             dtype="bf16"),
        # a training step over packed sequences of ragged lengths (empty and one-token ones among them)
        dict(name="swa_train_packed", op="swa_train", B=1, T=8191, past=0, Hq=12, Hkv=4, d=64, W=512, S=1, N=13,
             dtype="bf16"),
        # one decoding step of 32 requests of different lengths over rolling caches
        dict(name="swa_decode_batch", op="swa_decode", B=32, Hq=16, Hkv=4, d=128, W=2048, S=4, cap=2052, lo=0,
             hi=9000, rot=128, layout="half", dtype="bf16"),
        # one decoding step of one request: latency
        dict(name="swa_decode_one", op="swa_decode", B=1, Hq=16, Hkv=4, d=128, W=2048, S=4, cap=2052, lo=1500,
             hi=1500, rot=64, layout="interleaved", dtype="bf16"),
        # queries and keys of one layer
        dict(name="rope_layer", op="rope", B=8, T=2048, Hq=16, Hkv=4, d=128, rot=128, layout="half", pos0=0,
             scaling="none", dtype="bf16"),
        # gradients of far positions, half of each head rotated, frequencies scaled for a long context
        dict(name="rope_bwd_far", op="rope_bwd", B=1, T=32768, Hq=16, Hkv=4, d=128, rot=64, layout="interleaved",
             pos0=1000000, scaling="byparts", dtype="bf16"),
        # small and odd: a rotated part whose halves fill no vector, one key head
        dict(name="rope_odd", op="rope", B=3, T=77, Hq=5, Hkv=1, d=64, rot=36, layout="half", pos0=5,
             scaling="linear", dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["glr_fwd", "glr_train", "glr_step", "swa_fwd", "swa_train", "swa_train", "swa_decode",
                     "swa_decode", "rope", "rope_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op in ("glr_fwd", "glr_train"):
        top = 64 << 20 if dtype == "bf16" else 24 << 20
        D = rng.choice([_log_int(rng, 16, 8192), 64 * _log_int(rng, 1, 64)])
        B = _log_int(rng, 1, 16)
        T = _log_int(rng, 1, max(1, min(65536, top // (B * D))))
        return dict(op=op, B=B, T=T, D=D, dtype=dtype, gate=rng.random() < 0.6, h0=rng.random() < 0.5)
    if op == "glr_step":
        return dict(op=op, B=_log_int(rng, 1, 256), D=_log_int(rng, 64, 8192), dtype=dtype, gate=rng.random() < 0.7)
    if op in ("swa_fwd", "swa_train"):
        d = rng.choice([32, 64, 128, 128])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
        least = 2 if op == "swa_train" else 1     # a row that sees one key alone has no gradient to compare
        W = _log_int(rng, least, 4096)
        S = rng.choice([0, 1, 4, rng.randint(0, 64)])
        case = dict(op=op, B=1, T=1, past=0, Hq=Hq, Hkv=Hkv, d=d, W=W, S=S, N=0, dtype=dtype)
        # at most a third of the largest listed case's products (fp32: a fortieth)
        budget = 4 * 128 * 16 * 32768 * 2048 / (3 if dtype == "bf16" else 40)
        per = (4 if op == "swa_fwd" else 14) * d * Hq
        for _ in range(64):
            case["T"] = _log_int(rng, least, 16384)
            case["B"] = _log_int(rng, 1, 16)
            if per * case["B"] * case["T"] * min(case["T"], W + S) <= budget and \
                    case["B"] * case["T"] * Hq * d <= 1 << 27:
                break
        else:
            case["T"], case["B"] = 257, 1
        if rng.random() < 0.3:                       # packed sequences
            case["B"], case["N"] = 1, rng.randint(1, 24)
        elif op == "swa_fwd" and rng.random() < 0.3:   # a later piece of a prompt
            case["past"] = _log_int(rng, 1, 4096)
        return case
    if op == "swa_decode":
        d = rng.choice([32, 64, 128, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        S = rng.choice([0, 1, 4, rng.randint(0, 64)])
        W = _log_int(rng, 1, 4096)
        cap = S + W + rng.choice([0, 0, _log_int(rng, 1, 1000)])
        lo = rng.choice([0, 0, rng.randint(0, 5000)])
        B = _log_int(rng, 1, 128)
        while B > 1 and B * Hkv * cap * d * _es(dict(dtype=dtype)) > 1 << 28:
            B //= 2
        return dict(op=op, B=B, Hq=Hkv * rng.choice([1, 2, 3, 4, 8, 16]), Hkv=Hkv, d=d, W=W, S=S, cap=cap, lo=lo,
                    hi=lo + _log_int(rng, 1, 20000), rot=rng.choice([0, d, d // 2, d, 2 * rng.randint(1, d // 2)]),
                    layout=rng.choice(["half", "interleaved"]), dtype=dtype)
    d = rng.choice([32, 64, 128, 8 * rng.randint(1, 32)])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
    B = _log_int(rng, 1, 16)
    T = _log_int(rng, 1, max(1, min(32768, (1 << 26) // (B * (Hq + Hkv) * d))))
    return dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, rot=rng.choice([d, d // 2 * 2, 2 * rng.randint(1, d // 2)]),
                layout=rng.choice(["half", "interleaved"]), pos0=rng.choice([0, _log_int(rng, 1, 10 ** 6)]),
                scaling=rng.choice(["none", "linear", "byparts"]), dtype=dtype)


# ------------------------------------------------------- what a case is made of
def _freqs(rot, scaling):
    """Angle per position of each rotated pair, radians, 64 bits, and the factor on the rotated part."""
    n = rot // 2
    base = [10000.0 ** (-2.0 * j / rot) for j in range(n)]
    if scaling == "none":
        return base, 1.0
    if scaling == "linear":          # positions stretched by 4
        return [w / 4.0 for w in base], 1.0
    # by parts: fast pairs (more than 32 turns in 4096 positions) keep their angle, slow ones (less than one) are
    # stretched by 8, those between are blended
    out = []
    for w in base:
        turns = 4096.0 * w / (2.0 * math.pi)
        keep = min(max((turns - 1.0) / 31.0, 0.0), 1.0)
        out.append(w * keep + w / 8.0 * (1.0 - keep))
    return out, 0.1 * math.log(8.0) + 1.0


def _lens(case):
    """Tokens in each request's cache before the step: spread over lo .. hi."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    if B == 1:
        return [hi]
    r = random.Random(B * 1000003 + lo * 101 + hi)
    return [lo + (hi - lo) * j // (B - 1) if j % 3 else r.randint(lo, hi) for j in range(B)]


def _cu(case):
    """Offsets of the packed sequences: ragged, with an empty and a one-token one where there are enough."""
    N, T = case["N"], case["T"]
    r = random.Random(N * 7919 + T)
    cuts = sorted(r.randint(0, T) for _ in range(N - 1))
    if N >= 4:
        cuts[1] = cuts[0]
        cuts[2] = max(cuts[2], min(cuts[1] + 1, T))
        cuts = sorted(cuts)
    return [0] + cuts + [T]


def _spans(case):
    """(batch, first row, rows, first key, keys) of every sequence of an attention case."""
    if case["N"]:
        cu = _cu(case)
        return [(0, a, b - a, a, b - a) for a, b in zip(cu[:-1], cu[1:]) if b > a]
    return [(b, 0, case["T"], 0, case["T"] + case["past"]) for b in range(case["B"])]


def _pairs(n, past, W, S):
    """Visible (query, key) pairs of n queries that stand at positions past .. past + n - 1."""
    def upto(m):          # sum over positions p < m of the keys they see
        full = min(m, W + S)
        tot = full * (full + 1) // 2
        return tot + (m - full) * (W + S)
    return upto(past + n) - upto(past)


def _seen(case):
    return sum(min(p + 1, case["W"] + case["S"]) for p in _lens(case))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    dt, op = _dt(case), case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)

    st = dict(case=case)
    if op.startswith("glr"):
        B, D = case["B"], case["D"]
        sh = (B, D) if op == "glr_step" else (B, case["T"], D)
        st["x"] = normal(*sh).to(dt)
        # forget gates as the mixer makes them: sigmoid(N(3, 1)) to a power per channel
        e = torch.exp(torch.rand(D, generator=g, device=DEV) * 2 - 1)
        st["f"] = torch.sigmoid(normal(*sh) + 3.0).pow(e).to(dt)
        st["i"] = torch.sigmoid(normal(*sh)).to(dt) if case["gate"] else None
        st["h0"] = normal(B, D) if op == "glr_step" or case["h0"] else None
        if op == "glr_train":
            st["dh"] = normal(*sh).to(dt)
            st["dhT"] = normal(B, D) if case["h0"] else None
        if op == "glr_step":
            st["h1"] = torch.empty(B, D, device=DEV)
        return st
    if op in ("swa_fwd", "swa_train"):
        T, Tk = case["T"], case["T"] + case["past"]
        lead = () if case["N"] else (case["B"],)
        st["q"] = normal(*lead, T, case["Hq"], case["d"]).to(dt)
        st["k"] = normal(*lead, Tk, case["Hkv"], case["d"]).to(dt)
        st["v"] = normal(*lead, Tk, case["Hkv"], case["d"]).to(dt)
        if op == "swa_train":
            st["do"] = normal(*lead, T, case["Hq"], case["d"]).to(dt)
        st["cu"] = torch.tensor(_cu(case), dtype=torch.int32, device=DEV) if case["N"] else None
        return st
    if op == "swa_decode":
        B, d, cap = case["B"], case["d"], case["cap"]
        st["q"] = normal(B, case["Hq"], d).to(dt)
        st["k"] = normal(B, case["Hkv"], d).to(dt)
        st["v"] = normal(B, case["Hkv"], d).to(dt)
        lens = _lens(case)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        used = torch.tensor([min(p, cap) for p in lens], device=DEV)
        live = (torch.arange(cap, device=DEV)[None, :] < used[:, None])[:, :, None, None]
        # slots that no token has reached yet hold zeros
        st["kc"] = torch.where(live, normal(B, cap, case["Hkv"], d), 0.0).to(dt)
        st["vc"] = torch.where(live, normal(B, cap, case["Hkv"], d), 0.0).to(dt)
        st["freqs"] = torch.tensor(_freqs(case["rot"], "none")[0], dtype=torch.float64, device=DEV) \
            if case["rot"] else None
        if own:    # a serving loop keeps the workspace of its decoding steps
            st["ws"] = _kd().swa_decode_workspace(st["q"], st["kc"])
        return st
    B, T = case["B"], case["T"]
    st["q"] = normal(B, T, case["Hq"], case["d"]).to(dt)
    st["k"] = normal(B, T, case["Hkv"], case["d"]).to(dt)
    fr, st["mscale"] = _freqs(case["rot"], case["scaling"])
    st["freqs"] = torch.tensor(fr, dtype=torch.float64, device=DEV)
    st["pos"] = case["pos0"] + torch.arange(T, dtype=torch.int64, device=DEV)
    return st


# ----------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    kd, case, op = _kd(), st["case"], st["case"]["op"]
    if op == "glr_fwd":
        h, hT = kd.glr_fwd(st["x"], st["f"], st["i"], st["h0"])
        return dict(h=h, hT=hT)
    if op == "glr_train":
        h, hT, hs = kd.glr_fwd(st["x"], st["f"], st["i"], st["h0"], save_states=True)
        gr = kd.glr_bwd(st["x"], st["f"], st["i"], hs, st["dh"], st["dhT"])
        out = dict(h=h, hT=hT, dx=gr["dx"], df=gr["df"], dh0=gr["dh0"])
        if case["gate"]:
            out["di"] = gr["di"]
        return out
    if op == "glr_step":
        y = kd.glr_step(st["x"], st["f"], st["i"], st["h0"], h_out=st["h1"])
        return dict(y=y, h=st["h1"])
    if op == "swa_fwd":
        return dict(o=kd.swa_fwd(st["q"], st["k"], st["v"], case["W"], case["S"], cu_seqlens=st["cu"]))
    if op == "swa_train":
        o, lse = kd.swa_fwd(st["q"], st["k"], st["v"], case["W"], case["S"], cu_seqlens=st["cu"], return_lse=True)
        gr = kd.swa_bwd(st["q"], st["k"], st["v"], o, lse, st["do"], case["W"], case["S"], cu_seqlens=st["cu"])
        return dict(o=o, lse=lse, dq=gr["dq"], dk=gr["dk"], dv=gr["dv"])
    if op == "swa_decode":
        o = kd.swa_decode(st["q"], st["k"], st["v"], st["kc"], st["vc"], st["lens"], case["W"], case["S"],
                          freqs=st["freqs"], layout=case["layout"], workspace=st["ws"])
        return dict(o=o, k_cache=st["kc"], v_cache=st["vc"])
    f = kd.rope if op == "rope" else kd.rope_bwd
    q, k = f(st["q"], st["k"], st["pos"], st["freqs"], layout=case["layout"], scale=st["mscale"])
    return dict(q=q, k=k)


def _shift_scan(a, b):
    """y_t = a_t y_{t-1} + b_t along dim 1 by doubling (a is consumed)."""
    s, T = 1, b.shape[1]
    while s < T:
        b = torch.cat([b[:, :s], b[:, s:] + a[:, s:] * b[:, :-s]], 1)
        if 2 * s < T:
            a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
        s *= 2
    return b


def _plain_glr(st):
    dt, case = _dt(st["case"]), st["case"]
    x, f = st["x"].float(), st["f"].float()
    i = st["i"].float() if st["i"] is not None else None
    b = x if i is None else i * x
    h0 = st["h0"]
    if h0 is not None:
        b = torch.cat([b[:, :1] + f[:, :1] * h0[:, None], b[:, 1:]], 1)
    h = _shift_scan(f, b)
    out = dict(h=h.to(dt), hT=h[:, -1].contiguous())
    if case["op"] == "glr_fwd":
        return out
    dh = st["dh"].float()
    if st["dhT"] is not None:
        dh = torch.cat([dh[:, :-1], dh[:, -1:] + st["dhT"][:, None]], 1)
    fn = torch.cat([f[:, 1:], torch.zeros_like(f[:, :1])], 1)     # the gate that carries t into t + 1
    lam = _shift_scan(fn.flip(1), dh.flip(1)).flip(1)
    first = h0[:, None] if h0 is not None else torch.zeros_like(h[:, :1])
    prev = torch.cat([first, h[:, :-1]], 1)
    out["dx"] = (lam if i is None else lam * i).to(dt)
    out["df"] = (lam * prev).to(dt)
    out["dh0"] = f[:, 0] * lam[:, 0]
    if i is not None:
        out["di"] = (lam * x).to(dt)
    return out


def _plain_attn_span(q, k, v, W, S, do, dq, dk, dv, o, lse):
    """q, do, o, dq [b, Hkv, G, n, d]; k, v, dk, dv [b, Hkv, m, d]; lse [b, Hkv, G, n]; queries stand at the end."""
    b, H, G, n, d = q.shape
    m = k.shape[2]
    past, scale = m - n, 1.0 / math.sqrt(d)
    rows = max(32, min(1024, (1 << 29) // max(1, b * H * G * min(m, W + S + 1024))))
    for r0 in range(0, n, rows):
        r1 = min(n, r0 + rows)
        lo = max(0, past + r0 - W + 1)
        hi, ns = past + r1, min(S, lo)
        idx = torch.cat([torch.arange(0, ns, device=DEV), torch.arange(lo, hi, device=DEV)])
        pos = torch.arange(past + r0, past + r1, device=DEV)[:, None]
        vis = (idx[None] <= pos) & ((pos - idx[None] < W) | (idx[None] < S))
        kk = torch.cat([k[:, :, :ns], k[:, :, lo:hi]], 2)
        vv = torch.cat([v[:, :, :ns], v[:, :, lo:hi]], 2)
        qq = q[:, :, :, r0:r1].reshape(b, H, -1, d)
        s = torch.matmul(qq, kk.transpose(2, 3).contiguous()).view(b, H, G, r1 - r0, -1) * scale
        s = s.masked_fill(~vis, float("-inf"))
        mx = s.amax(-1, keepdim=True)
        p = torch.exp(s - mx)
        l = p.sum(-1, keepdim=True)
        p = (p / l).view(b, H, G * (r1 - r0), -1)
        oo = torch.matmul(p, vv)
        o[:, :, :, r0:r1] = oo.view(b, H, G, r1 - r0, d)
        lse[:, :, :, r0:r1] = (mx + torch.log(l)).squeeze(-1)
        if do is None:
            continue
        dd = do[:, :, :, r0:r1].reshape(b, H, -1, d)
        dp = torch.matmul(dd, vv.transpose(2, 3).contiguous())
        ds = p * (dp - (dd * oo).sum(-1, keepdim=True)) * scale
        dq[:, :, :, r0:r1] = torch.matmul(ds, kk).view(b, H, G, r1 - r0, d)
        gk = torch.matmul(ds.transpose(2, 3).contiguous(), qq)
        gv = torch.matmul(p.transpose(2, 3).contiguous(), dd)
        dk[:, :, :ns] += gk[:, :, :ns]
        dk[:, :, lo:hi] += gk[:, :, ns:]
        dv[:, :, :ns] += gv[:, :, :ns]
        dv[:, :, lo:hi] += gv[:, :, ns:]


def _plain_swa(st):
    case, dt = st["case"], _dt(st["case"])
    Hkv, G, d = case["Hkv"], case["Hq"] // case["Hkv"], case["d"]
    packed = case["N"] > 0

    def heads(t, grouped):       # [B, T, H, d] -> [B, Hkv, (G,) T, d] in 32 bits
        t = (t[None] if packed else t).float()
        if grouped:
            return t.view(t.shape[0], t.shape[1], Hkv, G, d).permute(0, 2, 3, 1, 4).contiguous()
        return t.permute(0, 2, 1, 3).contiguous()

    q, k, v = heads(st["q"], True), heads(st["k"], False), heads(st["v"], False)
    train = case["op"] == "swa_train"
    do = heads(st["do"], True) if train else None
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:-1], device=DEV)
    dq, dk, dv = (torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)) if train else (None, None, None)
    spans = _spans(case)
    if not packed:               # equal sequences go together
        spans = [(slice(None), 0, case["T"], 0, case["T"] + case["past"])]
    else:
        spans = [(slice(0, 1),) + s[1:] for s in spans]
    for bs, r0, n, k0, m in spans:
        rs, ks = slice(r0, r0 + n), slice(k0, k0 + m)
        _plain_attn_span(q[bs, :, :, rs], k[bs, :, ks], v[bs, :, ks], case["W"], case["S"],
                         do[bs, :, :, rs] if train else None, dq[bs, :, :, rs] if train else None,
                         dk[bs, :, ks] if train else None, dv[bs, :, ks] if train else None,
                         o[bs, :, :, rs], lse[bs, :, :, rs])

    def back(t, grouped):
        t = t.permute(0, 3, 1, 2, 4).flatten(2, 3) if grouped else t.permute(0, 2, 1, 3)
        t = t.to(dt).contiguous()
        return t[0] if packed else t

    if not train:
        return dict(o=back(o, True))
    lse = lse.flatten(1, 2)
    return dict(o=back(o, True), lse=lse[0].contiguous() if packed else lse, dq=back(dq, True), dk=back(dk, False),
                dv=back(dv, False))


def _rotate(x, ang, layout, sign, mscale):
    """x [..., d] in 32 bits; ang [..., rot / 2] in 64 bits, broadcast against x's leading dims."""
    n = ang.shape[-1]
    c, s = (torch.cos(ang) * mscale).float(), (torch.sin(ang) * (sign * mscale)).float()
    r, rest = x[..., :2 * n], x[..., 2 * n:]
    if layout == "half":
        a, b = r[..., :n], r[..., n:]
        return torch.cat([a * c - b * s, b * c + a * s, rest], -1)
    a, b = r[..., 0::2], r[..., 1::2]
    return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), rest], -1)


def _slots(pos, S, cap):
    return torch.where(pos < S, pos, S + (pos - S) % max(cap - S, 1))


def _plain_decode(st):
    case, dt = st["case"], _dt(st["case"])
    B, Hkv, G, d, W, S, cap = (case[n] for n in ("B", "Hkv", "Hq", "d", "W", "S", "cap"))
    G = G // Hkv
    q, k, lens = st["q"].float(), st["k"].float(), st["lens"].long()
    if case["rot"]:
        ang = lens.double()[:, None, None] * st["freqs"]
        q, k = _rotate(q, ang, case["layout"], 1.0, 1.0), _rotate(k, ang, case["layout"], 1.0, 1.0)
    rows = torch.arange(B, device=DEV)
    at = _slots(lens, S, cap)
    st["kc"][rows, at] = k.to(dt)
    st["vc"][rows, at] = st["v"]
    # the first S positions, then the W last ones
    pos = torch.cat([torch.arange(S, device=DEV)[None].expand(B, S),
                     lens[:, None] - W + 1 + torch.arange(W, device=DEV)[None]], 1)
    new = torch.arange(S + W, device=DEV)[None] >= S
    vis = (pos <= lens[:, None]) & (pos >= 0) & (~new | (pos >= S))
    sl = _slots(pos.clamp(min=0), S, cap)
    kk = st["kc"][rows[:, None], sl].float().permute(0, 2, 1, 3).contiguous()     # [B, Hkv, S + W, d]
    vv = st["vc"][rows[:, None], sl].float().permute(0, 2, 1, 3).contiguous()
    s = torch.matmul(q.view(B, Hkv, G, d), kk.transpose(2, 3).contiguous()) / math.sqrt(d)
    s = s.masked_fill(~vis[:, None, None], float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul(p, vv) / p.sum(-1, keepdim=True)
    return dict(o=o.view(B, Hkv * G, d).to(dt), k_cache=st["kc"], v_cache=st["vc"])


def _run_plain(st):
    case, op, dt = st["case"], st["case"]["op"], _dt(st["case"])
    if op in ("glr_fwd", "glr_train"):
        return _plain_glr(st)
    if op == "glr_step":
        u = st["x"].float() if st["i"] is None else st["i"].float() * st["x"].float()
        st["h1"].copy_(st["f"].float() * st["h0"] + u)
        return dict(y=st["h1"].to(dt), h=st["h1"])
    if op in ("swa_fwd", "swa_train"):
        return _plain_swa(st)
    if op == "swa_decode":
        return _plain_decode(st)
    ang = (st["pos"].double()[:, None] * st["freqs"])[:, None, :]
    sign = 1.0 if op == "rope" else -1.0
    return dict(q=_rotate(st["q"].float(), ang, case["layout"], sign, st["mscale"]).to(dt),
                k=_rotate(st["k"].float(), ang, case["layout"], sign, st["mscale"]).to(dt))


# ------------------------------------------------------------- the least work
def work(case):
    op, es = case["op"], _es(case)
    if op.startswith("glr"):
        B, D = case["B"], case["D"]
        n = B * D * case.get("T", 1)
        gate = 1 if case["gate"] else 0
        fwd, state = n * es * (3 + gate), 4 * B * D
        if op == "glr_fwd":
            return dict(bytes=fwd + state * (2 if case["h0"] else 1), flops=n * (2 + gate))
        if op == "glr_step":
            return dict(bytes=fwd + 2 * state, flops=n * (2 + gate))
        # dh read, dx, df and di written; h0 and dhT read, hT and dh0 written
        return dict(bytes=fwd + n * es * (3 + gate) + state * (4 if case["h0"] else 2), flops=n * (5 + 3 * gate))
    if op in ("swa_fwd", "swa_train"):
        d, Hq, Hkv = case["d"], case["Hq"], case["Hkv"]
        sp = _spans(case)
        pairs = sum(_pairs(n, m - n, case["W"], case["S"]) for _, _, n, _, m in sp)
        nq, nk = sum(s[2] for s in sp) * Hq * d, sum(s[4] for s in sp) * Hkv * d
        if op == "swa_fwd":
            return dict(bytes=es * (2 * nq + 2 * nk), flops=4 * d * Hq * pairs)
        return dict(bytes=es * (4 * nq + 4 * nk) + 4 * nq // d, flops=14 * d * Hq * pairs)
    if op == "swa_decode":
        d, Hq, Hkv, B = case["d"], case["Hq"], case["Hkv"], case["B"]
        seen = _seen(case)
        # the visible keys and values but the new one's from the cache; q, k, v in, o and the new rows out
        return dict(bytes=es * d * (2 * Hkv * (seen - B) + 2 * B * Hq + 4 * B * Hkv), flops=4 * d * Hq * seen)
    n = case["B"] * case["T"] * (case["Hq"] + case["Hkv"])
    return dict(bytes=2 * es * n * case["d"] + 8 * (case["T"] + case["rot"] // 2), flops=3 * n * case["rot"])


# ------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "glr_step":
        h = st["f"].double() * st["h0"].double()
        h += st["x"].double() * (st["i"].double() if case["gate"] else 1.0)
        return dict(y=h, h=h)
    if op in ("glr_fwd", "glr_train"):
        return _exact_glr(case, st)
    if op in ("swa_fwd", "swa_train"):
        return _exact_swa(case, st)
    if op == "swa_decode":
        return _exact_decode(case, st)
    # a rotation of each pair, as a product of complex numbers
    turn = torch.polar(torch.full((case["T"], 1, case["rot"] // 2), st["mscale"], dtype=torch.float64, device=DEV),
                       (1 if op == "rope" else -1) * st["pos"].double()[:, None, None] * st["freqs"])
    return dict(q=_exact_turn(st["q"], turn, case["layout"]), k=_exact_turn(st["k"], turn, case["layout"]))


def _exact_turn(x, turn, layout):
    y, n = x.double(), turn.shape[-1]
    first = torch.arange(n, device=DEV) * (1 if layout == "half" else 2)
    second = first + (n if layout == "half" else 1)
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_glr(case, st):
    # token by token
    x, f = st["x"].double(), st["f"].double()
    i = st["i"].double() if case["gate"] else torch.ones((), dtype=torch.float64, device=DEV).expand_as(x)
    T = case["T"]
    h = st["h0"].double() if case["h0"] else torch.zeros(case["B"], case["D"], dtype=torch.float64, device=DEV)
    hs = torch.empty(T + 1, case["B"], case["D"], dtype=torch.float64, device=DEV)
    hs[0] = h
    for t in range(T):
        torch.addcmul(x[:, t] * i[:, t], f[:, t], hs[t], out=hs[t + 1])
    out = dict(h=hs[1:].transpose(0, 1), hT=hs[T])
    if case["op"] == "glr_fwd":
        return out
    lam = st["dhT"].double() if case["h0"] else torch.zeros_like(hs[0])
    dx, df, di = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    for t in reversed(range(T)):
        lam = lam + st["dh"][:, t].double()
        dx[:, t], df[:, t], di[:, t] = lam * i[:, t], lam * hs[t], lam * x[:, t]
        lam = lam * f[:, t]
    out.update(dx=dx, df=df, dh0=lam)
    if case["gate"]:
        out["di"] = di
    return out


def _exact_swa(case, st):
    train, packed = case["op"] == "swa_train", case["N"] > 0
    spans = _spans(case)
    G = case["Hq"] // case["Hkv"]
    names = ("q", "k", "v") + (("do",) if train else ())
    t = {n: (st[n][None] if packed else st[n]) for n in names}
    o = torch.zeros(t["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(o.shape[0], o.shape[2], o.shape[1], dtype=torch.float64, device=DEV)
    gr = {n: torch.zeros(t[n].shape, dtype=torch.float64, device=DEV) for n in ("q", "k", "v")} if train else None
    for b, r0, n, k0, m in spans:
        for h in range(case["Hq"]):
            q = t["q"][b, r0:r0 + n, h].double()
            k = t["k"][b, k0:k0 + m, h // G].double()
            v = t["v"][b, k0:k0 + m, h // G].double()
            # rows in groups only where the whole table of scores would be large
            step = n if n * m <= 1 << 27 else max(1, (1 << 26) // m)
            for a in range(0, n, step):
                e = min(n, a + step)
                first = 0 if case["S"] else max(0, m - n + a - case["W"] + 1)
                last = m - n + e
                at = torch.arange(m - n + a, m - n + e, device=DEV)[:, None]
                key = torch.arange(first, last, device=DEV)[None]
                hidden = (key > at) | ((key <= at - case["W"]) & (key >= case["S"]))
                kk, vv, qq = k[first:last], v[first:last], q[a:e]
                score = (qq @ kk.T).mul_(1.0 / math.sqrt(case["d"])).masked_fill_(hidden, -math.inf)
                z = torch.logsumexp(score, 1)
                w = score.sub_(z[:, None]).exp_()
                o[b, r0 + a:r0 + e, h] = w @ vv
                lse[b, h, r0 + a:r0 + e] = z
                if train:
                    g = t["do"][b, r0 + a:r0 + e, h].double()
                    gr["v"][b, k0 + first:k0 + last, h // G] += w.T @ g
                    dw = g @ vv.T
                    dw = w * (dw - (w * dw).sum(1, keepdim=True)) / math.sqrt(case["d"])
                    gr["q"][b, r0 + a:r0 + e, h] = dw @ kk
                    gr["k"][b, k0 + first:k0 + last, h // G] += dw.T @ qq
    if not train:
        return dict(o=o[0] if packed else o)
    out = dict(o=o, lse=lse, dq=gr["q"], dk=gr["k"], dv=gr["v"])
    return {n: a[0] for n, a in out.items()} if packed else out


def _exact_decode(case, st):
    S, cap, W = case["S"], case["cap"], case["W"]
    q, k = st["q"].double(), st["k"].double()
    if case["rot"]:
        turn = torch.exp(1j * (st["lens"].double()[:, None, None] * st["freqs"]))
        q, k = _exact_turn(q, turn, case["layout"]), _exact_turn(k, turn, case["layout"])
    kc, vc = st["kc"].double(), st["vc"].double()
    o = torch.empty_like(q)
    for b, p in enumerate(_lens(case)):
        see = sorted(set(range(min(S, p + 1))) | set(range(max(0, p - W + 1), p + 1)))
        slot = torch.tensor([s if s < S else S + (s - S) % max(cap - S, 1) for s in see], device=DEV)
        # the cache holds the new key in its own type, and the step reads it from there
        kc[b, slot[-1]], vc[b, slot[-1]] = k[b].to(_dt(case)).double(), st["v"][b].double()
        kk = kc[b, slot].repeat_interleave(case["Hq"] // case["Hkv"], 1)       # [keys, Hq, d]
        vv = vc[b, slot].repeat_interleave(case["Hq"] // case["Hkv"], 1)
        w = torch.softmax((kk * q[b]).sum(-1) / math.sqrt(case["d"]), 0)
        o[b] = (w[..., None] * vv).sum(0)
        kc[b, slot[-1]] = k[b]
    return dict(o=o, k_cache=kc, v_cache=vc)
