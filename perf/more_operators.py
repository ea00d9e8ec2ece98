"""Training a recurrent layer of a hybrid, and serving the hybrid to requests that share a prompt, as cases to measure.

Three operators, each in the forms that training and serving call:

* the gated delta rule  S <- e^g S,  S <- S + beta (v - S k) k^T,  o = scale S q  (``gdr_fwd``, ``gdr_bwd`` over
  sequences, ``gdr_step`` for one token);
* keys and values into a paged cache, turned to their positions on the way (``paged_append``);
* attention of a batch over a prefix that all of it shares and over each request's own pages (``prefix_attn``).

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
        # prefill of one layer, the states kept for decoding: the sizes of the package's gdn2_step workload
        dict(name="gdr_prefill", op="gdr_fwd", B=8, T=2048, Hk=16, Hv=16, dk=128, dv=128, N=0, S0=False, dtype="bf16"),
        # prefill of one long prompt: the sizes of the package's long_ctx workload
        dict(name="gdr_long", op="gdr_fwd", B=1, T=32768, Hk=16, Hv=16, dk=128, dv=128, N=0, S0=False, dtype="bf16"),
        # a training step: the sizes of the package's fwd_bwd workload
        dict(name="gdr_train", op="gdr_train", B=4, T=2048, Hk=16, Hv=16, dk=128, dv=128, N=0, S0=False, dtype="bf16"),
        # a training step over packed sequences of ragged lengths, key heads shared by three value heads
        dict(name="gdr_train_packed", op="gdr_train", B=1, T=8191, Hk=4, Hv=12, dk=64, dv=64, N=13, S0=False,
             dtype="bf16"),
        # odd sizes in fp32, carried on from a state, with the gradient of that state
        dict(name="gdr_train_odd", op="gdr_train", B=3, T=333, Hk=1, Hv=2, dk=48, dv=80, N=0, S0=True, dtype="fp32"),
        # one decoding step of 32 requests: the sizes of the package's decode_step workload
        dict(name="gdr_step", op="gdr_step", B=32, Hk=16, Hv=16, dk=128, dv=128, dtype="bf16"),
        # 24 prompts of ragged lengths into the pages, their queries turned with them
        dict(name="append_prompts", op="paged_append", B=24, n=1100, lo=0, hi=0, Hq=16, Hkv=4, d=128, page=64, rot=128,
             layout="half", offset=0, dtype="bf16"),
        # one decoding step of 32 requests behind a shared prompt, half of each head rotated: latency
        dict(name="append_step", op="paged_append", B=32, n=0, lo=0, hi=1000, Hq=16, Hkv=4, d=128, page=16, rot=64,
             layout="interleaved", offset=32768, dtype="bf16"),
        # one decoding step of 64 requests behind a long shared prompt
        dict(name="prefix_decode", op="prefix_attn", B=64, n=0, P=32768, lo=0, hi=1000, Hq=16, Hkv=4, d=128, page=64,
             dtype="bf16"),
        # the same of a few requests behind a short one: latency
        dict(name="prefix_few", op="prefix_attn", B=3, n=0, P=2000, lo=5, hi=200, Hq=16, Hkv=4, d=128, page=16,
             dtype="bf16"),
        # the requests' own questions, ragged, behind the shared prompt
        dict(name="prefix_prompts", op="prefix_attn", B=16, n=300, P=8192, lo=0, hi=0, Hq=16, Hkv=4, d=128, page=64,
             dtype="bf16"),
        # pages that end inside a tile, a prefix that ends inside a page, fp32
        dict(name="prefix_odd", op="prefix_attn", B=5, n=7, P=1003, lo=0, hi=90, Hq=6, Hkv=2, d=64, page=24,
             dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["gdr_fwd", "gdr_fwd", "gdr_train", "gdr_train", "gdr_step", "paged_append", "paged_append",
                     "prefix_attn", "prefix_attn", "prefix_attn"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op.startswith("gdr"):
        Hk = rng.choice([1, 2, 4, 8, 16])
        Hv = Hk * rng.choice([1, 1, 2, 3, 4])
        dk = rng.choice([64, 128, 128, 8 * rng.randint(1, 16)])
        dv = rng.choice([dk, 64, 128, 8 * rng.randint(1, 32)])
        if op == "gdr_step":
            B = _log_int(rng, 1, 128)
            while B > 1 and B * Hv * dk * dv > 32 * 16 * 128 * 128 * 4:
                B //= 2
            return dict(op=op, B=B, Hk=Hk, Hv=Hv, dk=dk, dv=dv, dtype=dtype)
        top = (16384 if op == "gdr_fwd" else 6000) * 16 * 128 // (1 if dtype == "bf16" else 8)
        T, B = _log_int(rng, 1, 8192), _log_int(rng, 1, 16)
        while B > 1 and B * T * Hv * max(dk, dv) > top:
            B //= 2
        while T > 1 and B * T * Hv * max(dk, dv) > top:
            T //= 2
        case = dict(op=op, B=B, T=T, Hk=Hk, Hv=Hv, dk=dk, dv=dv, N=0, S0=False, dtype=dtype)
        if rng.random() < 0.3 and T >= 16:
            case.update(B=1, N=rng.randint(1, 16))
        elif dtype == "fp32" or op == "gdr_fwd":
            case["S0"] = rng.random() < 0.5
        return case
    d = rng.choice([32, 64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([1, 16, 16, 32, 64, 128, rng.randint(1, 200)])
    lo = rng.choice([0, 0, rng.randint(0, 200)])
    hi = lo + _log_int(rng, 1, 1500)
    if op == "paged_append":
        n = rng.choice([0, 1, _log_int(rng, 2, 2000)])
        B = _log_int(rng, 1, 256 if n < 2 else 32)
        while B > 1 and B * max(n, 1) * (Hq + Hkv) * d > 24 * 1100 * 20 * 128:
            B //= 2
        return dict(op=op, B=B, n=n, lo=lo, hi=hi, Hq=rng.choice([0, Hq]), Hkv=Hkv, d=d, page=page,
                    rot=rng.choice([0, d, d, d // 2, 2 * rng.randint(1, d // 2)]),
                    layout=rng.choice(["half", "interleaved"]), offset=rng.choice([0, _log_int(rng, 1, 10 ** 6)]),
                    dtype=dtype)
    n = rng.choice([0, 0, _log_int(rng, 1, 400)])
    case = dict(op=op, B=_log_int(rng, 1, 96), n=n, P=rng.choice([0, _log_int(rng, 1, 32768), _log_int(rng, 1, 32768)]),
                lo=lo, hi=hi, Hq=Hq, Hkv=Hkv, d=d, page=page, dtype=dtype)
    # at most two thirds of the largest listed case's products (fp32: a fifteenth), and bounded caches
    budget = 4 * 128 * 16 * 16 * 150 * 8192 / (1.5 if dtype == "bf16" else 15)
    while case["B"] > 1 and (4 * d * Hq * case["B"] * max(1, n // 2) * (case["P"] + hi) > budget or
                             case["B"] * (hi + n) * Hkv * d > 1 << 27):
        case["B"] //= 2
    while 4 * d * Hq * case["B"] * max(1, n // 2) * (case["P"] + hi) > budget and case["P"] > 64:
        case["P"] //= 2
    return case


# ------------------------------------------------------- what a case is made of
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


def _held(case):
    """Own tokens of each request before the call: spread over lo .. hi."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    if B == 1:
        return [hi]
    r = random.Random(B * 1000003 + lo * 101 + hi)
    return [lo + (hi - lo) * j // (B - 1) if j % 3 else r.randint(lo, hi) for j in range(B)]


def _new(case):
    """New tokens of each request: one (n = 0: not packed), or ragged ones up to n, one of them none."""
    B, n = case["B"], case["n"]
    if n == 0:
        return [1] * B
    r = random.Random(B * 31337 + n)
    out = [r.randint(1, n) for _ in range(B)]
    out[B // 2] = n
    if B > 3:
        out[2] = 0
    return out


def _table(case, tokens, first, g):
    """A table of shuffled pages for requests of so many tokens, from page `first` on, and the pages used."""
    per = [max(1, -(-t // case["page"])) for t in tokens]
    ids = torch.randperm(sum(per), generator=g, device=DEV).to(torch.int32) + first
    table = torch.full((len(tokens), max(per)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, p in enumerate(per):
        table[b, :p] = ids[at:at + p]
        at += p
    return table, at


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 23)
    dt, op = _dt(case), case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)

    st = dict(case=case)
    if op.startswith("gdr"):
        B, Hk, Hv, dk, dv = (case[n] for n in ("B", "Hk", "Hv", "dk", "dv"))
        lead = (B,) if op == "gdr_step" else (case["T"],) if case["N"] else (B, case["T"])

        def unit(*shape):      # as the mixer makes its queries and keys: SiLU, then the L2 norm
            x = torch.nn.functional.silu(normal(*shape))
            return x / x.norm(dim=-1, keepdim=True).clamp(min=1e-6)

        st["q"], st["k"] = unit(*lead, Hk, dk).to(dt), unit(*lead, Hk, dk).to(dt)
        st["v"] = torch.nn.functional.silu(normal(*lead, Hv, dv)).to(dt)
        # log decays as the mixer makes its gates: sigmoid(N(3, 1)) to a power per head; write strengths sigmoid(N(0, 1))
        e = torch.exp(torch.rand(Hv, generator=g, device=DEV) * 2 - 1)
        st["g"] = (torch.nn.functional.logsigmoid(normal(*lead, Hv) + 3.0) * e).to(dt)
        st["beta"] = torch.sigmoid(normal(*lead, Hv)).to(dt)
        n = case.get("N", 0) or B
        st["S0"] = 0.3 * normal(n, Hv, dv, dk) if op == "gdr_step" or case["S0"] else None
        if op == "gdr_step":
            st["S1"] = torch.empty_like(st["S0"])
            return st
        if op == "gdr_train":
            st["dO"] = normal(*lead, Hv, dv).to(dt)
            st["dST"] = 0.3 * normal(n, Hv, dv, dk) if case["S0"] else None
        st["cu"] = torch.tensor(_cu(case), dtype=torch.int32, device=DEV) if case["N"] else None
        return st
    held, new = _held(case), _new(case)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    rows, Hq, Hkv, d, page = cu[-1], case["Hq"], case["Hkv"], case["d"], case["page"]
    st["lens"] = torch.tensor(held, dtype=torch.int32, device=DEV)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV) if case["n"] else None
    st["q"] = normal(rows, Hq, d).to(dt) if Hq else None
    tokens = [a + n for a, n in zip(held, new)]
    if op == "paged_append":
        st["k"], st["v"] = normal(rows, Hkv, d).to(dt), normal(rows, Hkv, d).to(dt)
        st["table"], used = _table(case, tokens, 0, g)
        rot = case["rot"]
        st["freqs"] = torch.tensor([10000.0 ** (-2.0 * j / rot) for j in range(rot // 2)], dtype=torch.float64,
                                   device=DEV) if rot else None
    else:
        P = case["P"]
        n = -(-P // page)
        st["ptable"] = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
        st["table"], used = _table(case, tokens, n, g)
        used += n
    st["kp"], st["vp"] = normal(used, page, Hkv, d).to(dt), normal(used, page, Hkv, d).to(dt)
    if op == "prefix_attn" and own:    # a serving loop keeps the workspace of its steps
        st["ws"] = _kd().prefix_attn_workspace(st["q"], st["kp"], case["P"], st["table"])
    return st


# ----------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    kd, case, op = _kd(), st["case"], st["case"]["op"]
    if op == "gdr_fwd":
        o, ST = kd.gdr_fwd(st["q"], st["k"], st["v"], st["g"], st["beta"], st["S0"], cu_seqlens=st["cu"])
        return dict(o=o, ST=ST)
    if op == "gdr_train":
        o, ST, saved = kd.gdr_fwd(st["q"], st["k"], st["v"], st["g"], st["beta"], st["S0"], cu_seqlens=st["cu"],
                                  return_state=case["S0"], save_states=True)
        gr = kd.gdr_bwd(st["q"], st["k"], st["v"], st["g"], st["beta"], saved, st["dO"], st["dST"],
                        cu_seqlens=st["cu"], return_dS0=case["S0"])
        out = dict(o=o, dq=gr["dq"], dk=gr["dk"], dv=gr["dv"], dg=gr["dg"], dbeta=gr["dbeta"])
        if case["S0"]:
            out.update(ST=ST, dS0=gr["dS0"])
        return out
    if op == "gdr_step":
        o = kd.gdr_step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["S0"], S_out=st["S1"])
        return dict(o=o, S=st["S1"])
    if op == "paged_append":
        q = kd.paged_append(st["k"], st["v"], st["kp"], st["vp"], st["table"], st["lens"], q=st["q"],
                            cu_seqlens=st["cu"], freqs=st["freqs"], layout=case["layout"], offset=case["offset"])
        out = dict(k_pages=st["kp"], v_pages=st["vp"])
        if q is not None:
            out["q"] = q
        return out
    return dict(o=kd.prefix_attn(st["q"], st["kp"], st["vp"], st["ptable"], case["P"], st["table"], st["lens"],
                                 cu_seqlens=st["cu"], workspace=st["ws"]))


CHUNK = 64


def _plain_gdr(q, k, v, g, beta, S, scale):
    """q, k [n, Hv, T, dk], v [n, Hv, T, dv], g, beta [n, Hv, T], S [n, Hv, dk, dv] in 32 bits, chunk by chunk."""
    n, H, T, dk = q.shape
    C, NC = CHUNK, -(-T // CHUNK)

    def chunks(x):
        x = torch.cat([x, x.new_zeros(*x.shape[:2], NC * C - T, *x.shape[3:])], 2)
        return x.view(n, H, NC, C, *x.shape[3:])

    q, k, v, g, beta = (chunks(x) for x in (q * scale, k, v, g, beta))
    b = g.cumsum(-1)
    low = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    decay = torch.exp((b[..., :, None] - b[..., None, :]).masked_fill(~low, float("-inf")))
    kt = k.transpose(-1, -2).contiguous()
    x = -(beta[..., None] * decay * torch.matmul(k, kt)).tril(-1)
    inv = torch.eye(C, device=q.device) + x
    for _ in range(5):           # (I - x)^-1 = (I + x) (I + x^2) (I + x^4) ...
        x = torch.matmul(x, x)
        inv = inv + torch.matmul(inv, x)
    attn = torch.matmul(q, kt) * decay
    eb = torch.exp(b)[..., None]
    w, u = torch.matmul(inv, k * eb * beta[..., None]), torch.matmul(inv, v * beta[..., None])
    qe, last = q * eb, b[..., -1:]
    ke = (k * torch.exp(last - b)[..., None]).transpose(-1, -2).contiguous()
    o = []
    for c in range(NC):
        un = u[:, :, c] - torch.matmul(w[:, :, c], S)
        o.append(torch.matmul(qe[:, :, c], S) + torch.matmul(attn[:, :, c], un))
        S = torch.exp(last[:, :, c, :, None]) * S + torch.matmul(ke[:, :, c], un)
    return torch.cat(o, 2)[:, :, :T], S


def _plain_gdr_case(st):
    case, dt = st["case"], _dt(st["case"])
    Hk, Hv, dk, dv = (case[n] for n in ("Hk", "Hv", "dk", "dv"))
    train = case["op"] == "gdr_train"
    leaves = [st[n].float() for n in ("q", "k", "v", "g", "beta")]
    n = case["N"] or case["B"]
    S0 = st["S0"] if st["S0"] is not None else torch.zeros(n, Hv, dv, dk, device=DEV)
    if train:
        leaves, S0 = [x.clone().requires_grad_() for x in leaves], S0.clone().requires_grad_()
    with torch.set_grad_enabled(train):
        x = leaves
        if case["N"]:             # the sequences side by side, padded by tokens that change nothing
            cu = _cu(case)
            long = max(b - a for a, b in zip(cu[:-1], cu[1:]))
            at = st["cu"][:-1].long()[:, None] + torch.arange(long, device=DEV)[None]
            live = at < st["cu"][1:].long()[:, None]
            at = at.clamp(max=case["T"] - 1)
            x = [t[at] * live.view(n, long, *[1] * (t.dim() - 1)) for t in x]
        q, k, v, g, b = (t.transpose(1, 2) for t in x)
        q, k = (t.repeat_interleave(Hv // Hk, 1) for t in (q, k))
        o, S = _plain_gdr(q, k, v, g, b, S0.transpose(-1, -2), 1.0 / math.sqrt(dk))
        o, ST = o.transpose(1, 2), S.transpose(-1, -2)
        if case["N"]:
            o = o[live]
    out = dict(o=o.detach().to(dt))
    if case["op"] == "gdr_fwd" or case["S0"]:
        out["ST"] = ST.detach().contiguous()
    if not train:
        return out
    ys, dys = [o], [st["dO"].float()]
    if case["S0"]:
        ys, dys = ys + [ST], dys + [st["dST"]]
    gr = torch.autograd.grad(ys, leaves + [S0], dys)
    out.update({"d" + m: t.to(dt) for m, t in zip(("q", "k", "v", "g", "beta"), gr)})
    if case["S0"]:
        out["dS0"] = gr[5]
    return out


def _plain_step(st):
    case = st["case"]
    G = case["Hv"] // case["Hk"]
    q, k = (st[n].float().repeat_interleave(G, 1) for n in ("q", "k"))
    v, g, beta = (st[n].float() for n in ("v", "g", "beta"))
    S = torch.exp(g)[..., None, None] * st["S0"]
    u = beta[..., None] * (v - (S * k[:, :, None]).sum(-1))
    st["S1"].copy_(S + u[..., None] * k[:, :, None])
    o = (st["S1"] * q[:, :, None]).sum(-1) / math.sqrt(case["dk"])
    return dict(o=o.to(_dt(case)), S=st["S1"])


def _rotate(x, ang, layout):
    """x [rows, H, d] in 32 bits; ang [rows, rot / 2] in 64 bits."""
    n = ang.shape[-1]
    c, s = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    r, rest = x[..., :2 * n], x[..., 2 * n:]
    if layout == "half":
        a, b = r[..., :n], r[..., n:]
        return torch.cat([a * c - b * s, b * c + a * s, rest], -1)
    a, b = r[..., 0::2], r[..., 1::2]
    return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), rest], -1)


def _owners(st, rows):
    """Request and own position of every row."""
    if st["cu"] is None:
        b = torch.arange(rows, device=DEV)
        return b, st["lens"].long()
    r = torch.arange(rows, device=DEV)
    b = torch.searchsorted(st["cu"][1:].long(), r, right=True)
    return b, st["lens"].long()[b] + r - st["cu"].long()[b]


def _plain_append(st):
    case, dt = st["case"], _dt(st["case"])
    b, at = _owners(st, st["k"].shape[0])
    k, q = st["k"].float(), st["q"].float() if case["Hq"] else None
    if case["rot"]:
        ang = (at + case["offset"]).double()[:, None] * st["freqs"]
        k = _rotate(k, ang, case["layout"])
        q = _rotate(q, ang, case["layout"]) if case["Hq"] else None
    page = st["table"].long()[b, at // case["page"]]
    st["kp"][page, at % case["page"]] = k.to(dt)
    st["vp"][page, at % case["page"]] = st["v"]
    out = dict(k_pages=st["kp"], v_pages=st["vp"])
    if case["Hq"]:
        out["q"] = q.to(dt)
    return out


def _plain_prefix(st):
    case, dt = st["case"], _dt(st["case"])
    B, Hq, Hkv, d, P, page = (case[n] for n in ("B", "Hq", "Hkv", "d", "P", "page"))
    G, q = Hq // Hkv, st["q"].float()
    rows = q.shape[0]
    owner, at = _owners(st, rows)
    # the queries of all requests side by side against the prefix
    qh = q.view(rows, Hkv, G, d).permute(1, 0, 2, 3).reshape(Hkv, rows * G, d)
    kp = st["kp"][st["ptable"].long()].flatten(0, 1)[:P].float().permute(1, 2, 0).contiguous()
    vp = st["vp"][st["ptable"].long()].flatten(0, 1)[:P].float().permute(1, 0, 2).contiguous()
    # and each request's own, padded to the most new tokens
    new = _new(case)
    most, width = max(new), st["table"].shape[1] * page
    slot = torch.arange(rows, device=DEV) - (st["cu"].long()[owner] if case["n"] else owner)
    qb = q.new_zeros(B, most, Hkv, G, d)
    qb[owner, slot] = q.view(rows, Hkv, G, d)
    pos = torch.full((B, most), -1, device=DEV)
    pos[owner, slot] = at
    pages = st["table"].long().clamp(min=0)
    kb = st["kp"][pages].flatten(1, 2).float().permute(0, 2, 3, 1).contiguous()     # [B, Hkv, d, width]
    vb = st["vp"][pages].flatten(1, 2).float().permute(0, 2, 1, 3).contiguous()
    qb = qb.permute(0, 2, 1, 3, 4).reshape(B, Hkv, most * G, d)
    hidden = torch.arange(width, device=DEV) > pos[:, None, :, None, None]          # [B, 1, most, 1, width]
    sb = torch.matmul(qb, kb).view(B, Hkv, most, G, width).masked_fill(hidden, float("-inf")) / math.sqrt(d)
    sp = torch.matmul(qh, kp).view(Hkv, rows, G, P) / math.sqrt(d)
    top = sb.permute(0, 2, 1, 3, 4)[owner, slot].amax(-1).transpose(0, 1)            # [Hkv, rows, G]
    if P:
        top = torch.maximum(top, sp.amax(-1))
    mb = sb.new_zeros(B, most, Hkv, G)
    mb[owner, slot] = top.transpose(0, 1)
    wb = torch.exp(sb - mb.permute(0, 2, 1, 3)[..., None])
    ob = torch.matmul(wb.view(B, Hkv, most * G, width), vb).view(B, Hkv, most, G, d).permute(0, 2, 1, 3, 4)[owner, slot]
    l = wb.sum(-1).permute(0, 2, 1, 3)[owner, slot]                                  # [rows, Hkv, G]
    wp = torch.exp(sp - top[..., None])
    op = torch.matmul(wp.view(Hkv, rows * G, P), vp).view(Hkv, rows, G, d).transpose(0, 1)
    l = l + wp.sum(-1).transpose(0, 1)
    return dict(o=((ob + op) / l[..., None]).reshape(rows, Hq, d).to(dt))


def _run_plain(st):
    op = st["case"]["op"]
    if op == "gdr_step":
        return _plain_step(st)
    if op.startswith("gdr"):
        return _plain_gdr_case(st)
    return _plain_append(st) if op == "paged_append" else _plain_prefix(st)


# ------------------------------------------------------------- the least work
def work(case):
    op, es = case["op"], _es(case)
    if op.startswith("gdr"):
        B, Hk, Hv, dk, dv = (case[n] for n in ("B", "Hk", "Hv", "dk", "dv"))
        rows, n = B * case.get("T", 1), case.get("N", 0) or B
        ins, outs, state = rows * (2 * Hk * dk + Hv * (dv + 2)) * es, rows * Hv * dv * es, 4 * n * Hv * dk * dv
        # a token: S k, the update and S q (2 dk dv each), and as much for each of the gradients' six
        if op == "gdr_step":
            return dict(bytes=ins + outs + 2 * state, flops=7 * rows * Hv * dk * dv)
        if op == "gdr_fwd":
            return dict(bytes=ins + outs + state * (2 if case["S0"] else 1), flops=6 * rows * Hv * dk * dv)
        return dict(bytes=2 * ins + 2 * outs + state * (4 if case["S0"] else 0), flops=20 * rows * Hv * dk * dv)
    held, new = _held(case), _new(case)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    rows = sum(new)
    if op == "paged_append":
        n = rows * (Hq + 2 * Hkv) * d
        return dict(bytes=2 * es * n + 4 * rows, flops=3 * rows * (Hq + Hkv) * max(case["rot"], 1))
    P = case["P"]
    pairs = sum(n * (P + a) + n * (n + 1) // 2 for a, n in zip(held, new))
    keys = P + sum(a + n for a, n in zip(held, new) if n)
    return dict(bytes=2 * es * d * (Hkv * keys + Hq * rows), flops=4 * d * Hq * pairs)


# ------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op.startswith("gdr"):
        return _exact_gdr(case, st)
    held, new = _held(case), _new(case)
    first, page = 0, case["page"]
    table = st["table"].tolist()
    if op == "paged_append":
        kc, vc = st["kp"].double(), st["vp"].double()
        q = st["q"].double() if case["Hq"] else None
        for b, (p, n) in enumerate(zip(held, new)):
            at = torch.arange(p, p + n, device=DEV)
            r = slice(first, first + n)
            where = torch.tensor([table[b][i // page] for i in range(p, p + n)], dtype=torch.long, device=DEV)
            k = st["k"][r].double()
            if case["rot"]:
                turn = torch.exp(1j * ((at + case["offset"]).double()[:, None, None] * st["freqs"]))
                k = _exact_turn(k, turn, case["layout"])
                if case["Hq"]:
                    q[r] = _exact_turn(q[r], turn, case["layout"])
            kc[where, at % page], vc[where, at % page] = k, st["v"][r].double()
            first += n
        out = dict(k_pages=kc, v_pages=vc)
        if case["Hq"]:
            out["q"] = q
        return out
    G, P = case["Hq"] // case["Hkv"], case["P"]
    if sum(new) * case["Hq"] * (P + case["hi"]) > 3 << 30:
        return None
    o = torch.empty(st["q"].shape, dtype=torch.float64, device=DEV)
    pt = st["ptable"].tolist()
    for b, (p, n) in enumerate(zip(held, new)):
        if n == 0:
            continue
        spots = [(pt[i // page], i % page) for i in range(P)] + [(table[b][i // page], i % page) for i in range(p + n)]
        where, off = torch.tensor(spots, device=DEV).unbind(1)
        late = torch.arange(P + p + n, device=DEV)[None] > torch.arange(P + p, P + p + n, device=DEV)[:, None]
        for h in range(case["Hq"]):
            kk, vv = st["kp"][where, off, h // G].double(), st["vp"][where, off, h // G].double()
            s = (st["q"][first:first + n, h].double() @ kk.T) / math.sqrt(case["d"])
            o[first:first + n, h] = torch.softmax(s.masked_fill(late, -math.inf), 1) @ vv
        first += n
    return dict(o=o)


def _exact_turn(x, turn, layout):
    y, n = x.clone(), turn.shape[-1]
    first = torch.arange(n, device=DEV) * (1 if layout == "half" else 2)
    second = first + (n if layout == "half" else 1)
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_gdr(case, st):
    # token by token; the states of a stretch are made again on the way back
    G = case["Hv"] // case["Hk"]
    scale, op = 1.0 / math.sqrt(case["dk"]), case["op"]
    q, k, v, g, beta = (st[n].double() for n in ("q", "k", "v", "g", "beta"))
    if op == "gdr_step":
        q, k, v, g, beta = (t[:, None] for t in (q, k, v, g, beta))
    packed = bool(case.get("N"))
    if packed:
        q, k, v, g, beta = (t[None] for t in (q, k, v, g, beta))
    q, k = q.repeat_interleave(G, 2), k.repeat_interleave(G, 2)
    decay = torch.exp(g)[..., None, None]
    n = case.get("N", 0) or case["B"]
    S0 = st["S0"].double() if st["S0"] is not None else \
        torch.zeros(n, case["Hv"], case["dv"], case["dk"], dtype=torch.float64, device=DEV)
    spans = [(slice(0, 1), slice(i, i + 1), a, b) for i, (a, b) in enumerate(zip(_cu(case)[:-1], _cu(case)[1:]))] \
        if packed else [(slice(None), slice(None), 0, q.shape[1])]
    if op == "gdr_train" and sum(b - a for _, _, a, b in spans) > 12000:
        return None
    o, ST = torch.empty_like(v), S0.clone()
    gr = {m: torch.zeros_like(t) for m, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta))}
    dS0 = torch.zeros_like(S0)
    if op == "gdr_train":
        dO = st["dO"].double()
        dO = dO[None] if packed else dO
        dST = st["dST"].double() if st["dST"] is not None else torch.zeros_like(S0)

    def token(S, r, t):
        Sb = decay[r, t] * S
        u = beta[r, t][..., None] * (v[r, t] - (Sb @ k[r, t][..., None])[..., 0])
        return Sb, u, torch.addcmul(Sb, u[..., None], k[r, t][..., None, :])

    for r, s, a, b in spans:
        S, kept = S0[s], {}
        for t in range(a, b):
            if (t - a) % 64 == 0:
                kept[t] = S
            S = token(S, r, t)[2]
            o[r, t] = scale * (S @ q[r, t][..., None])[..., 0]
        ST[s] = S
        if op != "gdr_train":
            continue
        dS = dST[s].clone()
        for start in sorted(kept, reverse=True):
            states = [kept.pop(start)]
            for t in range(start, min(start + 64, b) - 1):
                states.append(token(states[-1], r, t)[2])
            for t in reversed(range(start, min(start + 64, b))):
                before = states.pop()
                Sb, u, S = token(before, r, t)
                do = dO[r, t][..., None]
                gr["q"][r, t] = scale * (do * S).sum(-2)
                dS = dS + scale * do * q[r, t][..., None, :]
                du = (dS @ k[r, t][..., None])[..., 0]
                gr["v"][r, t] = beta[r, t][..., None] * du
                gr["beta"][r, t] = (du * (v[r, t] - (Sb @ k[r, t][..., None])[..., 0])).sum(-1)
                bu = gr["v"][r, t][..., None]
                gr["k"][r, t] = (dS * u[..., None]).sum(-2) - (Sb * bu).sum(-2)
                dS = decay[r, t] * (dS - bu * k[r, t][..., None, :])
                gr["g"][r, t] = (dS * before).sum((-1, -2))
        dS0[s] = dS
    if op == "gdr_step":
        return dict(o=o[:, 0], S=ST)
    lose = (lambda t: t[0]) if packed else (lambda t: t)
    out = dict(o=lose(o))
    if op == "gdr_fwd" or case["S0"]:
        out["ST"] = ST
    if op == "gdr_train":
        for m in ("q", "k"):
            gr[m] = gr[m].unflatten(2, (case["Hk"], G)).sum(3)
        out.update({"d" + m: lose(t) for m, t in gr.items()})
        if case["S0"]:
            out["dS0"] = dS0
    return out
