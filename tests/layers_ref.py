"""References of the layers beside the mixer in 64 bits (numpy), with bounds on what the kernels' arithmetic may
add.  u is the unit rounding error of the tensors' type (2^-8 for bf16, 2^-24 for fp32), W = 2^-24 that of the fp32
arithmetic."""
import numpy as np

W = 2.0 ** -24


def unit(dtype):
    return 2.0 ** -8 if dtype == "bf16" else W


# ------------------------------------------------- gated linear recurrence
def glr(x, f, i, h0):
    """h [B, T, D] with the state before every token in h[:, t] of the [B, T + 1, D] result."""
    B, T, D = x.shape
    h = np.zeros((B, T + 1, D))
    if h0 is not None:
        h[:, 0] = h0
    for t in range(T):
        h[:, t + 1] = f[:, t] * h[:, t] + (x[:, t] if i is None else i[:, t] * x[:, t])
    return h


def glr_bwd(x, f, i, h, dh, dhT):
    """g (gradient of h_t through all its uses), dx, df, di, dh0 from h = glr(...)."""
    B, T, D = x.shape
    g = np.zeros((B, T, D))
    m = np.zeros((B, D)) if dhT is None else dhT.copy()
    for t in reversed(range(T)):
        g[:, t] = dh[:, t] + m
        m = f[:, t] * g[:, t]
    return g, g if i is None else i * g, g * h[:, :-1], None if i is None else x * g, m


def glr_bounds(x, f, i, h0, dh=None, dhT=None):
    """Bounds on the error of the fp32 state and of g.  One step rounds its product and its sum (2 W of the magnitudes
    H that add up in it); a state carried over a tile of 128 tokens is a product of up to 128 gates times the
    entering state, each factor rounded once."""
    a = np.abs
    H = glr(a(x), a(f), None if i is None else a(i), None if h0 is None else a(h0))
    eh = glr(3 * W * H[:, 1:], a(f), None, None) + 136 * W * H
    if dh is None:
        return eh
    G = glr_bwd(a(x), a(f), None, H, a(dh), None if dhT is None else a(dhT))[0]
    eg = glr_bwd(a(x), a(f), None, H, 3 * W * G, None)[0] + 136 * W * G
    return eh, eg, H, G


# ---------------------------------------------------------- rotary positions
def rope(x, pos, freqs, layout, scale, inverse=False):
    """x [B, T, H, d], pos [B, T] integers; freqs float64."""
    n = len(freqs)
    ang = np.longdouble(pos)[..., None, None] * np.longdouble(freqs)
    c, s = np.cos(ang) * scale, np.sin(ang) * scale * (-1 if inverse else 1)
    y = np.longdouble(x).copy()
    ia = np.arange(n) if layout == "half" else 2 * np.arange(n)
    ib = ia + (n if layout == "half" else 1)
    a, b = np.longdouble(x[..., ia]), np.longdouble(x[..., ib])
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    # both products, their sum, and the sine and cosine (fraction of a turn to fp32: 2 pi 2^-25; the functions and
    # their scaling: 4 W) round
    e = np.zeros_like(x)
    mag = scale * (np.abs(x[..., ia]) + np.abs(x[..., ib]))
    e[..., ia] = e[..., ib] = 12 * W * mag
    return np.float64(y), e


# ------------------------------------------------- sliding-window attention
def visible(Tq, Tk, window, sinks):
    p = Tk - Tq + np.arange(Tq)[:, None]
    s = np.arange(Tk)[None]
    return (s <= p) & ((p - s < window) | (s < sinks))


def attention(q, k, v, window, sinks, scale, dO=None, u=W):
    """One head: q [Tq, d], k, v [Tk, d].  Returns dicts of values and of error bounds (o, lse, dq, dk, dv)."""
    d = q.shape[1]
    vis = visible(len(q), len(k), window, sinks)
    some = vis.any(1)
    s = np.where(vis, (q @ k.T) * scale, -np.inf)
    m = np.where(some, s.max(1, initial=-np.inf), 0.0)
    e = np.where(vis, np.exp(np.where(vis, s - m[:, None], 0.0)), 0.0)
    l = e.sum(1)
    P = e / np.where(some, l, 1.0)[:, None]
    with np.errstate(divide="ignore"):
        lse = np.where(some, m + np.log(np.where(some, l, 1.0)), -np.inf)
    o = P @ v
    a = np.abs
    # a score: d products and sums of fp32, its scaling, and the argument and value of exp2; as a relative error of
    # every weight (and of their sum)
    smax = a(s[vis]).max() if vis.any() else 0.0
    ds_ = 2 * W * (d * (np.where(vis, a(q) @ a(k).T, 0.0)).max(initial=0.0) * scale + 8 * smax + 8)
    n = max(int(vis.sum(1).max(initial=1)), 1)
    # weights rounded to the type (u), summed over n keys in fp32, the result rounded to the type (u)
    eo = (u + 2 * ds_ + n * W) * (P @ a(v)) + u * a(o)
    val, err = dict(o=o, lse=lse), dict(o=eo, lse=ds_ + n * W + 4 * W * (1 + np.where(some, a(lse), 0.0)))
    if dO is None:
        return val, err
    dP = dO @ v.T
    D = (dO * o).sum(1)
    dS = P * (dP - D[:, None])
    val.update(dq=scale * dS @ k, dk=scale * dS.T @ q, dv=P.T @ dO)
    # delta is taken from the o that the forward pass returned
    eD = (a(dO) * eo).sum(1) + d * W * (a(dO) * a(o)).sum(1)
    edS = (u + W) * a(dS) + P * (eD[:, None] + d * W * (a(dO) @ a(v).T) + 4 * ds_ * (a(dP) + a(D)[:, None]))
    nq = max(int(vis.sum(0).max(initial=1)), 1)
    mdS = a(dS) + edS
    err.update(dq=scale * (edS + n * W * mdS) @ a(k) + u * a(val["dq"]),
               dk=scale * (edS + nq * W * mdS).T @ a(q) + u * a(val["dk"]),
               dv=(u + 4 * ds_ + nq * W) * (P.T @ a(dO)) + u * a(val["dv"]))
    return val, err


def attention_heads(q, k, v, window, sinks, scale, dO=None, u=W):
    """[T, H, d] tensors with grouped heads; lse [Hq, Tq].  dk, dv are sums over a group's query heads."""
    Tq, Hq, d = q.shape
    Tk, Hkv, _ = k.shape
    G = Hq // Hkv
    names = ("o", "dq", "dk", "dv") if dO is not None else ("o",)
    shp = dict(o=q.shape, dq=q.shape, dk=k.shape, dv=k.shape)
    val, err = {n: np.zeros(shp[n]) for n in names}, {n: np.zeros(shp[n]) for n in names}
    val["lse"], err["lse"] = np.zeros((Hq, Tq)), np.zeros((Hq, Tq))
    for h in range(Hq):
        a, b = attention(q[:, h], k[:, h // G], v[:, h // G], window, sinks, scale,
                         None if dO is None else dO[:, h], u)
        for src, dst in ((a, val), (b, err)):
            dst["lse"][h] = src["lse"]
            for n in names:
                if n in ("dk", "dv"):
                    dst[n][:, h // G] += src[n]
                else:
                    dst[n][:, h] = src[n]
    return val, err


# ---------------------------------------------------------------- decoding
def slot(s, sinks, cap):
    return s if s < sinks else sinks + (s - sinks) % (cap - sinks)


def seen(p, window, sinks):
    return sorted(set(range(min(sinks, p + 1))) | set(range(max(0, p - window + 1), p + 1)))
