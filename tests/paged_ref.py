"""Plain paged cache and attention over a shared prefix in 64 bits (numpy), with bounds on what the kernels' arithmetic
may add.  u is the unit rounding error of the tensors' type, W = 2^-24 that of fp32."""
import numpy as np

W = 2.0 ** -24


def rows_of(lens, cu, T):
    """(sequence, own position) of every row: None for a row that no sequence holds, position None for an unused one."""
    if cu is None:
        return [(b, None if lens[b] < 0 else int(lens[b])) for b in range(T)]
    out = [None] * T
    for b in range(len(lens)):
        for r in range(cu[b], cu[b + 1]):
            out[r] = (b, None if lens[b] < 0 else int(lens[b]) + r - int(cu[b]))
    return out


def slot(table, page, pages, i):
    """(page id, slot) of own token i, None where there is no page."""
    if i // page >= len(table) or not 0 <= table[i // page] < pages:
        return None
    return int(table[i // page]), i % page


def keys_of(row, lens, cu, ptable, prefix, table, page, pages):
    """Slots that a row sees: the prefix's, then its sequence's own up to itself (page ids clamped)."""
    b, p = row
    at = [(min(max(int(ptable[i // page]), 0), pages - 1), i % page) for i in range(prefix)]
    n = min(p + 1, len(table[b]) * page)
    return at + [(min(max(int(table[b][i // page]), 0), pages - 1), i % page) for i in range(n)]


def attend(q, k, v, scale, u):
    """One query [d] over its keys k, v [n, d]: o, its bound, lse, its bound."""
    d, n = k.shape[1], len(k)
    if n == 0:
        return np.zeros(d), np.zeros(d), -np.inf, 0.0
    a = np.abs
    s = (k @ q) * scale
    m = s.max()
    e = np.exp(s - m)
    P = e / e.sum()
    o, lse = P @ v, m + np.log(e.sum())
    # a score: d products and sums of fp32, its scaling, and the argument and value of exp2; as a relative error of
    # every weight and of their sum, in the parts and again where parts are joined
    ds = 2 * W * (d * (a(k) @ a(q)).max() * scale + 8 * a(s).max() + 16)
    # weights rounded to the type (u), summed over n keys in fp32 (64 parts more), the result rounded to the type (u)
    eo = (u + 2 * ds + (n + 64) * W) * (P @ a(v)) + u * a(o)
    return o, 1.01 * eo, lse, 1.01 * (ds + (n + 64) * W + 4 * W * (1 + a(lse)))
