"""The gated delta rule token by token in 64 bits (numpy), its gradients, and bounds on what the kernels' chunked
arithmetic may add.

Bounds: u is half a step of the tensors' type (2^-8 for bf16), W = 2^-24 that of the fp32 sums (at most dk + dv + 128
terms in any of them).  The forward pass holds states, U and A to a rounded part and its remainder (each at most 2^-9 of
the value before it, what is left 2^-17, and the product of two remainders, 2^-18, is left out: below 2^-16 a use);
P is rounded to the type, and so are, in the gradients, the states that are kept, X, U, E and F."""
import numpy as np

W = 2.0 ** -24


def tokens(q, k, v, g, beta, S0, scale):
    """One head: q, k [T, dk], v [T, dv], g, beta [T], S0 [dv, dk].  o and the states before every token (T + 1)."""
    T, S = len(q), S0.copy()
    o, states = np.zeros(v.shape), [S.copy()]
    for t in range(T):
        Sb = np.exp(g[t]) * S
        S = Sb + np.outer(beta[t] * (v[t] - Sb @ k[t]), k[t])
        o[t] = scale * S @ q[t]
        states.append(S)
    return o, states


def tokens_bwd(q, k, v, g, beta, states, dO, dST, scale):
    """dq, dk, dv, dg, dbeta, and the gradients of the states before every token (T + 1; the first is dS0)."""
    T = len(q)
    dq, dk, dv, dg, db = (np.zeros(x.shape) for x in (q, k, v, g, beta))
    dS, grads = dST.copy(), [None] * T + [dST.copy()]
    for t in reversed(range(T)):
        a = np.exp(g[t])
        Sb = a * states[t]
        r = v[t] - Sb @ k[t]
        u = beta[t] * r
        dq[t] = scale * dO[t] @ states[t + 1]
        dS = dS + scale * np.outer(dO[t], q[t])
        du = dS @ k[t]
        db[t], dv[t] = du @ r, beta[t] * du
        dk[t] = u @ dS - dv[t] @ Sb
        dSb = dS - np.outer(dv[t], k[t])
        dg[t] = a * (dSb * states[t]).sum()
        dS = a * dSb
        grads[t] = dS
    return dq, dk, dv, dg, db, grads


def chunk(q, k, v, g, beta, S0, scale):
    """Matrices of one chunk: Gam, P, A, U, W and the decays e^b, e^(bC - b)."""
    b = np.cumsum(np.maximum(g, -1e3))
    low = np.tril(np.ones((len(g), len(g)), bool))
    Gam = np.where(low, np.exp(np.where(low, b[:, None] - b[None], 0.0)), 0.0)
    A = np.linalg.inv(np.eye(len(g)) + np.tril(beta[:, None] * Gam * (k @ k.T), -1))
    eb = np.exp(b)
    Wv = v - eb[:, None] * (k @ S0.T)
    return Gam, scale * Gam * (q @ k.T), A, A @ (beta[:, None] * Wv), Wv, eb, np.exp(b[-1] - b)


def bounds(q, k, v, g, beta, states, scale, u, dO=None, grads=None):
    """Bounds without the results' own rounding: o, and with dO dq, dk, dv, dg, dbeta; then those of the states."""
    T, a = len(q), np.abs
    dk_, dv_ = q.shape[1], v.shape[1]
    w = (dk_ + dv_ + 128) * W
    eta, u = 2.0 ** -16 * (u > W) + w, u * (u > W) + w
    nc = -(-T // 64)
    names = ("o", "dq", "dk", "dv", "dg", "dbeta")
    out = {n: np.zeros(x.shape) for n, x in zip(names, (v, q, k, v, g, beta))}
    big = lambda x: a(x) + np.sqrt(np.mean(x * x)) + 1e-30  # noqa: E731
    for c in range(nc):
        s = slice(64 * c, min(64 * c + 64, T))
        Q, K, V, be = q[s], k[s], v[s], beta[s][:, None]
        S0, C = states[64 * c], s.stop - s.start
        Gam, P, A, U, Wv, eb, ec = chunk(Q, K, V, g[s], beta[s], S0, scale)
        e1, ec1 = eb[:, None], ec[:, None]
        # what the chunks before have left in the state: a few uses each, none amplified (the map of a token does not
        # lengthen anything for keys of at most length 1)
        eS = 8 * eta * (c + 1) * big(S0)
        eW = e1 * a(K) @ (eS + eta * a(S0)).T + eta * a(V)
        eU = a(A) @ (be * eW) + 8 * eta * a(A) @ (be * (a(V) + e1 * a(K) @ a(S0).T))
        out["o"][s] = u * a(P) @ a(U) + a(P) @ eU + scale * e1 * (a(Q) @ (eS + eta * a(S0)).T)
        if dO is None:
            continue
        D, dS = dO[s], grads[s.stop]
        eD = 8 * eta * (nc - c) * big(dS)
        dU = P.T @ D + ec1 * (K @ dS.T)
        edU = u * a(P).T @ a(D) + ec1 * (a(K) @ (eD + eta * a(dS)).T)
        X = A.T @ dU
        eX = a(A).T @ edU + 8 * eta * a(A).T @ (a(P).T @ a(D) + ec1 * (a(K) @ a(dS).T))
        out["dv"][s] = be * eX
        # the chunk's own pass: the kept states, X and U are rounded
        eX = eX + u * a(X)
        eS, eD = eS + u * a(S0), eD + u * a(dS)
        eW = e1 * a(K) @ (eS + w * a(S0)).T + w * a(V)
        eU = a(A) @ (be * eW) + 8 * eta * a(A) @ (be * (a(V) + e1 * a(K) @ a(S0).T)) + u * a(U)
        Gs = np.tril(Gam, -1)
        E, F = scale * Gam * (D @ U.T), be * Gs * (X @ U.T)
        eE = u * a(E) + scale * Gam * (a(D) @ eU.T + w * a(D) @ a(U).T)
        eF0 = Gs * (a(X) @ eU.T + eX @ a(U).T + w * a(X) @ a(U).T)
        eF = u * a(F) + be * eF0
        eQi = scale * e1 * (a(D) @ (eS + w * a(S0)))
        eKs = ec1 * (eU @ a(dS) + a(U) @ (eD + w * a(dS)))
        eKe = be * e1 * (eX @ a(S0) + a(X) @ (eS + w * a(S0)))
        out["dq"][s] = eE @ a(K) + eQi
        out["dk"][s] = eE.T @ a(Q) + (eF + eF.T) @ a(K) + eKs + eKe
        KK, QK = a(K) @ a(K).T, a(Q) @ a(K).T
        out["dbeta"][s] = (eX * a(Wv) + a(X) * eW).sum(1) + (eF0 * KK).sum(1)
        # dg sums thousands of roundings whose signs are independent of each other: they add in squares.  Each is at most
        # its bound x, a deviation of x / sqrt(3); six deviations of the sum
        p2 = lambda x: x * x  # noqa: E731
        rU = p2(A) @ (be ** 2 * (p2(e1 * K) @ p2(eS).T)) + p2(u * U)
        rX = p2(A).T @ (p2(u * P).T @ p2(D) + p2(ec1) * (p2(K) @ p2(eD).T)) + p2(u * X)
        rE = p2(u * E) + p2(scale * Gam) * (p2(D) @ rU.T)
        rF = p2(u * F) + p2(be * Gs) * (p2(X) @ rU.T + rX @ p2(U).T)
        rK = p2(ec1) * (rU @ p2(dS) + p2(U) @ p2(eD))
        m2 = rE * p2(Q @ K.T) + rF * p2(K @ K.T) + p2(w) * (p2(E) * p2(QK) + p2(F) * p2(KK))
        send = (p2(K) * (rK + p2(w * ec1) * (p2(U) @ p2(dS)))).sum(1)
        db = m2.sum(1) + m2.sum(0) + send + (p2(Q) * p2(scale * e1) * (p2(D) @ p2(eS))).sum(1) + \
            (p2(K) * p2(be * e1) * (rX @ p2(S0) + p2(X) @ p2(eS))).sum(1)
        end = send.sum() + eb[-1] ** 2 * (p2(eS * dS) + p2(S0 * eD)).sum()
        out["dg"][s] = 6 / np.sqrt(3) * np.sqrt(np.cumsum(db[::-1])[::-1] + end)
    eST = 8 * eta * (nc + 1) * (big(states[-1]) + np.sqrt(np.mean(v * v)))
    edS0 = None if grads is None else 8 * eta * (nc + 1) * (big(grads[0]) + np.sqrt(np.mean(dO * dO)))
    if grads is not None and u > 2 * w:      # P rounded in dU reaches the gradient of the state
        edS0 = edS0 + 4 * u * np.sqrt(np.mean(dO * dO)) + 4 * u * big(grads[0])
    return out, eST, edS0
