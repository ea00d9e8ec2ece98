"""The gated delta rule in the kernels' chunks with exactly their roundings to bf16 and nothing else (numpy, 64 bits for
everything between), so that tests can tell what each of the kept remainders is worth.

A matrix that enters a bf16 product is a sum of parts: the rounded matrix, its rounded remainder, and so on.
`Keep` says how many there are of each: what the kernels hold, or less for a mistake planted on purpose."""
from dataclasses import dataclass

import numpy as np


@dataclass
class Keep:
    added: int = 3      # parts of what is added to a state: U before A and after it, dU, X, and dO with its factor
    state: int = 2      # of a state and of its gradient where they meet K and Q
    A: int = 2
    P_bwd: int = 2      # of P in dU (in o it has one)
    X: int = 2          # of X and U in the chunk's gradients
    U: int = 2
    segment: int = 0    # chunks of a segment (0: not cut)
    plant: str = ""     # of the segments' maps: "zero", "transposed", "order"


def bf16(x):
    """Nearest bf16, ties to even."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(np.float64)


def parts(x, n):
    out = []
    for _ in range(n):
        out.append(bf16(x))
        x = x - out[-1]
    return out


def twice(a, x):
    """a x for sums of parts, without products of two remainders."""
    return a[0] @ sum(x) + sum(a[1:], 0 * a[0]) @ x[0]


class Chunks:
    """One head: q, k [T, dk], v [T, dv], g, beta [T]."""

    def __init__(self, q, k, v, g, beta, scale, keep=Keep()):
        self.q, self.k, self.v, self.g, self.beta, self.scale, self.keep = q, k, v, g, beta, scale, keep
        self.at = [slice(i, min(i + 64, len(q))) for i in range(0, len(q), 64)]
        self.mats = [self.matrices(s) for s in self.at]

    def matrices(self, s):
        b = np.cumsum(np.maximum(self.g[s], -120.0))
        low = np.tril(np.ones((len(b), len(b)), bool))
        gam = np.where(low, np.exp(np.where(low, b[:, None] - b[None], 0.0)), 0.0)
        K, Q, be = self.k[s], self.q[s], self.beta[s]
        A = np.linalg.inv(np.eye(len(b)) + np.tril(be[:, None] * gam * (K @ K.T), -1))
        P = self.scale * gam * (Q @ K.T)
        return dict(gam=gam, A=parts(A, self.keep.A), P=parts(P, 2), be=be[:, None], bb=(be * np.exp(b))[:, None],
                    bc=np.exp(b[-1] - b)[:, None], se=self.scale * np.exp(b)[:, None], eC=np.exp(b[-1]))

    def through(self, c, S, v, out=None):
        """The state behind chunk c from the one before it; outputs to `out`."""
        K, m, kp = self.k[self.at[c]], self.mats[c], self.keep
        s = parts(S, kp.state)
        U = twice(m["A"], parts(m["be"] * v - m["bb"] * (K @ sum(s).T), kp.added))
        if out is not None:
            out[self.at[c]] = m["se"] * (self.q[self.at[c]] @ sum(s).T) + m["P"][0] @ sum(parts(U, 2))
        return m["eC"] * S + sum(parts(m["bc"] * U, kp.added)).T @ K

    def forward(self, S0):
        """o and the states before every chunk and behind the last."""
        kp, n = self.keep, len(self.at)
        o, S, states = np.zeros(self.v.shape), S0, []
        entering = {0: S0}
        if kp.segment:
            for c0 in range(0, n - kp.segment, kp.segment):
                N = S0 if c0 == 0 else 0 * S0
                M = np.eye(S0.shape[1])
                for c in range(c0, c0 + kp.segment):
                    N, M = self.through(c, N, self.v[self.at[c]]), self.through(c, M, 0.0)
                if c0 > 0:
                    M = {"zero": 0 * M, "transposed": M.T}.get(kp.plant, M)
                    N = N + entering[c0 if kp.plant != "order" else max(c0 - kp.segment, 0)] @ M
                entering[c0 + kp.segment] = N
        for c in range(n):
            S = entering.get(c, S)
            states.append(S)
            S = self.through(c, S, self.v[self.at[c]], o)
        return o, states + [S]

    def backward(self, states, dO, dST):
        """dq, dk, dv, dg, dbeta and dS0 from the states before every chunk."""
        kp, a = self.keep, np.sum
        dq, dk, dv = (np.zeros(x.shape) for x in (self.q, self.k, self.v))
        dg, dbeta, dS = np.zeros(self.g.shape), np.zeros(self.g.shape), dST
        for c in reversed(range(len(self.at))):
            s, m = self.at[c], self.mats[c]
            Q, K, V, D = self.q[s], self.k[s], self.v[s], dO[s]
            At = [x.T for x in m["A"]]
            d = parts(dS, kp.state)
            dU = m["bc"] * (K @ sum(d).T) + sum(m["P"][:kp.P_bwd]).T @ D
            X = twice(At, parts(dU, kp.added))
            nextS = m["eC"] * dS + sum(parts(m["se"] * D, kp.added)).T @ Q - sum(parts(m["bb"] * X, kp.added)).T @ K
            dv[s] = m["be"] * sum(parts(X, 2))
            # the chunk's gradients: kept states rounded
            S0, d1, x = bf16(states[c]), d[0], parts(X, kp.X)
            u = parts(twice(m["A"], parts(m["be"] * V - m["bb"] * (K @ S0.T), 2)), kp.U)
            dP = D @ sum(u).T
            dT = x[0] @ sum(u).T + sum(x[1:], 0 * x[0]) @ u[0].T
            e, y = self.scale * m["gam"] * dP, -np.tril(m["gam"], -1) * dT
            f = bf16(m["be"] * y)
            qi, ke, ks = m["se"] * (D @ S0), -m["bb"] * (sum(x) @ S0), m["bc"] * (sum(u) @ d1)
            dq[s] = bf16(e) @ K + qi
            dk[s] = bf16(e).T @ Q + (f + f.T) @ K + ks + ke
            dbeta[s] = np.diag(dT) / self.beta[s]
            both = e * (Q @ K.T) + m["be"] * y * (K @ K.T)
            ys = a(K * ks, 1)
            db = a(both, 1) - a(both, 0) + a(Q * qi, 1) + a(K * ke, 1) - ys
            dg[s] = np.cumsum(db[::-1])[::-1] + a(ys) + m["eC"] * a(S0 * d1)
            dS = nextS
        return dict(dq=dq, dk=dk, dv=dv, dg=dg, dbeta=dbeta, dS0=dS)


def problem(T, dk, dv, gates, seed, unit=bf16):
    """One head's inputs in the tensors' type (gates in fp32), its states and the gradients that come in.  gates: "fast"
    (a chunk forgets nearly all), "slow" (the first state still matters at the end)."""
    r = np.random.default_rng(seed)
    f32 = lambda x: np.asarray(x, np.float32).astype(np.float64)  # noqa: E731
    k = r.normal(size=(T, dk))
    x = dict(q=unit(r.normal(size=(T, dk)) / np.sqrt(dk)), k=unit(0.99 * k / np.linalg.norm(k, axis=1, keepdims=True)),
             v=unit(r.normal(size=(T, dv))))
    if gates == "fast":
        x["g"], x["beta"] = f32(-np.log1p(np.exp(-r.normal(size=T) - 3))), f32(1 / (1 + np.exp(-r.normal(size=T))))
    else:
        x["g"], x["beta"] = f32(-r.uniform(0, 2 / 4096, size=T)), f32(r.uniform(0.001, 0.04, size=T))
    return x, f32(r.normal(size=(dv, dk))), unit(r.normal(size=(T, dv))), f32(r.normal(size=(dv, dk)))


def off(got, ref):
    """Relative to the reference, in the root of the sum of squares."""
    return float(np.linalg.norm(np.asarray(got, np.float64) - ref) / np.linalg.norm(ref))
