"""The references of the gated delta rule against each other, closed forms and differences (CPU)."""
import numpy as np
import pytest

import gdr_ref as R


def case(T, dk, dv, seed=0):
    r = np.random.default_rng(seed)
    k = r.normal(size=(T, dk))
    k /= np.linalg.norm(k, axis=1, keepdims=True)
    q = r.normal(size=(T, dk)) / np.sqrt(dk)
    return (q, k, r.normal(size=(T, dv)), -r.gamma(1.0, 0.2, size=T), r.uniform(0, 1, size=T), r.normal(size=(dv, dk)),
            r.normal(size=(T, dv)), r.normal(size=(dv, dk)))


def test_chunks_agree_with_tokens():
    q, k, v, g, beta, S0, _, _ = case(100, 16, 24)
    o, states = R.tokens(q, k, v, g, beta, S0, 0.3)
    for c in (0, 64):
        s = slice(c, min(c + 64, 100))
        Gam, P, A, U, W, eb, ec = R.chunk(q[s], k[s], v[s], g[s], beta[s], states[c], 0.3)
        assert np.allclose(P @ U + 0.3 * eb[:, None] * (q[s] @ states[c].T), o[s])
        assert np.allclose(eb[-1] * states[c] + U.T @ (ec[:, None] * k[s]), states[s.stop])


def test_closed_forms():
    q, k, v, g, beta, S0, _, _ = case(3, 8, 8)
    o, st = R.tokens(q, k, v, np.array([-np.inf, 0.0, 0.0]), np.array([1.0, 0.0, 1.0]), S0, 1.0)
    assert np.allclose(st[1], np.outer(v[0], k[0])) and np.array_equal(st[2], st[1])
    assert np.allclose(st[3] @ k[2], v[2])          # a full write answers with its value
    assert np.allclose(o[0], v[0] * (k[0] @ q[0]))


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "S0"])
def test_gradients_against_differences(name):
    args = dict(zip(("q", "k", "v", "g", "beta", "S0", "dO", "dST"), case(7, 6, 5, seed=3)))

    def loss(**x):
        a = {**args, **x}
        o, st = R.tokens(a["q"], a["k"], a["v"], a["g"], a["beta"], a["S0"], 0.4)
        return (o * a["dO"]).sum() + (st[-1] * a["dST"]).sum()

    _, st = R.tokens(*(args[n] for n in ("q", "k", "v", "g", "beta", "S0")), 0.4)
    gr = R.tokens_bwd(*(args[n] for n in ("q", "k", "v", "g", "beta")), st, args["dO"], args["dST"], 0.4)
    got = dict(zip(("q", "k", "v", "g", "beta", "S0"), gr[:5] + (gr[5][0],)))[name]
    r = np.random.default_rng(5)
    for _ in range(3):
        d = r.normal(size=args[name].shape)
        h = 1e-5
        num = (loss(**{name: args[name] + h * d}) - loss(**{name: args[name] - h * d})) / (2 * h)
        assert abs(num - (got * d).sum()) <= 1e-7 * max(1.0, abs(num))


def test_bounds_are_small_against_the_results():
    q, k, v, g, beta, S0, dO, dST = case(150, 64, 64, seed=7)
    o, st = R.tokens(q, k, v, g, beta, S0, 0.125)
    gr = R.tokens_bwd(q, k, v, g, beta, st, dO, dST, 0.125)
    for u, most in ((2.0 ** -8, 0.25), (R.W, 0.05)):
        e, eST, edS0 = R.bounds(q, k, v, g, beta, st, 0.125, u, dO, gr[5])
        for n, x in zip(("o", "dq", "dk", "dv", "dg", "dbeta"), (o,) + gr[:5]):
            assert np.sqrt(np.mean(e[n] ** 2)) <= most * np.sqrt(np.mean(x ** 2)), (n, u)
