"""The references of the layers beside the mixer against what defines them: finite differences, closed forms,
and plain loops (CPU)."""
import numpy as np
import pytest

from tests import layers_ref as R



def test_glr_closed_forms():
    r = np.random.default_rng(0)
    x, f = r.standard_normal((2, 9, 3)), r.random((2, 9, 3))
    h0 = r.standard_normal((2, 3))
    # gates of 1: a running sum; gates of 0: the input itself
    assert np.allclose(R.glr(x, np.ones_like(f), None, h0)[:, 1:], h0[:, None] + np.cumsum(x, 1))
    assert np.allclose(R.glr(x, np.zeros_like(f), f, h0)[:, 1:], f * x)
    # a decayed state alone
    assert np.allclose(R.glr(0 * x, f, None, h0)[:, -1], h0 * f.prod(1))


@pytest.mark.parametrize("gate", [False, True])
def test_glr_gradients_by_differences(gate):
    r = np.random.default_rng(1)
    x, f, i, dh = r.standard_normal((2, 6, 3)), r.random((2, 6, 3)), r.random((2, 6, 3)), r.standard_normal((2, 6, 3))
    h0, dhT = r.standard_normal((2, 3)), r.standard_normal((2, 3))
    i = i if gate else None

    def loss(x, f, i, h0):
        h = R.glr(x, f, i, h0)
        return (dh * h[:, 1:]).sum() + (dhT * h[:, -1]).sum()

    _, dx, df, di, dh0 = R.glr_bwd(x, f, i, R.glr(x, f, i, h0), dh, dhT)
    args = [x, f, i, h0]
    for n, got in ((0, dx), (1, df), (2, di), (3, dh0)):
        if args[n] is None:
            continue
        for at in np.ndindex(args[n].shape):
            lo, hi = [None if a is None else a.copy() for a in args], [None if a is None else a.copy() for a in args]
            lo[n][at] -= 1e-6
            hi[n][at] += 1e-6
            assert abs((loss(*hi) - loss(*lo)) / 2e-6 - got[at]) < 1e-7 * (1 + abs(got[at]))


def test_attention_against_a_loop_and_differences():
    r = np.random.default_rng(2)
    for Tq, Tk, window, sinks in ((5, 5, 2, 1), (4, 7, 3, 0), (6, 4, 2, 1), (1, 1, 1, 0), (6, 6, 100, 0)):
        q, k, v, dO = (r.standard_normal((n, 3)) for n in (Tq, Tk, Tk, Tq))

        def fwd(q, k, v):
            o = np.zeros((Tq, 3))
            for t in range(Tq):
                p = Tk - Tq + t
                ks = [s for s in range(Tk) if s <= p and (p - s < window or s < sinks)]
                if ks:
                    w = np.exp([0.7 * q[t] @ k[s] for s in ks])
                    o[t] = (w[:, None] * v[ks]).sum(0) / w.sum()
            return o

        val, err = R.attention(q, k, v, window, sinks, 0.7, dO)
        assert np.allclose(val["o"], fwd(q, k, v), atol=1e-12)
        for n, x in (("dq", q), ("dk", k), ("dv", v)):
            for at in np.ndindex(x.shape):
                a = [y.copy() for y in (q, k, v)]
                j = ("dq", "dk", "dv").index(n)
                a[j][at] += 1e-6
                up = (fwd(*a) * dO).sum()
                a[j][at] -= 2e-6
                assert abs((up - (fwd(*a) * dO).sum()) / 2e-6 - val[n][at]) < 1e-7 * (1 + abs(val[n][at]))
        assert all((e >= 0).all() for e in err.values())


def test_rope_is_a_rotation():
    r = np.random.default_rng(3)
    x = r.standard_normal((1, 4, 2, 8))
    pos, fr = np.array([[0, 1, 7, 10 ** 6]]), 10000.0 ** (-np.arange(3) / 3.0)
    for layout in ("half", "interleaved"):
        y, _ = R.rope(x, pos, fr, layout, 1.5)
        assert np.allclose((y[..., :6] ** 2).sum(-1), 2.25 * (x[..., :6] ** 2).sum(-1))
        assert np.array_equal(y[..., 6:], x[..., 6:]) and np.allclose(y[:, 0, :, :6], 1.5 * x[:, 0, :, :6])
        z, _ = R.rope(y, pos, fr, layout, 1 / 1.5, inverse=True)
        assert np.allclose(z[..., :6], x[..., :6], atol=1e-9)
    # relative positions: a turned query against a turned key depends on their distance
    a, _ = R.rope(x, np.array([[5, 6, 7, 8]]), fr, "half", 1.0)
    b, _ = R.rope(x, np.array([[105, 106, 107, 108]]), fr, "half", 1.0)
    assert np.allclose(np.einsum("bthd,bshd->bhts", a, a), np.einsum("bthd,bshd->bhts", b, b))


def test_slots_keep_every_visible_position_apart():
    for sinks, window, cap in ((0, 1, 1), (2, 3, 5), (4, 8, 15), (1, 5, 6)):
        for p in range(60):
            at = [R.slot(s, sinks, cap) for s in R.seen(p, window, sinks)]
            assert len(set(at)) == len(at) and max(at) < cap
