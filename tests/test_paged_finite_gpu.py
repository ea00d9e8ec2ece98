"""Attention over a shared prefix where queries, keys and values are not finite, and where rows are nobody's."""
import math

import numpy as np
import pytest

import paged_ref as R
from test_paged_gpu import Case, _torch, check, f64

pytestmark = pytest.mark.gpu

# packed or one row per sequence; rows see the prefix and own keys, own keys alone, one own key alone
BATCHES = [(False, [3, 0, 200, 70], [1] * 4, 100), (False, [3, 0, 200, 70], [1] * 4, 0), (False, [0, 0], [1, 1], 0),
           (True, [3, 0, 9], [20, 40, 2], 300), (True, [3, 0, 9], [20, 40, 2], 0), (True, [0, 0], [1, 1], 0)]


def compare(c, o, lse, scale=None, atol=0.0):
    """Against plain arithmetic in 64 bits: scores that are NaN or +infinity make NaNs; keys of score -infinity weigh
    nothing, and a row that sees no other has no weights (0 / 0) and the logarithm of 0."""
    scale = 1.0 / math.sqrt(c.d) if scale is None else scale
    q, k, v = f64(c.q), f64(c.kp), f64(c.vp)
    u = 2.0 ** -8 if c.dt == _torch().bfloat16 else R.W
    for r, owner in enumerate(R.rows_of(c.lens, c.cu, c.T)):
        if owner is None or owner[1] is None:
            continue
        at = R.keys_of(owner, c.lens, c.cu, c.ptable, c.P, c.table, c.page, c.pages)
        pg, sl = (np.array([x[i] for x in at], int) for i in (0, 1))
        for h in range(c.Hq):
            hk = h // (c.Hq // c.Hkv)
            with np.errstate(invalid="ignore"):
                s = (k[pg, sl, hk] @ q[r, h]) * scale
                ro, eo, rl, el = R.attend(q[r, h], k[pg, sl, hk], v[pg, sl, hk], scale, u)
            if np.isneginf(s).all():
                ro, rl = np.full(c.d, np.nan), -np.inf
            elif np.isneginf(s).any() and np.isfinite(s).any() and not np.isnan(s).any():
                live = np.isfinite(s)      # (the bounds come from the keys that weigh something)
                ro, eo, rl, el = R.attend(q[r, h], k[pg, sl, hk][live], v[pg, sl, hk][live], scale, u)
            check("o of row %d, head %d" % (r, h), o[r, h], ro, eo)
            check("lse of row %d, head %d" % (r, h), np.float64(lse[h, r].item()), np.float64(rl), el)


def case(i, dtype, seed):
    packed, lens, new, P = BATCHES[i]
    print("batch", BATCHES[i], dtype, flush=True)
    return Case(lens, new, P, 16, 4, 2, 64, dtype, seed=seed, packed=packed)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("i", range(len(BATCHES)))
def test_a_query_that_is_not_finite_shows(i, value, dtype):
    c = case(i, dtype, 40 + i)
    c.q[1, 2, 5] = float(value)
    o, lse = c.run(return_lse=True)
    compare(c, o, lse)
    assert np.isnan(f64(o)[1, 2]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("i", range(len(BATCHES)))
def test_keys_that_are_not_finite_show(i, value, dtype):
    """All keys of one head in pages that the second sequence alone sees."""
    c = case(i, dtype, 50 + i)
    own = [int(p) for p in c.table[1] if p >= 0]
    c.kp[own, :, 1, 3] = float(value)
    o, lse = c.run(return_lse=True)
    compare(c, o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("packed", [False, True])
def test_rows_whose_scores_are_all_minus_infinity(packed, dtype):
    c = Case([3, 40], [1, 1], 70, 16, 4, 2, 64, dtype, seed=60, packed=packed)
    c.kp[..., 7] = c.kp[..., 7].abs() + 0.5
    c.q[0, 1, 7] = float("-inf")
    o, lse = c.run(return_lse=True)
    compare(c, o, lse)
    assert np.isnan(f64(o)[0, 1]).all() and np.isneginf(lse[1, 0].item())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("where", ["own", "prefix"])
def test_an_infinite_value_of_no_weight_shows(where, packed, dtype):
    """Weights below fp32's range: e^-400 of infinity is not 0."""
    c = Case([5, 2], [1, 1], 40, 16, 2, 1, 64, dtype, seed=61, packed=packed)
    big = [int(p) for p in c.ptable] if where == "own" else [int(p) for p in c.table[0] if p >= 0]
    c.q[0] = 0
    c.q[0, :, 0] = 20
    c.kp[:, :, :, 0] = 0
    c.kp[big, :, :, 0] = 160        # scores of 400 there, of 0 elsewhere
    pg, sl = (int(c.table[0, 0]), 1) if where == "own" else (int(c.ptable[1]), 2)
    c.vp[pg, sl, 0, 9] = float("inf")
    o = f64(c.run())
    assert not np.isfinite(o[0, :, 9]).any() and np.isfinite(np.delete(o[0], 9, -1)).all()


FILLS = ["nan", "inf", "-inf", 1e30, -3.0]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("packed", [False, True])
def test_rows_that_are_nobodys_change_nothing(packed, dtype):
    """Rows of unused sequences and rows that no sequence holds: other rows have the same bits whatever is there."""
    torch = _torch()
    if packed:
        c = Case([3, -1, 0, 50, -2], [20, 5, 3, 1, 1], 700, 16, 4, 2, 64, dtype, seed=62, packed=True, gap=9)
    else:
        c = Case([3, -1, 0, 50, -2], [1] * 5, 700, 16, 4, 2, 64, dtype, seed=62)
    held = torch.tensor([o is not None and o[1] is not None for o in R.rows_of(c.lens, c.cu, c.T)], device="cuda")
    c.q *= 4
    c.q[~held] = 0
    ref, rl = c.run(return_lse=True)
    c.check(ref, rl, rows=[0, 1])
    for fill in FILLS:
        c.q[~held] = float(fill)
        o, lse = c.run(return_lse=True)
        assert torch.equal(o[held], ref[held]) and torch.equal(lse[:, held], rl[:, held]), fill


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("packed", [False, True])
def test_another_rows_nan_changes_nothing(packed, dtype):
    """A request whose queries are NaN beside others: theirs have the same bits as with queries of 0 there."""
    torch = _torch()
    lens, new = ([3, 6, 0, 50], [20, 5, 3, 1]) if packed else ([3, 6, 0, 50], [1] * 4)
    c = Case(lens, new, 700, 16, 4, 2, 64, dtype, seed=63, packed=packed)
    mine = torch.tensor([o[0] == 1 for o in R.rows_of(c.lens, c.cu, c.T)], device="cuda")
    c.q[mine] = 0
    ref, rl = c.run(return_lse=True)
    c.q[mine] = float("nan")
    o, lse = c.run(return_lse=True)
    assert torch.equal(o[~mine], ref[~mine]) and torch.equal(lse[:, ~mine], rl[:, ~mine])
    assert torch.isnan(o[mine]).all() and torch.isnan(lse[:, mine]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_sequences_with_unused_ones_between(dtype):
    """More sequences than lanes, some empty, some unused."""
    torch = _torch()
    rng = np.random.default_rng(64)
    lens = [int(x) if x > 4 else -1 for x in rng.integers(0, 30, 150)]
    new = [int(x) for x in rng.integers(0, 5, 150)]
    c = Case(lens, new, 130, 16, 2, 1, 32, dtype, seed=64, packed=True, gap=4)
    held = torch.tensor([o is not None and o[1] is not None for o in R.rows_of(c.lens, c.cu, c.T)], device="cuda")
    c.q[~held] = 0
    ref, rl = c.run(return_lse=True)
    c.check(ref, rl, rows=range(0, c.T - 4, 7))
    c.q[~held] = float("nan")
    o, lse = c.run(return_lse=True)
    assert torch.equal(o[held], ref[held]) and torch.equal(lse[:, held], rl[:, held])
