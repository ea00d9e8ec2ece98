"""What attention over a shared prefix is off by, against 64 bits, in the root of the sum of squares: its output's
rounding, and the weights' where they have no remainder.  The tolerances tell the one from the other (CPU)."""
import math

import numpy as np
import pytest

import paged_ref as R
from gdr_rounded import bf16, off


def problem(n, rows, d, seed):
    """`rows` queries over n keys, all of which they see."""
    r = np.random.default_rng(seed)
    return tuple(bf16(r.normal(size=s)) for s in ((rows, d), (n, d), (n, d)))


def attend(q, k, v, weights):
    """With the weights rounded to bf16 as they are used (those of the sum are not), or not."""
    s = (k @ q.T).T / math.sqrt(q.shape[1])
    p = np.exp(s - s.max(1, keepdims=True))
    return (weights(p) @ v) / p.sum(1, keepdims=True)


def tolerance(q, k, v, remainder):
    """fp32: scores of d terms, sums of n + 64."""
    exact = attend(q, k, v, lambda p: p)
    e = off(bf16(attend(q, k, v, (lambda p: p) if remainder else bf16)), exact)
    return exact, 1.05 * e + 4 * R.W * (q.shape[1] + len(k) + 64) ** 0.5


# (The reference of the exponents is not always the maximum, so the weights that are rounded are others: a tenth more.)
def test_the_tolerances_tell_rounded_weights():
    for n, d in ((700, 64), (40, 128), (3000, 32)):
        x = problem(n, 64, d, n)
        exact, with_ = tolerance(*x, True)
        once = off(bf16(attend(*x, bf16)), exact)
        assert once > 1.1 * with_, (n, d, once, with_)


@pytest.mark.gpu
@pytest.mark.parametrize("n,d", [(700, 64), (40, 128), (3000, 32)])
def test_own_keys_of_single_rows_keep_their_weights(n, d):
    import torch

    import delta_rule_recurrent_chunk_amd as kd
    q, k, v = problem(n, 64, d, n)
    dev = lambda x: torch.tensor(x, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    page = 16
    pages = -(-n // page)
    kp, vp = (torch.zeros(pages, page, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kp.view(-1, d)[:n], vp.view(-1, d)[:n] = dev(k), dev(v)
    # 64 heads of one row: two blocks of heads
    o = kd.prefix_attn(dev(q)[None], kp, vp, i32([]), 0, i32([list(range(pages))]), i32([n - 1]))
    exact, tol = tolerance(q, k, v, True)
    got = off(o[0].double().cpu().numpy(), exact)
    print("own keys of a row: %.3e, tolerance %.3e" % (got, tol), flush=True)
    assert got <= tol
    # the same keys as a prefix, and no table of own ones: weights rounded once
    o = kd.prefix_attn(dev(q)[None], kp, vp, i32(list(range(pages))), n, torch.zeros(1, 0, dtype=torch.int32, device="cuda"),
                       i32([0]))
    exact, tol = tolerance(q, k, v, False)
    got = off(o[0].double().cpu().numpy(), exact)
    print("a prefix: %.3e, tolerance %.3e" % (got, 1.1 * tol), flush=True)
    assert got <= 1.1 * tol
