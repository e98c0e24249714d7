"""Sums of block means at their limits: rows that cancel, sums beyond fp32, subnormal rows.

Tolerance of a mean, from the arithmetic: a sum carried as two fp32 numbers is off by at most ((n - 1) 2^-24)^2 of the sum
of |x|, n <= 128 rows: 2^-34; and the mean is rounded to fp32, 2^-24 of it (2^-150 where it is subnormal).  The largest
mean gives the scale: one more product, 2^-24.
"""
import itertools

import numpy as np
import pytest
import torch

from speculative_decoding_tree_05_gb300 import ddtree
from parity_util import require_cuda

pytestmark = pytest.mark.gpu
C = np.float64(np.float32(1) / np.float32(127))


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    require_cuda()
    from speculative_decoding_tree_05_gb300 import build
    build.build()


def summarise(rows, block):
    """rows [n, 576] fp64 of bf16 values, in this order: one request of one block (or its first ones)."""
    kv = torch.tensor(rows, dtype=torch.float64).to(torch.bfloat16).cuda()
    assert torch.equal(kv.double().cpu(), torch.tensor(rows, dtype=torch.float64))
    n = kv.shape[0]
    i32 = dict(dtype=torch.int32, device="cuda")
    s, c = ddtree.block_summary(kv, torch.arange(n, **i32)[None].contiguous(), torch.tensor([n], **i32), block)
    return s[0, 0].double().cpu().numpy(), float(c[0, 0])


def check(rows, block=16):
    got, scale = summarise(rows, block)
    n = len(rows)
    mean, mass = rows.sum(0) / n, np.abs(rows).sum(0) / n
    tol = 2.0 ** -34 * mass + 2.0 ** -24 * np.abs(mean) + 2.0 ** -150
    top, at = np.abs(mean).max(), np.abs(mean).argmax()
    assert abs(scale - top * C) <= tol.max() * C + 2.0 ** -24 * top * C + 2.0 ** -150
    if scale == 0:
        assert not got.any()
        return scale
    # an integer is the nearest one to a quotient that is off by the mean's and the scale's error
    quot = mean / scale
    assert (np.abs(got - quot) <= 0.5 + tol / scale + 2.0 ** -22 * np.abs(quot)).all()
    assert abs(abs(got[at]) - 127) <= 1
    return scale


def spread(values):
    """The values as rows: each dim has them times its own sign, one dim in four doubled."""
    sign = np.where(np.arange(576) % 3 == 0, -1.0, 1.0) * np.where(np.arange(576) % 4 == 1, 0.5, 1.0)
    return np.asarray(values, np.float64)[:, None] * sign[None]


BIG = 255 * 2.0 ** 119   # close to the largest bf16 value, 255 * 2^120


def test_partial_sums_beyond_fp32_in_any_order():
    """2 BIG + 2 BIG is more than fp32 holds, the sum of all is not."""
    x = [2 * BIG, 2 * BIG, -2 * BIG, 1.0, -2 * BIG, 2 * BIG]
    for order in sorted(set(itertools.permutations(range(6))))[::37]:
        assert np.isfinite(check(spread([x[i] for i in order])))


@pytest.mark.parametrize("n,block", [(2, 16), (16, 16), (17, 32), (64, 64), (127, 128), (128, 128)])
def test_sums_beyond_fp32_with_means_within(n, block):
    scale = check(spread([2 * BIG] * n), block)
    assert scale == float(np.float32(np.float32(2 * BIG) * np.float32(C)))
    mixed = [2 * BIG if i % 3 else -BIG for i in range(n)]
    check(spread(mixed), block)


@pytest.mark.parametrize("seed", range(4))
def test_rows_that_cancel(seed):
    """Pairs of opposite rows over many binades beside small ones, in random orders."""
    g = np.random.default_rng(seed)
    big = np.exp2(g.integers(-20, 41, 24)) * g.choice([1, 1.5, -1.25], 24)
    x = np.concatenate([big, -big, np.exp2(g.integers(-12, -4, 16))])
    for _ in range(6):
        check(spread(x[g.permutation(64)]), 64)


def test_small_example_of_cancellation():
    for order in ([40, 16, -9, 140, 116], [-9, 40, 140, 16, 116]):
        x = [np.exp2(e) if e < 100 else -np.exp2(e - 100) for e in order]
        check(spread(x))


@pytest.mark.parametrize("n", [1, 3, 16])
def test_subnormal_rows(n):
    """bf16 values from 2^-133 on: still exact at 2^-7 of their size."""
    check(spread([2.0 ** -132 * (1 + i % 5) for i in range(n)]))
    check(spread([2.0 ** -126 * (1 if i % 2 else -1) + 0.0 for i in range(n)]))


@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
def test_a_row_that_is_not_finite(value):
    rows = spread([1.0, 2.0, 3.0])
    kv = torch.tensor(rows, dtype=torch.float64).to(torch.bfloat16).cuda()
    kv[1, 77] = value
    i32 = dict(dtype=torch.int32, device="cuda")
    s, c = ddtree.block_summary(kv, torch.arange(3, **i32)[None].contiguous(), torch.tensor([3], **i32), 16)
    assert bool(torch.isnan(c).all()) and not bool(s.any())
