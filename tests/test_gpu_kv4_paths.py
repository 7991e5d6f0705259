"""Attention over a cache in 4 bits by each of its two kernels: groups of at most 32 (row, head) pairs take fragments,
larger ones query tiles; prefixes likewise by the rows behind them."""
import math

import pytest

import attn_ref as R
import kv4_ref as K
from test_gpu_kv4 import Case4

pytestmark = pytest.mark.gpu


def restate(c, k_factor, v_factor):
    """What the same codes stand for under other factors."""
    c.factors = (k_factor, v_factor)
    c.kc, c.vc = (K.values(x, s, f) for x, s, f in zip(c.codes, c.scales, c.factors))


def check(c, rows=None, ref=None, **more):
    """A call against 64 bits, with the probabilities' own rounding beside the output's.

    Both kernels round a probability to F16 after a power of two that brings a row's largest to 2^6 or more: by 2^-11 of it, or,
    below F16's normal numbers, by 2^-25, which is 2^-31 of the largest.  Where the results are divided by the sum of the rounded
    ones, sum p (1 + d) v / sum p (1 + d) differs from o = sum p v by sum p d (v - o) / (1 + d'): 2^-11 (sum p |v| + |o|) and a
    2^-10th of that.  Scores are off as they are for attend (see attn_ref)."""
    out, lse, st = c.run(**more)
    assert st == 0, hex(st)
    rows = slice(0, c.indptr[-1]) if rows is None else rows
    o, want_lse, mag, bound, count, vmax = (x[rows] for x in ref or c.ref())
    tol = R.U[c.dtype] * o.abs() + (2.0 ** -11 + 2.0 ** -20 + 2 * bound + 2.0 ** -18)[..., None] * (mag + o.abs())
    tol = tol + (2.0 ** -30 * count * vmax)[..., None] + R.STEP[c.dtype]
    err = (out[rows].double() - o).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), int((~(err <= tol)).sum()))
    none = want_lse == -math.inf
    got = lse[rows].double()
    assert bool((got[none] == -math.inf).all()) and bool((out[rows][none] == 0).all())
    off = (got - want_lse).abs()[~none]
    assert bool((off <= (bound + 2.0 ** -18)[~none]).all()), float(off.max())
    return out, lse


@pytest.mark.parametrize("dtype,d", [("f16", 128), ("f16", 64), ("bf16", 128)])
@pytest.mark.parametrize("n,hq", [([2, 3], 4), ([12, 20], 8)])  # fragments; query tiles (more than 32 pairs a group)
@pytest.mark.parametrize("scale,factor", [(2.0 ** -100, 2.0 ** -100), (2.0 ** -149, 1.0), (2.0 ** -3, 2.0 ** -149)])
def test_attend4_scores_whose_factor_vanishes(dtype, d, n, hq, scale, factor):
    """scale * k_factor below FP32's range: every score is 0 to within the bound, and tokens past a length stay out."""
    c = Case4(dtype=dtype, d=d, hq=hq, hk=1, n=n, lens=[40, 300], prefixes=[70])
    c.scale = scale
    restate(c, factor, 1.0)
    check(c)


@pytest.mark.parametrize("dtype,d", [("f16", 128), ("f16", 64), ("bf16", 128)])
@pytest.mark.parametrize("n,hq", [([2, 3], 4), ([12, 20], 8)])
def test_attend4_scores_of_zero_under_a_factor_past_the_range(dtype, d, n, hq):
    """scale * k_factor past FP32's range: a score of 0 is 0."""
    import torch
    c = Case4(dtype=dtype, d=d, hq=hq, hk=1, n=n, lens=[40, 300], prefixes=[70])
    c.q = torch.zeros_like(c.q)
    c.scale = 2.0 ** 80
    restate(c, 2.0 ** 80, 1.0)
    check(c)


@pytest.mark.parametrize("n,hq", [([2, 3], 4), ([12, 20], 8)])
@pytest.mark.parametrize("size,scale,factor", [
    (2.0 ** -105, 2.0 ** 40, 2.0 ** 62), (2.0 ** -128, 2.0 ** 70, 2.0 ** 58), (2.0 ** -110, 1.75 * 2.0 ** 127, 2.0 ** -20),
    (2.0 ** 100, 2.0 ** -60, 2.0 ** -43), (2.0 ** 100, 2.0 ** 20, 2.0 ** -123),
])
def test_attend4_factors_that_bring_one_another_back(size, scale, factor, n, hq):
    """BF16 queries far from 1 under a scale and a factor that bring their scores back, whatever the products on the way."""
    c = Case4(hq=hq, hk=1, n=n, lens=[40, 300], prefixes=[70])
    c.q = (c.q.float() * size).bfloat16()
    c.scale = scale
    restate(c, factor, 1.0)
    check(c)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64)])
@pytest.mark.parametrize("n,hq", [([2], 4), ([12], 8)])
@pytest.mark.parametrize("factor", [2.0 ** -126, 2.0 ** -128, 2.0 ** -131, 2.0 ** 116])
def test_attend4_values_under_a_factor_at_the_ends_of_the_range(dtype, d, n, hq, factor):
    """Values of 2,688 factor, which BF16 holds: the factor alone, divided by the sum of 5,000 probabilities, would leave FP32's normal numbers."""
    import torch
    c = Case4(dtype=dtype, d=d, hq=hq, hk=1, n=n, lens=[5001])
    c.raw[1][~c.raw[1].isnan()] = 2688.0
    c.quantise()
    restate(c, 1.0, factor)
    out, _ = check(c)
    assert torch.equal(out.double(), torch.full_like(out, 2688.0 * factor).double())
