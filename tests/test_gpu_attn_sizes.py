"""Attention over packed sequences at the ends of fp32's range: scores that are larger than what separates them from the
running maximum can be, and in fp32, whose kernel for many rows takes each factor as two f16 on a power of two of its row,
queries, keys and values near both ends. Against attention in 64 bits (attn_dense, which derives the bounds)."""
import numpy as np
import pytest
import torch

import attn_dense as ad
from gpu_harness import DEV, say
from test_gpu_attn import DT, ints, rows, run, wide
from test_gpu_attn_many import is_many
from activation_residual_compression_amd import librescomp as rc

pytestmark = pytest.mark.gpu
DTYPES = pytest.mark.parametrize("dtype", ["bf16", "f32"])
# few rows, in one part and in several; many, the keys in one part, in several
SIZES = pytest.mark.parametrize("dim,nq,nk", [(64, 7, 300), (128, 5, 9000), (64, 1900, 1900), (128, 200, 9000)])


@DTYPES
@SIZES
@pytest.mark.parametrize("power", [10, 20, 30, 90])
def test_large_scores_choose_one_key(dtype, dim, nq, nk, power):
    """Scores are +-2^power * 0, 1, 2, ... in some order, all exact: each row's output is the value of its largest one seen,
    its lse that score (the next one is 2^10 / sqrt(128) lower at least, a weight of 2^-127 or less). Bounds: in bf16 the
    weight's rounding (it is 2^r for the r that the score differs from its own rounding by) and the output's, in fp32
    products of 22 bits; the lse's product with the scale and its two roundings."""
    assert is_many([nq], [nk], 2, 2, dim) == (nq > 100)
    rng = np.random.default_rng(power)
    say("[gpu] one key, 2^%d %s %s" % (power, dtype, (dim, nq, nk)))
    order = rng.permutation(nk)
    q, k = np.zeros((nq, 2, dim)), np.zeros((nk, 2, dim))
    sign = rng.choice([-1.0, 1.0], (nq, 2))
    q[:, :, 3], q[:, :, dim - 1] = sign * 128 * 2.0 ** (power // 2), sign * 2.0 ** (power // 2)
    k[:, :, 3], k[:, :, dim - 1] = (order // 128 * 2.0 ** (power - power // 2))[:, None], (order % 128 * 2.0 ** (power - power // 2))[:, None]
    q, k = (torch.from_numpy(x).to(DT[dtype]).to(DEV) for x in (q, k))
    v = rows(rng, nk, 2, dim, dtype)
    for causal in (False, True):
        out, lse = torch.full_like(q, float("nan")), torch.full((nq, 2), float("nan"), device=DEV)
        with rc.AttnPlan(2, 2, dim, dtype, max_seqs=1, max_queries=nq, max_keys=nk, causal=causal) as p:
            p.attend(q, k, v, ints([0, nq]), out, lse, kv_offsets=ints([0, nk]))
            torch.cuda.synchronize()
        seen = np.arange(nk - nq + 1, nk + 1) if causal else np.full(nq, nk)
        high, low = np.maximum.accumulate(order)[seen - 1], np.minimum.accumulate(order)[seen - 1]
        best = np.where(sign > 0, high[:, None], low[:, None])
        at = np.empty(nk, int)
        at[order] = np.arange(nk)
        want = wide(v)[at[best], np.arange(2)]
        assert (np.abs(wide(out) - want) <= np.abs(want) * (2 * 2.0 ** -8 if dtype == "bf16" else 2.0 ** -20)).all()
        score = sign * best * 2.0 ** power / np.sqrt(dim)
        assert (np.abs(wide(lse) - score) <= np.abs(score) * 2.0 ** -21).all()


@DTYPES
@SIZES
@pytest.mark.parametrize("up,down", [(20, 6), (20, 12), (40, -4), (60, 50)])
def test_large_scores_stay_finite(dtype, dim, nq, nk, up, down):
    rng = np.random.default_rng(up)
    say("[gpu] scores of 2^%d %s %s" % (up + down, dtype, (dim, nq, nk)))
    q, k, v = rows(rng, nq, 2, dim, dtype) * 2.0 ** up, rows(rng, nk, 2, dim, dtype) * 2.0 ** down, rows(rng, nk, 2, dim, dtype)
    for causal in (False, True):
        run(q, k, v, [nq], [nk], causal, dtype)


@pytest.mark.parametrize("dim,nq,nk", [(64, 1900, 1900), (128, 200, 9000)])
@pytest.mark.parametrize("up,down", [(118, -70), (124, -60)])
def test_large_queries(dim, nq, nk, up, down):
    """The queries' power of two and the plan's factor pass fp32, the scores do not: each row's lse is its largest score."""
    rng = np.random.default_rng(up)
    say("[gpu] queries of 2^%d, keys of 2^%d, %d" % (up, down, dim))
    q, k, v = (rows(rng, n, 2, dim, "f32") * 2.0 ** x for n, x in ((nq, up), (nk, down), (nk, 0)))
    q[5] = 0
    q[7] *= 2.0 ** -90
    for causal in (False, True):
        run(q, k, v, [nq], [nk], causal, "f32")
    run(q * 2.0 ** -60, k * 2.0 ** -10, v, [nq], [nk], False, "f32", scale=2.0 ** 68)


@DTYPES
@SIZES
def test_small_scale(dtype, dim, nq, nk):
    """A factor of the scores under fp32's normal range: all weights are 1, hidden keys stay hidden."""
    rng = np.random.default_rng(nq)
    say("[gpu] scale 2^-126 %s %s" % (dtype, (dim, nq, nk)))
    q, k, v = rows(rng, nq, 2, dim, dtype) * 2.0 ** -50, rows(rng, nk, 2, dim, dtype), rows(rng, nk, 2, dim, dtype)
    for causal in (False, True):
        run(q, k, v, [nq], [nk], causal, dtype, scale=2.0 ** -126)


@pytest.mark.parametrize("dim,nq,nk", [(64, 1900, 1900), (128, 200, 9000)])
@pytest.mark.parametrize("what", ["small, then large", "large, then small", "any", "small after rising scores"])
def test_values_of_very_different_sizes(dim, nq, nk, what):
    """Tokens whose values differ by more than fp32 has powers of two between 1 and its end: each counts in the sum of the
    weights, and so in lse, by its score alone."""
    rng = np.random.default_rng(dim)
    say("[gpu] values %s %d" % (what, dim))
    q, k, v = (rows(rng, n, 2, dim, "f32") for n in (nq, nk, nk))
    at = torch.arange(nk, device=DEV)[:, None, None]
    if what == "any":
        power = torch.from_numpy(rng.integers(-75, 110, (nk, 1, 1))).to(DEV)
    elif what == "small after rising scores":            # weights of 1, then of 2^80 and more, then large values
        q, k = q * 0.1, k * 0.1
        q[:, :, 3] = 8.0
        k[:, :, 3] = torch.where(at[:, :, 0] > nk // 3, 7.0 * dim ** 0.5, 0.0)
        power = torch.where(at < nk // 3, 0, torch.where(at < nk // 2, -75, 60))
    else:
        power = torch.where((at < nk // 2) == (what[0] == "s"), -75, 100)
    v = v * torch.exp2(power.float())
    for causal in (False, True):
        run(q, k, v, [nq], [nk], causal, "f32")


@pytest.mark.parametrize("dim,nq,nk", [(64, 1900, 1900), (128, 200, 9000)])
@pytest.mark.parametrize("qp,kp,vp", [(110, -110, 0), (-110, 110, 0), (118, -118, 0), (0, 0, -85), (0, 0, -100), (0, 0, -116)])
def test_rows_of_tiny_values(dim, nq, nk, qp, kp, vp):
    """Queries, keys or values whose largest are far under 1 have the precision of others; checked with the values and
    outputs, which are proportional, on a scale at which the bounds' absolute term is nothing."""
    rng = np.random.default_rng(abs(dim - qp - vp))
    say("[gpu] 2^%d 2^%d 2^%d, %d" % (qp, kp, vp, dim))
    q, k, v = (rows(rng, n, 2, dim, "f32") * 2.0 ** x for n, x in ((nq, qp), (nk, kp), (nk, vp)))
    up = torch.linspace(0, 100, nk, device=DEV)[:, None]
    for rising in (False, True):                 # scores that rise by 140 and more in base 2, under small weights
        if rising:
            q[:, :, 1], k[:, :, 1] = dim ** 0.5 * 2.0 ** qp, up * 2.0 ** kp
        for causal in (False, True):
            out, lse = torch.full_like(q, float("nan")), torch.full((nq, 2), float("nan"), device=DEV)
            with rc.AttnPlan(2, 2, dim, "f32", max_seqs=1, max_queries=nq, max_keys=nk, causal=causal) as p:
                p.attend(q, k, v, ints([0, nq]), out, lse, kv_offsets=ints([0, nk]))
                torch.cuda.synchronize()
            ref = ad.attend(wide(q), wide(k), wide(v) * 2.0 ** -vp, causal, dim ** -0.5)
            ad.check(wide(out) * 2.0 ** -vp, wide(lse), ref, nk, dim, True, (qp, kp, vp, rising, causal))


@pytest.mark.parametrize("dim,nq,nk", [(64, 1900, 1900), (128, 200, 9000)])
@pytest.mark.parametrize("power", [0, -20, -40, -110])
def test_values_beside_zeros(dim, nq, nk, power):
    """Tokens whose values are all zero, at a sequence's start and among others: what the others add has its bits, however
    small they are; checked on a scale at which the bounds' absolute term is nothing."""
    rng = np.random.default_rng(dim - power)
    say("[gpu] zeros and values of 2^%d, %d" % (power, dim))
    q, k, v = (rows(rng, n, 2, dim, "f32") for n in (nq, nk, nk))
    zero = torch.from_numpy(rng.random(nk) < 0.5).to(DEV)
    zero[:300] = True
    v = torch.where(zero[:, None, None], 0.0, v * 2.0 ** power)
    # the zeros' scores are 72 above in base 2: outputs of 2^-72 times the values, which fp32 has for values of 2^-70 and more
    for rising in (False, True) if power > -70 else (False,):
        if rising:
            q[:, :, 1], k[:, :, 1] = dim ** 0.5, torch.where(zero, 50.0, 0.0)[:, None]
        for causal in (False, True):
            out, lse = torch.full_like(q, float("nan")), torch.full((nq, 2), float("nan"), device=DEV)
            with rc.AttnPlan(2, 2, dim, "f32", max_seqs=1, max_queries=nq, max_keys=nk, causal=causal) as p:
                p.attend(q, k, v, ints([0, nq]), out, lse, kv_offsets=ints([0, nk]))
                torch.cuda.synchronize()
            ref = ad.attend(wide(q), wide(k), wide(v) * 2.0 ** -power, causal, dim ** -0.5)
            ad.check(wide(out) * 2.0 ** -power, wide(lse), ref, nk, dim, True, (power, rising, causal))


@pytest.mark.parametrize("dim,nq,nk", [(64, 1900, 1900), (128, 200, 9000)])
@pytest.mark.parametrize("power", [100, 118, 125])
def test_huge_values(dim, nq, nk, power):
    """Values of one sign whose sum over the keys passes fp32 and whose mean does not; also of large scores, of which one
    key's value is the result."""
    rng = np.random.default_rng(power)
    say("[gpu] values of 2^%d, %d" % (power, dim))
    q, k = rows(rng, nq, 2, dim, "f32"), rows(rng, nk, 2, dim, "f32")
    v = (1 + torch.from_numpy(rng.random((nk, 2, dim)).astype(np.float32)).to(DEV)) * 2.0 ** power
    for causal in (False, True):
        run(q, k, v, [nq], [nk], causal, "f32")
        run(q * 2.0 ** 15, k * 2.0 ** 15, v, [nq], [nk], causal, "f32")
