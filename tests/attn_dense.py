"""Attention over packed sequences and the join in 64 bits, for the tests; no code of the
library.

Bounds of an output, for A = sum p |v| of it, S = the largest sum_d |q_d k_d| * scale of its
row, L keys and u = 2^-24 (half a step of fp32):
  scores   bf16 products are exact in fp32; fp32 inputs enter products as sums of two f16
           (each good to 2^-22, and the product of the two low parts, 2^-22, is left out):
           3 * 2^-22. Accumulation over D products (three of each for fp32), the factor and
           the exponent's argument: |ds| <= S * (3 * 2^-22 * fp32 + (2 D + 8) u), with 6 D
           for fp32. The hardware exponential is good to 2^-21.
  weights  rounded to bf16 (half a step: 2^-8), or to two f16 (2^-21), where those lose what
           lies under 2^-32 of the largest (2^-32 per key)
  values   fp32 as two f16, and without the product of the low parts: 3 * 2^-22
  sums     at most L + 64 fp32 additions
so with r = 2 |ds| + 2^-20 + 2 (L + 64) u (numerator and denominator)
  |out - ref| <= A (r + 2^-8, or 2^-21 + 3 * 2^-22) + fp32 * L 2^-32 max|v| + |ref| (2^-8, or 4 u)
  |lse - ref| <= |ds| + 2^-20 + (L + 64) u + 4 u |ref|
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def limits(nq, nk, causal):
    return np.clip(nk - nq + 1 + np.arange(nq), 0, None) if causal else np.full(nq, nk)


def attend(q, k, v, causal, scale):
    """One sequence: q [queries, q_heads, D], k, v [keys, kv_heads, D] float64. Returns out, lse and
    what the bounds need (A, S), and where a value that is not finite is seen."""
    nq, qh, d = q.shape
    nk, kh, _ = k.shape
    out, lse = np.zeros((nq, qh, d)), np.full((nq, qh), -np.inf)
    weight, logit, strange = np.zeros((nq, qh, d)), np.zeros((nq, qh)), np.zeros((nq, qh, d), bool)
    if nk == 0:
        return out, lse, weight, logit, strange
    see = np.arange(nk) < limits(nq, nk, causal)[:, None]
    some = see.any(1)
    for h in range(qh):
        kk, vv = k[:, h * kh // qh], v[:, h * kh // qh]
        odd = ~np.isfinite(vv)
        vv = np.where(odd, 0.0, vv)
        with np.errstate(all="ignore"):
            s = np.where(see, q[:, h] @ kk.T * scale, -np.inf)
            m = s.max(1, initial=-np.inf, keepdims=True)
            m0 = np.where(np.isneginf(m), 0.0, m)
            p = np.where(see, np.exp(s - m0), 0.0)
            total = p.sum(1)
            none = total == 0
            out[:, h] = p @ vv / np.where(none, 1.0, total)[:, None]
            lse[:, h] = np.where(none, -np.inf, m0[:, 0] + np.log(np.where(none, 1.0, total)))
            weight[:, h] = p @ np.abs(vv) / np.where(none, 1.0, total)[:, None]
            # a score of -infinity has no error (its weight is zero), one of +infinity or NaN makes its row NaN
            logit[:, h] = np.where(see & np.isfinite(s), np.abs(q[:, h]) @ np.abs(kk).T * scale, 0.0).max(1, initial=0.0)
        strange[:, h] = ((see & some[:, None]).astype(float) @ odd) > 0
    return out, lse, weight, logit, strange


def check(got, lse, ref, keys, dim, f32, what=""):
    """got, lse float64 against attend's return. NaN outputs and lse of the reference (a query or key that is NaN, a
    score of +infinity) have to be NaN."""
    want, want_lse, weight, logit, strange = ref
    bad = np.isnan(want_lse) | np.isposinf(want_lse)
    assert np.isnan(lse[bad]).all() and np.isnan(got[bad]).all(), (what, "rows that have to be NaN")
    ok = ~bad
    assert not np.isnan(lse[ok]).any(), (what, "lse that must not be NaN", np.argwhere(np.isnan(lse) & ok)[:4])
    empty = np.isneginf(want_lse) & ok
    assert np.array_equal(np.isneginf(lse) & ok, empty), (what, "rows that see nothing")
    assert (got[empty] == 0).all(), (what, "outputs of rows that see nothing")
    odd = strange & ok[..., None]
    assert not np.isfinite(got[odd]).any(), (what, "outputs that see a value that is not finite")
    plain = ok[..., None] & ~strange
    assert np.isfinite(got[plain]).all(), (what, "outputs that must be finite", np.argwhere(plain & ~np.isfinite(got))[:4])
    some = ok & ~empty
    ds = np.where(some, logit, 0.0) * ((3 * 2.0 ** -22 + (6 * dim + 8) * U) if f32 else (2 * dim + 8) * U)
    r = 2 * ds + 2.0 ** -20 + 2 * (keys + 64) * U
    weight = np.where(plain, weight, 0.0)
    bound = weight * (r[..., None] + (2.0 ** -21 + 3 * 2.0 ** -22 if f32 else 2.0 ** -8)) + \
        (keys * 2.0 ** -32 * weight.max(initial=0.0) if f32 else 0.0) + \
        np.where(plain, np.abs(want), 0.0) * (4 * U if f32 else 2.0 ** -8) + 1e-30
    err = np.where(plain, np.abs(np.where(plain, got, 0.0) - np.where(plain, want, 0.0)), 0.0)
    assert (err <= bound).all(), (what, "outputs", np.argwhere(err > bound)[:4], (err / bound).max())
    with np.errstate(invalid="ignore"):
        off = np.where(some, np.abs(lse - want_lse), 0.0)
    most = ds + 2.0 ** -20 + (keys + 64) * U + 4 * U * np.abs(np.where(some, want_lse, 0.0))
    assert (off <= most).all(), (what, "lse", np.argwhere(off > most)[:4], (off / most).max())


def join(outs, lses):
    """outs [parts][rows, D], lses [parts][rows] float64: out, lse and A = sum w |out_i| of each output."""
    lse = np.stack(lses)
    bad = np.isnan(lse).any(0) | np.isposinf(lse).any(0)
    m = np.where(bad, 0.0, np.where(np.isnan(lse), 0.0, lse).max(0))
    none = np.isneginf(m)
    with np.errstate(all="ignore"):
        w = np.exp(lse - np.where(none, 0.0, m))
        total = w.sum(0)
        w = np.where(np.isneginf(lse), 0.0, w / np.where(none, 1.0, total))
        part = [np.where((x == 0)[:, None], 0.0, x[:, None] * o) for x, o in zip(w, outs)]
        out, weight = sum(part), sum(np.abs(x) for x in part)
        log = np.where(none, -np.inf, m + np.log(np.where(none, 1.0, total)))
    out[bad], log[bad] = np.nan, np.nan
    return out, log, weight
