"""Attention over the 8-bit cache of kv_oracle in 64 bits by dense products, with what
kv_oracle.attend leaves out: NaN and infinities, lists in any order, entries that
repeat. For the tests; no code of the library."""
from __future__ import annotations

import numpy as np

import kv_oracle as ko

U = 2.0 ** -24


def attend(cache, row, length, q, causal, scale, lists=None, q_tile=0):
    """One sequence: q [queries, heads, dim] float64, row its table, lists [kv_heads,
    tiles, keep]. A list ends at its first entry that is negative or not below the
    number of blocks that its tile sees; an entry that repeats counts again. Returns
    out, lse, what the bounds need (weight = sum p |v|, logit = the largest sum |q k| *
    scale), and where a NaN among values that a query does not see lies in a block that
    its tile reads."""
    nq, qh, d = q.shape
    pool, kh = cache.k_scale.shape
    out, lse = np.zeros((nq, qh, d)), np.full((nq, qh), -np.inf)
    weight, logit, near = np.zeros((nq, qh, d)), np.zeros((nq, qh)), np.zeros((nq, qh, d), bool)
    lim = ko.limits(length, nq, causal)
    step = q_tile if lists is not None else nq
    group = qh // kh
    for h in range(kh):
        for t in range(-(-nq // step)):
            rows = slice(t * step, min(nq, (t + 1) * step))
            reach = -(-lim[rows][-1] // ko.BLOCK)
            blocks = list(range(reach))
            if lists is not None:
                entries = [int(j) for j in lists[h, t]]
                blocks = entries[:next((i for i, j in enumerate(entries) if not 0 <= j < reach), len(entries))]
            blocks = [j for j in blocks if 0 <= row[j] < pool]
            if not blocks:
                continue
            pos = np.concatenate([np.arange(j * ko.BLOCK, (j + 1) * ko.BLOCK) for j in blocks])
            k = np.concatenate([ko.TABLE[cache.k_codes(row[j], h)] * float(cache.k_scale[row[j], h]) for j in blocks])
            v = np.concatenate([ko.TABLE[cache.v_codes(row[j], h)] * float(cache.v_scale[row[j], h]) for j in blocks])
            k, v, pos = k[pos < length], v[pos < length], pos[pos < length]
            see = pos < lim[rows][:, None]
            nan = np.isnan(v)
            v = np.where(nan, 0.0, v)
            for g in range(group):
                hq = h * group + g
                with np.errstate(all="ignore"):
                    x = q[rows, hq]
                    s = np.where(see, x @ k.T * scale, -np.inf)
                    m = s.max(1, initial=-np.inf, keepdims=True)
                    p = np.where(see, np.exp(s - m), 0.0)
                    total = np.where(see.any(1), p.sum(1), 1.0)
                    out[rows, hq] = p @ v / total[:, None]
                    lse[rows, hq] = np.where(see.any(1), m[:, 0] + np.log(total), -np.inf)
                    weight[rows, hq] = p @ np.abs(v) / total[:, None]
                    logit[rows, hq] = np.where(see, np.abs(x) @ np.abs(k).T * scale, 0.0).max(1, initial=0.0)
                out[rows, hq][(see.astype(float) @ nan) > 0] = np.nan
                near[rows, hq] = ((~see).astype(float) @ nan) > 0
    return out, lse, weight, logit, near


def check(got, lse, ref, length, dim, f32):
    """got, lse (float64 arrays) against attend's return, by the bounds that test_gpu_kv
    derives. Where the reference is NaN they have to be; nothing else may be, but for
    the outputs for which a masked value that is NaN was read."""
    want, want_lse, weight, logit, near = ref
    ds = logit * ((2.0 ** -22 if f32 else 0.0) + (2 * dim + 8) * U)
    r = 2 * ds + 2.0 ** -20 + 2 * (length + 64) * U
    vmax = np.nanmax(weight, initial=0.0)
    bound = weight * (r[..., None] + (2.0 ** -21 if f32 else 2.0 ** -11)) + length * 2.0 ** -32 * vmax + \
        np.abs(want) * (4 * U if f32 else 2.0 ** -8) + 1e-30
    nan = np.isnan(want)
    assert np.isnan(got[nan]).all(), ("outputs that have to be NaN", np.argwhere(nan & ~np.isnan(got))[:4], got[nan][:4])
    open_ = nan | (near & np.isnan(got))
    assert not np.isnan(got[~open_]).any(), ("outputs that must not be NaN", np.argwhere(np.isnan(got) & ~open_)[:4])
    err = np.where(open_, 0.0, np.abs(got - np.where(nan, 0.0, want)))
    assert (err <= np.where(open_, 1.0, bound)).all(), (np.argwhere(err > np.where(open_, 1.0, bound))[:4], err.max())
    nan, empty = np.isnan(want_lse), np.isneginf(want_lse)
    assert np.isnan(lse[nan]).all(), ("sums that have to be NaN", np.argwhere(nan & ~np.isnan(lse))[:4], lse[nan][:4])
    assert np.array_equal(np.isneginf(lse), empty), "rows without tokens"
    assert (got[empty] == 0).all()
    some = ~nan & ~empty
    assert (np.abs(lse[some] - want_lse[some]) <=
            (ds + 2.0 ** -20 + (length + 64) * U + 4 * U * np.abs(np.where(some, want_lse, 0.0)))[some]).all()


def choose(cache, row, length, q, causal, q_tile, keep):
    """The choice of blocks of one sequence, q [queries, heads, dim] float32: every block
    that is there and that a query of the tile sees can be chosen; a score that is NaN
    counts as -infinity, a NaN in a query as 0."""
    nq, qh, _ = q.shape
    pool, kh = cache.k_scale.shape
    nb = -(-length // ko.BLOCK)
    lim = ko.limits(length, nq, causal)
    f, group = np.float32, qh // kh
    got = np.full((kh, -(-nq // q_tile), keep), -1, np.int32)
    there = np.array([0 <= row[j] < pool for j in range(nb)], bool)
    at = np.where(there, row[:nb], 0)
    begins = np.arange(nb) * ko.BLOCK
    with np.errstate(all="ignore"):
        for h in range(kh):
            x = np.where(np.isnan(q), f(0), q)[:, h * group:(h + 1) * group]
            top = np.abs(x).max(-1, keepdims=True)
            up = f(127) * (f(1) / top)
            codes = np.rint(x * np.where(np.isfinite(up), up, f(0)))
            codes = np.where(np.isnan(codes), 0, codes).astype(np.int64)
            dot = (codes @ cache.k_mean[at, h].astype(np.int64).T).astype(f)
            score = (dot * cache.k_mean_scale[at, h]).astype(f) * top
            score = np.where(np.isnan(score), f(-np.inf), score).max(1)                 # [queries, blocks]
            score = np.where(begins < lim[:, None], score, f(-np.inf))
            for t in range(got.shape[1]):
                ln = lim[t * q_tile:(t + 1) * q_tile]
                best = score[t * q_tile:(t + 1) * q_tile].max(0).astype(np.float64)
                rank = best.copy()
                own = np.zeros(nb, bool)
                if causal and ln[-1] > 0:
                    own[(max(ln[0], 1) - 1) // ko.BLOCK:(ln[-1] - 1) // ko.BLOCK + 1] = True
                able = [j for j in range(nb) if there[j] and begins[j] < ln[-1]]
                order = sorted(able, key=lambda j: (not own[j], 0 if own[j] else -rank[j], j))[:keep]
                got[h, t, :len(order)] = sorted(order)
    return got
