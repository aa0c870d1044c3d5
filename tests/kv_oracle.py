"""The 8-bit key/value cache in plain form on the CPU (numpy, 64 bits), for the
tests: e4m3 rounding by hand, loops over blocks, no code of the library."""
from __future__ import annotations

import math

import numpy as np

BLOCK = 64
E_MIN, E_MAX = -40, 44


def e4m3_table():
    """The value of each of the 256 codes."""
    t = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, c >> 3 & 15, c & 7
        v = math.nan if (e == 15 and m == 7) else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        t[c] = -v if s else v
    return t


TABLE = e4m3_table()


def e4m3_encode(x):
    """Codes of the nearest e4m3 values (ties to even), |x| clamped to 448."""
    x = np.asarray(x, np.float64)
    y = np.clip(np.nan_to_num(np.abs(x), nan=0.0, posinf=448.0), 0.0, 448.0)
    ex = np.maximum(np.floor(np.log2(np.maximum(y, 2.0 ** -9))), -6)
    r = np.rint(y / 2.0 ** (ex - 3)) * 2.0 ** (ex - 3)
    code = np.searchsorted(TABLE[:127], r).astype(np.uint8)
    assert np.array_equal(TABLE[code], r)
    code = np.where(np.isnan(x), 255, code).astype(np.uint8)   # NaN has one code
    return code | (np.signbit(x).astype(np.uint8) << 7)


def exponent(amax):
    """Smallest e in range with amax <= 448 * 2^e."""
    e = E_MIN
    while e < E_MAX and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


class Cache:
    """The library's arrays on the host, with the orders inside a block undone by
    `k_codes` / `v_codes` ([64, D] code arrays of one block and head)."""

    def __init__(self, pool, heads, dim, fill=0):
        self.k = np.full((pool, heads, dim // 16, BLOCK, 16), fill, np.uint8)
        self.v = np.full((pool, heads, 4, dim, 16), fill, np.uint8)
        self.k_scale = np.ones((pool, heads), np.float32)
        self.v_scale = np.ones((pool, heads), np.float32)
        self.k_mean = np.zeros((pool, heads, dim), np.int8)
        self.k_mean_scale = np.zeros((pool, heads), np.float32)
        self.dim = dim

    def k_codes(self, p, h):
        return self.k[p, h].transpose(1, 0, 2).reshape(BLOCK, self.dim)

    def v_codes(self, p, h):
        return self.v[p, h].transpose(0, 2, 1).reshape(BLOCK, self.dim)

    def put(self, p, h, k=None, v=None):
        if k is not None:
            self.k[p, h] = k.reshape(BLOCK, self.dim // 16, 16).transpose(1, 0, 2)
        if v is not None:
            self.v[p, h] = v.reshape(4, 16, self.dim).transpose(0, 2, 1)

    def store(self, table, start, count, k, v):
        """k, v: [batch, tokens, heads, dim] float64 (exact input values)."""
        pool, heads = self.k_scale.shape
        for b in range(k.shape[0]):
            n, s = count[b], start[b]
            if s < 0:
                continue
            for j in range(s // BLOCK, min(-(-(s + n) // BLOCK), table.shape[1])):
                p = table[b, j]
                if not 0 <= p < pool:
                    continue
                first, last = max(0, s - j * BLOCK), min(BLOCK, s + n - j * BLOCK)
                for h in range(heads):
                    for name, x, codes in (("k", k, self.k_codes(p, h)), ("v", v, self.v_codes(p, h))):
                        x = x[b, j * BLOCK + first - s:j * BLOCK + last - s, h]
                        fin = np.abs(x[np.isfinite(x)])
                        e = exponent(fin.max() if fin.size else 0.0)
                        scale = getattr(self, name + "_scale")
                        codes = codes.copy() if first else np.zeros_like(codes)
                        if first:
                            was = int(np.log2(scale[p, h]))
                            if e > was:
                                codes[:first] = e4m3_encode(TABLE[codes[:first]] * 2.0 ** (was - e))
                            e = max(e, was)
                        codes[first:last] = e4m3_encode(x * 2.0 ** -e)
                        scale[p, h] = 2.0 ** e
                        self.put(p, h, **{name: codes})
                        if name == "k":
                            total = np.nan_to_num(TABLE[codes[:last]]).sum(0).astype(np.float32)
                            a = np.abs(total).max()
                            up = np.float32(127) * (np.float32(1) / a) if a > 0 else np.float32(0)
                            self.k_mean[p, h] = np.rint(total * up).astype(np.int8)
                            self.k_mean_scale[p, h] = a / np.float32(127 * last) * np.float32(2.0 ** e)


def limits(length, queries, causal):
    i = np.arange(queries)
    return np.maximum(0, length - queries + i + 1) if causal else np.full(queries, length)


def attend(cache, table, length, q, causal, scale, blocks=None, q_tile=0):
    """One sequence: q [queries, heads, dim] float64. Returns out, lse, and what the
    error bounds need: weight = sum p |v| per output, logit = max sum |q k| * scale."""
    nq, qh, d = q.shape
    pool, kh = cache.k_scale.shape
    nb = -(-length // BLOCK)
    out, lse = np.zeros((nq, qh, d)), np.full((nq, qh), -np.inf)
    weight, logit = np.zeros((nq, qh, d)), np.zeros((nq, qh))
    lim = limits(length, nq, causal)
    for h in range(kh):
        k, v = np.zeros((nb * BLOCK, d)), np.zeros((nb * BLOCK, d))
        there = np.zeros(nb * BLOCK, bool)
        for j in range(nb):
            p = table[j]
            if 0 <= p < pool:
                n = min(BLOCK, length - j * BLOCK)
                at = slice(j * BLOCK, j * BLOCK + n)
                k[at] = TABLE[cache.k_codes(p, h)[:n]] * float(cache.k_scale[p, h])
                v[at] = TABLE[cache.v_codes(p, h)[:n]] * float(cache.v_scale[p, h])
                there[at] = True
        for i in range(nq):
            see = there & (np.arange(nb * BLOCK) < lim[i])
            if blocks is not None:
                mine = np.zeros(nb, bool)
                lst = blocks[h, i // q_tile]
                mine[lst[(lst >= 0) & (lst < nb)]] = True
                see = see & np.repeat(mine, BLOCK)
            if not see.any():
                continue
            for g in range(qh // kh):
                hq = h * (qh // kh) + g
                s = k[see] @ q[i, hq] * scale
                m = s.max()
                p = np.exp(s - m)
                out[i, hq] = p @ v[see] / p.sum()
                lse[i, hq] = m + np.log(p.sum())
                weight[i, hq] = p @ np.abs(v[see]) / p.sum()
                logit[i, hq] = (np.abs(k[see]) @ np.abs(q[i, hq])).max() * scale
    return out, lse, weight, logit


def select(cache, table, length, q, causal, q_tile, keep):
    """One sequence: q [queries, heads, dim] float32. [kv_heads, tiles, keep] int32."""
    nq, qh, d = q.shape
    pool, kh = cache.k_scale.shape
    nb = -(-length // BLOCK)
    lim = limits(length, nq, causal)
    f = np.float32
    got = np.full((kh, -(-nq // q_tile), keep), -1, np.int32)
    for h in range(kh):
        for t in range(got.shape[1]):
            rows = range(t * q_tile, min(nq, (t + 1) * q_tile))
            best = np.full(nb, -np.inf)
            for i in rows:
                for g in range(qh // kh):
                    x = q[i, h * (qh // kh) + g]
                    top = np.abs(x).max()
                    c = np.rint(x * (f(127) * (f(1) / top)) if top > 0 else x * f(0)).astype(np.int64)
                    for j in range(-(-lim[i] // BLOCK)):
                        p = table[j]
                        if 0 <= p < pool:
                            dot = int(c @ cache.k_mean[p, h].astype(np.int64))
                            best[j] = max(best[j], f(f(dot) * cache.k_mean_scale[p, h]) * top)
            if causal:
                lo, hi = max(lim[rows[0]], 1) - 1, lim[rows[-1]] - 1
                for j in range(lo // BLOCK, hi // BLOCK + 1 if hi >= 0 else 0):
                    if 0 <= table[j] < pool:
                        best[j] = np.inf
            order = sorted((j for j in range(nb) if best[j] > -np.inf), key=lambda j: (-best[j], j))[:keep]
            got[h, t, :len(order)] = sorted(order)
    return got
