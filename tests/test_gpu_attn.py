"""Attention over packed sequences and the join of attentions on the GPU, against attention in
64 bits (attn_dense, which derives the bounds)."""
import numpy as np
import pytest
import torch

import attn_dense as ad
from gpu_harness import DEV, say
from activation_residual_compression_amd import librescomp as rc

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def rows(rng, n, heads, dim, dtype, spread=1.0):
    return torch.from_numpy((rng.standard_normal((n, heads, dim)) * spread).astype(np.float32)).to(DT[dtype]).to(DEV)


def wide(x):
    return x.double().cpu().numpy()


def offsets(lengths, first=0):
    return np.concatenate([[first], first + np.cumsum(lengths)]).astype(np.int64)


def check_all(q, k, v, qo, ko, causal, scale, out, lse, dtype, what=""):
    """Every sequence of a call against the dense reference."""
    q, k, v, out, lse = (wide(x) for x in (q, k, v, out, lse))
    for i in range(len(qo) - 1):
        a, b, c, d = qo[i], qo[i + 1], ko[i], ko[i + 1]
        ref = ad.attend(q[a:b], k[c:d], v[c:d], causal, scale)
        ad.check(out[a:b], lse[a:b], ref, max(d - c, 1), q.shape[2], dtype == "f32", (what, "sequence", i))


def run(q, k, v, lq, lk, causal, dtype, scale=0.0, same=False, **kw):
    """One call over sequences of lengths lq, lk, with outputs that begin as NaN."""
    qo, ko = offsets(lq), offsets(lk)
    out = torch.full((q.shape[0], q.shape[1], q.shape[2]), float("nan"), dtype=DT[dtype], device=DEV)
    lse = torch.full((q.shape[0], q.shape[1]), float("nan"), device=DEV)
    with rc.AttnPlan(q.shape[1], k.shape[1], q.shape[2], dtype, max_seqs=len(lq), max_queries=max(q.shape[0], 1),
                     max_keys=max(k.shape[0], 1), causal=causal, scale=scale) as p:
        p.attend(q, k, v, ints(qo), out, lse, kv_offsets=None if same else ints(ko), max_q=max(lq), max_kv=max(lk), **kw)
        torch.cuda.synchronize()
    check_all(q, k, v, qo, ko, causal, scale or q.shape[2] ** -0.5, out, lse, dtype)
    return out, lse


HEADS = [(3, 3, 64), (2, 2, 128), (8, 2, 64), (6, 2, 128), (20, 1, 128)]
LENGTHS = [
    ([1], [1]), ([1], [333]), ([2, 1, 3], [64, 65, 63]), ([5, 0, 64, 3, 129], [5, 7, 64, 0, 130]),
    ([300, 1, 17, 0], [300, 1, 500, 0]), ([70], [3]), ([257, 31], [1025, 40]), ([0, 0], [5, 0]), ([511, 130], [511, 130])]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("causal", [False, True])
def test_attend_equals_dense(dtype, heads, causal):
    qh, kh, dim = heads
    rng = np.random.default_rng(dim + qh + causal)
    for lq, lk in LENGTHS:
        say("[gpu] attend %s %s causal %s lengths %s %s" % (dtype, heads, causal, lq, lk))
        q, k, v = (rows(rng, sum(n), h, dim, dtype) for n, h in ((lq, qh), (lk, kh), (lk, kh)))
        run(q, k, v, lq, lk, causal, dtype, same=lq == lk)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
def test_scores_of_every_size(dtype, dim):
    """Scores that grow along the keys (the maximum rises in every step), fall, spread over 2^20, are all zero, all the
    lowest; keys and values of very different sizes in neighbouring tokens; a scale of the caller's."""
    rng = np.random.default_rng(dim)
    n = 300
    up = torch.linspace(0, 6, n, device=DEV)[:, None, None]
    for what, kf, vf, scale in (("rising", lambda x: x + up, None, 0.0), ("falling", lambda x: x - up, None, 0.0),
                                ("large", lambda x: x * 30, None, 0.0), ("small", lambda x: x * 2.0 ** -60, None, 0.0),
                                ("zero", lambda x: x * 0, None, 0.0), ("scale", lambda x: x, None, 0.7),
                                ("mixed", lambda x: x * torch.exp2(torch.randint(-8, 3, (n, 1, 1), device=DEV).float()),
                                 lambda x: x * torch.exp2(torch.randint(-3, 4, (n, 1, 1), device=DEV).float()), 0.0),
                                ("values of 2^60", None, lambda x: x * 2.0 ** 60, 0.0),
                                ("values of 2^-90", None, lambda x: x * 2.0 ** -90, 0.0)):
        say("[gpu] scores %s %s %d" % (what, dtype, dim))
        q, k, v = rows(rng, n, 2, dim, dtype) * 0.5 + 0.5, rows(rng, n, 2, dim, dtype), rows(rng, n, 2, dim, dtype)
        k = kf(k.float()).to(DT[dtype]) if kf else k
        v = vf(v.float()).to(DT[dtype]) if vf else v
        for causal in (False, True):
            run(q, k, v, [n], [n], causal, dtype, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("queries", [1, 3, 150])
def test_nan_and_infinities_reach_only_who_sees_them(dtype, dim, queries):
    rng = np.random.default_rng(queries)
    n, m = queries, queries + 67
    say("[gpu] not finite %s %d %d" % (dtype, dim, queries))
    for bad in (float("nan"), float("inf"), -float("inf")):
        q, k, v = rows(rng, 2 * n, 4, dim, dtype), rows(rng, 2 * m, 2, dim, dtype), rows(rng, 2 * m, 2, dim, dtype)
        v[m - 1, 0, 5] = bad                 # the first sequence's last value: its last query alone sees it
        v[m + 2, 1, 3] = bad                 # the second's early one: all its queries do
        if n > 40:
            v[m - 33, 1, 60] = bad
            v[2 * m - 20, 0] = bad
            k[2 * m - 7, 1, 2] = float("nan")
            q[n + 9, 2, 11] = bad
        run(q, k, v, [n, n], [m, m], True, dtype)
        run(q, k, v, [n, n], [m, m], False, dtype)
    # behind a sequence's last key, in no sequence at all
    q, k, v = rows(rng, n, 4, dim, dtype), rows(rng, 200, 2, dim, dtype), rows(rng, 200, 2, dim, dtype)
    k[77:] = float("nan")
    v[77:] = float("nan")
    run(q, k, v, [n], [77], False, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [False, True])
def test_strides_and_rows_of_no_sequence(dtype, causal):
    """Queries, keys and values side by side in one row of a token; head-major keys; outputs with gaps; tokens before the
    first and behind the last sequence. Nothing but the sequences' rows is written."""
    rng = np.random.default_rng(5)
    lq, first, tail = [40, 0, 300, 7], 3, 21
    n = first + sum(lq) + tail
    qo = offsets(lq, first)
    for qh, kh, dim in ((4, 2, 64), (4, 4, 128)):
        say("[gpu] strides %s causal %s %s" % (dtype, causal, (qh, kh, dim)))
        qkv = rows(rng, n, qh + 2 * kh, dim, dtype)
        q, k = qkv[:, :qh], qkv[:, qh:qh + kh]
        v = qkv[:, qh + kh:].permute(1, 0, 2).contiguous().permute(1, 0, 2)      # [head][token][dim]
        space = torch.full((n, qh + 1, dim + 8), 7.0, dtype=DT[dtype], device=DEV)
        out = space[:, :qh, :dim]
        lse = torch.full((n, qh), 7.0, device=DEV)
        with rc.AttnPlan(qh, kh, dim, dtype, max_seqs=9, max_queries=n + 5, max_keys=n + 9, causal=causal) as p:
            p.attend(q, k, v, ints(qo), out, lse)
            torch.cuda.synchronize()
        check_all(q, k, v, qo, qo, causal, dim ** -0.5, out, lse, dtype)
        assert (space[:, qh:] == 7).all() and (space[:, :, dim:] == 7).all()
        for part in (slice(0, first), slice(n - tail, n)):
            assert (space[part] == 7).all() and (lse[part] == 7).all()


def test_bounds_cut_sequences_and_bad_offsets_stay_inside():
    rng = np.random.default_rng(6)
    q, k, v = rows(rng, 100, 4, 64, "bf16"), rows(rng, 200, 2, 64, "bf16"), rows(rng, 200, 2, 64, "bf16")
    with rc.AttnPlan(4, 2, 64, "bf16", max_seqs=4, max_queries=100, max_keys=200, causal=True) as p:
        for qo, ko, mq, mk, rows_q, rows_k in (
                ([0, 60, 100], [0, 120, 200], 50, 90, [(0, 50), (60, 100)], [(0, 90), (120, 200)]),
                ([-5, 20, 10, 400], [0, 50, 40, 300], 0, 0, [(0, 20), (20, 20), (10, 100)], [(0, 50), (50, 50), (40, 200)]),
                ([70, 70, 2000000000], [-2000000000, 30, 2000000000], 0, 0, [(70, 70), (70, 100)], [(0, 30), (30, 200)])):
            say("[gpu] offsets %s %s" % (qo, ko))
            out = torch.full((100, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
            lse = torch.full((100, 4), 7.0, device=DEV)
            p.attend(q, k, v, ints(qo), out, lse, kv_offsets=ints(ko), max_q=mq, max_kv=mk)
            torch.cuda.synchronize()
            seen = np.zeros(100, int)
            for a, b in rows_q:
                seen[a:b] += 1
            for (a, b), (c, d) in zip(rows_q, rows_k):
                ref = ad.attend(wide(q)[a:b], wide(k)[c:d], wide(v)[c:d], True, 0.125)
                one = seen[a:b] == 1          # where offsets descend, rows may be of two sequences: either's results
                ad.check(wide(out)[a:b][one], wide(lse)[a:b][one], [x[one] for x in ref], 200, 64, False, (qo, a))
            left = torch.from_numpy(seen == 0)
            assert (out.cpu()[left] == 7).all() and (lse.cpu()[left] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,lq,lk", [
    ((2, 2, 128), [1], [20011]), ((8, 2, 64), [1, 1, 1], [9000, 1, 5003]), ((4, 1, 128), [40], [7001]),
    ((2, 2, 64), [200, 3], [6001, 12000]), ((6, 2, 128), [64, 0, 1, 90], [4097, 33, 8192, 0])])
def test_long_keys_are_split_and_joined_alike(dtype, heads, lq, lk):
    """Few queries over long keys run in parts; the result is the same every time, also where other calls of the plan ran
    in between, and where a captured graph replays it."""
    qh, kh, dim = heads
    rng = np.random.default_rng(sum(lk))
    say("[gpu] long %s %s %s %s" % (dtype, heads, lq, lk))
    q, k, v = (rows(rng, sum(n), h, dim, dtype) for n, h in ((lq, qh), (lk, kh), (lk, kh)))
    for causal in (False, True):
        out, lse = run(q, k, v, lq, lk, causal, dtype)
        qo, ko = ints(offsets(lq)), ints(offsets(lk))
        again, sums = torch.empty_like(out), torch.empty_like(lse)
        with rc.AttnPlan(qh, kh, dim, dtype, max_seqs=len(lq), max_queries=q.shape[0], max_keys=k.shape[0], causal=causal) as p:
            kw = dict(kv_offsets=ko, max_q=max(lq), max_kv=max(lk))
            p.attend(q, k, v, qo, again, sums, **kw)
            torch.cuda.synchronize()
            stream = torch.cuda.Stream()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                p.attend(q, k, v, qo, again, sums, **kw)
            for _ in range(3):
                again.fill_(3)
                sums.fill_(3)
                graph.replay()
                torch.cuda.synchronize()
                assert torch.equal(again, out) and torch.equal(sums, lse)
                p.attend(q[:1], k[:5], v[:5], ints([0, 1]), again[:1], kv_offsets=ints([0, 5]))
                torch.cuda.synchronize()


def test_calls_on_two_streams_with_plans_of_their_own():
    rng = np.random.default_rng(9)
    cases = []
    for i in range(2):
        q, k, v = rows(rng, 3, 4, 128, "bf16"), rows(rng, 12000, 2, 128, "bf16"), rows(rng, 12000, 2, 128, "bf16")
        out, lse = run(q, k, v, [2, 1], [7000, 5000], True, "bf16")
        plan = rc.AttnPlan(4, 2, 128, "bf16", max_seqs=2, max_queries=3, max_keys=12000, causal=True)
        cases.append((plan, torch.cuda.Stream(), (q, k, v, ints([0, 2, 3])), torch.empty_like(out), torch.empty_like(lse), out, lse))
    ko = ints([0, 7000, 12000])
    torch.cuda.synchronize()
    say("[gpu] two streams")
    for _ in range(20):
        for plan, stream, args, o, s, *_ in cases:
            plan.attend(*args, o, s, kv_offsets=ko, max_q=2, max_kv=7000, stream=stream)
    torch.cuda.synchronize()
    for plan, _, _, o, s, out, lse in cases:
        assert torch.equal(o, out) and torch.equal(s, lse)
        plan.close()


def test_rows_more_than_2_to_the_31_elements_apart():
    say("[gpu] far rows")
    rng = np.random.default_rng(10)
    n, step = 150, 1 << 24
    far = torch.empty(n * step, dtype=torch.bfloat16, device=DEV)        # 5 GB
    k, v = (torch.as_strided(far, (n, 2, 64), (step, 64, 1), at) for at in (0, 4096))
    q = torch.as_strided(far, (n, 2, 64), (step, 64, 1), 8192)
    out = torch.as_strided(far, (n, 2, 64), (step, 64, 1), 12288)
    for x in (q, k, v):
        x.copy_(rows(rng, n, 2, 64, "bf16"))
    lse = torch.empty(n, 2, device=DEV)
    with rc.AttnPlan(2, 2, 64, "bf16", max_seqs=1, max_queries=n, max_keys=n, causal=True) as p:
        p.attend(q, k, v, ints([0, n]), out, lse)
        torch.cuda.synchronize()
    check_all(q, k, v, [0, n], [0, n], True, 0.125, out, lse, "bf16")


def test_plan_refuses_wrong_tensors():
    rng = np.random.default_rng(11)
    q, k = rows(rng, 6, 4, 64, "bf16"), rows(rng, 9, 2, 64, "bf16")
    with rc.AttnPlan(4, 2, 64, "bf16", max_seqs=2, max_queries=6, max_keys=9) as p:
        qo, ko = ints([0, 3, 6]), ints([0, 4, 9])
        for args, kw in [((q.float(), k, k, qo, q), {}), ((q, k, k[:5], qo, q), {}), ((q, k[:, :1], k, qo, q), {}),
                         ((q, k, k, qo.long(), q), {}), ((q, k, k, qo, q[:5]), {}), ((q[None], k, k, qo, q), {}),
                         ((q, k, k, qo, q, torch.empty(6, 3, device=DEV)), {}), ((q, k, k, qo, q), dict(kv_offsets=ko[:2])),
                         ((q.transpose(1, 2), k, k, qo, q), {}), ((q, k, k, qo.cpu(), q), {})]:
            with pytest.raises(ValueError):
                p.attend(*args, **kw)
        with pytest.raises(rc.RcError):
            p.attend(q, k, k, qo, q[:1].expand(6, 4, 64), kv_offsets=ko)       # outputs that overlap


# ------------------------------------------------------------------ join
@pytest.mark.parametrize("in_dtype,out_dtype", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("dim", [64, 128])
def test_join_equals_dense(in_dtype, out_dtype, dim):
    """Bound: weights to 2^-21 and the roundings of their argument (the lse's differences up to 40: 40 * 2 u), sums over the
    parts, and the output's rounding: A (2^-20 + 80 u * 2 + 16 u) + |ref| (2^-8 or 4 u)."""
    rng = np.random.default_rng(dim)
    for parts, shape in ((1, (3, 5)), (2, (1, 1)), (3, (70, 3)), (8, (33, 7)), (2, (4, 9, 5))):
        say("[gpu] join %s %s dim %d parts %d shape %s" % (in_dtype, out_dtype, dim, parts, shape))
        space = torch.from_numpy(rng.standard_normal((parts, *shape, dim + 8)).astype(np.float32)).to(DT[in_dtype]).to(DEV)
        outs = [x[..., :dim] for x in space]
        lses = [torch.from_numpy((rng.standard_normal(shape) * 6 + 3).astype(np.float32)).to(DEV) for _ in range(parts)]
        flat = [x.view(-1) for x in lses]
        for x in flat:
            x[torch.from_numpy(rng.random(x.numel()) < 0.2).to(DEV)] = -float("inf")
        if flat[0].numel() > 4:
            for x in flat:
                x[1] = -float("inf")
            flat[0][2], flat[-1][3] = float("nan"), float("inf")
            for x, y in zip(outs, lses):      # parts that saw nothing hold anything
                x[y == -float("inf")] = float("nan")
        to = torch.full((*shape, dim + 8), 7.0, dtype=DT[out_dtype], device=DEV)
        out, lse = to[..., :dim], torch.empty(shape, device=DEV)
        rc.join_attention(outs, lses, out, lse)
        torch.cuda.synchronize()
        want, log, weight = ad.join([wide(x).reshape(-1, dim) for x in outs], [wide(x).reshape(-1) for x in lses])
        got, sums = wide(out).reshape(-1, dim), wide(lse).reshape(-1)
        nan = np.isnan(log)
        assert np.isnan(got[nan]).all() and np.isnan(sums[nan]).all()
        ok = ~nan
        assert np.isfinite(got[ok]).all() and np.array_equal(np.isneginf(sums[ok]), np.isneginf(log[ok]))
        assert (got[np.isneginf(log) & ok] == 0).all()
        bound = weight * (2.0 ** -20 + 176 * U) + np.abs(want) * (4 * U if out_dtype == "f32" else 2.0 ** -8) + 1e-30
        assert (np.abs(got - want) <= bound)[ok].all()
        some = ok & ~np.isneginf(log)
        assert (np.abs(sums - log)[some] <= 2.0 ** -20 + 176 * U + 4 * U * np.abs(log[some])).all()
        assert (to[..., dim:] == 7).all()


def test_join_in_place_and_of_attention_over_parts_of_the_keys():
    """Attention over two parts of the keys, joined into the first one's buffers, is attention over all: each part's
    rounding to bf16 (2^-8 of it) comes on top of the bounds of attention."""
    rng = np.random.default_rng(3)
    n, m, qh, kh, dim = 50, 700, 6, 2, 128
    say("[gpu] join in place")
    for dtype in ("bf16", "f32"):
        q, k, v = rows(rng, n, qh, dim, dtype), rows(rng, m, kh, dim, dtype), rows(rng, m, kh, dim, dtype)
        parts = [run(q, k[a:b], v[a:b], [n], [b - a], False, dtype) for a, b in ((0, 301), (301, m))]
        outs, lses = zip(*parts)
        rc.join_attention(outs, lses, outs[0], lses[0])
        torch.cuda.synchronize()
        want, log, weight, logit, _ = ad.attend(wide(q), wide(k), wide(v), False, dim ** -0.5)
        ds = logit * ((3 * 2.0 ** -22 + (6 * dim + 8) * U) if dtype == "f32" else (2 * dim + 8) * U)
        r = 4 * ds + 2.0 ** -18 + 4 * (m + 64) * U
        bound = weight * (r[..., None] + (2.0 ** -19 if dtype == "f32" else 2 * 2.0 ** -8)) + np.abs(want) * (4 * U if dtype == "f32" else 2.0 ** -8) + \
            (m * 2.0 ** -32 * weight.max() if dtype == "f32" else 0)
        assert (np.abs(wide(outs[0]) - want) <= bound).all()
        assert (np.abs(wide(lses[0]) - log) <= 2 * ds + 2.0 ** -18 + (m + 64) * U).all()


def test_join_refuses_wrong_tensors():
    x, s = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(3, 4, device=DEV)
    for args in [([x, x.float()], [s, s], x), ([x, x[:2]], [s, s], x), ([x], [s[:2]], x), ([x], [s.double()], x),
                 ([x.half()], [s], x), ([x], [s], x[0]), ([x], [s], x, s[:1]), ([x], [s.cpu()], x)]:
        with pytest.raises((ValueError, rc.RcError)):
            rc.join_attention(*args)
    with pytest.raises(rc.RcError):
        rc.join_attention([x] * 9, [s] * 9, x)
