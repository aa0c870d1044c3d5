"""Attention over packed sequences for many query rows, at sizes for which the kernels for many rows
run (they are chosen by what the kernel for few rows would read: 100 MB of keys and values), against
attention in 64 bits (attn_dense, which derives the bounds)."""
import numpy as np
import pytest
import torch

import attn_dense as ad
from gpu_harness import DEV, say
from test_gpu_attn import DT, check_all, ints, offsets, rows, run, wide
from activation_residual_compression_amd import librescomp as rc

pytestmark = pytest.mark.gpu
DTYPES = pytest.mark.parametrize("dtype", ["bf16", "f32"])


def is_many(lq, lk, qh, kh, dim):
    return -(-max(lq) * (qh // kh) // 16) * sum(lk) * kh * dim * 4 > 100 << 20


SHORT = [1 + 7 * i % 41 for i in range(131)]
CASES = [
    ((8, 2, 64), [700, 1, 0, 33, 64], [1200, 5, 7, 0, 65]),            # shared heads, empty sequences, one key
    ((3, 3, 64), [1100, 129, 128], [1900, 100, 130]),                  # fewer keys than queries: rows that see none
    ((6, 2, 128), [700, 2, 257], [700, 1, 257]), ((20, 1, 128), [300, 0, 77], [500, 3, 97]),
    ((2, 2, 128), [1500], [1300]),                                     # causal: 200 rows that see none
    ((4, 4, 128), SHORT + [900], SHORT[::-1] + [901]),                 # more than 64 sequences
    ((4, 2, 64), [1000] + SHORT, [1003] + SHORT),
    ((2, 2, 128), [200], [9000]), ((8, 2, 64), [100], [9001]),         # few tiles of rows: the keys in many parts
    ((2, 2, 64), [5000], [700]), ((5, 5, 128), [2100], [513]),         # many tiles, few keys
]


@DTYPES
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attend_equals_dense(dtype, causal, case):
    (qh, kh, dim), lq, lk = CASES[case]
    assert is_many(lq, lk, qh, kh, dim)
    rng = np.random.default_rng(case)
    say("[gpu] many rows %s causal %s case %d" % (dtype, causal, case))
    q, k, v = (rows(rng, sum(n), h, dim, dtype) for n, h in ((lq, qh), (lk, kh), (lk, kh)))
    out, lse = run(q, k, v, lq, lk, causal, dtype)
    again, sums = run(q, k, v, lq, lk, causal, dtype)
    assert torch.equal(out, again) and torch.equal(lse, sums)


@DTYPES
@pytest.mark.parametrize("dim,n", [(64, 1900), (128, 1300)])
def test_scores_and_values_of_every_size(dtype, dim, n):
    """As for few rows; and tokens of very different sizes next to each other."""
    assert is_many([n], [n], 2, 2, dim)
    rng = np.random.default_rng(dim)
    up = torch.linspace(0, 6, n, device=DEV)[:, None, None]

    def powers(lo, hi):
        return torch.from_numpy(np.exp2(rng.integers(lo, hi, (n, 1, 1))).astype(np.float32)).to(DEV)
    for what, qf, kf, vf, scale in (
            ("rising", None, lambda x: x + up, None, 0.0), ("falling", None, lambda x: x - up, None, 0.0),
            ("large", None, lambda x: x * 30, None, 0.0), ("small", None, lambda x: x * 2.0 ** -60, None, 0.0),
            ("zero", None, lambda x: x * 0, None, 0.0), ("scale", None, None, None, 0.7),
            ("mixed", None, lambda x: x * powers(-8, 3), lambda x: x * powers(-3, 4), 0.0),
            ("queries of every size", lambda x: x * powers(-60, 3), None, None, 0.0),
            ("keys of every size", None, lambda x: x * powers(-60, 3), None, 0.0),
            ("large queries, small keys", lambda x: x * 2.0 ** 70, lambda x: x * 2.0 ** -70, None, 0.0),
            ("small queries, large keys", lambda x: x * 2.0 ** -70, lambda x: x * 2.0 ** 70, None, 0.0),
            ("values of every size", None, None, lambda x: x * powers(-60, 30), 0.0),
            ("values of 2^60", None, None, lambda x: x * 2.0 ** 60, 0.0), ("no values", None, None, lambda x: x * 0, 0.0),
            ("values of 2^-90", None, None, lambda x: x * 2.0 ** -90, 0.0)):
        say("[gpu] many rows, scores %s %s %d" % (what, dtype, dim))
        x = [rows(rng, n, 2, dim, dtype) * 0.5 + 0.5, rows(rng, n, 2, dim, dtype), rows(rng, n, 2, dim, dtype)]
        q, k, v = (f(y.float()).to(DT[dtype]) if f else y for f, y in zip((qf, kf, vf), x))
        for causal in (False, True):
            run(q, k, v, [n], [n], causal, dtype, scale=scale)


@DTYPES
@pytest.mark.parametrize("dim,n", [(64, 1900), (128, 1300)])
def test_what_a_query_does_not_see_does_not_touch_its_result(dtype, dim, n):
    """Hidden keys and values that are huge, infinite or NaN: the rows before them have their result within the bounds
    of what they see, and where their tile does not read them to the bit."""
    rng = np.random.default_rng(n)
    q, k, v = (rows(rng, n, 2, dim, dtype) for _ in range(3))
    at = n - 333
    want, sums = run(q, k, v, [n], [n], True, dtype)
    for bad in (2.0 ** 100, -2.0 ** 100, float("inf"), float("nan")):
        say("[gpu] hidden %s %s %d" % (bad, dtype, dim))
        for kb, vb in ((False, True), (True, False), (True, True)):
            k2, v2 = k.clone(), v.clone()
            if kb:
                k2[at:] = bad
            if vb:
                v2[at:] = bad
            out, lse = torch.empty_like(q), torch.empty((n, 2), device=DEV)
            with rc.AttnPlan(2, 2, dim, dtype, max_seqs=1, max_queries=n, max_keys=n, causal=True) as p:
                p.attend(q, k2, v2, ints([0, n]), out, lse)
                torch.cuda.synchronize()
            whole = at // 256 * 256              # of no tile of rows that reads such a key
            assert torch.equal(out[:whole], want[:whole]) and torch.equal(lse[:whole], sums[:whole])
            ref = ad.attend(wide(q)[whole:at], wide(k)[:at], wide(v)[:at], True, dim ** -0.5)
            ad.check(wide(out)[whole:at], wide(lse)[whole:at], ref, n, dim, dtype == "f32", (bad, kb, vb))


@DTYPES
@pytest.mark.parametrize("dim", [64, 128])
def test_nan_and_infinities_reach_only_who_sees_them(dtype, dim):
    n = 1000
    m = n + 67
    assert is_many([n, n], [m, m], 4, 2, dim)
    rng = np.random.default_rng(dim)
    for bad in (float("nan"), float("inf"), -float("inf")):
        say("[gpu] many rows, not finite %s %d %s" % (dtype, dim, bad))
        q, k, v = rows(rng, 2 * n, 4, dim, dtype), rows(rng, 2 * m, 2, dim, dtype), rows(rng, 2 * m, 2, dim, dtype)
        v[m - 1, 0, 5] = bad
        v[m + 2, 1, 3] = bad
        v[m - 33, 1, 60] = bad
        v[2 * m - 20, 0] = bad
        k[2 * m - 7, 1, 2] = bad
        k[300, 0, 7] = -bad
        q[n + 9, 2, 11] = bad
        q[17, 0] = bad
        for causal in (False, True):
            run(q, k, v, [n, n], [m, m], causal, dtype)


@DTYPES
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("qh,kh,dim", [(4, 2, 64), (2, 2, 128)])
def test_strides_and_rows_of_no_sequence(dtype, causal, qh, kh, dim):
    rng = np.random.default_rng(5)
    lq, first, tail = [40, 0, 1700, 7], 3, 21
    n = first + sum(lq) + tail
    qo = offsets(lq, first)
    assert is_many([n], [n], qh, kh, dim)
    say("[gpu] many rows, strides %s causal %s %s" % (dtype, causal, (qh, kh, dim)))
    qkv = rows(rng, n, qh + 2 * kh, dim, dtype)
    q, k = qkv[:, :qh], qkv[:, qh:qh + kh]
    v = qkv[:, qh + kh:].permute(1, 0, 2).contiguous().permute(1, 0, 2)      # [head][token][dim]
    space = torch.full((n, qh + 1, dim + 8), 7.0, dtype=DT[dtype], device=DEV)
    out = space[:, :qh, :dim]
    lse = torch.full((n, qh), 7.0, device=DEV)
    with rc.AttnPlan(qh, kh, dim, dtype, max_seqs=9, max_queries=n + 5, max_keys=n + 9, causal=causal) as p:
        p.attend(q, k, v, ints(qo), out, lse)
        one = torch.full_like(out, 7.0)
        p.attend(q, k[:, :1].expand(-1, kh, -1), v[:1].expand(n, -1, -1), ints(qo), one)     # strides of zero
        torch.cuda.synchronize()
    check_all(q, k, v, qo, qo, causal, dim ** -0.5, out, lse, dtype)
    assert (space[:, qh:] == 7).all() and (space[:, :, dim:] == 7).all()
    for part in (slice(0, first), slice(n - tail, n)):
        assert (space[part] == 7).all() and (lse[part] == 7).all() and (one[part] == 7).all()
    for i in range(len(lq)):                     # every token's value is the first one's: outputs are it
        a, b = qo[i], qo[i + 1]
        for h in range(qh):
            got, want = wide(one[a:b, h]), wide(v[0, h * kh // qh])
            assert (np.abs(got - want) <= np.abs(want) * (2 * 2.0 ** -8 if dtype == "bf16" else 2.0 ** -17)).all()


@DTYPES
def test_bad_offsets_stay_inside(dtype):
    """Offsets that leave the tensors or descend, so that sequences claim more than there is: nothing outside the outputs
    is written, and the plan's next call is right (few rows over long keys run in parts that count each other)."""
    rng = np.random.default_rng(6)
    n, m = 1500, 2000
    q, k, v = rows(rng, n, 4, 64, dtype), rows(rng, m, 2, 64, dtype), rows(rng, m, 2, 64, dtype)
    with rc.AttnPlan(4, 2, 64, dtype, max_seqs=100, max_queries=n, max_keys=m) as p:
        want = torch.empty_like(q)
        p.attend(q[:1], k, v, ints([0, 1]), want[:1], kv_offsets=ints([0, m]))
        for qo, ko, mq, mk in (([-5, 1000, 10, 2 ** 31 - 1], [0, 1900, -3, 2 ** 31 - 1], 0, 0), ([0, 1, 0, 1], [0, m, 0, m], 1, m),
                               ([0, 1] * 50, [0, m] * 50, 1, m), ([0, 700, 1500], [5, 2000, 1], 800, 0)):
            say("[gpu] bad offsets %s %s" % (dtype, qo[:4]))
            space = torch.full((n + 2, 4, 64), 7.0, dtype=DT[dtype], device=DEV)
            p.attend(q, k, v, ints(qo), space[1:-1], kv_offsets=ints(ko), max_q=mq, max_kv=mk)
            torch.cuda.synchronize()
            assert (space[0] == 7).all() and (space[-1] == 7).all()
            again = torch.empty_like(want[:1])
            p.attend(q[:1], k, v, ints([0, 1]), again, kv_offsets=ints([0, m]))
            torch.cuda.synchronize()
            assert torch.equal(again, want[:1])


@DTYPES
@pytest.mark.parametrize("lq,lk", [([1300, 5], [1300, 5]), ([130], [9000])])
def test_captured_calls_replay(dtype, lq, lk):
    """Two graphs of one plan, replayed in turn, with the program's own calls between: the outputs are the eager ones."""
    rng = np.random.default_rng(7)
    say("[gpu] many rows, graphs %s %s" % (dtype, lq))
    q, k, v = (rows(rng, sum(n), 2, 128, dtype) for n in (lq, lk, lk))
    out, lse = run(q, k, v, lq, lk, False, dtype)
    qo, ko = ints(offsets(lq)), ints(offsets(lk))
    with rc.AttnPlan(2, 2, 128, dtype, max_seqs=len(lq), max_queries=q.shape[0], max_keys=k.shape[0]) as p:
        kw = dict(kv_offsets=ko, max_q=max(lq), max_kv=max(lk))
        graphs = []
        for _ in range(2):
            o, s = torch.empty_like(out), torch.empty_like(lse)
            p.attend(q, k, v, qo, o, s, **kw)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                p.attend(q, k, v, qo, o, s, **kw)
            graphs.append((g, o, s))
        for _ in range(3):
            for g, o, s in graphs:
                o.fill_(3)
                s.fill_(3)
                g.replay()
                p.attend(q[:1], k[:5], v[:5], ints([0, 1]), torch.empty_like(q[:1]), kv_offsets=ints([0, 5]))
                torch.cuda.synchronize()
                assert torch.equal(o, out) and torch.equal(s, lse)


@DTYPES
def test_calls_on_two_streams_with_plans_of_their_own(dtype):
    rng = np.random.default_rng(9)
    n, cases = 1400, []
    for i in range(2):
        q, k, v = (rows(rng, n, 2, 128, dtype) for _ in range(3))
        out, lse = run(q, k, v, [n], [n], True, dtype)
        plan = rc.AttnPlan(2, 2, 128, dtype, max_seqs=1, max_queries=n, max_keys=n, causal=True)
        cases.append((plan, torch.cuda.Stream(), (q, k, v, ints([0, n])), torch.empty_like(out), torch.empty_like(lse), out, lse))
    torch.cuda.synchronize()
    say("[gpu] many rows, two streams %s" % dtype)
    for _ in range(10):
        for plan, stream, args, o, s, *_ in cases:
            plan.attend(*args, o, s, stream=stream)
    torch.cuda.synchronize()
    for plan, _, _, o, s, out, lse in cases:
        assert torch.equal(o, out) and torch.equal(s, lse)
        plan.close()


@pytest.mark.parametrize("n,dim,step", [(1900, 64, 1 << 21), (1300, 128, 1 << 24)])
def test_rows_more_than_2_to_the_31_elements_apart(n, dim, step):
    say("[gpu] many rows, far rows %d" % step)
    rng = np.random.default_rng(10)
    far = torch.empty(n * step, dtype=torch.bfloat16, device=DEV)        # 8 and 44 GB
    k, v = (torch.as_strided(far, (n, 2, dim), (step, dim, 1), at) for at in (0, 4096))
    q = torch.as_strided(far, (n, 2, dim), (step, dim, 1), 8192)
    out = torch.as_strided(far, (n, 2, dim), (step, dim, 1), 12288)
    for x in (q, k, v):
        x.copy_(rows(rng, n, 2, dim, "bf16"))
    lse = torch.empty(n, 2, device=DEV)
    with rc.AttnPlan(2, 2, dim, "bf16", max_seqs=1, max_queries=n, max_keys=n, causal=True) as p:
        p.attend(q, k, v, ints([0, n]), out, lse)
        torch.cuda.synchronize()
    check_all(q, k, v, [0, n], [0, n], True, dim ** -0.5, out, lse, "bf16")
    del far, k, v, q, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("max_keys", [40000, 1 << 20])
def test_fp32_with_and_without_room_for_halves(max_keys):
    """A plan for more keys than their halves have room for (4 GB) runs the kernel for few rows."""
    say("[gpu] fp32 plan for %d keys" % max_keys)
    rng = np.random.default_rng(12)
    n = 1300
    q, k, v = (rows(rng, n, 8, 128, "f32") for _ in range(3))
    out, lse = torch.empty_like(q), torch.empty((n, 8), device=DEV)
    with rc.AttnPlan(8, 8, 128, "f32", max_seqs=1, max_queries=n, max_keys=max_keys, causal=True) as p:
        assert p.workspace_bytes < (6 << 30) and (p.workspace_bytes > max_keys * 8 * 128 * 8) == (max_keys == 40000)
        p.attend(q, k, v, ints([0, n]), out, lse)
        torch.cuda.synchronize()
    check_all(q[:, :1], k[:, :1], v[:, :1], [0, n], [0, n], True, 128 ** -0.5, out[:, :1], lse[:, :1], "f32")


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("f32", 128)])
def test_join_of_more_than_the_caches_hold(dtype, dim):
    """Against the sum in 64 bits on the GPU; bounds as in test_gpu_attn's join."""
    g = torch.Generator(device=DEV)
    g.manual_seed(dim)
    parts, shape = 3, (2, 1500, 1 + (150 << 20) // (3 * 3000 * dim * (2 if dtype == "bf16" else 4)))
    say("[gpu] join of large parts %s %s" % (dtype, shape))
    outs = [torch.randn((*shape, dim), generator=g, device=DEV).to(DT[dtype]) for _ in range(parts)]
    lses = [torch.randn(shape, generator=g, device=DEV) * 4 for _ in range(parts)]
    lses[1][1, 3:9] = -float("inf")
    assert sum(x.numel() * x.element_size() for x in outs) > 128 << 20
    want = torch.softmax(torch.stack(lses).double(), 0)
    weight = sum(w[..., None] * x.double().abs() for w, x in zip(want, outs))
    total = sum(w[..., None] * x.double() for w, x in zip(want, outs))
    out, lse = torch.empty_like(outs[0]), torch.empty(shape, device=DEV)
    rc.join_attention(outs, lses, out, lse)
    torch.cuda.synchronize()
    bound = weight * (2.0 ** -20 + 176 * 2.0 ** -24) + total.abs() * (4 * 2.0 ** -24 if dtype == "f32" else 2.0 ** -8) + 1e-30
    assert ((out.double() - total).abs() <= bound).all()
    log = torch.logsumexp(torch.stack(lses).double(), 0)
    assert ((lse.double() - log).abs() <= 2.0 ** -20 + 176 * 2.0 ** -24 + 4 * 2.0 ** -24 * log.abs()).all()
    rc.join_attention(outs, lses, outs[0], lses[0])          # in place
    torch.cuda.synchronize()
    assert torch.equal(outs[0], out) and torch.equal(lses[0], lse)


@DTYPES
@pytest.mark.parametrize("qh,kh,dim,lq,bounds", [
    (4, 4, 128, [100 + 7 * i % 31 for i in range(200)], True),        # as many blocks for each sequence
    (4, 4, 128, [100 + 7 * i % 31 for i in range(200)], False),
    (2, 1, 128, [i % 41 for i in range(1100)] + [900], True),         # more sequences than a wave's registers hold
    (4, 2, 64, [1] * 70, False), (4, 2, 64, [1, 0, 2] * 50, False),   # few rows, far fewer than the bounds
])
def test_many_sequences(dtype, qh, kh, dim, lq, bounds):
    rng = np.random.default_rng(len(lq))
    lk = [n + i % 5 for i, n in enumerate(lq)]
    say("[gpu] %d sequences %s bounds %s" % (len(lq), dtype, bounds))
    q, k, v = (rows(rng, sum(n), h, dim, dtype) for n, h in ((lq, qh), (lk, kh), (lk, kh)))
    qo, ko = offsets(lq), offsets(lk)
    out, lse = torch.full_like(q, float("nan")), torch.full((q.shape[0], qh), float("nan"), device=DEV)
    with rc.AttnPlan(qh, kh, dim, dtype, max_seqs=len(lq), max_queries=q.shape[0], max_keys=k.shape[0], causal=True) as p:
        p.attend(q, k, v, ints(qo), out, lse, kv_offsets=ints(ko), **(dict(max_q=max(lq), max_kv=max(lk)) if bounds else {}))
        torch.cuda.synchronize()
    check_all(q, k, v, qo, ko, True, dim ** -0.5, out, lse, dtype)


@DTYPES
@pytest.mark.parametrize("causal", [False, True])
def test_single_tokens_of_many_ragged_sequences(dtype, causal):
    """Few rows in parts, numbered over more than 64 sequences."""
    rng = np.random.default_rng(70)
    say("[gpu] 70 ragged sequences of one token %s" % dtype)
    lk = [1 + i * 977 % 6000 for i in range(70)]
    lk[3], lk[69] = 0, 6001
    q, k, v = rows(rng, 70, 6, 64, dtype), rows(rng, sum(lk), 2, 64, dtype), rows(rng, sum(lk), 2, 64, dtype)
    out, lse = run(q, k, v, [1] * 70, lk, causal, dtype)
    again, sums = run(q, k, v, [1] * 70, lk, causal, dtype)
    assert torch.equal(out, again) and torch.equal(lse, sums)
