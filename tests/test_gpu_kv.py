"""GPU parity of the 8-bit key/value cache (store, select, attend) with the plain
implementation in 64 bits (kv_oracle).

Stores and selections are defined to the bit and compared exactly. Bounds of an
attention output, for A = sum p |v| of that output, S = the largest
sum_d |q_d k_d| * scale of its row, L tokens seen and u = 2^-24 (fp32 rounding):
  scores   q as one f16 (bf16 input: exact) or two (fp32: 2^-22 relative), fp32
           accumulation over D products (twice D for fp32) and three more
           roundings: |ds| <= S * (2^-22 * fp32 + (2 D + 4) u); the exponent's
           argument is rounded once more (its size is at most 2 S / ln 2): + 4 S u,
           and the hardware exponential is good to 2^-21
  p        rounded to f16 (2^-11) or two f16 (2^-21), or lost below 2^-32 of the
           largest (2^-32 per token)
  sums     at most L + 64 fp32 additions: (L + 64) u
so with r = 2 |ds| + 2^-20 + 2 (L + 64) u (numerator and denominator)
  |out - ref| <= A (r + 2^-11 or 2^-21) + L 2^-32 max|v| + |ref| 2^-8 (bf16 output) or 4 u
  |lse - ref| <= |ds| + 2^-20 + (L + 64) u + 4 u |ref|
"""
import numpy as np
import pytest
import torch

import kv_oracle as ko
from gpu_harness import DEV, say
from activation_residual_compression_amd import librescomp as rc

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
FIELDS = ("k", "v", "k_scale", "v_scale", "k_mean", "k_mean_scale")


def to_gpu(cache):
    """KvCache with the contents of an oracle cache."""
    return rc.KvCache(**{n: torch.from_numpy(getattr(cache, n)).to(DEV) for n in FIELDS})


def assert_same(kv, cache, what=""):
    for n in FIELDS:
        got, want = getattr(kv, n).view(torch.uint8 if n in ("k", "v") else getattr(kv, n).dtype).cpu().numpy(), getattr(cache, n)
        assert np.array_equal(got, want), (what, n, np.argwhere(got != want)[:5])


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def values(rng, shape, dtype, spread=1.0):
    """fp32 array and its tensor; bf16 values are exact in both."""
    x = torch.from_numpy((rng.standard_normal(shape) * spread).astype(np.float32))
    t = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return t.float().numpy(), t.to(DEV)


def filled(rng, pool, heads, dim, v_exponents=(-1, 0), k_exponents=(-5, -4)):
    """An oracle cache of random finite codes, scales and consistent means."""
    c = ko.Cache(pool, heads, dim)
    for name in ("k", "v"):
        a = getattr(c, name)
        a[...] = ko.e4m3_encode(rng.standard_normal(a.shape) * 60).reshape(a.shape)
    c.k_scale[...] = 2.0 ** rng.integers(k_exponents[0], k_exponents[1] + 1, c.k_scale.shape)
    c.v_scale[...] = 2.0 ** rng.integers(v_exponents[0], v_exponents[1] + 1, c.v_scale.shape)
    c.k_mean[...] = rng.integers(-127, 128, c.k_mean.shape)
    c.k_mean_scale[...] = rng.random(c.k_mean_scale.shape) + 0.1
    return c


def check_attend(cache, kv, plan_kw, table, lens, q32, q, causal, blocks=None, max_len=0, oracle_blocks=None,
                 gpu_table=None, out=None):
    B, nq, qh, d = q32.shape
    f32 = q.dtype == torch.float32
    plan = rc.KvPlan(batch=B, q_heads=qh, kv_heads=cache.k_scale.shape[1], head_dim=d,
                     pool_blocks=cache.k_scale.shape[0], seq_blocks=table.shape[1], dtype="f32" if f32 else "bf16",
                     causal=causal, **{"max_queries": nq, **plan_kw})
    out = torch.full(q32.shape, 77.0, dtype=q.dtype, device=DEV) if out is None else out
    lse = torch.full(q32.shape[:3], 77.0, device=DEV)
    plan.attend(kv, ints(lens), q, out, lse, table=ints(table) if gpu_table is None else gpu_table, blocks=blocks,
                max_len=max_len)
    torch.cuda.synchronize()
    plan.close()
    got, glse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    scale = plan_kw.get("scale") or 1.0 / np.float64(np.sqrt(np.float32(d)))
    for b in range(B):
        n = max(0, min(lens[b], 64 * table.shape[1], max_len or 1 << 40))
        ob = None if blocks is None else (blocks.cpu().numpy() if oracle_blocks is None else oracle_blocks)[b]
        ref, rlse, A, S = ko.attend(cache, table[b], n, q32[b].astype(np.float64), causal, scale, ob,
                                    plan_kw.get("q_tile", 0))
        ds = S * ((2.0 ** -22 if f32 else 0.0) + (2 * d + 8) * U)
        r = 2 * ds + 2.0 ** -20 + 2 * (n + 64) * U
        vmax = A.max() if A.size else 0.0
        bound = A * (r[..., None] + (2.0 ** -21 if f32 else 2.0 ** -11)) + n * 2.0 ** -32 * vmax + \
            np.abs(ref) * (4 * U if f32 else 2.0 ** -8) + 1e-30
        empty = np.isinf(rlse)
        assert np.array_equal(np.isneginf(glse[b]), empty), "rows without tokens"
        assert (got[b][empty] == 0).all()
        err = np.abs(got[b] - ref)
        assert (err <= bound).all(), (b, np.argwhere(err > bound)[:4], (err / bound).max())
        le = np.abs(np.where(empty, 0, glse[b]) - np.where(empty, 0, rlse))
        assert (le <= ds + 2.0 ** -20 + (n + 64) * U + 4 * U * np.abs(np.where(empty, 0, rlse))).all(), le.max()
    return out, lse


# ------------------------------------------------------------------ store
@pytest.mark.parametrize("dim,heads", [(64, 3), (128, 2)])
@pytest.mark.parametrize("kd,vd", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_store_whole_and_append(dim, heads, kd, vd):
    rng = np.random.default_rng(dim + heads)
    pool, nb = 14, 4
    cache = ko.Cache(pool, heads, dim, fill=0x7F)          # stale codes are NaN
    kv = to_gpu(cache)
    table = rng.permutation(pool)[:3 * nb].reshape(3, nb).astype(np.int32)
    plan = rc.KvPlan(batch=3, q_heads=heads, kv_heads=heads, head_dim=dim, pool_blocks=pool, seq_blocks=nb)
    # (starts, tokens, counts, spread): whole, appends inside and across blocks, growing scales, rollback, past the end
    steps = [((0, 0, 0), 130, (130, 64, 1), 1.0), ((130, 64, 1), 1, None, 1.0), ((131, 65, 2), 3, None, 40.0),
             ((134, 68, 5), 1, None, 3000.0), ((100, 67, 0), 70, (70, 0, 61), 0.01), ((170, 67, 61), 5, None, 1.0),
             ((250, 256, -3), 9, None, 1.0), ((5, 63, 64), 1, None, 1e-3)]
    for starts, n, counts, spread in steps:
        say("[gpu] store %d at %s" % (n, starts))
        k32, kt = values(rng, (3, n, heads, dim), kd, spread)
        v32, vt = values(rng, (3, n, heads, dim), vd, spread)
        cache.store(table, starts, counts or (n,) * 3, k32.astype(np.float64), v32.astype(np.float64))
        plan.store(kv, ints(starts), kt, vt, table=ints(table), count=None if counts is None else ints(counts))
        torch.cuda.synchronize()
        assert_same(kv, cache, starts)
    plan.close()


def test_store_ranges_and_non_finite():
    """Zero blocks, values at and past the range of scales, ties at 448 * 2^e, infinities and NaN."""
    rng = np.random.default_rng(3)
    for spread, special in ((0.0, ()), (1e-30, ()), (3e14, ()), (1e30, ()), (1.0, (np.inf, -np.inf, np.nan)),
                            (1e-3, (448.0, 448.0 * (1 + 2 ** -23), -448.0))):
        cache = ko.Cache(2, 1, 64)
        kv = to_gpu(cache)
        x = (rng.standard_normal((1, 70, 1, 64)) * spread).astype(np.float32)
        for i, s in enumerate(special):
            x[0, 5 + i, 0, 3 * i] = s
        t = torch.from_numpy(x).to(DEV)
        say("[gpu] store range %g %s" % (spread, special))
        with rc.KvPlan(batch=1, q_heads=1, kv_heads=1, head_dim=64, pool_blocks=2, seq_blocks=2) as plan:
            plan.store(kv, ints([0]), t, t)
            torch.cuda.synchronize()
        with np.errstate(all="ignore"):
            cache.store(np.array([[0, 1]]), [0], [70], x.astype(np.float64), x.astype(np.float64))
        assert_same(kv, cache, spread)


def test_store_strided_views_missing_blocks_and_no_tokens():
    rng = np.random.default_rng(9)
    heads, dim, n = 2, 128, 100
    cache = ko.Cache(4, heads, dim)
    kv = to_gpu(cache)
    table = np.array([[3, -1], [9, 1]], np.int32)           # two entries outside the pool
    x32, x = values(rng, (n, 2, 3 * heads + 1, dim), "bf16")   # tokens first, q | k | v side by side
    k, v = x[:, :, 1:1 + heads].transpose(0, 1), x[:, :, 1 + heads:1 + 2 * heads].transpose(0, 1)
    with rc.KvPlan(batch=2, q_heads=heads, kv_heads=heads, head_dim=dim, pool_blocks=4, seq_blocks=2) as plan:
        plan.store(kv, ints([0, 10]), k[:, :0], v[:, :0], table=ints(table))
        plan.store(kv, ints([0, 10]), k, v, table=ints(table))
        torch.cuda.synchronize()
    k64 = x32[:, :, 1:1 + heads].transpose(1, 0, 2, 3).astype(np.float64)
    v64 = x32[:, :, 1 + heads:1 + 2 * heads].transpose(1, 0, 2, 3).astype(np.float64)
    cache.store(table, [0, 10], [n, n], k64, v64)
    assert_same(kv, cache)


# ------------------------------------------------------------------ attend
LAYOUTS = [(1, 1), (4, 1), (6, 2), (3, 3), (20, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("qh,kh", LAYOUTS)
@pytest.mark.parametrize("nq,causal", [(1, True), (2, False), (17, True), (65, False), (130, True)])
def test_attend_layouts_and_lengths(dtype, dim, qh, kh, nq, causal):
    rng = np.random.default_rng(qh * 100 + nq)
    lens = [0, 1, 63, 64, 65, 200, 256, 1000]                # 1000: past the table, cut to 256
    nb, B = 4, 8
    cache = filled(rng, B * nb + 3, kh, dim)
    table = rng.permutation(B * nb + 3)[:B * nb].reshape(B, nb).astype(np.int32)
    table[5, 1], table[6, 0], table[6, 3] = -1, 10 ** 6, -5  # blocks that are not there
    for b in (1, 3, 5):                                      # stale codes after a sequence's end are NaN
        last = table[b, lens[b] // 64]
        if 0 <= last and lens[b] % 64:
            for h in range(kh):
                kc, vc = cache.k_codes(last, h).copy(), cache.v_codes(last, h).copy()
                kc[lens[b] % 64:], vc[lens[b] % 64:] = 0x7F, 0xFF
                cache.put(last, h, kc, vc)
    q32, q = values(rng, (B, nq, qh, dim), dtype, 0.7)
    q32[2], q[2] = 0.0, 0.0                                  # a row of zeros: equal weights
    say("[gpu] attend %s %d heads %d/%d queries %d causal %d" % (dtype, dim, qh, kh, nq, causal))
    check_attend(cache, to_gpu(cache), {}, table, lens, q32, q, causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 5, 70, 300])
def test_attend_long_split_over_keys(dtype, nq):
    """One sequence, one head: the keys are split over many blocks of threads and joined."""
    rng = np.random.default_rng(nq)
    n = 64 * 41 + 13
    cache = filled(rng, 42, 1, 128)
    q32, q = values(rng, (1, nq, 1, 128), dtype, 1.5)
    table = rng.permutation(42).reshape(1, 42).astype(np.int32)
    kv = to_gpu(cache)
    say("[gpu] attend split %s %d" % (dtype, nq))
    a = check_attend(cache, kv, {}, table, [n], q32, q, False)
    b = check_attend(cache, kv, {}, table, [n], q32, q, False)
    assert all(torch.equal(x, y) for x, y in zip(a, b))      # the order of every sum is fixed
    check_attend(cache, kv, {"max_queries": 400, "scale": 0.3}, table, [n], q32, q, True, max_len=n)
    check_attend(cache, kv, {}, table, [n], q32, q, False, max_len=777)


@pytest.mark.parametrize("nq", [3, 129])
def test_attend_block_scales_far_apart(nq):
    """Values whose block scales differ by up to 2^84 (what fp32 holds of them), and large scores."""
    rng = np.random.default_rng(nq)
    cache = filled(rng, 8, 2, 64, v_exponents=(-40, 44), k_exponents=(-6, -2))
    cache.v_scale[0], cache.v_scale[7] = 2.0 ** 44, 2.0 ** -40
    q32, q = values(rng, (1, nq, 2, 64), "f32", 0.5)
    q32[:, :, 1] *= 30
    q[:, :, 1] *= 30
    say("[gpu] attend scales %d" % nq)
    check_attend(cache, to_gpu(cache), {}, np.arange(8, dtype=np.int32)[None], [500], q32, q, False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [3, 129])
def test_attend_zero_rows_and_blocks_at_a_small_scale(dtype, nq):
    """Masked tokens weigh nothing where the factor of the scores underflows: rows of zeros,
    blocks of zeros at the smallest scale, and a scale of 1e-12."""
    rng = np.random.default_rng(nq)
    cache = filled(rng, 4, 1, 64, k_exponents=(-40, -40))
    cache.k[1:] = 0
    kv = to_gpu(cache)
    q32, q = values(rng, (1, nq, 1, 64), dtype)
    q32[:, ::2] = 0
    q[:, ::2] = 0
    for causal in (True, False):
        say("[gpu] zero rows %s %d causal %s" % (dtype, nq, causal))
        check_attend(cache, kv, dict(scale=1e-12), np.array([[1, 0, 3, 2]], np.int32), [230], q32, q, causal)


@pytest.mark.parametrize("nq", [2, 140])
def test_attend_strided_queries_and_outputs(nq):
    rng = np.random.default_rng(nq)
    qh, kh, d = 4, 2, 64
    cache = filled(rng, 6, kh, d)
    x32, x = values(rng, (nq, 2, qh + 3, d), "bf16")
    big = torch.full((qh + 1, 2, nq, d), 5.0, dtype=torch.bfloat16, device=DEV)
    say("[gpu] attend strides %d" % nq)
    check_attend(cache, to_gpu(cache), {}, np.arange(6, dtype=np.int32).reshape(2, 3), [150, 190],
                 x32[:, :, 2:2 + qh].transpose(1, 0, 2, 3), x[:, :, 2:2 + qh].transpose(0, 1), False,
                 out=big[1:].permute(1, 2, 0, 3))
    assert (big[0] == 5.0).all()                             # nothing outside the view is written


def test_attend_broadcast_queries_without_lse():
    rng = np.random.default_rng(1)
    cache = filled(rng, 4, 2, 128)
    kv = to_gpu(cache)
    q32, q = values(rng, (1, 1, 1, 128), "bf16")
    q = q.expand(2, 3, 2, 128)
    out = torch.empty(2, 3, 2, 128, dtype=torch.bfloat16, device=DEV)
    with rc.KvPlan(batch=2, q_heads=2, kv_heads=2, head_dim=128, pool_blocks=4, seq_blocks=2, max_queries=3) as plan:
        plan.attend(kv, ints([100, 100]), q, out)            # table: None, blocks in order
        torch.cuda.synchronize()
    check_attend(cache, kv, {}, np.arange(4, dtype=np.int32).reshape(2, 2), [100, 100],
                 np.broadcast_to(q32, (2, 3, 2, 128)), q, False)
    assert torch.equal(out[:, 0], out[:, 2])


def test_attend_block_past_32_bits():
    """Blocks whose bytes lie beyond 2^32 in the cache."""
    heads, dim = 8, 128
    pool = 2 ** 32 // (heads * 64 * dim) + 3
    rng = np.random.default_rng(2)
    small = filled(rng, 3, heads, dim)
    kv = rc.KvCache.empty(pool, heads, dim, DEV)
    q32, q = values(rng, (1, 1, heads, dim), "bf16")
    for n in FIELDS:
        getattr(kv, n).view(torch.uint8 if n in ("k", "v") else getattr(kv, n).dtype)[pool - 3:] = \
            torch.from_numpy(getattr(small, n)).to(DEV)
    k32, k = values(rng, (1, 5, heads, dim), "bf16")
    lse, out = torch.empty(1, 1, heads, device=DEV), torch.empty_like(q)
    say("[gpu] attend past 2^32 bytes, pool %d" % pool)
    with rc.KvPlan(batch=1, q_heads=heads, kv_heads=heads, head_dim=dim, pool_blocks=pool, seq_blocks=3, q_tile=1,
                   keep_blocks=2) as plan:
        table = ints([[pool - 1, pool - 3, pool - 2]])
        plan.store(kv, ints([126]), k, k, table=table)
        blocks = torch.empty(1, heads, 1, 2, dtype=torch.int32, device=DEV)
        plan.select(kv, ints([131]), q, blocks, table=table)
        plan.attend(kv, ints([131]), q, out, lse, table=table)
        torch.cuda.synchronize()
    order = np.array([[2, 0, 1]], np.int32)
    small.store(order, [126], [5], k32.astype(np.float64), k32.astype(np.float64))
    for n in FIELDS:
        got = getattr(kv, n).view(torch.uint8 if n in ("k", "v") else getattr(kv, n).dtype)[pool - 3:].cpu().numpy()
        assert np.array_equal(got, getattr(small, n)), n
    assert np.array_equal(blocks.cpu().numpy()[0], ko.select(small, order[0], 131, q32[0], False, 1, 2))
    got, glse = check_attend(small, to_gpu(small), {}, order, [131], q32, q, False)
    assert torch.equal(got, out) and torch.equal(glse, lse)


# ------------------------------------------------------------------ select
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("qh,kh,dim", [(1, 1, 64), (6, 2, 64), (8, 1, 128), (3, 3, 128)])
@pytest.mark.parametrize("nq,q_tile,keep,causal", [(1, 1, 3, True), (3, 1, 5, False), (5, 1, 1, True),
                                                   (130, 128, 4, False), (200, 128, 3, True), (7, 128, 64, True)])
def test_select_and_attend(dtype, qh, kh, dim, nq, q_tile, keep, causal):
    rng = np.random.default_rng(nq + dim + keep)
    lens, nb, B = [640, 0, 333, 129], 10, 4
    cache = filled(rng, B * nb, kh, dim)
    cache.k_mean[cache.k_scale.shape[0] // 2:] = cache.k_mean[0]                 # equal scores: ties
    cache.k_mean_scale[cache.k_scale.shape[0] // 2:] = cache.k_mean_scale[0]
    table = rng.permutation(B * nb).reshape(B, nb).astype(np.int32)
    table[0, 4], table[2, 0] = -1, B * nb
    kv = to_gpu(cache)
    q32, q = values(rng, (B, nq, qh, dim), dtype)
    if nq > 2:
        q32[3, 1], q[3, 1] = 0.0, 0.0                                            # scores of zero
    want = np.stack([ko.select(cache, table[b], lens[b], q32[b], causal, q_tile, keep) for b in range(B)])
    blocks = torch.full(want.shape, 12345, dtype=torch.int32, device=DEV)
    say("[gpu] select %s %d/%d %d queries %d tile %d keep %d causal %d" % (dtype, qh, kh, dim, nq, q_tile, keep, causal))
    kw = dict(q_tile=q_tile, keep_blocks=keep)
    with rc.KvPlan(batch=B, q_heads=qh, kv_heads=kh, head_dim=dim, pool_blocks=B * nb, seq_blocks=nb, dtype=dtype,
                   max_queries=nq, causal=causal, **kw) as plan:
        plan.select(kv, ints(lens), q, blocks, table=ints(table))
        torch.cuda.synchronize()
    assert np.array_equal(blocks.cpu().numpy(), want)
    check_attend(cache, kv, kw, table, lens, q32, q, causal, blocks=blocks)


def test_select_many_blocks_and_close_scores():
    """Thousands of blocks, scores that share their leading bits, and long runs of ties at the last place."""
    rng = np.random.default_rng(4)
    nb, dim = 5000, 64
    cache = ko.Cache(nb, 1, dim)
    cache.k_mean[...] = rng.integers(-2, 3, cache.k_mean.shape)
    cache.k_mean[1000:3000] = cache.k_mean[17]
    cache.k_mean_scale[...] = 0.5
    q32, q = values(rng, (1, 1, 1, dim), "f32")
    kv = to_gpu(cache)
    table = np.arange(nb, dtype=np.int32)[None]
    for keep in (1, 100, 1000):
        want = ko.select(cache, table[0], 64 * nb - 5, q32[0], False, 1, keep)
        blocks = torch.empty(1, 1, 1, keep, dtype=torch.int32, device=DEV)
        say("[gpu] select %d of %d" % (keep, nb))
        with rc.KvPlan(batch=1, q_heads=1, kv_heads=1, head_dim=dim, pool_blocks=nb, seq_blocks=nb, dtype="f32",
                       q_tile=1, keep_blocks=keep) as plan:
            plan.select(kv, ints([64 * nb - 5]), q, blocks)
            torch.cuda.synchronize()
        assert np.array_equal(blocks.cpu().numpy()[0], want)


def test_attend_lists_that_hold_anything():
    """Entries past a sequence's end and past the table end a list; no list, no output."""
    rng = np.random.default_rng(8)
    cache = filled(rng, 4, 1, 64)
    kv = to_gpu(cache)
    table = np.arange(4, dtype=np.int32)[None]
    for nq in (1, 128):
        for lst in ([-1, 5, 6], [0, 2, 2 ** 30], [1, 4, 3], [2, 3, -7]):
            q32, q = values(rng, (1, nq, 1, 64), "bf16")
            blocks = ints([[[lst]]])
            end = next((i for i, j in enumerate(lst) if not 0 <= j < 4), 3)
            ob = np.array([[[lst[:end] + [-1] * (3 - end)]]])
            check_attend(cache, kv, dict(q_tile=1 if nq == 1 else 128, keep_blocks=3), table, [250], q32, q, False,
                         blocks=blocks, oracle_blocks=ob)


# ------------------------------------------------------------------ streams, graphs, refusals on the device
def test_streams_and_graph_replays():
    """A decode step (store one token, select, attend) on a stream of its own and as a captured graph, replayed
    with the lengths moving on in between, equals the eager calls each time."""
    rng = np.random.default_rng(6)
    B, qh, kh, d, nb = 3, 4, 2, 128, 6
    lens = [5, 200, 300]
    side = torch.cuda.Stream()
    eager, graphed = (rc.KvCache.empty(B * nb, kh, d, DEV) for _ in range(2))
    kw = dict(batch=B, q_heads=qh, kv_heads=kh, head_dim=d, pool_blocks=B * nb, seq_blocks=nb, causal=True)
    pe, pg = rc.KvPlan(**kw, q_tile=1, keep_blocks=3), rc.KvPlan(**kw, q_tile=1, keep_blocks=3)
    _, full = values(rng, (B, max(lens), kh, d), "bf16")
    at, blocks = ints(lens), [torch.empty(B, kh, 1, 3, dtype=torch.int32, device=DEV) for _ in range(2)]
    q, k, v = (torch.empty(B, 1, h, d, dtype=torch.bfloat16, device=DEV) for h in (qh, kh, kh))
    out, lse = [torch.empty_like(q) for _ in range(2)], [torch.empty(B, 1, qh, device=DEV) for _ in range(2)]
    grown = torch.empty_like(at)
    torch.cuda.synchronize()

    def step(plan, cache, i, stream):
        plan.store(cache, at, k, v, stream=stream)
        plan.select(cache, grown, q, blocks[i], stream=stream)
        plan.attend(cache, grown, q, out[i], lse[i], blocks=blocks[i], stream=stream)

    for cache, plan in ((eager, pe), (graphed, pg)):
        plan.store(cache, ints([0] * B), full, full, count=at)
    grown.copy_(at + 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(pg, graphed, 1, torch.cuda.current_stream())
    for n in range(4):
        q.copy_(values(rng, q.shape, "bf16")[1])
        k.copy_(values(rng, k.shape, "bf16")[1])
        v.copy_(values(rng, v.shape, "bf16")[1])
        grown.copy_(at + 1)
        torch.cuda.synchronize()
        step(pe, eager, 0, side)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], out[1]) and torch.equal(lse[0], lse[1]) and torch.equal(blocks[0], blocks[1]), n
        for f in FIELDS:
            assert torch.equal(getattr(eager, f).view(torch.uint8), getattr(graphed, f).view(torch.uint8)), (n, f)
        at.add_(1)
        torch.cuda.synchronize()
    pe.close()
    pg.close()


def test_binding_refusals_on_device_tensors():
    kv = rc.KvCache.empty(4, 2, 64, DEV)
    x = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device=DEV)
    lens = ints([1, 2])
    with rc.KvPlan(batch=2, q_heads=4, kv_heads=2, head_dim=64, pool_blocks=4, seq_blocks=2, max_queries=3, q_tile=1,
                   keep_blocks=2) as p:
        for bad in (x[:1], x[:, :, :3], x[..., :32], x.float(), x.transpose(2, 3), x.double()):
            with pytest.raises(ValueError):
                p.attend(kv, lens, bad, x.clone())
        with pytest.raises(ValueError):
            p.attend(kv, lens, x, x[:, :2].clone())
        for ln in (lens.long(), lens[:1], lens.cpu(), ints([1, 0, 2, 0])[::2]):
            with pytest.raises(ValueError):
                p.attend(kv, ln, x, x.clone())
        with pytest.raises(ValueError):
            p.attend(kv, lens, x, x.clone(), table=ints([[0, 1, 2], [0, 1, 2]]))
        with pytest.raises(ValueError):
            p.attend(kv, lens, x, x.clone(), lse=torch.zeros(2, 3, 3, device=DEV))
        with pytest.raises(ValueError):
            p.attend(kv, lens, x, x.clone(), blocks=torch.zeros(2, 2, 3, 1, dtype=torch.int32, device=DEV))
        with pytest.raises(ValueError):
            p.store(kv, lens, x[:, :, :2], x[:, :2, :2])
        with pytest.raises(ValueError):
            p.store(rc.KvCache.empty(5, 2, 64, DEV), lens, x[:, :, :2], x[:, :, :2])
        with pytest.raises(rc.RcError) as ei:                # rows that are not 16-byte aligned
            wide = torch.zeros(2, 3, 4, 68, dtype=torch.bfloat16, device=DEV)
            p.attend(kv, lens, wide[..., 2:66], x.clone())
        assert ei.value.status == rc.RC_ERR_ALIGNMENT
