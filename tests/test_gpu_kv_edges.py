"""The 8-bit key/value cache at its edges, against 64 bits (kv_dense; the bounds are the
ones that test_gpu_kv derives)."""
import numpy as np
import pytest
import torch

import kv_dense
import kv_oracle as ko
from gpu_harness import DEV, say
from activation_residual_compression_amd import librescomp as rc
from test_gpu_kv import filled, ints, to_gpu, values

pytestmark = pytest.mark.gpu


def as_query(x, dtype):
    """fp32 array -> (what the library sees, device tensor)."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return t.float().numpy(), t.to(DEV)


def new_plan(cache, table, q, causal, **kw):
    B, nq, qh, d = q.shape
    return rc.KvPlan(batch=B, q_heads=qh, kv_heads=cache.k_scale.shape[1], head_dim=d, pool_blocks=cache.k_scale.shape[0],
                     seq_blocks=table.shape[1], dtype="f32" if q.dtype == torch.float32 else "bf16", causal=causal,
                     **{"max_queries": nq, **kw})


def run(plan, kv, table, lens, q, blocks=None, max_len=0):
    out = torch.full(q.shape, 77.0, dtype=q.dtype, device=DEV)
    lse = torch.full(q.shape[:3], 77.0, device=DEV)
    plan.attend(kv, ints(lens), q, out, lse, table=ints(table), blocks=blocks, max_len=max_len)
    torch.cuda.synchronize()
    return out, lse


def check(cache, table, lens, q32, causal, out, lse, lists=None, q_tile=0, scale=0.0, which=None, max_len=0):
    """What run returned, for all sequences or those of `which`."""
    d = q32.shape[3]
    for b in range(q32.shape[0]) if which is None else which:
        n = max(0, min(int(lens[b]), 64 * table.shape[1], max_len or 1 << 40))
        ref = kv_dense.attend(cache, table[b], n, q32[b].astype(np.float64), causal,
                              float(np.float32(scale)) or 1.0 / np.float64(np.sqrt(np.float32(d))),
                              None if lists is None else lists[b], q_tile)
        kv_dense.check(out[b].double().cpu().numpy(), lse[b].double().cpu().numpy(), ref, n, d, out.dtype == torch.float32)


# ------------------------------------------------------------------ not finite
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nq,n", [(3, 200), (3, 64 * 40 + 13), (130, 300), (130, 64 * 40 + 13)])
@pytest.mark.parametrize("what", ["key", "value", "query", "infinite query"])
def test_nan_reaches_the_queries_that_see_it(dtype, dim, nq, n, what):
    """In the output and in its log-sum-exp (a value's in the output alone), and no other
    query: one part of the keys and several, few rows and many."""
    rng = np.random.default_rng(nq + n)
    nb = -(-n // 64)
    cache = filled(rng, nb, 2, dim)
    table = rng.permutation(nb).reshape(1, nb).astype(np.int32)
    q32, _ = values(rng, (1, nq, 4, dim), dtype, 0.7)
    at = n - nq // 2 - 1                                        # with a causal mask half of the queries see it
    kc, vc = (c(table[0, at // 64], 0).copy() for c in (cache.k_codes, cache.v_codes))
    if what == "key":
        kc[at % 64, 7] = 0xFF
    elif what == "value":
        vc[at % 64, 3], vc[at % 64, dim - 1] = 0xFF, 0x7F
    else:
        q32[0, 1, 2, 5] = np.nan if what == "query" else np.inf
    cache.put(table[0, at // 64], 0, kc, vc)
    kv = to_gpu(cache)
    q32, q = as_query(q32, dtype)
    for causal in (True, False):
        say("[gpu] %s nan %s %d queries %d over %d causal %d" % (what, dtype, dim, nq, n, causal))
        with new_plan(cache, table, q, causal) as plan:
            out, lse = run(plan, kv, table, [n], q)
        check(cache, table, [n], q32, causal, out, lse)


@pytest.mark.parametrize("nq,n", [(3, 200), (3, 64 * 40 + 13), (130, 300), (130, 64 * 40 + 13)])
@pytest.mark.parametrize("bits", [0x7F81, 0x7FFF, -1, -127])
def test_nan_of_any_payload_stays_nan_in_bf16(nq, n, bits):
    """bf16 queries that hold a NaN of any sign and payload (int16 bits)."""
    rng = np.random.default_rng(nq + n)
    nb = -(-n // 64)
    cache = filled(rng, nb, 2, 64)
    table = rng.permutation(nb).reshape(1, nb).astype(np.int32)
    q32, q = values(rng, (1, nq, 4, 64), "bf16", 0.7)
    q.view(torch.int16)[0, 1, 2] = bits
    q32[0, 1, 2] = np.nan
    say("[gpu] nan bits %x, %d queries over %d" % (bits & 0xFFFF, nq, n))
    with new_plan(cache, table, q, True) as plan:
        out, lse = run(plan, to_gpu(cache), table, [n], q)
    check(cache, table, [n], q32, True, out, lse)


# ------------------------------------------------------------------ the range of queries
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [3, 130])
@pytest.mark.parametrize("exponent", [127, 120, 116, 115, -86, -90, -110])
def test_queries_at_the_ends_of_the_range(dtype, nq, exponent):
    """Rows whose largest value is 2^exponent or a little less, at a scale of the scores
    that brings them to ordinary sizes (for small ones, with large keys)."""
    rng = np.random.default_rng(nq)
    cache = filled(rng, 4, 2, 64, k_exponents=(-5, -4) if exponent > 0 else (20, 21))
    q32 = rng.uniform(-0.99, 0.99, (1, nq, 2, 64)) * 2.0 ** (exponent + (0 if exponent > 126 else 1))
    q32, q = as_query(q32, dtype)
    table = np.array([[2, 0, 3, 1]], np.int32)
    scale = 2.0 ** -min(exponent + 5, 126) if exponent > 0 else 2.0 ** -(exponent + 30)
    say("[gpu] queries of 2^%d %s %d" % (exponent, dtype, nq))
    for causal in (True, False):
        with new_plan(cache, table, q, causal, scale=scale) as plan:
            out, lse = run(plan, to_gpu(cache), table, [250], q)
        check(cache, table, [250], q32, causal, out, lse, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [3, 130])
def test_keys_of_zero_at_the_largest_scale_weigh_alike(dtype, nq):
    """Scores of zero, where the row's power of two times the block's passes fp32."""
    rng = np.random.default_rng(nq)
    cache = filled(rng, 4, 1, 64, k_exponents=(44, 44))
    cache.k[...] = 0
    q32, q = as_query(rng.uniform(-0.99, 0.99, (1, nq, 1, 64)) * 2.0 ** 127, dtype)
    table = np.arange(4, dtype=np.int32)[None]
    say("[gpu] zero keys, queries of 2^127, %s %d" % (dtype, nq))
    with new_plan(cache, table, q, True, scale=1.0) as plan:
        out, lse = run(plan, to_gpu(cache), table, [250], q)
    check(cache, table, [250], q32, True, out, lse, scale=1.0)


# ------------------------------------------------------------------ choice of blocks
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,kh", [(64, 1), (128, 2)])
@pytest.mark.parametrize("nq,q_tile,keep,causal", [(1, 1, 3, True), (3, 1, 3, False), (5, 1, 1, True), (3, 1, 40, True),
                                                   (130, 128, 4, True), (130, 128, 4, False), (7, 128, 64, False)])
@pytest.mark.parametrize("what", ["infinite query", "nan query", "scores past fp32", "mean of scale nan"])
def test_select_scores_that_are_not_finite(dtype, dim, kh, nq, q_tile, keep, causal, what):
    """A block that is there and seen can be chosen whatever its score, and the tile's own
    come first: a query that holds an infinity reaches attention, and its output is NaN."""
    rng = np.random.default_rng(nq + dim + keep)
    lens, nb = [640, 333], 10
    cache = filled(rng, 2 * nb, kh, dim)
    table = rng.permutation(2 * nb).reshape(2, nb).astype(np.int32)
    table[0, 4] = -1
    q32, _ = values(rng, (2, nq, 2 * kh, dim), dtype)
    if what == "infinite query":
        q32[:, nq // 2, :, 3] = np.inf
        q32[:, 0, 0, 9] = -np.inf
    elif what == "nan query":
        q32[:, nq // 2, :, 3] = np.nan
        q32[:, 0, 0] = np.nan
    elif what == "scores past fp32":
        q32[:, ::2] *= np.float32(2.0 ** 115)
        cache.k_mean_scale[...] *= np.float32(2.0 ** 5)
    else:
        cache.k_mean_scale[table[0, 1]] = np.nan
        cache.k_mean_scale[table[1, 5]] = np.nan
    kv = to_gpu(cache)
    q32, q = as_query(q32, dtype)
    want = np.stack([kv_dense.choose(cache, table[b], lens[b], q32[b], causal, q_tile, keep) for b in range(2)])
    blocks = torch.full(want.shape, 12345, dtype=torch.int32, device=DEV)
    say("[gpu] select %s %s %d/%d queries %d tile %d keep %d causal %d" % (what, dtype, dim, kh, nq, q_tile, keep, causal))
    with new_plan(cache, table, q, causal, q_tile=q_tile, keep_blocks=keep) as plan:
        plan.select(kv, ints(lens), q, blocks, table=ints(table))
        torch.cuda.synchronize()
        assert np.array_equal(blocks.cpu().numpy(), want)
        out, lse = run(plan, kv, table, lens, q, blocks=blocks)
    if what != "scores past fp32":                              # there the scores of attention are as large
        check(cache, table, lens, q32, causal, out, lse, want, q_tile)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_select_rows_near_the_smallest_numbers(dtype):
    """Rows whose factor 127 / max|q| passes fp32 score 0: ties, the lowest blocks."""
    rng = np.random.default_rng(12)
    cache = filled(rng, 8, 1, 64)
    kv = to_gpu(cache)
    table = np.arange(8, dtype=np.int32)[None]
    q32, _ = values(rng, (1, 4, 1, 64), dtype)
    for i, size in enumerate((2.0 ** -120, 2.0 ** -124, 1e-38, 2e-40)):
        q32[0, i] *= np.float32(size) / np.abs(q32[0, i]).max()
    q32, q = as_query(q32, dtype)
    want = kv_dense.choose(cache, table[0], 512, q32[0], False, 1, 3)
    assert np.array_equal(want[0, 1:], np.tile([0, 1, 2], (3, 1)))
    blocks = torch.empty((1,) + want.shape, dtype=torch.int32, device=DEV)
    say("[gpu] select of tiny rows %s" % dtype)
    with new_plan(cache, table, q, False, q_tile=1, keep_blocks=3) as plan:
        plan.select(kv, ints([512]), q, blocks)
        torch.cuda.synchronize()
    assert np.array_equal(blocks.cpu().numpy()[0], want)


# ------------------------------------------------------------------ lists
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("qh,nq,n", [(1, 60, 300), (1, 128, 640), (2, 128, 640), (4, 16, 300)])
@pytest.mark.parametrize("entries", [[-1, 0], [-1, -2, 0], [-2, -1, -3], [1, 1, 0], [0, -1, 0, -1], [-1, 0, 99, 1], [-1]])
def test_lists_in_any_order(dtype, qh, nq, n, entries):
    """A tile's list, counted from the last block that the tile sees where negative, in the
    order given, with entries that repeat: rows that do not see a block yet go on after it."""
    rng = np.random.default_rng(nq + n)
    nb = 11
    cache = filled(rng, nb, 1, 64)
    table = rng.permutation(nb).reshape(1, nb).astype(np.int32)
    q32, q = values(rng, (1, nq, qh, 64), dtype)
    last = -(-n // 64)
    lst = [last + j if j < 0 else j for j in entries]
    keep = 5
    lists = np.full((1, 1, 1, keep), -1, np.int32)
    lists[0, 0, 0, :len(lst)] = lst
    say("[gpu] list %s %s %d queries of %d heads" % (lst, dtype, nq, qh))
    with new_plan(cache, table, q, True, q_tile=128, keep_blocks=keep) as plan:
        out, lse = run(plan, to_gpu(cache), table, [n], q, blocks=ints(lists))
    check(cache, table, [n], q32, True, out, lse, lists, 128)


# ------------------------------------------------------------------ keys split over blocks of threads
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("qh,kh", [(4, 2), (3, 3), (20, 1)])
def test_one_plan_many_calls_in_several_parts(dtype, dim, qh, kh):
    """Several sequences of very different lengths, heads and groups, one plan for calls of
    changing numbers of queries and bounds of the lengths: each against 64 bits."""
    rng = np.random.default_rng(dim + qh)
    nb, lens = 40, [64 * 40, 0, 1, 700, 64 * 39 + 5]
    B = len(lens)
    cache = filled(rng, 2 * nb, kh, dim)
    table = rng.integers(0, 2 * nb, (B, nb)).astype(np.int32)      # sequences may share what they read
    table[3, 2], table[4, 20] = -1, 2 * nb
    kv = to_gpu(cache)
    for causal in (True, False):
        q32, q = values(rng, (B, 150, qh, dim), dtype)
        with new_plan(cache, table, q, causal) as plan:
            assert plan.workspace_bytes > 0                       # it has several parts at these sizes
            for nq, max_len in ((1, 0), (1, 0), (150, 0), (2, 0), (150, 1000), (1, 1500), (70, 0), (1, 100), (150, 0), (1, 0)):
                say("[gpu] parts %s %d heads %d/%d queries %d max %d causal %d" % (dtype, dim, qh, kh, nq, max_len, causal))
                i = int(rng.integers(0, 151 - nq))
                out, lse = run(plan, kv, table, lens, q[:, i:i + nq], max_len=max_len)
                check(cache, table, lens, q32[:, i:i + nq], causal, out, lse, max_len=max_len)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ascending", [True, False])
@pytest.mark.parametrize("nq,q_tile", [(1, 1), (3, 1), (128, 128), (200, 128)])
def test_long_lists_in_several_parts(dtype, nq, q_tile, ascending):
    """Lists of more than 64 entries, some missing, for ragged sequences; twice on one plan."""
    rng = np.random.default_rng(nq)
    nb, keep, lens = 130, 100, [64 * 130, 64 * 70 + 3, 0]
    cache = filled(rng, 140, 2, 64)
    table = np.stack([rng.permutation(140)[:nb] for _ in lens]).astype(np.int32)
    table[0, 3] = -1
    q32, q = values(rng, (3, nq, 4, 64), dtype)
    tiles = -(-nq // q_tile)
    lists = np.full((3, 2, tiles, keep), -1, np.int32)
    for b, n in enumerate(lens):
        for h in range(2):
            for t in range(tiles):
                some = rng.permutation(max(1, -(-n // 64)))[:keep - 7 * t]
                some = np.sort(some) if ascending else some
                lists[b, h, t, :len(some)] = some
    kv = to_gpu(cache)
    with new_plan(cache, table, q, True, q_tile=q_tile, keep_blocks=keep) as plan:
        for again in range(2):
            say("[gpu] long lists %s queries %d call %d" % (dtype, nq, again))
            out, lse = run(plan, kv, table, lens, q, blocks=ints(lists))
            check(cache, table, lens, q32, True, out, lse, lists, q_tile)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,nq", [(768, 1), (512, 65)])
def test_more_than_256_blocks_in_one_part(dtype, B, nq):
    """A wave walks more than 64 blocks: so many sequences that none is split. All but the
    last two are the same one, and equal to the bit."""
    rng = np.random.default_rng(B)
    nb, n = 300, 64 * 300 - 9
    cache = filled(rng, nb, 1, 64)
    table = np.tile(rng.permutation(nb).astype(np.int32), (B, 1))
    table[B - 2] = rng.permutation(nb)
    table[B - 1, 4:280] = -1
    lens = [n] * (B - 1) + [64 * 290]
    q32, q = values(rng, (1, nq, 1, 64), dtype)
    q, q32 = q.expand(B, nq, 1, 64), np.broadcast_to(q32, (B, nq, 1, 64))
    say("[gpu] %d sequences of %d blocks, %d queries, %s" % (B, nb, nq, dtype))
    with new_plan(cache, table, q, False) as plan:
        out, lse = run(plan, to_gpu(cache), table, lens, q)
    assert all(torch.equal(x[1:B - 2], x[:1].expand_as(x[1:B - 2])) for x in (out, lse))
    check(cache, table, lens, q32, False, out, lse, which=(0, B - 2, B - 1))


@pytest.mark.parametrize("nq,q_tile", [(1, 0), (1, 1), (70, 0)])
def test_graph_replays_of_calls_in_several_parts(nq, q_tile):
    """A captured call whose keys are split, replayed while the lengths move, with the
    plan's own eager calls between the replays."""
    rng = np.random.default_rng(nq + q_tile)
    nb, kh, qh, d = 40, 2, 4, 64
    cache = filled(rng, 2 * nb, kh, d)
    table = rng.permutation(2 * nb).reshape(2, nb).astype(np.int32)
    kv = to_gpu(cache)
    q32, q = values(rng, (2, nq, qh, d), "bf16")
    kw = dict(q_tile=1, keep_blocks=30) if q_tile else {}
    lens, tab = ints([64 * nb, 900]), ints(table)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    blocks = torch.empty(2, kh, nq, 30, dtype=torch.int32, device=DEV) if q_tile else None
    with new_plan(cache, table, q, True, **kw) as plan:
        def step():
            if q_tile:
                plan.select(kv, lens, q, blocks, table=tab)
            plan.attend(kv, lens, q, out, lse, table=tab, blocks=blocks)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for i in range(5):
            now = [64 * nb - 7 * i, 900 + 130 * i if i % 2 else 3]
            lens.copy_(ints(now))
            torch.cuda.synchronize()
            out.fill_(77.0)
            lse.fill_(77.0)
            graph.replay()
            torch.cuda.synchronize()
            say("[gpu] replay %d of %d queries, lists %d" % (i, nq, q_tile))
            lists = blocks.cpu().numpy() if q_tile else None
            check(cache, table, now, q32, True, out, lse, lists, q_tile)
            kept = out.clone(), lse.clone()
            step()
            torch.cuda.synchronize()
            assert torch.equal(out, kept[0]) and torch.equal(lse, kept[1])
