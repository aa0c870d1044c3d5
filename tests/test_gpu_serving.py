"""Packed attention, the join, the pages and the 8-bit cache in one serving run: prompts, samples that
share them, tokens one by one, sequences that end, a pool that is compacted."""
import numpy as np
import pytest
import torch

import attn_dense as ad
import kv_oracle as ko
from gpu_harness import DEV, say
from test_gpu_attn import DT, check_all, ints, offsets, rows, wide
from activation_residual_compression_amd import librescomp as rc

pytestmark = pytest.mark.gpu
FIELDS = ("k", "v", "k_scale", "v_scale", "k_mean", "k_mean_scale")


def cached(cache, row, length):
    """Keys and values that the cache holds of a sequence, [length, heads, dim] float64."""
    c = ko.Cache(cache.pool_blocks, cache.kv_heads, cache.head_dim)
    for f in FIELDS:
        x = getattr(cache, f)
        getattr(c, f)[...] = (x.view(torch.uint8) if f in ("k", "v") else x).cpu().numpy()
    k = np.empty((-(-length // 64) * 64, cache.kv_heads, cache.head_dim))
    v = np.empty_like(k)
    for j in range(k.shape[0] // 64):
        for h in range(cache.kv_heads):
            p, at = row[j], slice(64 * j, 64 * j + 64)
            k[at, h] = ko.TABLE[c.k_codes(p, h)] * float(c.k_scale[p, h])
            v[at, h] = ko.TABLE[c.v_codes(p, h)] * float(c.v_scale[p, h])
    return k[:length], v[:length]


@pytest.mark.parametrize("dtype,qh,kh,dim", [("bf16", 8, 2, 128), ("f32", 4, 4, 64)])
def test_prompts_samples_and_tokens(dtype, qh, kh, dim):
    """Each step's output of a sequence is exact attention over the tokens since its prompt, joined with attention over
    the cached prompt. Bounds: those of the join's test in test_gpu_attn, and of the cache's attention its weights' 11
    bits (bf16) or 22, all on the weighted mean of |v|, doubled for the two stages of sums."""
    rng = np.random.default_rng(dim)
    slots, pool, width, steps = 6, 64, 12, 5
    prompts = [130, 0, 701, 64]
    scale = dim ** -0.5
    pages = rc.PagePlan(slots, kh, dim, pool, width)
    cache = rc.KvCache.empty(pool, kh, dim, DEV)
    refs, table = pages.empty(DEV)
    lacking = torch.zeros(1, dtype=torch.int32, device=DEV)
    say("[gpu] serving %s: prompts" % dtype)
    # prompts: causal attention in full precision, and their keys and values into the cache
    n = sum(prompts)
    q, k, v = rows(rng, n, qh, dim, dtype), rows(rng, n, kh, dim, dtype), rows(rng, n, kh, dim, dtype)
    out, lse = torch.empty_like(q), torch.empty((n, qh), device=DEV)
    off = offsets(prompts)
    with rc.AttnPlan(qh, kh, dim, dtype, max_seqs=4, max_queries=n, max_keys=n, causal=True) as p:
        p.attend(q, k, v, ints(off), out, lse, max_q=max(prompts), max_kv=max(prompts))
        torch.cuda.synchronize()
    check_all(q, k, v, off, off, True, scale, out, lse, dtype)
    lengths = prompts + [0, 0]
    start = ints([0] * slots)
    pages.reserve(cache, refs, table, start, ints(lengths), missing=lacking)
    padded = [torch.zeros((slots, max(prompts), kh, dim), dtype=DT[dtype], device=DEV) for _ in range(2)]
    for i, m in enumerate(prompts):
        for to, x in zip(padded, (k, v)):
            to[i, :m] = x[off[i]:off[i + 1]]
    with rc.KvPlan(slots, qh, kh, dim, pool, width, dtype, max_queries=1) as kv, \
            rc.AttnPlan(qh, kh, dim, dtype, max_seqs=slots, max_queries=slots, max_keys=slots * steps) as own:
        kv.store(cache, start, *padded, table=table, count=ints(lengths))
        torch.cuda.synchronize()
        assert int(lacking) == 0
        # two more samples of the third prompt, one of the first
        pages.fork(refs, table, ints([-1, 0, -1, -1, 2, 2]), ints([130, 130, 701, 64, 701, 701]))
        lengths = [130, 130, 701, 64, 701, 701]
        rows_ = table.cpu().numpy()
        held = [cached(cache, rows_[i], m) for i, m in enumerate(lengths)]
        assert all(np.array_equal(held[2][x], held[i][x]) for i in (4, 5) for x in (0, 1))
        used = -(-130 // 64) + -(-701 // 64) + 1
        assert int((refs > 0).sum()) == used and int(refs.sum()) == 2 * 3 + 3 * 11 + 1
        kv_len = ints(lengths)
        tail_k, tail_v = (torch.empty((slots, steps, kh, dim), dtype=DT[dtype], device=DEV) for _ in range(2))
        far, far_lse = torch.empty((slots, qh, dim), dtype=DT[dtype], device=DEV), torch.empty((slots, qh), device=DEV)
        near, near_lse = torch.empty_like(far), torch.empty_like(far_lse)
        for t in range(steps):
            say("[gpu] serving %s: token %d" % (dtype, t))
            q, tail_k[:, t], tail_v[:, t] = (rows(rng, slots, h, dim, dtype) for h in (qh, kh, kh))
            if t == 3:     # a sequence ends; the others' blocks move
                pages.free(refs, table, ints([10 ** 6, 0, 10 ** 6, 10 ** 6, 10 ** 6, 0]))
                before = torch.empty_like(far)
                kv.attend(cache, kv_len, q[:, None], before[:, None], far_lse[:, None], table=table)
                pages.compact(cache, refs, table, used=lacking)
                kv.attend(cache, kv_len, q[:, None], far[:, None], far_lse[:, None], table=table)
                torch.cuda.synchronize()
                live = [0, 2, 3, 4]
                assert int(lacking) == used and torch.equal(before[live], far[live])
                assert sorted(set(table.cpu().numpy().ravel()) - {-1}) == list(range(used))
            else:
                live = list(range(slots)) if t < 3 else [0, 2, 3, 4]
                kv.attend(cache, kv_len, q[:, None], far[:, None], far_lse[:, None], table=table)
            m = t + 1
            own.attend(q, tail_k[:, :m].reshape(-1, kh, dim), tail_v[:, :m].reshape(-1, kh, dim), ints(range(slots + 1)), near,
                       near_lse, kv_offsets=ints([m * i for i in range(slots + 1)]), max_q=1, max_kv=m)
            rc.join_attention([near, far], [near_lse, far_lse], far, far_lse)
            torch.cuda.synchronize()
            for i in live:
                keys = np.concatenate([held[i][0], wide(tail_k[i, :m])])
                vals = np.concatenate([held[i][1], wide(tail_v[i, :m])])
                want, log, weight, logit, _ = ad.attend(wide(q[i:i + 1]), keys, vals, False, scale)
                ds = logit * ((3 * 2.0 ** -22 + (6 * dim + 8) * ad.U) if dtype == "f32" else (2 * dim + 8) * ad.U)
                r = 4 * ds + 2.0 ** -18 + 4 * (len(keys) + 64) * ad.U
                bound = weight * (r[..., None] + (2.0 ** -19 if dtype == "f32" else 3 * 2.0 ** -8)) + \
                    np.abs(want) * (4 * ad.U if dtype == "f32" else 2.0 ** -8)
                assert (np.abs(wide(far[i:i + 1]) - want) <= bound).all(), (t, i)
                assert (np.abs(wide(far_lse[i:i + 1]) - log) <= 2 * ds + 2.0 ** -18 + (len(keys) + 64) * ad.U).all()
    pages.close()


def test_samples_that_go_on_writing_are_as_if_alone():
    """Two samples of a prompt that write into the cache token by token hold and read what each would alone."""
    rng = np.random.default_rng(8)
    heads, dim, pool, width, prompt, steps = 2, 64, 24, 6, 100, 40
    kv0 = [torch.from_numpy(rng.standard_normal((1, prompt, heads, dim))).to(DEV, torch.bfloat16) for _ in range(2)]
    tokens = [[torch.from_numpy(rng.standard_normal((2, 1, heads, dim))).to(DEV, torch.bfloat16) for _ in range(3)] for _ in range(steps)]

    def serve(shared, captured=False):
        cache = rc.KvCache.empty(pool, heads, dim, DEV)
        pages = rc.PagePlan(2, heads, dim, pool, width)
        refs, table = pages.empty(DEV)
        outs = []
        with rc.KvPlan(2, heads, heads, dim, pool, width, max_queries=1) as kv:
            pages.reserve(cache, refs, table, ints([0, 0]), ints([prompt, 0 if shared else prompt]))
            kv.store(cache, ints([0, 0]), *(x.expand(2, -1, -1, -1) for x in kv0), table=table,
                     count=ints([prompt, 0 if shared else prompt]))
            if shared:
                pages.fork(refs, table, ints([-1, 0]), ints([0, prompt]))
            if captured:      # one step as a graph, whose position moves on by itself
                at, one = ints([prompt, prompt]), ints([1, 1])
                q, k, v = (torch.empty_like(x) for x in tokens[0])
                out, after = torch.empty_like(q), torch.empty_like(at)
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    pages.reserve(cache, refs, table, at, one)
                    kv.store(cache, at, k, v, table=table)
                    torch.add(at, 1, out=after)
                    kv.attend(cache, after, q, out, table=table)
                    at.copy_(after)
                for x in tokens:
                    for to, y in zip((q, k, v), x):
                        to.copy_(y)
                    graph.replay()
                    outs.append(out.clone())
                    torch.cuda.synchronize()
            for t, (q, k, v) in enumerate(() if captured else tokens):
                at = ints([prompt + t] * 2)
                pages.reserve(cache, refs, table, at, ints([1, 1]))
                kv.store(cache, at, k, v, table=table)
                out = torch.empty_like(q)
                kv.attend(cache, at + 1, q, out, table=table)
                outs.append(out)
            torch.cuda.synchronize()
        pages.close()
        return outs, int((refs > 0).sum())
    say("[gpu] two samples of a prompt")
    alone, blocks = serve(False)
    together, fewer = serve(True)
    assert len(together) == steps and all(torch.equal(x, y) for x, y in zip(alone, together))
    assert blocks == 6 and fewer == 5
    replayed, fewer = serve(True, captured=True)
    assert len(replayed) == steps and all(torch.equal(x, y) for x, y in zip(alone, replayed))
    assert fewer == 5
