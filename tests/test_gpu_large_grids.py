"""Calls that take more blocks of threads than one launch can have (2^32 threads, 2^24 blocks of 256): copies of pages,
and the join."""
import pytest
import torch

from gpu_harness import DEV, say
from test_gpu_pages import filled, ints, raw
from activation_residual_compression_amd import librescomp as rc

pytestmark = pytest.mark.gpu


def test_reserve_with_copies_for_many_slots_of_many_heads():
    """65535 slots x 258 pieces of a block: the written block is the first one's, and its contents come with it."""
    slots, heads, pool = 65535, 257, 6
    say("[gpu] reserve, %d slots, %d heads" % (slots, heads))
    cache = filled(pool, heads, 128)
    before = [x.clone() for x in raw(cache)]
    plan = rc.PagePlan(slots, heads, 128, pool, 1)
    refs, table = plan.empty()
    start, tokens, missing = (torch.zeros(n, dtype=torch.int32, device=DEV) for n in (slots, slots, 1))
    table[5] = table[65534] = table[77] = 2
    refs[2] = 3
    start[5] = start[65534] = 10
    tokens[5] = tokens[65534] = 1
    plan.reserve(cache, refs, table, start, tokens, missing)
    torch.cuda.synchronize()
    assert missing.item() == 0 and [table[s].item() for s in (5, 77, 65534)] == [0, 2, 1]
    assert (table >= 0).sum().item() == 3 and refs.tolist() == [1, 1, 1, 0, 0, 0]
    for x, y in zip(raw(cache), before):
        assert torch.equal(x, y[[2, 2, 2, 3, 4, 5]])
    plan.close()


def test_copy_of_many_pairs():
    """2^23 + 5 pairs of two pieces each, most of them of no block."""
    count, pool = (1 << 23) + 5, 9
    say("[gpu] copy, %d pairs" % count)
    cache, to = filled(pool, 1, 64), filled(pool, 1, 64, 1)
    before = [x.clone() for x in raw(to)]
    src, dst = (torch.full((count,), -1, dtype=torch.int32, device=DEV) for _ in range(2))
    at = ints([0, 1 << 22, (1 << 23) - 1, 1 << 23, count - 1]).long()
    src[at], dst[at] = ints([8, 0, 3, 3, 5]), ints([1, 0, 7, 6, 2])
    with rc.PagePlan(1, 1, 64, pool, 1) as plan:
        plan.copy(cache, src, dst, to=to)
        torch.cuda.synchronize()
    for x, y, z in zip(raw(cache), raw(to), before):
        z[[1, 0, 7, 6, 2]] = x[[8, 0, 3, 3, 5]]
        assert torch.equal(y, z)


def test_join_of_many_rows():
    """2^27 + 3 rows of 128 in fp32, 8 to a block of threads: two parts, each of one row for all, weighted by the rows'
    own lse. Bound: as in test_gpu_attn's join, |x| <= 4 and lse up to 1."""
    n = (1 << 27) + 3
    say("[gpu] join, %d rows" % n)
    x, y = torch.linspace(-4, 4, 128, device=DEV), torch.linspace(1, -2, 128, device=DEV)
    parts = [z[None, None].expand(n, 1, 128) for z in (x, y)]
    ls = torch.arange(n, device=DEV, dtype=torch.int32).remainder_(251).float().div_(251).view(n, 1)
    lr = torch.zeros(n, 1, device=DEV)
    out = torch.full((n, 1, 128), float("nan"), dtype=torch.bfloat16, device=DEV)        # 34 GB
    lse = torch.full((n, 1), float("nan"), device=DEV)
    rc.join_attention(parts, [ls, lr], out, lse)
    torch.cuda.synchronize()
    step = 1 << 21
    for i in range(0, n, step):
        a = ls[i:i + step].double()
        w = torch.sigmoid(a)
        want = w * x.double() + (1 - w) * y.double()
        bound = 4 * (2.0 ** -20 + 176 * 2.0 ** -24) + want.abs() * 2.0 ** -8
        assert ((out[i:i + step, 0].double() - want).abs() <= bound).all(), i
        log = torch.logaddexp(a, torch.zeros_like(a))
        assert ((lse[i:i + step].double() - log).abs() <= 2.0 ** -20 + 176 * 2.0 ** -24 + 4 * 2.0 ** -24 * log).all(), i
    del out, parts
    torch.cuda.empty_cache()
