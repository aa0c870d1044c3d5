"""Pages of the cache on the GPU against their definition (pages_oracle): tables, counts and
contents to the bit."""
import numpy as np
import pytest
import torch

import pages_oracle as po
from gpu_harness import DEV, say
from activation_residual_compression_amd import librescomp as rc

pytestmark = pytest.mark.gpu
FIELDS = ("k", "v", "k_scale", "v_scale", "k_mean", "k_mean_scale")


def ints(x):
    return torch.tensor(np.asarray(x).astype(np.int64).clip(-2 ** 31, 2 ** 31 - 1), dtype=torch.int32, device=DEV)


def raw(cache):
    return [getattr(cache, f).reshape(cache.pool_blocks, -1).view(torch.uint8) for f in FIELDS]


def filled(pool, heads, dim, seed=0):
    """A cache of random bytes."""
    c = rc.KvCache.empty(pool, heads, dim)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    for x in raw(c):
        x.copy_(torch.randint(0, 256, x.shape, generator=g, dtype=torch.uint8, device=DEV))
    return c


class Pair:
    """The library and the oracle side by side."""

    def __init__(self, slots, heads, dim, pool, width, seed=0):
        self.plan = rc.PagePlan(slots, heads, dim, pool, width)
        self.cache = filled(pool, heads, dim, seed)
        self.first = [x.clone() for x in raw(self.cache)]
        self.refs, self.table = self.plan.empty()
        self.o = po.Pages(slots, pool, width)
        self.count = torch.full((1,), 77, dtype=torch.int32, device=DEV)
        self.moved = torch.full((pool,), 77, dtype=torch.int32, device=DEV)

    def set(self, table, refs):
        self.table.copy_(ints(table))
        self.refs.copy_(ints(refs))
        self.o.table[...] = table
        self.o.refs[...] = refs

    def check(self, what):
        torch.cuda.synchronize()
        assert np.array_equal(self.table.cpu().numpy(), self.o.table), (what, "table")
        assert np.array_equal(self.refs.cpu().numpy(), self.o.refs), (what, "refs")
        held = torch.from_numpy(self.o.held).to(DEV)
        for f, x, y in zip(FIELDS, raw(self.cache), self.first):
            assert torch.equal(x, y[held]), (what, f)

    def reserve(self, start, tokens):
        self.plan.reserve(self.cache, self.refs, self.table, ints(start), ints(tokens), missing=self.count)
        lacking = self.o.reserve(start, tokens)
        self.check(("reserve", start, tokens))
        assert int(self.count) == lacking
        return lacking

    def fork(self, source, length):
        self.plan.fork(self.refs, self.table, ints(source), ints(length))
        self.o.fork(source, length)
        self.check(("fork", source, length))

    def free(self, keep):
        self.plan.free(self.refs, self.table, ints(keep))
        self.o.free(keep)
        self.check(("free", keep))

    def compact(self):
        self.plan.compact(self.cache, self.refs, self.table, used=self.count, moved=self.moved)
        n, moved = self.o.compact()
        self.check("compact")
        assert int(self.count) == n and np.array_equal(self.moved.cpu().numpy(), moved)


@pytest.mark.parametrize("slots,heads,dim,pool,width", [
    (1, 1, 64, 1, 1), (3, 2, 64, 9, 4), (6, 3, 128, 40, 8), (40, 1, 64, 300, 20), (5, 30, 64, 64, 300)])
def test_long_use_equals_the_definition(slots, heads, dim, pool, width):
    rng = np.random.default_rng(pool)
    p = Pair(slots, heads, dim, pool, width)
    lengths = np.zeros(slots, int)
    for step in range(40):
        kind = rng.choice(["grow", "grow", "grow", "fork", "free", "compact"])
        say("[gpu] pages %s step %d %s" % ((slots, heads, dim, pool, width), step, kind))
        if kind == "grow":
            more = np.minimum(rng.integers(0, [2, 70, 400][rng.integers(3)], slots), 64 * width - lengths)
            if p.reserve(lengths, more) == 0:
                lengths = lengths + more
        elif kind == "fork":
            source = np.where(rng.random(slots) < 0.5, rng.integers(0, slots, slots), -1)
            lengths = np.where(source >= 0, (lengths[source] * rng.choice([1, rng.random()])).astype(int), lengths)
            p.fork(source, lengths)
        elif kind == "free":
            lengths = np.where(rng.random(slots) < 0.4, (lengths * rng.random(slots)).astype(int), lengths)
            p.free(lengths)
        else:
            p.compact()
        assert np.array_equal(po.counts(p.o.table, pool), p.o.refs)


def test_shared_blocks():
    """Who keeps a block that several write, and which contents are copied."""
    say("[gpu] shared blocks")
    p = Pair(5, 2, 64, 30, 6)
    p.reserve([0] * 5, [150, 0, 0, 0, 0])
    p.fork([-1, 0, 0, 0, -1], [0, 150, 150, 128, 0])
    p.reserve([150, 150, 150, 128, 0], [0, 1, 70, 1, 0])    # a holder does not write: every writer copies
    p.fork([-1, 0, 0, -1, 0], [0, 150, 150, 0, 150])
    p.free([0, 999, 999, 0, 999])
    p.reserve([0, 150, 150, 0, 150], [0, 5, 5, 0, 5])       # every holder writes: the first keeps it
    p.fork([1, 2, 4, 1, 3], [155, 155, 155, 64, 0])         # exchanged, all rows as they were
    p.reserve([0] * 5, [400] * 5)                           # not enough: nothing changes
    p.reserve([0] * 5, [64] * 5)                            # written from their first token: nothing is copied
    p.free([0] * 5)
    assert (p.o.refs == 0).all()


def test_entries_and_lengths_outside_the_allowed():
    say("[gpu] outside")
    p = Pair(4, 1, 64, 12, 3)
    p.set(np.array([[3, 99, -7], [-1, 3, 5], [12, 2 ** 31 - 1, 0], [-2 ** 31, 1, 1]]),
          np.array([1, 2, 0, 2, -3, 1, 0, 0, 0, 0, 0, 1]))
    p.reserve([2 ** 31 - 1, -5, 60, 100], [2 ** 31 - 1, 50, 2 ** 31 - 1, -9])
    p.reserve([64 * 3, 0, 0, 0], [5, 64 * 4, 0, 1])
    p.fork([7, -2, 1, 2 ** 31 - 1], [3, 3, 2 ** 31 - 1, 0])
    p.compact()
    p.fork([3, 0, 2, -1], [-5, 100, 64, 0])
    p.free([-1, 2 ** 31 - 1, 64, 65])
    p.compact()


@pytest.mark.parametrize("pool", [1, 1023, 1024, 1025, 5000, 20011])
def test_compact_and_reserve_of_large_pools(pool):
    rng = np.random.default_rng(pool)
    say("[gpu] pool of %d" % pool)
    p = Pair(3, 1, 64, pool, 8192)
    for share in (0.0, 0.02, 0.5, 0.97, 1.0):
        used = np.flatnonzero(rng.random(pool) < share)
        table = np.full((3, 8192), -1)
        table.reshape(-1)[rng.permutation(table.size)[:used.size]] = rng.permutation(used)
        p.first = [x.clone() for x in raw(p.cache)]
        p.o.held[...] = np.arange(pool)
        p.set(table, po.counts(table, pool))
        p.reserve([0, 3000 * 64, 5], [64 * 40, 64 * 2000, 64 * 8000])
        p.reserve([0, 3000 * 64, 5], [64 * 4, 64 * 20, 64])
        p.compact()


def test_more_than_1024_slots_and_entries():
    rng = np.random.default_rng(1)
    say("[gpu] many slots")
    p = Pair(2500, 1, 64, 9000, 4)
    lengths = rng.integers(0, 200, 2500) * (rng.random(2500) < 0.7)
    p.reserve(np.zeros(2500, int), lengths)
    source = np.where(rng.random(2500) < 0.3, rng.integers(0, 2500, 2500), -1)
    lengths = np.where(source >= 0, lengths[source], lengths)
    p.fork(source, lengths)
    p.reserve(lengths, np.full(2500, 3))
    p.compact()


@pytest.mark.parametrize("heads,dim", [(1, 64), (2, 128), (30, 64)])
def test_copy(heads, dim):
    say("[gpu] copy %d %d" % (heads, dim))
    rng = np.random.default_rng(heads)
    a, b = filled(50, heads, dim, 1), filled(50, heads, dim, 2)
    src, dst = rng.permutation(50)[:20], rng.permutation(50)[:20]
    before = [x.clone() for x in raw(b)]
    with rc.PagePlan(1, heads, dim, 50, 1) as plan:
        plan.copy(a, ints([-1, *src, 50, 3]), ints([7, *dst, 3, -9]), to=b)
        torch.cuda.synchronize()
        for x, y, z in zip(raw(a), raw(b), before):
            want = z.clone()
            want[torch.from_numpy(dst).to(DEV)] = x[torch.from_numpy(src).to(DEV)]
            assert torch.equal(y, want)
        before = [x.clone() for x in raw(a)]
        plan.copy(a, ints([0, 1, 2, 3]), ints([10, 11, 12, 3]))
        plan.copy(a, ints([]), ints([]))
        torch.cuda.synchronize()
        for x, z in zip(raw(a), before):
            z[10:13] = z[0:3]
            assert torch.equal(x, z)
        with pytest.raises(ValueError):
            plan.copy(a, ints([0, 1]), ints([2]))
        with pytest.raises(ValueError):
            plan.copy(a, ints([0]), ints([2]), to=filled(49, heads, dim))


def test_captured_calls_replay():
    """A decoding step's calls in a graph: their results follow the state, not the capture."""
    say("[gpu] captured pages")
    p = Pair(4, 2, 64, 40, 6)
    p.reserve([0] * 4, [130, 0, 70, 0])
    start, tokens, source, length, keep = (ints([0] * 4) for _ in range(5))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        p.plan.free(p.refs, p.table, keep)
        p.plan.fork(p.refs, p.table, source, length)
        p.plan.reserve(p.cache, p.refs, p.table, start, tokens, missing=p.count)
        p.plan.compact(p.cache, p.refs, p.table, used=p.count)
    for k, s, n, a, t in (([130, 0, 70, 0], [-1, 0, -1, 2], [0, 130, 0, 70], [0, 130, 0, 70], [0, 1, 0, 64]),
                          ([0, 131, 70, 134], [1, -1, -1, -1], [131, 0, 0, 0], [131, 131, 70, 134], [1, 1, 1, 1]),
                          ([132, 0, 0, 135], [-1, 0, 0, 0], [0, 132, 60, 0], [132, 132, 60, 0], [64, 64, 64, 64])):
        for x, y in ((keep, k), (source, s), (length, n), (start, a), (tokens, t)):
            x.copy_(ints(y))
        graph.replay()
        p.o.free(k)
        p.o.fork(s, n)
        p.o.reserve(a, t)
        used, _ = p.o.compact()
        p.check((k, s, n, a, t))
        assert int(p.count) == used
        torch.zeros(1000, device=DEV).sum().item()


def test_plan_refuses_wrong_tensors():
    p = Pair(3, 2, 64, 8, 4)
    good = ints([0, 0, 0])
    for call, args in ((p.plan.free, (p.refs, p.table, good[:2])), (p.plan.free, (p.refs[:7], p.table, good)),
                       (p.plan.free, (p.refs, p.table[:2], good)), (p.plan.free, (p.refs, p.table, good.long())),
                       (p.plan.fork, (p.refs, p.table, good.cpu(), good)),
                       (p.plan.reserve, (filled(9, 2, 64), p.refs, p.table, good, good)),
                       (p.plan.reserve, (p.cache, p.refs, p.table.t(), good, good)),
                       (p.plan.compact, (p.cache, p.refs, p.table, good))):
        with pytest.raises(ValueError):
            call(*args)
