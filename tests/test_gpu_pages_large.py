"""Pages of the cache in calls of more entries and sequences than one block of threads has threads,
against their definition."""
import numpy as np
import pytest

from gpu_harness import say
from test_gpu_pages import Pair

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("slots,pool,width", [(3, 9000, 4000), (1024, 4000, 9), (1025, 4000, 9), (2100, 5000, 3)])
def test_reserve_fork_and_free_of_many_entries(slots, pool, width):
    rng = np.random.default_rng(slots)
    say("[gpu] pages of %d sequences, %d blocks" % (slots, pool))
    p = Pair(slots, 1, 64, pool, width)
    lengths = np.minimum(rng.integers(0, 64 * width, slots), 64 * pool // (2 * slots))
    assert p.reserve(np.zeros(slots, int), lengths) == 0
    source = np.where(rng.random(slots) < 0.6, rng.integers(0, slots, slots), -1)
    lengths = np.where(source >= 0, lengths[source], lengths)
    p.fork(source, lengths)
    more = np.where(rng.random(slots) < 0.7, rng.integers(1, 130, slots), 0)
    more = np.minimum(more, 64 * width - lengths)
    if p.reserve(lengths, more) == 0:
        lengths = lengths + more
    p.reserve(np.zeros(slots, int), np.full(slots, 64 * width))      # of all, shared ones too
    lengths = np.where(rng.random(slots) < 0.5, lengths // 3, lengths)
    p.free(lengths)
    p.compact()
    p.fork(rng.permutation(slots), np.full(slots, 64 * width))
    p.free(np.zeros(slots, int))
    assert (p.o.refs == 0).all()


@pytest.mark.parametrize("entries", [1023, 1024, 1025])
def test_reserve_around_a_thread_for_each_entry(entries):
    say("[gpu] reserve %d entries" % entries)
    p = Pair(2, 1, 64, 3000, 1500)
    assert p.reserve([0, 0], [64 * 500, 64 * (entries - 500)]) == 0
    p.fork([1, 0], [64 * (entries - 500), 64 * 500])
    p.fork([0, 0], [64 * 500, 64 * 500])
    assert p.reserve([0, 64], [64 * 500, 64 * (entries - 500)]) == 0      # shared: the first writer keeps them
    p.fork([1, 1], [64 * 1500, 64 * 1500])
    assert p.reserve([0, 0], [64 * 1500, 64 * 1500]) == 0                 # every block of the pool
    assert (p.o.refs == 1).all()
    p.compact()
