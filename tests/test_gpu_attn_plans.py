"""Attention over packed sequences by plans that are made for larger calls, as a serving program keeps one, against
attention in 64 bits (attn_dense, which derives the bounds)."""
import numpy as np
import pytest
import torch

from gpu_harness import DEV, say
from test_gpu_attn import DT, check_all, ints, rows
from activation_residual_compression_amd import librescomp as rc

pytestmark = pytest.mark.gpu


# heads, the plan's queries and keys, the calls': the workspace limits the parts of the first call
@pytest.mark.parametrize("dtype,heads,most,calls", [
    ("bf16", (32, 8, 128), (5, 8192), [(5, 7168), (3, 8100)]), ("bf16", (32, 8, 128), (16, 4000), [(14, 3744), (16, 3333)]),
    ("bf16", (24, 24, 128), (26, 4001), [(26, 3501), (17, 4001)]), ("f32", (12, 12, 64), (24, 5500), [(21, 5244), (24, 5001)])])
@pytest.mark.parametrize("causal", [False, True])
def test_calls_of_one_sequence_smaller_than_the_plan(dtype, heads, most, calls, causal):
    """Every call twice, the others between: the parts of a call are joined by the plan's counters."""
    qh, kh, dim = heads
    rng = np.random.default_rng(sum(most))
    say("[gpu] plan for %s, calls %s %s causal %s" % (most, calls, dtype, causal))
    inputs = [[rows(rng, n, h, dim, dtype) for n, h in ((nq, qh), (nk, kh), (nk, kh))] for nq, nk in calls]
    first = [None] * len(calls)
    with rc.AttnPlan(qh, kh, dim, dtype, max_seqs=1, max_queries=most[0], max_keys=most[1], causal=causal) as p:
        for _ in range(2):
            for i, (nq, nk) in enumerate(calls):
                out = torch.full((nq, qh, dim), float("nan"), dtype=DT[dtype], device=DEV)
                lse = torch.full((nq, qh), float("nan"), device=DEV)
                p.attend(*inputs[i], ints([0, nq]), out, lse, kv_offsets=ints([0, nk]), max_q=nq, max_kv=nk)
                torch.cuda.synchronize()
                check_all(*inputs[i], [0, nq], [0, nk], causal, dim ** -0.5, out, lse, dtype, (nq, nk))
                if first[i] is None:
                    first[i] = out, lse
                assert torch.equal(out, first[i][0]) and torch.equal(lse, first[i][1])
