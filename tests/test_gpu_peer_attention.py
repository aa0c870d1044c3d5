"""The sequence-parallel step that runs the exchange and the 8-bit cache together:
its cache is to the bit what the oracle stores of the reconstructions, its choice of
blocks the oracle's, and its outputs attention over that cache (bounds as in
test_gpu_kv)."""
import numpy as np
import pytest
import torch

import kv_oracle as ko
from activation_residual_compression_amd import librescomp as rc
from activation_residual_compression_amd.peer_attention import PeerAttention, Sender
from gpu_harness import say
from test_gpu_kv import FIELDS, check_attend, to_gpu, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,rank,heads,dim,dtype,keep", [
    ((100, 77, 64), 1, 2, 64, "bf16", 0), ((130, 200), 0, 1, 128, "f32", 2), ((70, 90), 1, 3, 64, "bf16", 1)])
def test_step_equals_oracle_over_the_reconstructions(tokens, rank, heads, dim, dtype, keep):
    rng = np.random.default_rng(sum(tokens))
    kw = dict(scheme="q2", group=64, dtype=dtype)
    senders = [Sender(n, heads, dim, **kw) for n in tokens]
    a = PeerAttention(tokens, rank, heads, dim, keep_blocks=keep, **kw)
    total = sum(tokens)
    nb = -(-total // 64)
    cache = ko.Cache(nb, heads, dim)
    table = np.arange(nb, dtype=np.int32)[None]
    for t in range(3):
        say("[gpu] peer attention %s step %d" % (tokens, t))
        kv = [(values(rng, (1, n, heads, dim), dtype)[1], values(rng, (1, n, heads, dim), dtype)[1]) for n in tokens]
        q32, q = values(rng, (1, tokens[rank], heads, dim), dtype)
        sent = {p: senders[p].step(*kv[p]) for p in range(len(tokens))}
        out, lse = a.step(q, *kv[rank], sent)
        torch.cuda.synchronize()
        for p, n in enumerate(tokens):
            k, v = kv[p] if p == rank else senders[p].ahat.view(2, 1, n, heads, dim)
            if p != rank:
                assert torch.equal(a.recon[p], senders[p].ahat)
            cache.store(table, [sum(tokens[:p])], [n], k.double().cpu().numpy(), v.double().cpu().numpy())
        for f in FIELDS:
            got = getattr(a.cache, f)
            assert np.array_equal((got.view(torch.uint8) if f in ("k", "v") else got).cpu().numpy(), getattr(cache, f)), f
        plan_kw, blocks = {}, None
        if keep:
            assert np.array_equal(a.blocks.cpu().numpy()[0], ko.select(cache, table[0], total, q32[0], False, 128, keep))
            plan_kw, blocks = dict(q_tile=rc.RC_KV_QTILE, keep_blocks=keep), a.blocks
        got, glse = check_attend(cache, to_gpu(cache), plan_kw, table, [total], q32, q, False, blocks=blocks)
        assert torch.equal(got, out) and torch.equal(glse, lse)
    for x in senders + [a]:
        x.close()


def test_example_runs(capsys):
    from activation_residual_compression_amd import peer_attention
    peer_attention.main(gpus=2, tokens=200, heads=2, head_dim=64, steps=2, keep_blocks=3)
    assert capsys.readouterr().out.count("off by") == 4
