"""The sequence-parallel step that attends to its own share in full precision and to the peers' through
the 8-bit cache."""
import numpy as np
import pytest
import torch

import attn_dense as ad
import kv_dense as kd
import kv_oracle as ko
from activation_residual_compression_amd.peer_attention import PeerAttention, Sender
from gpu_harness import say
from test_gpu_kv import FIELDS, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,rank,heads,dim,dtype,keep", [
    ((100, 77, 64), 1, 2, 64, "bf16", 0), ((130, 200), 0, 1, 128, "f32", 2), ((70, 90), 1, 3, 64, "bf16", 1),
    ((90,), 0, 2, 128, "bf16", 0)])
def test_own_share_is_exact_and_joined(tokens, rank, heads, dim, dtype, keep):
    """The cache holds the peers' tokens alone; the output is their attention (in 64 bits over what the cache holds)
    joined with that over the own ones. Bounds as in test_gpu_serving, with one key head for each query head."""
    rng = np.random.default_rng(sum(tokens))
    kw = dict(scheme="q2", group=64, dtype=dtype)
    senders = [Sender(n, heads, dim, **kw) for n in tokens]
    a = PeerAttention(tokens, rank, heads, dim, keep_blocks=keep, exact_own=True, **kw)
    total, scale = sum(tokens) - tokens[rank], dim ** -0.5
    nb = max(-(-total // 64), 1)
    cache = ko.Cache(nb, heads, dim)
    table = np.arange(nb, dtype=np.int32)[None]
    for t in range(3):
        say("[gpu] peer attention, own share exact, %s step %d" % (tokens, t))
        kv = [(values(rng, (1, n, heads, dim), dtype)[1], values(rng, (1, n, heads, dim), dtype)[1]) for n in tokens]
        q32, q = values(rng, (1, tokens[rank], heads, dim), dtype)
        sent = {p: senders[p].step(*kv[p]) for p in range(len(tokens))}
        out, lse = a.step(q, *kv[rank], sent)
        torch.cuda.synchronize()
        at = 0
        for p, n in enumerate(tokens):
            if p == rank:
                continue
            k, v = senders[p].ahat.view(2, 1, n, heads, dim)
            cache.store(table, [at], [n], k.double().cpu().numpy(), v.double().cpu().numpy())
            at += n
        for f in FIELDS if total else ():
            got = getattr(a.cache, f)
            assert np.array_equal((got.view(torch.uint8) if f in ("k", "v") else got).cpu().numpy(), getattr(cache, f)), f
        lists = a.blocks.cpu().numpy()[0] if keep else None
        x = q.double().cpu().numpy()[0]
        far = kd.attend(cache, table[0], total, x, False, scale, lists, 128 if keep else 0)
        near = ad.attend(x, *(y.double().cpu().numpy()[0] for y in kv[rank]), False, scale)
        want, log, _ = ad.join([near[0].reshape(-1, dim), far[0].reshape(-1, dim)], [near[1].ravel(), far[1].ravel()])
        _, _, weight = ad.join([near[2].reshape(-1, dim), far[2].reshape(-1, dim)], [near[1].ravel(), far[1].ravel()])
        ds = np.maximum(near[3], far[3]).ravel() * ((3 * 2.0 ** -22 + (6 * dim + 8) * ad.U) if dtype == "f32" else (2 * dim + 8) * ad.U)
        r = 4 * ds + 2.0 ** -18 + 4 * (sum(tokens) + 64) * ad.U
        bound = weight * (r[:, None] + (2.0 ** -19 if dtype == "f32" else 3 * 2.0 ** -8)) + \
            np.abs(want) * (4 * ad.U if dtype == "f32" else 2.0 ** -8)
        assert (np.abs(out.double().cpu().numpy().reshape(-1, dim) - want) <= bound).all()
        assert (np.abs(lse.double().cpu().numpy().ravel() - log) <= 2 * ds + 2.0 ** -18 + (sum(tokens) + 64) * ad.U).all()
    for y in senders + [a]:
        y.close()
