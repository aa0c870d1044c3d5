"""Attention of one GPU of a sequence-parallel group over every peer's tokens, with
the keys and values exchanged as compressed residuals and held in 8 bits.

A step of a layer: each GPU compresses the residual of its own keys and values
(`Sender`), the peers apply what they receive to their reconstructions, write all
parts in the order of the tokens into the 8-bit cache, and attend from their own
queries (`PeerAttention`), over the whole cache or over the blocks that a cheap
score selects. Step 0 is sent in full ("Limitations" of the CompactFusion notes).
A GPU's own keys and values need no exchange: it may attend to them as they are, in
full precision, and to the cache for the others' only (`exact_own`).

    python -m activation_residual_compression_amd.peer_attention

runs a group on one GPU and prints, for each step, how far the outputs are from
attention in fp32 over the uncompressed keys and values.
"""
from __future__ import annotations

import torch  # before the library: both then share the HIP runtime that torch brings

from activation_residual_compression_amd import librescomp as rc


def _exchange_plan(tokens, heads, head_dim, dtype, scheme, params):
    return rc.Plan((2, tokens, heads * head_dim), dtype, scheme, **params)


class Sender:
    """One GPU's side that sends: keys and values [1, tokens, heads, head_dim] of its
    share, as one batch of two activation tensors."""

    def __init__(self, tokens, heads, head_dim, dtype="bf16", scheme="q2", device="cuda", **params):
        self.plan = _exchange_plan(tokens, heads, head_dim, dtype, scheme, params)
        self.shape = (2, tokens, heads * head_dim)
        self.a = torch.empty(self.shape, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device=device)
        self.ahat = torch.zeros(self.shape, dtype=torch.float32, device=device)
        self.e = torch.zeros_like(self.ahat)
        self.packed = torch.empty(self.plan.packed_bytes, dtype=torch.uint8, device=device)
        self.started = False

    def step(self, k, v):
        """What is sent: the activations themselves at step 0, then packed residuals."""
        self.a[0].copy_(k.reshape(self.shape[1:]))
        self.a[1].copy_(v.reshape(self.shape[1:]))
        if not self.started:
            self.started = True
            self.ahat.copy_(self.a)
            return self.a
        self.plan.compress(self.a, self.ahat, self.e, self.packed)
        return self.packed

    def close(self):
        self.plan.close()


class PeerAttention:
    """One GPU's side that receives and attends. `tokens`: of every GPU's share, in the
    order of the sequence; `rank`: this GPU. keep_blocks > 0: attention over that many
    blocks for each tile of 128 queries, chosen anew at each step. exact_own: this GPU's
    keys and values stay out of the cache; attention over them in full precision (k and v
    then in `dtype`) is joined with that over the cache, or over the blocks chosen of it."""

    def __init__(self, tokens, rank, heads, head_dim, dtype="bf16", scheme="q2", keep_blocks=0, device="cuda",
                 exact_own=False, **params):
        self.tokens, self.rank, self.heads, self.head_dim = list(tokens), rank, heads, head_dim
        own = self.tokens[rank]
        cached = [0 if exact_own and p == rank else n for p, n in enumerate(self.tokens)]
        self.starts = [sum(cached[:p]) for p in range(len(cached))]
        total = sum(cached)
        blocks = max(-(-total // rc.RC_KV_BLOCK), 1)
        self.peers = [p for p in range(len(self.tokens)) if p != rank]
        self.exchange = {p: _exchange_plan(self.tokens[p], heads, head_dim, dtype, scheme, params) for p in self.peers}
        self.recon = {p: torch.zeros((2, self.tokens[p], heads * head_dim), dtype=torch.float32, device=device)
                      for p in self.peers}
        self.cache = rc.KvCache.empty(blocks, heads, head_dim, device)
        self.plan = rc.KvPlan(batch=1, q_heads=heads, kv_heads=heads, head_dim=head_dim, pool_blocks=blocks,
                              seq_blocks=blocks, dtype=dtype, max_queries=own,
                              q_tile=rc.RC_KV_QTILE if keep_blocks else 0, keep_blocks=keep_blocks)
        ints = dict(dtype=torch.int32, device=device)
        self.at = [torch.tensor([s], **ints) for s in self.starts]
        self.length = torch.tensor([total], **ints)
        self.out = torch.empty((1, own, heads, head_dim), dtype=torch.bfloat16 if dtype == "bf16" else torch.float32,
                               device=device)
        self.lse = torch.empty((1, own, heads), dtype=torch.float32, device=device)
        self.blocks = torch.empty((1, heads, -(-own // rc.RC_KV_QTILE), keep_blocks), **ints) if keep_blocks else None
        self.own_plan = None
        if exact_own:
            self.own_plan = rc.AttnPlan(heads, heads, head_dim, dtype, max_seqs=1, max_queries=own, max_keys=own)
            self.own_offsets = torch.tensor([0, own], **ints)
            self.own_out, self.own_lse = torch.empty_like(self.out), torch.empty_like(self.lse)
        self.started = False

    def step(self, q, k, v, received):
        """q, k, v: this GPU's [1, own, heads, head_dim]; received: {peer: what its Sender
        returned}. Returns out and lse, buffers of this object."""
        if self.own_plan is not None:  # needs nothing that is received
            self.own_plan.attend(q[0], k[0], v[0], self.own_offsets, self.own_out[0], self.own_lse[0])
        for p in self.peers:
            if self.started:
                self.exchange[p].decompress(received[p], self.recon[p])
            else:
                self.recon[p].copy_(received[p])
        self.started = True
        # in the order of the tokens: a store ends the sequence after its tokens
        for p, at in enumerate(self.at):
            if p == self.rank:
                if self.own_plan is None:
                    self.plan.store(self.cache, at, k, v)
            else:
                kv = self.recon[p].view(2, 1, self.tokens[p], self.heads, self.head_dim)
                self.plan.store(self.cache, at, kv[0], kv[1])
        if self.blocks is not None:
            self.plan.select(self.cache, self.length, q, self.blocks)
        self.plan.attend(self.cache, self.length, q, self.out, self.lse, blocks=self.blocks)
        if self.own_plan is not None:
            rc.join_attention([self.own_out, self.out], [self.own_lse, self.lse], self.out, self.lse)
        return self.out, self.lse

    def close(self):
        for p in self.exchange.values():
            p.close()
        self.plan.close()
        if self.own_plan is not None:
            self.own_plan.close()


def main(gpus=4, tokens=1152, heads=24, head_dim=128, steps=5, keep_blocks=18):
    g = torch.Generator(device="cuda")
    g.manual_seed(0)

    def noise(scale, n=tokens):
        return torch.randn(1, n, heads, head_dim, generator=g, device="cuda") * scale
    kw = dict(scheme="q2", group=128)
    senders = [Sender(tokens, heads, head_dim, **kw) for _ in range(gpus)]
    dense = PeerAttention([tokens] * gpus, 0, heads, head_dim, **kw)
    sparse = PeerAttention([tokens] * gpus, 0, heads, head_dim, keep_blocks=keep_blocks, **kw)
    exact = PeerAttention([tokens] * gpus, 0, heads, head_dim, exact_own=True, **kw)
    shared = noise(1.0, gpus * tokens // 48 + 1).repeat_interleave(48, 1)[:, :gpus * tokens]
    state = [(shared[:, i * tokens:(i + 1) * tokens] + noise(0.5), noise(1.0)) for i in range(gpus)]
    q = state[0][0] * 0.7 + noise(0.5)
    for t in range(steps):
        state = [(k + noise(0.05), v + noise(0.05)) for k, v in state]
        kv = [(k.bfloat16(), v.bfloat16()) for k, v in state]
        q = (q + noise(0.05)).bfloat16()
        sent = {p: senders[p].step(*kv[p]) for p in range(gpus)}
        k, v = (torch.cat([x[i] for x in kv], 1).float().transpose(1, 2) for i in (0, 1))
        s = q.float().transpose(1, 2) @ k.transpose(2, 3) * head_dim ** -0.5
        want = (torch.softmax(s, -1) @ v).transpose(1, 2)
        line = "step %d: %7d bytes from each peer" % (t, sent[1].numel() * sent[1].element_size())
        for name, a in (("all blocks", dense), ("%d of %d blocks" % (keep_blocks, sparse.cache.pool_blocks), sparse)):
            out, _ = a.step(q, *kv[0], sent)
            line += ", %s off by %.4f" % (name, (out.float() - want).norm().item() / want.norm().item())
        out, _ = exact.step(q, *kv[0], sent)
        line += " (%.4f with its own share as it is)" % ((out.float() - want).norm().item() / want.norm().item())
        print(line, flush=True)
    for x in senders + [dense, sparse, exact]:
        x.close()


if __name__ == "__main__":
    main()
