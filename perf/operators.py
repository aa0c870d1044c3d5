"""Cases of the 8-bit key/value cache operators, for measuring them.

A GPU that takes part in a sequence-parallel step attends from its own share of
the tokens to the keys and values of all peers, which it holds in a cache of
blocks of 64 tokens: 8-bit (e4m3) codes with one power-of-two scale per block
and head, and one 8-bit mean key per block and head. Three operators:

  store   writes new keys and values into the cache (quantise, append, block means)
  attend  attention of new queries over the whole cache, with the log-sum-exp
  sparse  the cheap score (8-bit query times mean key) selects blocks for each
          query (or each tile of 128 queries), and attention over those alone

`run` computes each operator in a plain form (elementary torch operations in
fp32) or, where `own` is true, by the library's calls. Layouts of a block and
head: K codes [D/16][64 tokens][16], V codes [4][D][16 tokens].
"""
import math

import torch

own = False

BLOCK = 64
QTILE = 128
E_MIN, E_MAX = -40, 44        # exponents a block's scale may have
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # serving: one new token of each of 16 sequences is appended to its ragged cache
        dict(name="store_token", op="store", dtype="bf16", batch=16, q_heads=32, kv_heads=8, dim=128, tokens=1,
             start=4095, paged=True),
        # a peer's share of the video workload (4444 tokens of 1920 channels, fp32 reconstruction), after another's
        dict(name="store_share_f32", op="store", dtype="f32", batch=1, q_heads=30, kv_heads=30, dim=64, tokens=4444,
             start=4444, paged=False),
        # four image sequences of 4 x 1152 tokens and 3072 channels, written whole
        dict(name="store_image", op="store", dtype="bf16", batch=4, q_heads=24, kv_heads=24, dim=128, tokens=4608,
             start=0, paged=False),
        # the smallest call: one query token over a short cache, no shared heads
        dict(name="attend_token_short", op="attend", dtype="bf16", batch=1, q_heads=24, kv_heads=24, dim=128,
             queries=1, length=333, ragged=False, causal=True, paged=False),
        # serving: one query token for each of 32 ragged sequences in shared pages, four query heads to a key head
        dict(name="attend_token_batch", op="attend", dtype="bf16", batch=32, q_heads=32, kv_heads=8, dim=128,
             queries=1, length=8192, ragged=True, causal=True, paged=True),
        # one GPU's share of the image workload (1152 of 4608 tokens), two images
        dict(name="attend_image", op="attend", dtype="bf16", batch=2, q_heads=24, kv_heads=24, dim=128,
             queries=1152, length=4608, ragged=False, causal=False, paged=False),
        # the same share with fp32 activations
        dict(name="attend_image_f32", op="attend", dtype="f32", batch=1, q_heads=24, kv_heads=24, dim=128,
             queries=1152, length=4608, ragged=False, causal=False, paged=False),
        # one GPU's share of the video workload (4444 of 17776 tokens)
        dict(name="attend_video", op="attend", dtype="bf16", batch=1, q_heads=30, kv_heads=30, dim=64,
             queries=4444, length=17776, ragged=False, causal=False, paged=False),
        # causal prompts of odd ragged lengths in pages, shared heads
        dict(name="attend_prompt", op="attend", dtype="bf16", batch=3, q_heads=16, kv_heads=4, dim=128,
             queries=1999, length=4001, ragged=True, causal=True, paged=True),
        # one query token over long ragged caches, 32 blocks of about a thousand
        dict(name="sparse_token", op="sparse", dtype="bf16", batch=8, q_heads=32, kv_heads=8, dim=128, queries=1,
             length=65536, ragged=True, causal=True, paged=True, keep=32, q_tile=1),
        # the video share, each tile of 128 queries with a quarter of the blocks
        dict(name="sparse_video", op="sparse", dtype="bf16", batch=1, q_heads=30, kv_heads=30, dim=64, queries=4444,
             length=17776, ragged=False, causal=False, paged=False, keep=70, q_tile=QTILE),
        # a causal prompt with shared heads and fp32 activations
        dict(name="sparse_prompt_f32", op="sparse", dtype="f32", batch=2, q_heads=16, kv_heads=4, dim=128,
             queries=2000, length=8000, ragged=True, causal=True, paged=True, keep=24, q_tile=QTILE),
    ]


HEADS = [(24, 24, 128), (30, 30, 64), (32, 8, 128), (16, 4, 128), (12, 12, 64), (16, 2, 64), (5, 5, 128)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    kind = rng.choice(["store_token", "store", "token", "queries", "sparse_token", "sparse"])
    qh, kh, d = rng.choice(HEADS)
    c = dict(dtype=rng.choice(["bf16", "bf16", "f32"]), q_heads=qh, kv_heads=kh, dim=d, paged=rng.random() < 0.5)
    if kind == "store_token":
        return dict(c, op="store", batch=_log(rng, 1, 32), tokens=rng.choice([1, 1, 2, 5]), start=_log(rng, 1, 4000))
    if kind == "store":
        return dict(c, op="store", batch=_log(rng, 1, 4), tokens=_log(rng, 64, 4608), start=rng.choice([0, _log(rng, 1, 4608)]))
    c.update(ragged=rng.random() < 0.5)
    if kind == "token":
        return dict(c, op="attend", batch=_log(rng, 1, 32), queries=rng.choice([1, 1, 2, 3]), length=_log(rng, 16, 8192),
                    causal=True)
    if kind == "queries":
        return dict(c, op="attend", batch=_log(rng, 1, 3), queries=_log(rng, 8, 4444), length=_log(rng, 512, 17776),
                    causal=rng.random() < 0.4)
    if kind == "sparse_token":
        return dict(c, op="sparse", batch=_log(rng, 1, 8), queries=rng.choice([1, 1, 2]), length=_log(rng, 2048, 65536),
                    causal=True, keep=_log(rng, 4, 64), q_tile=1)
    return dict(c, op="sparse", batch=_log(rng, 1, 2), queries=_log(rng, 128, 4444), length=_log(rng, 4444, 17776),
                causal=rng.random() < 0.4, keep=_log(rng, 8, 70), q_tile=QTILE)


def draw(rng):
    most = {}
    for c in listed():
        w, m = work(c), most.setdefault(c["op"], {"bytes": 0.0, "flops": 0.0})
        most[c["op"]] = {k: max(m[k], w[k]) for k in m}
    while True:
        c = _draw(rng)
        w, m = work(c), most[c["op"]]
        several = 3 if c["dtype"] == "f32" else 1       # an fp32 case does several products for one
        if w["bytes"] <= m["bytes"] and w["flops"] * several <= m["flops"]:
            return c


def _lengths(c):
    """Lengths of the sequences (starts of the new tokens, for a store), from the case alone."""
    n, top = c["batch"], c["start"] if c["op"] == "store" else c["length"]
    ragged = c["batch"] > 1 if c["op"] == "store" else c["ragged"]
    if not ragged:
        return [top] * n
    # the first is the longest, the others spread down to an eighth of it, mostly odd
    return [max(0, top - (i * 7 * top) // (8 * max(1, n - 1)) - (i % 3)) for i in range(n)] if n > 1 else [top]


def work(case):
    c = case
    b, qh, kh, d = c["batch"], c["q_heads"], c["kv_heads"], c["dim"]
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "store":
        new = b * c["tokens"] * kh * d
        blocks = sum((s + c["tokens"] + 63) // 64 - s // 64 for s in _lengths(c))
        return {"bytes": new * 2 * (es + 1) + blocks * kh * (12 + d), "flops": 6 * new}
    nq, moved, flops = c["queries"], 0, 0
    for n in _lengths(c):
        used = min(nq, n) if c["causal"] else nq
        pairs = nq * n if not c["causal"] else sum(max(0, n - nq + i + 1) for i in range(nq))
        nb = (n + 63) // 64
        moved += 2 * nq * qh * d * es + nq * qh * 4
        if c["op"] == "attend":
            moved += 2 * n * kh * d + 8 * nb * kh
        else:
            tiles = -(-nq // c["q_tile"])
            kept = min(c["keep"], nb)
            # each block is read once at most, and each tile reads no more than it keeps
            moved += nb * kh * (d + 4) + 2 * min(tiles * kept, nb) * 64 * kh * d + 4 * tiles * kh * c["keep"]
            flops += 2 * used * nb * qh * d
            pairs = min(pairs, nq * kept * 64)
        flops += 4 * pairs * qh * d
    return {"bytes": float(moved), "flops": float(flops)}


# ------------------------------------------------------------------ inputs
def _dt(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _keys(g, b, n, h, d):
    """Keys as a transformer has them: a part shared by neighbouring tokens, a part of the token's own, and
    channels of a head that are larger than the others or off zero."""
    runs = torch.randn(b, -(-n // 48) + 1, h, d, generator=g, device=DEV)
    x = runs.repeat_interleave(48, 1)[:, :n]
    x = 0.8 * x + 0.6 * torch.randn(b, n, h, d, generator=g, device=DEV)
    gain = 1 + 3 * (torch.rand(h, d, generator=g, device=DEV) > 0.96)
    return x * gain + 0.3 * torch.randn(h, d, generator=g, device=DEV)


def _values(g, b, n, h, d):
    return torch.randn(b, n, h, d, generator=g, device=DEV) * torch.exp2(torch.randint(-1, 3, (h, 1), generator=g, device=DEV).float())


def _queries(g, c):
    b, nq, qh, d = c["batch"], c["queries"], c["q_heads"], c["dim"]
    drift = torch.randn(b, -(-nq // 96) + 1, qh, d, generator=g, device=DEV).repeat_interleave(96, 1)[:, :nq]
    return (0.9 * drift + 0.7 * torch.randn(b, nq, qh, d, generator=g, device=DEV)).to(_dt(c))


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    b, kh, d = c["batch"], c["kv_heads"], c["dim"]
    at = _lengths(c)
    store = c["op"] == "store"
    width = -(-(max(at) + (c["tokens"] if store else 0)) // BLOCK) if max(at) or store else 1
    pool = b * width + (5 if c["paged"] else 0)
    if c["paged"]:
        table = torch.randperm(pool, generator=g, device=DEV)[:b * width].view(b, width).int()
    else:
        table = torch.arange(pool, device=DEV).view(b, width).int()
    s = dict(case=c, width=width, pool=pool, table=table, at=torch.tensor(at, device=DEV, dtype=torch.int32), most=max(at))
    cache = dict(k=torch.zeros(pool, kh, d // 16, BLOCK, 16, device=DEV).to(torch.float8_e4m3fn),
                 v=torch.zeros(pool, kh, 4, d, 16, device=DEV).to(torch.float8_e4m3fn),
                 k_scale=torch.ones(pool, kh, device=DEV), v_scale=torch.ones(pool, kh, device=DEV),
                 k_mean=torch.zeros(pool, kh, d, dtype=torch.int8, device=DEV),
                 k_mean_scale=torch.zeros(pool, kh, device=DEV))
    s["cache"] = cache
    if max(at):     # what the sequences hold already, all sequences as long as the longest (the rest is stale)
        zero = torch.zeros(1, dtype=torch.int32, device=DEV)
        for i in range(b):
            n = max(at) if not store else max(at[i], 1)
            _plain_store(cache, table[i:i + 1], zero, _keys(g, 1, n, kh, d), _values(g, 1, n, kh, d), _touched([0], n))
    if not store and s["most"]:
        # blocks whose last tokens are not the sequence's: their means are those of its own tokens
        _trim(cache, table, s["at"])
    if store:
        # keys and values as the projections leave them: side by side in one row of a token
        kv = torch.cat([_keys(g, b, c["tokens"], kh, d), _values(g, b, c["tokens"], kh, d)], 2).to(_dt(c))
        s["k_new"], s["v_new"], s["touched"] = kv[:, :, :kh], kv[:, :, kh:], _touched(at, c["tokens"])
    else:
        s["q"] = _queries(g, c)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(b, c["queries"], c["q_heads"], device=DEV)
        if c["op"] == "sparse":
            s["blocks"] = torch.empty(b, kh, -(-c["queries"] // c["q_tile"]), c["keep"], dtype=torch.int32, device=DEV)
    if own:
        from activation_residual_compression_amd import librescomp as rc
        s["plan"] = rc.KvPlan(batch=b, q_heads=c["q_heads"], kv_heads=kh, head_dim=d, pool_blocks=pool, seq_blocks=width,
                              dtype=c["dtype"], max_queries=c.get("queries", 1), causal=c.get("causal", False),
                              q_tile=c.get("q_tile", 0), keep_blocks=c.get("keep", 0))
        s["kv"] = rc.KvCache(**cache)
    return s


# ------------------------------------------------------------------ plain forms
def _exponent(amax):
    """The smallest e with amax <= 448 * 2^e, within the allowed range."""
    m, ex = torch.frexp(amax)
    return torch.where(amax > 0, ex - 9 + (m > 0.875), torch.full_like(ex, E_MIN)).clamp(E_MIN, E_MAX)


def _encode(x, e):
    return (x * torch.exp2(-e.float())).clamp(-448, 448).to(torch.float8_e4m3fn).float()


def _k_tokens(k):
    """K codes [..., D/16, 64, 16] -> values [..., 64, D]."""
    return k.float().transpose(-3, -2).flatten(-2)


def _v_tokens(v):
    """V codes [..., 4, D, 16] -> values [..., 64, D]."""
    return v.float().transpose(-2, -1).flatten(-3, -2)


def _means(codes, count, e):
    """8-bit mean keys of blocks: codes [..., 64, D] with dead tokens zero, count of live tokens."""
    total = codes.sum(-2)
    a = total.abs().amax(-1)
    inv = torch.where(a > 0, 127 / a, torch.zeros_like(a))
    return (total * inv[..., None]).round().to(torch.int8), a / (127 * count) * torch.exp2(e.float())


def _touched(starts, tokens):
    """(sequence, block) of every block that gets a new token."""
    pairs = [(i, j) for i, s in enumerate(starts) for j in range(s // BLOCK, -(-(s + tokens) // BLOCK))]
    return torch.tensor(pairs, device=DEV).T.contiguous()


def _plain_store(cache, table, start, k, v, touched):
    b, n, h, d = k.shape
    seq, which = touched                                                      # [T]
    phys = table.long()[seq, which]
    first = start.long()[seq][:, None]
    pos = which[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)            # [T, 64]
    new = ((pos >= first) & (pos < first + n))[:, None, :, None]
    old = (pos < first)[:, None, :, None]
    begun = (which * BLOCK < first[:, 0])[:, None]                            # the block holds earlier tokens
    row = (pos - first).clamp(0, n - 1)
    for name, x, tokens in (("k", k, _k_tokens), ("v", v, _v_tokens)):
        x = x[seq[:, None], row].float().transpose(1, 2)                      # [T, h, 64, d]
        fresh = torch.where(new & x.isfinite(), x, torch.zeros_like(x))
        e = _exponent(fresh.abs().amax((-2, -1)))
        was = tokens(cache[name][phys])
        e_was = torch.log2(cache[name + "_scale"][phys]).round().int()
        e = torch.where(begun, torch.maximum(e, e_was), e)
        kept = torch.where(old, _encode(was, (e - e_was)[..., None, None]),
                           torch.where(begun[..., None, None], was, torch.zeros_like(was)))
        codes = torch.where(new, _encode(x, e[..., None, None]), kept)
        if name == "k":
            laid = codes.unflatten(-1, (d // 16, 16)).transpose(-3, -2)
            count = (first + n - which[:, None] * BLOCK).clamp(1, BLOCK).float()
            mean, mean_scale = _means(torch.where(new | old, codes, torch.zeros_like(codes)), count, e)
            cache["k_mean"][phys] = mean
            cache["k_mean_scale"][phys] = mean_scale
        else:
            laid = codes.unflatten(-2, (4, 16)).transpose(-2, -1)
        cache[name].view(torch.uint8)[phys] = laid.to(torch.float8_e4m3fn).view(torch.uint8)
        cache[name + "_scale"][phys] = torch.exp2(e.float())


def _trim(cache, table, lengths):
    """Recomputes the mean key of each sequence's last block, for a length inside it."""
    last = (lengths - 1).clamp(min=0) // BLOCK
    at = table.long().gather(1, last.long()[:, None])[:, 0]
    count = (lengths - last * BLOCK).clamp(1, BLOCK)
    codes = _k_tokens(cache["k"][at])
    live = (torch.arange(BLOCK, device=DEV) < count[:, None])[:, None, :, None]
    mean, scale = _means(torch.where(live, codes, torch.zeros_like(codes)), count[:, None].float(),
                         torch.log2(cache["k_scale"][at]).round().int())
    cache["k_mean"][at] = mean
    cache["k_mean_scale"][at] = scale


def _weigh(s, v):
    """Softmax of scores over the last axis times v; rows with no score give 0 and -inf."""
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    return out, (m + torch.log(total))[..., 0]


def _limits(s):
    """The number of cached tokens that each query may see, [b, queries]."""
    c, n = s["case"], s["at"][:, None]
    if not c["causal"]:
        return n.expand(-1, c["queries"])
    return (n - c["queries"] + 1 + torch.arange(c["queries"], device=DEV)).clamp(min=0)


def _grouped(s):
    """Queries in fp32, by key head: [b, kh, queries, G, d]."""
    c = s["case"]
    return s["q"].float().unflatten(2, (c["kv_heads"], -1)).permute(0, 2, 1, 3, 4)


def _plain_attend(s):
    c, cache = s["case"], s["cache"]
    b, kh, nq, d = c["batch"], c["kv_heads"], c["queries"], c["dim"]
    phys = s["table"].long()
    k = (_k_tokens(cache["k"][phys]) * cache["k_scale"][phys][..., None, None]).transpose(1, 2).flatten(2, 3)
    v = (_v_tokens(cache["v"][phys]) * cache["v_scale"][phys][..., None, None]).transpose(1, 2).flatten(2, 3)
    q = _grouped(s) * (1 / math.sqrt(d))
    score = q.flatten(2, 3) @ k.transpose(-1, -2)                             # [b, kh, nq * G, L]
    lim = _limits(s).repeat_interleave(c["q_heads"] // kh, 1)
    seen = torch.arange(k.shape[2], device=DEV) < lim[:, None, :, None]
    score = torch.where(seen, score, torch.full((), -math.inf, device=DEV))
    out, lse = _weigh(score, v)
    out = out.view(b, kh, nq, -1, d).transpose(1, 2).flatten(2, 3)
    return out.to(_dt(c)), lse.view(b, kh, nq, -1).transpose(1, 2).flatten(2).contiguous()


def _plain_select(s):
    """Indices of the blocks kept for each sequence, key head and tile of queries, ascending, -1 where there are fewer."""
    c, cache = s["case"], s["cache"]
    b, kh, nq, tile, keep = c["batch"], c["kv_heads"], c["queries"], c["q_tile"], c["keep"]
    phys = s["table"].long()
    q = _grouped(s)
    top = q.abs().amax(-1, keepdim=True)
    codes = (q * torch.where(top > 0, 127 / top, torch.zeros_like(top))).round()
    mean = cache["k_mean"][phys].float().permute(0, 2, 3, 1)                  # [b, kh, d, nblocks]
    dot = codes.flatten(2, 3) @ mean                                          # whole numbers below 2^24: exact
    score = dot * cache["k_mean_scale"][phys].transpose(1, 2)[:, :, None] * top.flatten(2, 3) + 0.0
    score = score.unflatten(2, (nq, -1)).amax(3)                              # over the heads that share keys
    lim = _limits(s)
    blocks = torch.arange(phys.shape[1], device=DEV)
    seen = blocks * BLOCK < lim[:, None, :, None]
    score = torch.where(seen, score, torch.full((), -math.inf, device=DEV))
    tiles = -(-nq // tile)
    score = torch.nn.functional.pad(score, (0, 0, 0, tiles * tile - nq), value=-math.inf).unflatten(2, (tiles, tile)).amax(3)
    if c["causal"]:                                                           # blocks that hold the tile's own positions
        low = torch.nn.functional.pad(lim, (0, tiles * tile - nq), value=1 << 30).unflatten(1, (tiles, tile)).amin(2)
        high = torch.nn.functional.pad(lim, (0, tiles * tile - nq), value=0).unflatten(1, (tiles, tile)).amax(2)
        mine = ((blocks + 1) * BLOCK >= low[..., None]) & (blocks * BLOCK < high[..., None])
        score = torch.where(mine[:, None], torch.full((), math.inf, device=DEV), score)
    if phys.shape[1] < keep:
        score = torch.nn.functional.pad(score, (0, keep - phys.shape[1]), value=-math.inf)
    best, index = torch.sort(score, dim=-1, descending=True, stable=True)
    best, index = best[..., :keep], index[..., :keep]
    index = torch.where(best > -math.inf, index, torch.full_like(index, 1 << 30)).sort(-1).values
    return torch.where(index < (1 << 30), index, torch.full_like(index, -1)).int()


def _plain_sparse(s):
    c, cache = s["case"], s["cache"]
    b, kh, nq, d, tile, keep = c["batch"], c["kv_heads"], c["queries"], c["dim"], c["q_tile"], c["keep"]
    blocks = _plain_select(s)                                                 # [b, kh, tiles, keep]
    tiles = blocks.shape[2]
    phys = s["table"].long()[:, None, None].expand(-1, kh, tiles, -1).gather(3, blocks.clamp(min=0).long())
    head = torch.arange(kh, device=DEV)[None, :, None, None]
    k = (_k_tokens(cache["k"][phys, head]) * cache["k_scale"][phys, head][..., None, None]).flatten(3, 4)
    v = (_v_tokens(cache["v"][phys, head]) * cache["v_scale"][phys, head][..., None, None]).flatten(3, 4)
    pad = tiles * tile - nq
    q = torch.nn.functional.pad(_grouped(s) * (1 / math.sqrt(d)), (0, 0, 0, 0, 0, pad)).unflatten(2, (tiles, tile)).flatten(3, 4)
    score = q @ k.transpose(-1, -2)                                           # [b, kh, tiles, tile * G, keep * 64]
    pos = (blocks[..., None] * BLOCK + torch.arange(BLOCK, device=DEV)).flatten(3)
    pos = torch.where((blocks >= 0)[..., None].expand(-1, -1, -1, -1, BLOCK).flatten(3), pos, torch.full_like(pos, 1 << 30))
    lim = torch.nn.functional.pad(_limits(s), (0, pad)).unflatten(1, (tiles, tile)).repeat_interleave(c["q_heads"] // kh, 2)
    score = torch.where(pos[:, :, :, None] < lim[:, None, :, :, None], score, torch.full((), -math.inf, device=DEV))
    out, lse = _weigh(score, v)
    out = out.view(b, kh, tiles * tile, -1, d)[:, :, :nq].transpose(1, 2).flatten(2, 3)
    lse = lse.reshape(b, kh, tiles * tile, -1)[:, :, :nq].transpose(1, 2).flatten(2)
    return out.to(_dt(c)), lse.contiguous(), blocks


def run(state):
    s = state
    c, cache = s["case"], s["cache"]
    if c["op"] == "store":
        if own:
            s["plan"].store(s["kv"], s["at"], s["k_new"], s["v_new"], table=s["table"])
        else:
            _plain_store(cache, s["table"], s["at"], s["k_new"], s["v_new"], s["touched"])
        return dict(cache)
    if c["op"] == "attend":
        if own:
            s["plan"].attend(s["kv"], s["at"], s["q"], s["out"], s["lse"], table=s["table"], max_len=s["most"])
            return {"out": s["out"], "lse": s["lse"]}
        out, lse = _plain_attend(s)
        return {"out": out, "lse": lse}
    if own:
        s["plan"].select(s["kv"], s["at"], s["q"], s["blocks"], table=s["table"], max_len=s["most"])
        s["plan"].attend(s["kv"], s["at"], s["q"], s["out"], s["lse"], table=s["table"], max_len=s["most"], blocks=s["blocks"])
        return {"out": s["out"], "lse": s["lse"], "blocks": s["blocks"]}
    out, lse, blocks = _plain_sparse(s)
    return {"out": out, "lse": lse, "blocks": blocks}


# ------------------------------------------------------------------ in 64 bits
def _exact_codes(x, e):
    """x / 2^e rounded to the nearest e4m3 value (ties to even), in 64 bits."""
    y = (x / torch.exp2(e.double())).clamp(-448, 448)
    ex = torch.frexp(y)[1].clamp(min=-5) - 1
    step = torch.exp2((ex - 3).double())
    return (y / step).round() * step


def _exact_store(c, s):
    cache, table = s["cache"], s["table"].cpu().tolist()
    got = {n: cache[n].double() for n in ("k", "v", "k_scale", "v_scale", "k_mean_scale")}
    for i, at in enumerate(s["at"].tolist()):
        end = at + c["tokens"]
        for j in range(at // 64, (end + 63) // 64):
            lo, hi, p = max(at, j * 64), min(end, j * 64 + 64), table[i][j]
            for n in ("k", "v"):
                x = s[n + "_new"][i, lo - at:hi - at].double().transpose(0, 1)            # [h, new, d]
                amax = x.abs().amax((1, 2))
                e = torch.ceil(torch.log2(amax / 448)).clamp(-40, 44)
                e = e + (amax > 448 * torch.exp2(e)).double() - (amax <= 448 * torch.exp2(e - 1)).double()
                mine = got[n][p].transpose(1, 2).reshape(x.shape[0], 64, -1) if n == "k" else \
                    got[n][p].transpose(2, 3).reshape(x.shape[0], 64, -1)
                if lo > j * 64:
                    was = torch.log2(got[n + "_scale"][p])
                    e = torch.maximum(e, was)
                    mine[:, :lo - j * 64] = _exact_codes(mine[:, :lo - j * 64], (e - was)[:, None, None])
                else:
                    mine = torch.zeros_like(mine)
                mine[:, lo - j * 64:hi - j * 64] = _exact_codes(x, e[:, None, None])
                d = mine.shape[2]
                got[n][p] = mine.view(-1, 64, d // 16, 16).transpose(1, 2) if n == "k" else mine.view(-1, 4, 16, d).transpose(2, 3)
                got[n + "_scale"][p] = torch.exp2(e)
                if n == "k":
                    total = mine[:, :hi - j * 64].sum(1)
                    got["k_mean_scale"][p] = total.abs().amax(1) / (127 * (hi - j * 64)) * torch.exp2(e)
    return {**got, "k_mean": None}


def _exact_kept(c, s, i, h, lim, q):
    """For each tile of queries of sequence i and key head h, a truth value for each block: the selection as it is
    defined (whole-number products, two roundings to fp32), from q [queries, G, d]."""
    at = s["table"][i].long()
    nb = at.numel()
    top = q.float().abs().amax(-1)
    codes = torch.where(top > 0, 127 / top, torch.zeros_like(top))[..., None].mul(q.float()).round().double()
    dot = codes @ s["cache"]["k_mean"][at, h].double().T                                  # [queries, G, nb]
    score = (dot.float() * s["cache"]["k_mean_scale"][at, h] * top[..., None]).amax(1)
    begins = torch.arange(nb, device=DEV) * 64
    kept = []
    for t in range(0, c["queries"], c["q_tile"]):
        ln = lim[t:t + c["q_tile"]]
        see = begins < ln[:, None]
        best = torch.where(see, score[t:t + c["q_tile"]], torch.full((), -math.inf, device=DEV)).amax(0)
        if c["causal"]:
            best[(begins + 64 >= ln.min()) & (begins < ln.max())] = math.inf
        order = sorted(range(nb), key=lambda j, f=best.tolist(): (-f[j], j))[:c["keep"]]
        mask = torch.zeros(nb, dtype=torch.bool, device=DEV)
        mask[torch.tensor(order, device=DEV)] = True
        kept.append(mask & (best > -math.inf))
    return torch.stack(kept)


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if c["op"] == "store":
        return _exact_store(c, s)
    b, nq, qh, kh, d = c["batch"], c["queries"], c["q_heads"], c["kv_heads"], c["dim"]
    out = torch.zeros(b, nq, qh, d, dtype=torch.float64, device=DEV)
    lse = torch.full((b, nq, qh), -math.inf, dtype=torch.float64, device=DEV)
    cache = s["cache"]
    for i, n in enumerate(s["at"].tolist()):
        lim = torch.full((nq,), n, device=DEV) if not c["causal"] else (torch.arange(nq, device=DEV) + (n - nq + 1)).clamp(min=0)
        at = s["table"][i].long()
        seen = torch.arange(at.numel() * 64, device=DEV) < lim[:, None]
        for h in range(kh):
            k = cache["k"][at, h].double().transpose(1, 2).reshape(-1, d) * cache["k_scale"][at, h].double().repeat_interleave(64)[:, None]
            v = cache["v"][at, h].double().transpose(2, 3).reshape(-1, d) * cache["v_scale"][at, h].double().repeat_interleave(64)[:, None]
            heads = slice(h * (qh // kh), (h + 1) * (qh // kh))
            q = s["q"][i, :, heads]
            see = seen
            if c["op"] == "sparse":
                kept = _exact_kept(c, s, i, h, lim, q)
                see = seen & kept.repeat_interleave(c["q_tile"], 0)[:nq].repeat_interleave(64, 1)
            for g in range(qh // kh):
                x = (q[:, g].double() @ k.T) / math.sqrt(d)
                x = torch.where(see, x, torch.full((), -math.inf, dtype=torch.float64, device=DEV))
                some = see.any(1)
                log = torch.logsumexp(x, 1)
                p = torch.exp(x - torch.where(some, log, torch.zeros_like(log))[:, None])
                out[i, :, h * (qh // kh) + g] = p @ v
                lse[i, :, h * (qh // kh) + g] = log
    r = {"out": out, "lse": lse}
    return {**r, "blocks": None} if c["op"] == "sparse" else r
