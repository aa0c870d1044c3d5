"""Cases of attention over packed sequences, of the join of partial attentions and of
the pages of a key/value cache, for measuring them.

  attend  attention of packed sequences of different lengths over their own keys and
          values in full precision (bf16 or fp32), causal or not, shared key heads, with
          the log-sum-exp
  join    several attentions of the same queries over different tokens become one
  pages   the blocks of a paged 8-bit cache: reserving blocks for new tokens (with a copy
          where a shared block is written), forking sequences, freeing, compacting the
          pool, copying blocks between caches

`run` computes each operator in a plain form (elementary torch operations in fp32) or,
where `own` is true, by the library's calls.
"""
import math

import torch

own = False

BLOCK = 64
DEV = "cuda"
PARTS = ("k", "v", "k_scale", "v_scale", "k_mean", "k_mean_scale")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest call: one new token over the short prompt of its sequence, no shared heads
        dict(name="attend_token", op="attend", dtype="bf16", q_heads=24, kv_heads=24, dim=128, seqs=1, queries=1,
             keys=333, ragged=False, causal=True),
        # serving without a quantised cache: one token for each of 8 ragged long sequences, four query heads to a key head
        dict(name="attend_tokens_long", op="attend", dtype="bf16", q_heads=32, kv_heads=8, dim=128, seqs=8, queries=1,
             keys=32768, ragged=True, causal=True),
        # one GPU's share of the image workload (1152 of 4608 tokens) at the step that is sent in full, two images
        dict(name="attend_image", op="attend", dtype="bf16", q_heads=24, kv_heads=24, dim=128, seqs=2, queries=1152,
             keys=4608, ragged=False, causal=False),
        # one GPU's share of the video workload (4444 of 17776 tokens) at that step
        dict(name="attend_video", op="attend", dtype="bf16", q_heads=30, kv_heads=30, dim=64, seqs=1, queries=4444,
             keys=17776, ragged=False, causal=False),
        # whole causal prompts of odd ragged lengths, one of a single token, one empty; shared heads
        dict(name="attend_prompts", op="attend", dtype="bf16", q_heads=16, kv_heads=4, dim=128, seqs=6, queries=0,
             keys=4001, ragged=True, causal=True),
        # fp32 activations: the next parts of prompts of which the first ones are there
        dict(name="attend_prompts_f32", op="attend", dtype="f32", q_heads=16, kv_heads=2, dim=64, seqs=3, queries=777,
             keys=3001, ragged=True, causal=True),
        # a token of each of 32 sequences: its own recent tokens joined with the cached ones
        dict(name="join_tokens", op="join", dtype="bf16", batch=32, tokens=1, heads=32, dim=128, parts=2),
        # the video share, attended to in one part for each of four GPUs' tokens
        dict(name="join_video", op="join", dtype="f32", batch=1, tokens=4444, heads=30, dim=64, parts=4),
        # a decoding step with drafts: 64 sequences give back the last drafts and reserve five more tokens
        dict(name="pages_draft", op="pages", kind="draft", kv_heads=8, dim=128, slots=64, length=2000, tokens=5),
        # eight samples of each of four prompts: forks, whose first token copies the block that they share
        dict(name="pages_fork", op="pages", kind="fork", kv_heads=8, dim=128, slots=36, parents=4, length=4001, tokens=1),
        # a pool of which half is scattered free is compacted
        dict(name="pages_compact", op="pages", kind="compact", kv_heads=8, dim=128, slots=40, length=2700, pool=2048),
        # blocks of a sequence handed to another cache (24 key heads: image workload)
        dict(name="pages_copy", op="pages", kind="copy", kv_heads=24, dim=128, blocks=500, pool=601),
    ]


HEADS = [(24, 24, 128), (30, 30, 64), (32, 8, 128), (16, 4, 128), (12, 12, 64), (16, 2, 64), (5, 5, 128)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    kind = rng.choice(["token", "share", "prompt", "prompt", "join", "draft", "fork", "compact", "copy"])
    qh, kh, d = rng.choice(HEADS)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("token", "share", "prompt"):
        c = dict(op="attend", dtype=dtype, q_heads=qh, kv_heads=kh, dim=d, ragged=rng.random() < 0.6)
        if kind == "token":
            return dict(c, seqs=_log(rng, 1, 32), queries=rng.choice([1, 1, 2, 3]), keys=_log(rng, 16, 32768), causal=True)
        if kind == "share":
            return dict(c, seqs=_log(rng, 1, 4), queries=_log(rng, 8, 4444), keys=_log(rng, 333, 17776),
                        causal=rng.random() < 0.3)
        return dict(c, seqs=_log(rng, 1, 24), queries=0, keys=_log(rng, 16, 8888), causal=rng.random() < 0.8)
    if kind == "join":
        return dict(op="join", dtype=dtype, batch=_log(rng, 1, 32), tokens=rng.choice([1, 1, 2, _log(rng, 8, 4444)]),
                    heads=qh, dim=d, parts=rng.choice([2, 2, 3, 4, 8]))
    c = dict(op="pages", kind=kind, kv_heads=kh, dim=d)
    if kind == "draft":
        return dict(c, slots=_log(rng, 1, 128), length=_log(rng, 1, 4001), tokens=rng.choice([1, 1, 2, 5, 64, 333]))
    if kind == "fork":
        parents = _log(rng, 1, 8)
        return dict(c, slots=parents * (1 + _log(rng, 1, 8)), parents=parents, length=_log(rng, 1, 8001),
                    tokens=rng.choice([1, 1, 3, 100]))
    if kind == "compact":
        slots, length = _log(rng, 1, 32), _log(rng, 64, 4001)
        return dict(c, slots=slots, length=length, pool=int(rng.uniform(1.05, 3.0) * slots * -(-length // BLOCK)) + 1)
    n = _log(rng, 1, 1500)
    return dict(c, blocks=n, pool=n + _log(rng, 1, 200))


def _kind(c):
    return c["op"] + c.get("kind", "")


def draw(rng):
    most = {}
    for c in listed():
        w, m = work(c), most.setdefault(_kind(c), {"bytes": 0.0, "flops": 0.0})
        most[_kind(c)] = {k: max(m[k], w[k]) for k in m}
    while True:
        c = _draw(rng)
        w, m = work(c), most[_kind(c)]
        several = 3 if c.get("dtype") == "f32" and c["op"] == "attend" else 1   # an fp32 product costs several
        if w["bytes"] <= m["bytes"] and w["flops"] * several <= max(m["flops"], 1.0):
            return c


def _spread(n, top):
    """n lengths from `top` down to an eighth of it, mostly odd."""
    return [top] if n == 1 else [max(0, top - (i * 7 * top) // (8 * (n - 1)) - (i % 3)) for i in range(n)]


def _lengths(c):
    """(queries, keys) of every sequence, from the case alone."""
    keys = _spread(c["seqs"], c["keys"]) if c["ragged"] else [c["keys"]] * c["seqs"]
    if c["ragged"] and c["seqs"] >= 4:
        keys[1], keys[2] = 1, 0
    return [(c["queries"] or k, k) for k in keys]


def _held(c):
    """Tokens that every slot holds (for forks: the parents, which come first)."""
    return _spread(c.get("parents", c["slots"]), c["length"])


def _block_bytes(c):
    return c["kv_heads"] * (2 * BLOCK * c["dim"] + c["dim"] + 12)


def work(case):
    c = case
    if c["op"] == "attend":
        qh, kh, d = c["q_heads"], c["kv_heads"], c["dim"]
        es = 2 if c["dtype"] == "bf16" else 4
        moved = pairs = 0
        for nq, n in _lengths(c):
            moved += 2 * nq * qh * d * es + 4 * nq * qh + 2 * n * kh * d * es
            first = n - nq + 1     # tokens that the first query sees
            pairs += nq * n if not c["causal"] else sum(range(max(first, 0), n + 1)) if nq else 0
        return {"bytes": float(moved), "flops": 4.0 * pairs * qh * d}
    if c["op"] == "join":
        rows = c["batch"] * c["tokens"] * c["heads"]
        es = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": float(rows * (c["parts"] + 1) * (c["dim"] * es + 4)), "flops": 2.0 * rows * c["parts"] * c["dim"]}
    if c["kind"] == "copy":
        return {"bytes": float(c["blocks"] * (2 * _block_bytes(c) + 8)), "flops": 0.0}
    held = _held(c)
    used = sum(-(-n // BLOCK) for n in held)
    if c["kind"] == "compact":
        # every entry and count read and written; of the used blocks that share moves that lies past the end
        moves = used * (1 - used / c["pool"])
        return {"bytes": float(8 * used + 8 * c["pool"] + 2 * moves * _block_bytes(c)), "flops": 0.0}
    new = sum(-(-(n + c["tokens"]) // BLOCK) - n // BLOCK for n in held)
    if c["kind"] == "draft":
        return {"bytes": float(8 * c["slots"] + 16 * new), "flops": 0.0}
    each = c["slots"] // c["parents"] - 1
    copies = each * sum(n % BLOCK > 0 for n in held)
    return {"bytes": float(4 * used + each * (4 * used + 16 * new) + 2 * copies * _block_bytes(c)), "flops": 0.0}


# ------------------------------------------------------------------ inputs
def _dt(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _keys(g, n, h, d):
    """Keys as a transformer has them: a part shared by neighbouring tokens, a part of the token's own, and
    channels of a head that are larger than the others or off zero."""
    x = torch.randn(-(-n // 48) + 1, h, d, generator=g, device=DEV).repeat_interleave(48, 0)[:n]
    x = 0.8 * x + 0.6 * torch.randn(n, h, d, generator=g, device=DEV)
    gain = 1 + 3 * (torch.rand(h, d, generator=g, device=DEV) > 0.96)
    return x * gain + 0.3 * torch.randn(h, d, generator=g, device=DEV)


def _values(g, n, h, d):
    return torch.randn(n, h, d, generator=g, device=DEV) * torch.exp2(torch.randint(-1, 3, (h, 1), generator=g, device=DEV).float())


def _queries(g, n, h, d):
    drift = torch.randn(-(-n // 96) + 1, h, d, generator=g, device=DEV).repeat_interleave(96, 0)[:n]
    return 0.9 * drift + 0.7 * torch.randn(n, h, d, generator=g, device=DEV)


def _starts(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _cache(g, c, pool):
    kh, d = c["kv_heads"], c["dim"]

    def codes(shape):        # e4m3 codes, finite ones
        x = torch.randint(0, 254, shape, generator=g, device=DEV, dtype=torch.uint8)
        return torch.where(x < 127, x, x + 1).view(torch.float8_e4m3fn)

    def scale():
        return torch.exp2(torch.randint(-8, 2, (pool, kh), generator=g, device=DEV).float())
    return dict(k=codes((pool, kh, d // 16, BLOCK, 16)), v=codes((pool, kh, 4, d, 16)), k_scale=scale(), v_scale=scale(),
                k_mean=torch.randint(-127, 128, (pool, kh, d), generator=g, device=DEV, dtype=torch.int8),
                k_mean_scale=torch.rand(pool, kh, generator=g, device=DEV))


def _prepare_pages(c, g, s):
    if c["kind"] == "copy":
        pool = c["pool"]
        s["cache"], s["to"] = _cache(g, c, pool), _cache(g, c, pool)
        s["src"] = torch.randperm(pool, generator=g, device=DEV)[:c["blocks"]].int()
        s["dst"] = torch.randperm(pool, generator=g, device=DEV)[:c["blocks"]].int()
        slots, width = 1, pool
    else:
        held, slots = _held(c), c["slots"]
        more = c.get("tokens", 0)
        width = -(-(max(held) + more) // BLOCK) + 1
        used = sum(-(-n // BLOCK) for n in held)
        # a tenth more than will be needed
        pool = c.get("pool") or int(1.1 * (used + slots * (-(-more // BLOCK) + 1))) + 1
        s["cache"] = _cache(g, c, pool)
        order = torch.randperm(pool, generator=g, device=DEV).int()
        s["table"] = torch.full((slots, width), -1, dtype=torch.int32, device=DEV)
        at = 0
        for i, n in enumerate(held):
            nb = -(-n // BLOCK)
            s["table"][i, :nb] = order[at:at + nb]
            at += nb
        s["refs"] = torch.zeros(pool, dtype=torch.int32, device=DEV)
        s["refs"][order[:at].long()] = 1
        if c["kind"] == "draft":
            s["keep"] = s["start"] = _int(held)
            s["tokens"] = torch.full((slots,), more, dtype=torch.int32, device=DEV)
            s["copying"] = None
        elif c["kind"] == "fork":
            each = slots // c["parents"] - 1
            s["keep"] = _int([1 << 30] * c["parents"] + [0] * (slots - c["parents"]))
            s["source"] = _int([-1] * c["parents"] + [p for p in range(c["parents"]) for _ in range(each)])
            s["start"] = s["length"] = _int([0] * c["parents"] + [n for n in held for _ in range(each)])
            s["tokens"] = _int([0] * c["parents"] + [more] * (slots - c["parents"]))
            copying = [c["parents"] + p * each + i for p, n in enumerate(held) if n % BLOCK for i in range(each)]
            s["copying"] = torch.tensor(copying, device=DEV) if copying else None
        else:
            s["table0"], s["refs0"] = s["table"].clone(), s["refs"].clone()
            s["moves"] = int((s["refs"][int((s["refs"] > 0).sum()):] > 0).sum())
        s["lacking"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if own:
        from activation_residual_compression_amd import librescomp as rc
        s["plan"] = rc.PagePlan(slots=slots, kv_heads=c["kv_heads"], head_dim=c["dim"], pool_blocks=pool, seq_blocks=width)
        s["kv"] = rc.KvCache(**s["cache"])
        if c["kind"] == "copy":
            s["kv_to"] = rc.KvCache(**s["to"])


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(case=c)
    if c["op"] == "pages":
        _prepare_pages(c, g, s)
    elif c["op"] == "join":
        shape = (c["batch"], c["tokens"], c["heads"], c["dim"])
        s["outs"] = [torch.randn(shape, generator=g, device=DEV).to(_dt(c)) for _ in range(c["parts"])]
        # parts of which one mostly weighs more, some that saw nothing, rows where none did
        s["lses"] = [torch.randn(shape[:3], generator=g, device=DEV) * 2 + 7 for _ in range(c["parts"])]
        none = torch.rand(shape[:3], generator=g, device=DEV) < 0.01
        for x in s["lses"]:
            x[none | (torch.rand(shape[:3], generator=g, device=DEV) < 0.03)] = -math.inf
        s["out"] = torch.empty_like(s["outs"][0])
        s["lse"] = torch.empty_like(s["lses"][0])
    else:
        qh, kh, d = c["q_heads"], c["kv_heads"], c["dim"]
        lengths = _lengths(c)
        s["q_at"], s["k_at"] = _starts([q for q, _ in lengths]), _starts([k for _, k in lengths])
        nq, nk = s["q_at"][-1], s["k_at"][-1]
        if c["queries"]:
            kv = torch.cat([_keys(g, nk, kh, d), _values(g, nk, kh, d)], 1).to(_dt(c))
            s["q"], s["k"], s["v"] = _queries(g, nq, qh, d).to(_dt(c)), kv[:, :kh], kv[:, kh:]
        else:     # one projection leaves queries, keys and values of a token side by side
            qkv = torch.cat([_queries(g, nq, qh, d), _keys(g, nk, kh, d), _values(g, nk, kh, d)], 1).to(_dt(c))
            s["q"], s["k"], s["v"] = qkv[:, :qh], qkv[:, qh:qh + kh], qkv[:, qh + kh:]
        s["q_offsets"], s["kv_offsets"] = _int(s["q_at"]), _int(s["k_at"]) if c["queries"] else None
        s["max_q"], s["max_kv"] = max(q for q, _ in lengths), max(k for _, k in lengths)
        s["out"] = torch.empty(nq, qh, d, dtype=_dt(c), device=DEV)
        s["lse"] = torch.empty(nq, qh, device=DEV)
        if own:
            from activation_residual_compression_amd import librescomp as rc
            s["plan"] = rc.AttnPlan(q_heads=qh, kv_heads=kh, head_dim=d, dtype=c["dtype"], max_seqs=c["seqs"],
                                    max_queries=nq, max_keys=nk, causal=c["causal"])
    return s


# ------------------------------------------------------------------ plain forms
def _plain_attend(s):
    c = s["case"]
    kh, d = c["kv_heads"], c["dim"]
    outs, sums = [], []
    for i in range(c["seqs"]):
        q = s["q"][s["q_at"][i]:s["q_at"][i + 1]].float().unflatten(1, (kh, -1)) * (1 / math.sqrt(d))
        k, v = (s[x][s["k_at"][i]:s["k_at"][i + 1]].float() for x in ("k", "v"))
        nq, n = q.shape[0], k.shape[0]
        if n == 0:
            outs.append(torch.zeros(nq, c["q_heads"], d, device=DEV))
            sums.append(torch.full((nq, c["q_heads"]), -math.inf, device=DEV))
            continue
        score = q.permute(1, 0, 2, 3).flatten(1, 2) @ k.permute(1, 2, 0).contiguous()        # [kh, nq * G, n]
        if c["causal"]:
            limit = (n - nq + 1 + torch.arange(nq, device=DEV)).repeat_interleave(c["q_heads"] // kh)
            seen = torch.arange(n, device=DEV) < limit[:, None]
            score = torch.where(seen, score, torch.full((), -math.inf, device=DEV))
        m = score.amax(-1, keepdim=True)
        m = torch.where(m > -math.inf, m, torch.zeros_like(m))
        p = torch.exp(score - m)
        total = p.sum(-1, keepdim=True)
        out = (p @ v.transpose(0, 1).contiguous()) / torch.where(total > 0, total, torch.ones_like(total))
        outs.append(out.view(kh, nq, -1, d).transpose(0, 1).flatten(1, 2))
        sums.append((m + torch.log(total))[..., 0].view(kh, nq, -1).transpose(0, 1).flatten(1))
    return {"out": torch.cat(outs).to(_dt(c)), "lse": torch.cat(sums)}


def _plain_join(s):
    lse = torch.stack(s["lses"])
    m = lse.amax(0)
    w = torch.exp(lse - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    total = w.sum(0)
    w = w / torch.where(total > 0, total, torch.ones_like(total))
    out = sum(w[i][..., None] * x.float() for i, x in enumerate(s["outs"]))
    return {"out": out.to(_dt(s["case"])), "lse": m + torch.log(total)}


def _plain_free(s):
    table, refs = s["table"], s["refs"]
    j = torch.arange(table.shape[1], device=DEV)
    gone = (j >= (s["keep"][:, None] + (BLOCK - 1)) // BLOCK) & (table >= 0)
    refs.index_add_(0, table.clamp(min=0).long().flatten(), -gone.int().flatten())
    table.masked_fill_(gone, -1)


def _plain_fork(s):
    table, refs = s["table"], s["refs"]
    j = torch.arange(table.shape[1], device=DEV)
    new = table[s["source"].clamp(min=0).long()]
    new = torch.where(j < (s["length"][:, None] + (BLOCK - 1)) // BLOCK, new, torch.full_like(new, -1))
    new = torch.where(s["source"][:, None] >= 0, new, table)
    for rows, sign in ((table, -1), (new, 1)):
        refs.index_add_(0, rows.clamp(min=0).long().flatten(), sign * (rows >= 0).int().flatten())
    table.copy_(new)


def _plain_reserve(s):
    """Every entry that lacks a block, or shares the block that it will write, gets the next free one. (In these cases
    a shared block has holders that do not write, so none of those that do keeps it.)"""
    table, refs, cache = s["table"], s["refs"], s["cache"]
    slots, width = table.shape
    pool = refs.numel()
    first, last = s["start"] // BLOCK, (s["start"] + s["tokens"] + BLOCK - 1) // BLOCK
    j = torch.arange(width, device=DEV)
    mine = (j >= first[:, None]) & (j < last[:, None]) & (s["tokens"][:, None] > 0)
    shared = mine & (table >= 0) & (refs[table.clamp(min=0).long()] > 1)
    need = (mine & (table < 0)) | shared
    rank = torch.cumsum(need.flatten().long(), 0).view(slots, width) - 1
    free = torch.sort(torch.where(refs > 0, pool, torch.arange(pool, device=DEV)))[0]       # ascending, then `pool`
    new = free[rank.clamp(min=0, max=pool - 1)].int()
    s["lacking"].copy_((need.sum() - (refs <= 0).sum()).clamp(min=0))
    if s["copying"] is not None:      # the slots whose first new token goes into a shared block
        slot, at = s["copying"], first[s["copying"]].long()
        old, to = table[slot, at].long(), new[slot, at].long()
        for x in PARTS:
            raw = cache[x].view(torch.uint8) if x in ("k", "v") else cache[x]
            raw[to] = raw[old]
    refs.index_add_(0, table.clamp(min=0).long().flatten(), -shared.int().flatten())
    refs.index_add_(0, new.long().clamp(max=pool - 1).flatten(), need.int().flatten())
    table.copy_(torch.where(need, new, table))


def _plain_compact(s):
    table, refs, cache = s["table"], s["refs"], s["cache"]
    pool = refs.numel()
    used = refs > 0
    count = used.sum()
    at = torch.arange(pool, device=DEV)
    src = torch.sort(torch.where(used & (at >= count), at, pool))[0][:s["moves"]]
    dst = torch.sort(torch.where(~used & (at < count), at, pool))[0][:s["moves"]]
    moved = torch.where(used, at, torch.full_like(at, -1))
    moved[src] = dst
    for x in PARTS:
        raw = cache[x].view(torch.uint8) if x in ("k", "v") else cache[x]
        raw[dst] = raw[src]
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, moved[table.clamp(min=0).long()].int(), table))
    s["lacking"].copy_(count)


def run(state):
    s = state
    c = s["case"]
    if c["op"] == "attend":
        if not own:
            return _plain_attend(s)
        s["plan"].attend(s["q"], s["k"], s["v"], s["q_offsets"], s["out"], s["lse"], kv_offsets=s["kv_offsets"],
                         max_q=s["max_q"], max_kv=s["max_kv"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "join":
        if not own:
            return _plain_join(s)
        from activation_residual_compression_amd import librescomp as rc
        rc.join_attention(s["outs"], s["lses"], s["out"], s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["kind"] == "copy":
        if own:
            s["plan"].copy(s["kv"], s["src"], s["dst"], to=s["kv_to"])
        else:
            for x in PARTS:
                a, b = ((y[x].view(torch.uint8) if x in ("k", "v") else y[x]) for y in (s["cache"], s["to"]))
                b[s["dst"].long()] = a[s["src"].long()]
        return dict(s["to"])
    if c["kind"] == "compact":       # a pool as it is each time: the same blocks scattered in it
        s["table"].copy_(s["table0"])
        s["refs"].copy_(s["refs0"])
        if own:
            s["plan"].compact(s["kv"], s["refs"], s["table"], used=s["lacking"])
        else:
            _plain_compact(s)
    elif own:
        s["plan"].free(s["refs"], s["table"], s["keep"])
        if c["kind"] == "fork":
            s["plan"].fork(s["refs"], s["table"], s["source"], s["length"])
        s["plan"].reserve(s["kv"], s["refs"], s["table"], s["start"], s["tokens"], missing=s["lacking"])
    else:
        _plain_free(s)
        if c["kind"] == "fork":
            _plain_fork(s)
        _plain_reserve(s)
    return {**s["cache"], "table": s["table"], "refs": s["refs"], "count": s["lacking"]}


# ------------------------------------------------------------------ in 64 bits
def _exact_attend(c, s):
    qh, kh, d = c["q_heads"], c["kv_heads"], c["dim"]
    out = torch.zeros(s["q_at"][-1], qh, d, dtype=torch.float64, device=DEV)
    lse = torch.full((s["q_at"][-1], qh), -math.inf, dtype=torch.float64, device=DEV)
    for i in range(c["seqs"]):
        (qa, qb), (ka, kb) = s["q_at"][i:i + 2], s["k_at"][i:i + 2]
        n = kb - ka
        for h in range(qh if n else 0):
            k, v = (s[x][ka:kb, h * kh // qh].double() for x in ("k", "v"))
            for a in range(qa, qb, 2048):
                b = min(a + 2048, qb)
                x = (s["q"][a:b, h].double() @ k.T) / math.sqrt(d)
                if c["causal"]:
                    last = torch.arange(a - qa, b - qa, device=DEV) + n - (qb - qa)
                    x.masked_fill_(torch.arange(n, device=DEV) > last[:, None], -math.inf)
                log = torch.logsumexp(x, 1)
                some = log > -math.inf
                x = torch.exp(x - torch.where(some, log, torch.zeros_like(log))[:, None])
                out[a:b, h] = x @ v
                lse[a:b, h] = log
    return {"out": out, "lse": lse}


def _exact_join(c, s):
    lse = torch.stack(s["lses"], -1).double()
    log = torch.logsumexp(lse, -1)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for i, x in enumerate(s["outs"]):
        w = torch.exp(lse[..., i] - log)
        out += torch.where(log > -math.inf, w, torch.zeros_like(w))[..., None] * x.double()
    return {"out": out, "lse": log}


def _moved(into, cache, pairs):
    """The contents of `into` in 64 bits, once block p of `cache` has gone to block q for every pair (p, q)."""
    got = {x: into[x].double() for x in PARTS}
    if pairs:
        src, dst = (torch.tensor(x, device=DEV) for x in zip(*pairs))
        for x in PARTS:
            got[x].index_copy_(0, dst, cache[x].double().index_select(0, src))
    return got


def _exact_pages(c, s):
    """Table, counts of holders and the counter, entry by entry in the order of the definition, and where contents go."""
    if c["kind"] == "copy":
        return _moved(s["to"], s["cache"], list(zip(s["src"].tolist(), s["dst"].tolist())))
    table, refs, pairs = s["table"].tolist(), s["refs"].tolist(), []
    if c["kind"] == "compact":
        count = sum(r > 0 for r in refs)
        holes = (p for p in range(count) if refs[p] <= 0)
        to = {p: p if p < count else next(holes) for p in range(len(refs)) if refs[p] > 0}
        pairs = [(p, q) for p, q in to.items() if p != q]
        table = [[to.get(e, e) for e in row] for row in table]
        refs = [0] * len(refs)
        for row in table:
            for e in row:
                if e >= 0:
                    refs[e] += 1
    else:
        keep, start, tokens = (s[x].tolist() for x in ("keep", "start", "tokens"))
        for i, row in enumerate(table):
            for j in range(-(-keep[i] // BLOCK), len(row)):
                if row[j] >= 0:
                    refs[row[j]] -= 1
                    row[j] = -1
        if c["kind"] == "fork":
            before = [list(row) for row in table]
            for i, (p, n) in enumerate(zip(s["source"].tolist(), s["length"].tolist())):
                if p >= 0:
                    for e in table[i]:
                        if e >= 0:
                            refs[e] -= 1
                    nb = -(-n // BLOCK)
                    table[i] = before[p][:nb] + [-1] * (len(before[p]) - nb)
                    for e in table[i]:
                        if e >= 0:
                            refs[e] += 1
        free = (p for p in range(len(refs)) if refs[p] <= 0)
        free = iter(list(free))
        for i, row in enumerate(table):
            for j in range(start[i] // BLOCK, -(-(start[i] + tokens[i]) // BLOCK)) if tokens[i] > 0 else ():
                was = row[j]
                if was < 0 or refs[was] > 1:
                    row[j] = next(free)
                    refs[row[j]] = 1
                    if was >= 0:
                        refs[was] -= 1
                        if start[i] > j * BLOCK:     # it holds earlier tokens
                            pairs.append((was, row[j]))
        count = 0
    got = _moved(s["cache"], s["cache"], pairs)
    for name, x in (("table", table), ("refs", refs), ("count", [count])):
        got[name] = torch.tensor(x, dtype=torch.int64, device=DEV)
    return got


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    return {"attend": _exact_attend, "join": _exact_join, "pages": _exact_pages}[c["op"]](c, s)
