"""What bounds the cost of a long context, as cases to be measured: attention
over the blocks of a paged cache that a cheap score selects (bounds of the keys
of a block, the score, the selection, the attention), and eviction by
accumulated attention weight (the weights, the same selection, moving the kept
tokens to other pages).

``run`` computes a case in its plain form (elementary torch operations in
fp32) or, where ``own`` is true, with this library's calls.  Both work on the
same state: the cache is held in the library's documented record layout
(include/w4.h, "Paged key-value cache"), which the plain form packs and unpacks
with reshapes.  A block is a page of the cache.

Sizes come from the decoder shapes of the library's workloads: 28 query and 4
key/value heads of 128 (hidden 3584), and 14 query and 2 key/value heads of 64
(hidden 896), with pages of 16 tokens and multiples of it.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
BITS = {"bf16": 16, "int8": 8, "int4": 4}
DECAY = 0.875


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # One decode step of 64 requests: the block that each is in has a new key.
        dict(name="bounds.decode64.int4", op="bounds", fmt="int4", seqs=64, tokens=1, hkv=4,
             dim=128, page=64, longest=3000, ragged=True),
        # A prompt of 16384 tokens has been written: the bounds of all its blocks.
        dict(name="bounds.prompt16k.int8", op="bounds", fmt="int8", seqs=1, tokens=16384, hkv=4,
             dim=128, page=64, longest=16384, ragged=False),
        # A single request of the small shape, pages of 16: latency only.
        dict(name="scores.short", op="scores", seqs=1, tokens=1, hq=14, hkv=2, dim=64, page=16,
             longest=2011, ragged=False),
        # 64 ragged requests of up to 32768 tokens, blocks of 64.
        dict(name="scores.batch64", op="scores", seqs=64, tokens=1, hq=28, hkv=4, dim=128,
             page=64, longest=32768, ragged=True),
        # 64 of up to 2048 blocks for each of 64 x 4 heads: the first one, the last four and
        # the best others.
        dict(name="select.blocks", op="select", seqs=64, hkv=4, longest=131072, ragged=True,
             unit=64, first=1, last=4, count=64),
        # Four prompts of 131072 tokens cut down to 8192 tokens a head.
        dict(name="select.tokens", op="select", seqs=4, hkv=4, longest=131072, ragged=False,
             unit=1, first=4, last=512, count=8192),
        # A single request at 128 k tokens reads 64 blocks of 64.
        dict(name="sparse.single128k.bf16", op="sparse", fmt="bf16", seqs=1, tokens=1, hq=28,
             hkv=4, dim=128, page=64, longest=131072, ragged=False, count=64),
        # 64 ragged requests of up to 32768 tokens read 4096 each.
        dict(name="sparse.batch64.int8", op="sparse", fmt="int8", seqs=64, tokens=1, hq=28, hkv=4,
             dim=128, page=32, longest=32768, ragged=True, count=128),
        # What three draft tokens of the small shape attend to, at a short context.
        dict(name="weights.short.bf16", op="weights", fmt="bf16", seqs=1, tokens=3, hq=14, hkv=2,
             dim=64, page=16, longest=201, ragged=False, window=0),
        # One decode step of 64 ragged requests of up to 8192 tokens.
        dict(name="weights.batch64.int8", op="weights", fmt="int8", seqs=64, tokens=1, hq=28,
             hkv=4, dim=128, page=64, longest=8192, ragged=True, window=0),
        # Five short requests of the small shape, 256 tokens kept, read back.
        dict(name="gather.small.bf16", op="gather", fmt="bf16", seqs=5, hkv=2, dim=64, page=32,
             longest=1001, ragged=True, count=256),
        # 16 requests of 32768 tokens cut down to 4096 a head, read back.
        dict(name="gather.batch16.int4", op="gather", fmt="int4", seqs=16, hkv=4, dim=128,
             page=16, longest=32768, ragged=False, count=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["bounds", "scores", "select", "sparse", "sparse", "weights", "weights",
                     "gather"])
    dim, hkv, ratio = rng.choice([(128, 4, 7), (128, 4, 7), (64, 2, 7), (128, 8, 4), (64, 8, 1),
                                  (128, 2, 8), (64, 3, 5)])
    seqs = _log(rng, 1, 96)
    if op == "select":
        unit = rng.choice([1, 1, 16, 32, 64])
        longest = _log(rng, 30, min(131072 * unit, unit * 500000 // (seqs * hkv)))
        items = -(-longest // unit)
        count = _log(rng, 1, min(items, 8192))
        first = rng.choice([0, 1, 4]) if count > 4 else 0
        return dict(op=op, seqs=seqs, hkv=hkv, longest=longest, ragged=rng.random() < 0.6,
                    unit=unit, first=first, last=rng.randrange(0, (count - first) // 2 + 1),
                    count=count)
    fmt = rng.choice(["bf16", "int8", "int4"])
    page = rng.choice([16, 16, 32, 64, 128])
    tokens = rng.choice([1, 1, 1, 2, 3, 5, 8])
    # as many tokens as the largest listed case of the kind has
    most = {"bounds": 60000, "scores": 1000000, "sparse": 500000, "weights": 250000,
            "gather": 250000}[op] * 512 // (hkv * dim)
    longest = _log(rng, 30, min(131072, most // seqs))
    ragged = rng.random() < 0.6
    shape = dict(op=op, seqs=seqs, hkv=hkv, dim=dim, page=page, longest=longest, ragged=ragged)
    if op == "bounds":
        if rng.random() < 0.5:
            tokens = _log(rng, 1, longest)
        return dict(shape, fmt=fmt, tokens=tokens)
    if op == "scores":
        return dict(shape, hq=hkv * ratio, tokens=tokens)
    if op == "sparse":
        blocks = -(-longest // page)
        return dict(shape, fmt=fmt, hq=hkv * ratio, tokens=tokens,
                    count=_log(rng, 1, min(blocks, max(1, most // (4 * seqs * page)))))
    if op == "weights":
        # up to 56 rows a key: fewer keys for many of them
        shape["longest"] = max(30, min(longest, 4 * most // (tokens * ratio * seqs)))
        return dict(shape, fmt=fmt, hq=hkv * ratio, tokens=tokens,
                    window=rng.choice([0, 0, 0, 1000]))
    return dict(shape, fmt=fmt, count=_log(rng, 1, longest))


# ---- inputs ------------------------------------------------------------------

def _record_bytes(fmt, dim):
    return 64 * dim if fmt == "bf16" else 16 * dim * 2 * BITS[fmt] // 8 + 128


def _normal(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _channels(gen, heads, dim):
    """Some channels of keys carry larger values than the rest."""
    wide = torch.rand(heads, dim, generator=gen, device=DEV) < 1 / 16
    return torch.where(wide, 4.0, 1.0)


def _lens(gen, case):
    B, longest = case["seqs"], case["longest"]
    lens = torch.full((B,), longest, device=DEV, dtype=torch.int32)
    if case["ragged"]:
        lens = torch.randint(0, longest + 1, (B,), generator=gen, device=DEV, dtype=torch.int32)
        lens[B // 2] = longest
        if B > 3:
            lens[0] = 0                                         # a slot without a request
    return lens


def _block_table(gen, seqs, pages_each, first=0):
    """Every sequence's pages, in a random order of the pool's."""
    order = torch.randperm(seqs * pages_each, generator=gen, device=DEV) + first
    return order.view(seqs, pages_each).to(torch.int32)


def _fill(gen, pool, fmt, dim):
    """Normal keys and values in all records of pool [pages, heads, records, bytes]."""
    pages, hkv, records, _ = pool.shape
    chan = _channels(gen, hkv, dim)[:, None, None]
    step = max(1, (1 << 27) // (hkv * records * 16 * dim))
    for p in range(0, pages, step):                             # a part of the pool at a time
        n = min(step, pages - p)
        k = _normal(gen, n, hkv, records, 16, dim, dtype=torch.float32) * chan
        v = _normal(gen, n, hkv, records, 16, dim, dtype=torch.float32)
        pool[p:p + n] = _pack(k.to(torch.bfloat16).float(), v.to(torch.bfloat16).float(), fmt)


def _token_weights(gen, *shape):
    """Accumulated attention: spread over decades, some of it nothing at all."""
    w = torch.exp(3.0 * torch.randn(*shape, generator=gen, device=DEV) - 8.0)
    return torch.where(torch.rand(*shape, generator=gen, device=DEV) < 0.1, 0.0, w)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, B, hkv = case["op"], case["seqs"], case["hkv"]
    s = dict(case=case, lens=_lens(gen, case))
    if op == "select":
        n = -(-case["longest"] // case["unit"])
        s["scores"] = _token_weights(gen, B, hkv, n) if case["unit"] == 1 else \
            20.0 * _normal(gen, B, hkv, n, dtype=torch.float32)
        s["index"] = torch.full((B, hkv, case["count"]), -1, device=DEV, dtype=torch.int32)
        s["counts"] = torch.zeros(B, device=DEV, dtype=torch.int32)
        return s
    dim, page = case["dim"], case["page"]
    width = -(-case["longest"] // page)
    s["table"] = _block_table(gen, B, width)
    if op == "scores":
        # the cache's pool is there, but only the bounds are looked at
        s["pool"] = torch.zeros(B * width * hkv * (page // 16) * _record_bytes("int4", dim),
                                device=DEV, dtype=torch.uint8)
        a, b = (_normal(gen, B * width, hkv, 1, dim) * 2 for _ in "ab")
        s["bounds"] = torch.cat([torch.maximum(a, b), torch.minimum(a, b)], 2)
        s["q"] = _normal(gen, B * case["tokens"], case["hq"], dim)
        s["scores"] = torch.zeros(B, hkv, width, device=DEV)
        return s
    fmt = case["fmt"]
    to_pages = B * -(-case["count"] // page) if op == "gather" else 0
    pool = torch.zeros(B * width + to_pages, hkv, page // 16, _record_bytes(fmt, dim), device=DEV,
                       dtype=torch.uint8)
    _fill(gen, pool[:B * width], fmt, dim)
    s["pool"] = pool.view(-1)
    if op == "bounds":
        s["bounds"] = torch.zeros(B * width, hkv, 2, dim, device=DEV, dtype=torch.bfloat16)
        return s
    if op == "gather":
        n = case["count"]
        s["to"] = _block_table(gen, B, -(-n // page), B * width)
        s["weights"] = _token_weights(gen, B, hkv, case["longest"])
        s["index"], s["counts"] = _choose(s["weights"], s["lens"].long(), 4 if n > 4 else 0, 0, n)
        i = torch.arange(n, device=DEV, dtype=torch.int32)
        there = i < s["counts"][:, None]
        s["positions"] = torch.where(there, i, -1).reshape(-1)  # of what is read back
        s["weights_out"] = torch.zeros(B, hkv, n, device=DEV)
        s["k_out"], s["v_out"] = (torch.zeros(B * n, hkv, dim, device=DEV, dtype=torch.bfloat16)
                                  for _ in "kv")
        return s
    M, hq = case["tokens"], case["hq"]
    s["q"] = _normal(gen, B * M, hq, dim)
    if op == "sparse":
        blocks = (s["lens"].long() + page - 1) // page
        score = torch.rand(B, hkv, width, generator=gen, device=DEV)
        n = case["count"]
        s["blocks"], s["counts"] = _choose(score, blocks, 1 if n > 2 else 0, min(2, n), n)
        s["out"] = torch.empty(B * M, hq, dim, device=DEV, dtype=torch.bfloat16)
        s["lse"] = torch.empty(B * M, hq, device=DEV)
        return s
    # the log-sum-exp that the attention has returned
    s["lse"] = torch.empty(B * M, hq, device=DEV)
    for b, rows, seen, score in _all_scores(s):
        x = score.masked_fill(~seen, -math.inf)
        s["lse"][b * M:b * M + M] = torch.logsumexp(x, -1).view(hkv, M, -1).transpose(0, 1).flatten(1)
    s["before"] = _token_weights(gen, B, hkv, case["longest"])
    s["after"] = torch.zeros(B, hkv, case["longest"], device=DEV)
    return s


# ---- the record layout, packed and unpacked -------------------------------------

def _swizzle(fmt, dim, device):
    """16-byte piece of a token's row that is stored in place c', [16, pieces]."""
    pieces = dim * BITS[fmt] // 128
    r = torch.arange(16, device=device)[:, None]
    c = torch.arange(pieces, device=device)
    if fmt == "bf16":
        return c ^ (r & 7)
    return c ^ (4 * (r & 1)) if fmt == "int8" and dim == 128 else c.expand(16, pieces)


def _swap_pieces(rows, fmt, dim):
    """rows [..., 16, bytes]: the pieces of every row exchanged (its own inverse)."""
    at = _swizzle(fmt, dim, rows.device)
    x = rows.view(*rows.shape[:-1], -1, 16)
    return torch.take_along_dim(x, at[..., None].expand(*x.shape), -2).flatten(-2)


def _quantise(x, fmt):
    """Codes (uint8) and (scale, zero) per token: fp32, each operation rounded once."""
    top = (1 << BITS[fmt]) - 1
    lo = x.amin(-1, keepdim=True).clamp(max=0.0)
    hi = x.amax(-1, keepdim=True).clamp(min=0.0)
    s16 = ((hi - lo) / top).clamp(max=65504.0).half()
    s = s16.float()
    zero = s == 0
    s = torch.where(zero, 1.0, s)
    z = torch.where(zero, 0.0, torch.round(-lo / s).clamp(0, top))
    q = torch.where(zero, z, (torch.round(x / s) + z).clamp(0, top))
    meta = torch.cat([s16.view(torch.int16), z.to(torch.int16)], -1)
    return q.to(torch.uint8), meta


def _pack(k, v, fmt):
    """fp32 [..., 16, dim] keys and values -> records [..., bytes]."""
    if fmt == "bf16":
        return _join((k.to(torch.bfloat16), None), (v.to(torch.bfloat16), None), fmt)
    return _join(_quantise(k, fmt), _quantise(v, fmt), fmt)


def _join(k, v, fmt):
    """Keys and values as held, (codes [..., 16, dim], meta [..., 16, 2]) -> records."""
    (kq, km), (vq, vm) = k, v
    lead, dim = kq.shape[:-2], kq.shape[-1]
    if fmt == "bf16":
        return torch.cat([_swap_pieces(x.contiguous().view(torch.uint8), fmt, dim).flatten(-2)
                          for x in (kq, vq)], -1)
    axes = lambda *a: (*range(len(lead)), *(len(lead) + x for x in a))  # noqa: E731
    if fmt == "int8":
        kb = _swap_pieces(kq, fmt, dim).flatten(-2)
        w = vq.reshape(*lead, 2, 4, 2, dim // 32, 4, 8)          # h, t, r, i, e, g
    else:
        kb = (kq[..., 0::2] | (kq[..., 1::2] << 4)).flatten(-2)
        w = vq.reshape(*lead, 2, 4, 2, dim // 64, 4, 2, 8)       # h, t, r, i, e, high, g
        w = w[..., 0, :] | (w[..., 1, :] << 4)
    vb = w.permute(axes(3, 5, 1, 4, 2, 0)).reshape(*lead, -1)
    return torch.cat([kb, vb, *(m.contiguous().view(torch.uint8).flatten(-2) for m in (km, vm))],
                     -1)


def _split(rec, fmt, dim, keys_only=False):
    """Records [..., bytes] -> keys and values as held (see _join)."""
    lead = rec.shape[:-1]
    size = 16 * dim * BITS[fmt] // 8
    kb = rec[..., :size].reshape(*lead, 16, -1)
    vb = None if keys_only else rec[..., size:2 * size]
    if fmt == "bf16":
        held = lambda x: _swap_pieces(x.reshape(*lead, 16, -1), fmt, dim).view(torch.bfloat16)  # noqa: E731
        return (held(kb), None), None if keys_only else (held(vb), None)
    meta = rec[..., 2 * size:].contiguous().view(torch.int16).view(*lead, 2, 16, 2)
    if fmt == "int8":
        kq = _swap_pieces(kb, fmt, dim)
    else:
        kq = torch.stack([kb & 15, kb >> 4], -1).reshape(*lead, 16, dim)
    if keys_only:
        return (kq, meta[..., 0, :, :]), None
    vq = vb.reshape(*lead, -1, 8, 4, 4, 2, 2)                   # i, g, t, e, r, h
    order = (5, 2, 4, 0, 3, 1)
    if fmt == "int4":
        vq, order = torch.stack([vq & 15, vq >> 4], -1), (5, 2, 4, 0, 3, 6, 1)
    vq = vq.permute(*range(len(lead)), *(len(lead) + a for a in order)).reshape(*lead, 16, dim)
    return (kq, meta[..., 0, :, :]), (vq, meta[..., 1, :, :])


def _values(held):
    """fp32 values [..., 16, dim] of keys or values as held."""
    q, meta = held
    if meta is None:
        return q.float()
    s = meta[..., 0].contiguous().view(torch.float16).float()[..., None]
    return (q.float() - meta[..., 1].float()[..., None]) * s


def _records_of(s, table):
    """Records of a table's pages, [seqs, hkv, pages, page // 16, bytes]."""
    case = s["case"]
    pool = s["pool"].view(-1, case["hkv"], case["page"] // 16,
                          _record_bytes(case["fmt"], case["dim"]))
    return pool[table.long()].transpose(1, 2)


# ---- plain forms ----------------------------------------------------------------

def _plain_bounds(s):
    """The blocks that hold the last `tokens` tokens of every sequence."""
    case = s["case"]
    page, M = case["page"], case["tokens"]
    lens, width = s["lens"].long(), s["table"].shape[1]
    n = min(width, (M + page - 2) // page + 1)
    first = (lens - M).clamp(min=0) // page
    blk = first[:, None] + torch.arange(n, device=lens.device)
    there = blk * page < lens[:, None]                          # [B, n]
    pages = s["table"].long().gather(1, blk.clamp(max=width - 1))
    k = _values(_split(_records_of(s, pages), case["fmt"], case["dim"], True)[0])
    k = k.flatten(3, 4).to(torch.bfloat16)                      # [B, hkv, n, page, dim]
    pos = blk[..., None] * page + torch.arange(page, device=lens.device)
    out = (pos >= lens[:, None, None])[:, None, :, :, None]
    hi = k.masked_fill(out, -math.inf).amax(3)
    lo = k.masked_fill(out, math.inf).amin(3)
    s["bounds"][pages[there]] = torch.stack([hi, lo], 3).transpose(1, 2)[there]
    return s["bounds"]


def _plain_scores(s):
    case = s["case"]
    B, M, hkv, dim, page = (case[n] for n in ("seqs", "tokens", "hkv", "dim", "page"))
    G, lens = case["hq"] // hkv, s["lens"].long()
    both = s["bounds"][s["table"].long()].permute(0, 2, 3, 4, 1).float()   # [B, hkv, 2, dim, n]
    q = s["q"].float().view(B, M, hkv, G, dim).transpose(1, 2).flatten(2, 3)
    x = torch.matmul(q.clamp(min=0.0), both[:, :, 0]) + torch.matmul(q.clamp(max=0.0), both[:, :, 1])
    there = lens[:, None] - M + torch.arange(M, device=lens.device) >= 0
    x = x.masked_fill(~there.repeat_interleave(G, 1)[:, None, :, None], -math.inf).amax(2)
    block = torch.arange(x.shape[-1], device=lens.device)
    s["scores"].copy_(torch.where(block * page < lens[:, None, None], x, s["scores"]))
    return s["scores"]


def _choose(scores, items, first, last, count):
    """The first and the last ones of `items` [B] items, and of the others the
    largest, `count` in all; ascending, -1 past the end.  ([B, hkv, count], [B])"""
    n = scores.shape[-1]
    i = torch.arange(n, device=scores.device)
    total = items[:, None, None]
    x = scores.double().masked_fill((i < first) | (i >= total - last), math.inf)
    x = x.masked_fill(i >= total, -math.inf)
    # a place past the last item ranks behind any item, whatever that one's score
    order = torch.sort(x, stable=True, dim=-1, descending=True).indices[..., :count]
    counts = items.clamp(max=count)
    order = order.masked_fill(torch.arange(order.shape[-1], device=i.device) >= counts[:, None, None],
                              n).sort(-1).values
    index = torch.full((*scores.shape[:2], count), -1, device=i.device, dtype=torch.int32)
    index[..., :order.shape[-1]] = torch.where(order < n, order, -1).to(torch.int32)
    return index, counts.to(torch.int32)


def _plain_select(s):
    case = s["case"]
    items = (s["lens"].long() + case["unit"] - 1) // case["unit"]
    index, counts = _choose(s["scores"], items, case["first"], case["last"], case["count"])
    s["index"].copy_(torch.where(index >= 0, index, s["index"]))
    s["counts"].copy_(counts)
    return s["index"], s["counts"]


def _plain_sparse(s):
    case = s["case"]
    fmt, dim, hkv, page = case["fmt"], case["dim"], case["hkv"], case["page"]
    B, M, G = case["seqs"], case["tokens"], case["hq"] // case["hkv"]
    blocks = s["blocks"].long()                                 # [B, hkv, n]
    pages = s["table"].long()[:, None].expand(B, hkv, -1).gather(2, blocks.clamp(min=0))
    pool = s["pool"].view(-1, hkv, page // 16, _record_bytes(fmt, dim))
    rec = pool[pages, torch.arange(hkv, device=pages.device)[None, :, None]]
    k, v = (_values(x).flatten(2, 4) for x in _split(rec, fmt, dim))
    pos = (blocks[..., None] * page + torch.arange(page, device=pages.device)).flatten(2)
    listed_ = torch.arange(blocks.shape[2], device=pages.device) < s["counts"][:, None]
    pos = pos.masked_fill(~listed_.repeat_interleave(page, 1)[:, None], 1 << 40)
    q = s["q"].float().view(B, M, hkv, G, dim).transpose(1, 2).flatten(2, 3)
    score = torch.matmul(q, k.transpose(-1, -2)) * dim ** -0.5  # [B, hkv, M * G, keys]
    last = s["lens"].long()[:, None] - M + torch.arange(M, device=pages.device)
    seen = pos[:, :, None] <= last.repeat_interleave(G, 1)[:, None, :, None]
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    v = v.masked_fill((pos > 1 << 39)[..., None], 0.0)
    out = torch.matmul(p, v) / total.masked_fill(total == 0, 1.0)
    lse = top + torch.log(total)
    back = lambda x: x.view(B, hkv, M, G, -1).transpose(1, 2).reshape(B * M, hkv * G, -1)  # noqa: E731
    s["out"].copy_(back(out))
    s["lse"].copy_(back(lse).squeeze(-1))
    return s["out"], s["lse"]


def _all_scores(s):
    """Of every sequence with tokens: its number, the rows' new tokens, which keys
    they see, and the scores, [hkv, M * G, keys]."""
    case = s["case"]
    hkv, page, M, dim = case["hkv"], case["page"], case["tokens"], case["dim"]
    G = case["hq"] // hkv
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            s["lse"][b * M:b * M + M] = -math.inf
            continue
        rec = _records_of(s, s["table"][b:b + 1, :-(-n // page)])[0]
        k = _values(_split(rec, case["fmt"], dim, True)[0]).flatten(1, 3)[:, :n]
        q = s["q"][b * M:b * M + M].float().view(M, hkv, G, dim).transpose(0, 1).flatten(1, 2)
        last = n - M + torch.arange(M, device=q.device).repeat_interleave(G)[:, None]
        key = torch.arange(n, device=q.device)
        seen = key <= last
        if case["window"]:
            seen &= key > last - case["window"]
        yield b, last, seen, torch.matmul(q, k.transpose(-1, -2)) * dim ** -0.5


def _plain_weights(s):
    case = s["case"]
    hkv, page, B, M, dim = case["hkv"], case["page"], case["seqs"], case["tokens"], case["dim"]
    G, lens = case["hq"] // hkv, s["lens"].long()
    k = _values(_split(_records_of(s, s["table"]), case["fmt"], dim, True)[0]).flatten(2, 4)
    rows = lambda x: x.view(B, M, hkv, G, -1).transpose(1, 2).flatten(2, 3)  # noqa: E731
    score = torch.matmul(rows(s["q"].float()), k.transpose(-1, -2)) * dim ** -0.5
    last = (lens[:, None] - M + torch.arange(M, device=lens.device)).repeat_interleave(G, 1)
    key = torch.arange(score.shape[-1], device=lens.device)
    seen = key <= last[..., None]
    if case["window"]:
        seen &= key > last[..., None] - case["window"]
    lse = rows(s["lse"])
    x = (score - lse.masked_fill(lse == -math.inf, 0.0)).masked_fill(~seen[:, None], -math.inf)
    got = torch.exp(x).sum(2)[..., :case["longest"]]
    key = key[:case["longest"]]
    old = (key < lens[:, None, None] - M)
    new = torch.where(old, DECAY * s["before"], 0.0) + got
    s["after"].copy_(torch.where(key < lens[:, None, None], new, s["after"]))
    return s["after"]


def _plain_gather(s):
    """The kept tokens' codes, scales and zeros in new records, and what these hold."""
    case = s["case"]
    fmt, dim, hkv, page, B, n = (case[x] for x in ("fmt", "dim", "hkv", "page", "seqs", "count"))
    index = s["index"].long().clamp(min=0)
    there = torch.arange(n, device=index.device) < s["counts"][:, None]        # [B, n]
    old = _split(_records_of(s, s["table"]), fmt, dim)
    new = _split(_records_of(s, s["to"]), fmt, dim)
    out = []
    for (q0, m0), (q1, m1) in zip(old, new):
        pair = []
        for a, b in ((q0, q1), (m0, m1)):
            if a is None:
                pair.append(None)
                continue
            a, shape = a.flatten(2, 4), b.shape
            b = b.flatten(2, 4).clone()
            moved = a.gather(2, index[..., None].expand(*index.shape, a.shape[-1]))
            b[:, :, :n] = torch.where(there[:, None, :, None], moved, b[:, :, :n])
            pair.append(b.view(shape))
        out.append(tuple(pair))
    rec = _join(*out, fmt)                                      # [B, hkv, pages, page // 16, bytes]
    pool = s["pool"].view(-1, hkv, page // 16, rec.shape[-1])
    pool[s["to"].long()] = rec.transpose(1, 2)
    w = s["weights"].gather(2, index)
    s["weights_out"].copy_(torch.where(there[:, None], w, s["weights_out"]))
    for name, held in (("k_out", out[0]), ("v_out", out[1])):
        x = _values(held).flatten(2, 4)[:, :, :n].transpose(1, 2).reshape(B * n, hkv, dim)
        s[name].copy_(torch.where(there.reshape(-1, 1, 1), x.to(torch.bfloat16), s[name]))
    return s["k_out"], s["v_out"], s["weights_out"]


PLAIN = dict(bounds=_plain_bounds, scores=_plain_scores, select=_plain_select,
             sparse=_plain_sparse, weights=_plain_weights, gather=_plain_gather)


# ---- the library's calls ----------------------------------------------------------

def _cache(s):
    """What a program keeps beside its tensors: the cache."""
    from int4_weight_only_w4_gb300 import w4
    case = s["case"]
    fmt = {"bf16": w4.KV_BF16, "int8": w4.KV_INT8, "int4": w4.KV_INT4}[case.get("fmt", "int4")]
    return w4.PagedCache(s["pool"], fmt, case["hkv"], case["dim"], case["page"])


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return PLAIN[op](s)
    if op == "select":
        from int4_weight_only_w4_gb300 import w4
        w4.select(s["scores"], s["lens"], s["index"], s["counts"], unit=case["unit"],
                  first=case["first"], last=case["last"])
        return s["index"], s["counts"]
    cache = s.get("cache")
    if cache is None:
        cache = s["cache"] = _cache(s)
    if op == "bounds":
        return cache.key_bounds(s["bounds"], s["lens"], s["table"], tokens=case["tokens"])
    if op == "scores":
        return cache.block_scores(s["bounds"], s["q"], s["lens"], s["table"], scores=s["scores"])
    if op == "sparse":
        return cache.attend_blocks(s["q"], s["lens"], s["table"], s["blocks"], s["counts"],
                                   out=s["out"], lse=s["lse"])
    if op == "weights":
        return cache.attn_weights(s["q"], s["lse"], s["lens"], s["table"], window=case["window"],
                                  before=s["before"], decay=DECAY, weights=s["after"])
    cache.gather(s["table"], s["lens"], s["index"], s["counts"], s["to"], weights=s["weights"],
                 weights_out=s["weights_out"])
    k, v = cache.read(s["positions"], s["to"], k=s["k_out"], v=s["v_out"])
    return k, v, s["weights_out"]


# ---- what a pass cannot do without ------------------------------------------------

def _mean(case, most=None):
    """Mean of min(length, most) over the sequences of a case."""
    B, top = case["seqs"], case["longest"]
    w = min(most or top, top)
    if not case["ragged"]:
        return w
    mean = w - w * w / (2 * top)                                # lengths are uniform
    return (mean * (B - 2) + w) / B if B > 3 else mean


def work(case):
    op, B, H = case["op"], case["seqs"], case["hkv"]
    if op == "select":
        n = _mean(case) / case["unit"]
        return dict(bytes=4 * B * (H * (n + min(n, case["count"])) + 2), flops=B * H * n)
    dim, page = case["dim"], case["page"]
    if op == "scores":
        n, rows = B * H * _mean(case) / page, case["tokens"] * case["hq"] // H
        return dict(bytes=n * (4 * dim + 4) + 2 * B * case["tokens"] * case["hq"] * dim,
                    flops=4 * n * dim * rows)
    per_token = _record_bytes(case["fmt"], dim) / 16 * H
    if op == "bounds":
        # the blocks that hold the new tokens; half of the last one, on average
        n = min(_mean(case), case["tokens"] - 1 + page / 2)
        return dict(bytes=B * (n * per_token / 2 + max(1, n / page) * 4 * H * dim),
                    flops=2 * B * n * H * dim)
    if op == "gather":
        n = B * _mean(case, case["count"])
        # a token of the records in and out, and in again to be read; index, weights; k, v out
        return dict(bytes=n * (3 * per_token + 12 * H + 4 * H * dim), flops=2 * n * H * dim)
    rows = B * case["tokens"] * case["hq"]
    if op == "sparse":
        keys = B * _mean(case, case["count"] * page)
        return dict(bytes=keys * per_token + 4 * rows * (dim + 1),
                    flops=4 * keys * case["tokens"] * case["hq"] * dim)
    seen = B * (_mean(case, case["window"] + case["tokens"]) if case["window"] else _mean(case))
    return dict(bytes=seen * per_token / 2 + 8 * B * _mean(case) * H + 2 * rows * (dim + 2),
                flops=2 * seen * case["tokens"] * case["hq"] * dim)


# ---- 64 bits ------------------------------------------------------------------------

def _code_bytes(fmt, dim, token, which):
    """(byte in the record, shift) of every code of key (0) or value (1) of the tokens."""
    r, d = token[:, None], torch.arange(dim, device=token.device)
    half = 16 * dim * BITS[fmt] // 8
    none = torch.zeros_like(r + d)
    if fmt == "bf16":
        return which * half + r * 2 * dim + (((d // 8) ^ (r % 8)) * 16) + d % 8 * 2, none
    if which == 0 and fmt == "int8":
        return r * dim + (((d // 16) ^ (4 * (r % 2) if dim == 128 else 0)) * 16) + d % 16, none
    if which == 0:
        return r * (dim // 2) + d // 2, none + 4 * (d % 2)
    lane, byte = 4 * (d % 8) + (r % 8) // 2, 2 * (r % 2) + r // 8
    if fmt == "int8":
        return half + d // 32 * 512 + lane * 16 + d // 8 % 4 * 4 + byte, none
    return half + d // 64 * 512 + lane * 16 + d // 16 % 4 * 4 + byte, none + 4 * (d // 8 % 2)


def _held(s, b, h, j, which):
    """fp64 keys (0) or values (1) [n, dim] of tokens j of sequence b and head h."""
    case = s["case"]
    fmt, dim, page = case["fmt"], case["dim"], case["page"]
    pool, nb = s["pool"], _record_bytes(fmt, dim)
    record = (s["table"][b].long()[j // page] * case["hkv"] + h) * (page // 16) + j % page // 16
    base = record[:, None] * nb
    at, shift = _code_bytes(fmt, dim, j % 16, which)
    u16 = lambda a: pool[a].long() | (pool[a + 1].long() << 8)  # noqa: E731
    if fmt == "bf16":
        return (u16(base + at) << 16).to(torch.int32).view(torch.float32).double()
    code = (pool[base + at].long() >> shift) & ((1 << BITS[fmt]) - 1)
    m = base + nb - 128 + 64 * which + 4 * (j % 16)[:, None]
    scale = u16(m).to(torch.int16).view(torch.float16).double()
    return (code - u16(m + 2)).double() * scale


def _rows(s, b, h):
    """Queries of sequence b's rows of head h in 64 bits, and their new tokens."""
    case = s["case"]
    M, G = case["tokens"], case["hq"] // case["hkv"]
    q = s["q"][b * M:(b + 1) * M, h * G:(h + 1) * G].double().flatten(0, 1)
    return q, torch.arange(M, device=q.device).repeat_interleave(G)


def exact(case, seed):
    s = prepare(case, seed)
    op, B, hkv, lens = case["op"], case["seqs"], case["hkv"], s["lens"].tolist()
    if op == "select":
        index, counts = s["index"].tolist(), []
        scores = s["scores"].cpu().numpy()
        for b, n in enumerate(lens):
            n = -(-n // case["unit"])
            counts.append(min(n, case["count"]))
            for h in range(hkv):
                always = set(range(min(case["first"], n))) | set(range(max(0, n - case["last"]), n))
                rank = (-scores[b, h, :n]).argsort(kind="stable").tolist()
                rest = [i for i in rank if i not in always]
                kept = sorted(list(always) + rest[:max(0, case["count"] - len(always))]) \
                    if n > case["count"] else list(range(n))
                index[b][h][:len(kept)] = kept
        return (torch.tensor(index, dtype=torch.int32, device=DEV),
                torch.tensor(counts, dtype=torch.int32, device=DEV))
    dim, page = case["dim"], case["page"]
    if op == "bounds":
        out = s["bounds"].double()
        for b, n in enumerate(lens):
            for i in range(max(0, n - case["tokens"]) // page, -(-n // page)):
                j = torch.arange(i * page, min(n, i * page + page), device=DEV)
                for h in range(hkv):
                    k = _held(s, b, h, j, 0).to(torch.bfloat16).double()
                    out[int(s["table"][b, i]), h, 0] = k.max(0).values
                    out[int(s["table"][b, i]), h, 1] = k.min(0).values
        return out
    if op == "scores":
        out = s["scores"].double()
        for b, n in enumerate(lens):
            blocks = -(-n // page)
            pages = s["table"][b, :blocks].long()
            for h in range(hkv):
                q, i = _rows(s, b, h)
                q = q[n - case["tokens"] + i >= 0]
                if not blocks:
                    continue
                both = s["bounds"][pages, h].double()            # [blocks, 2, dim]
                for r in range(0, blocks, 256):
                    part = both[r:r + 256, None]
                    x = torch.where(q >= 0, q * part[:, :, 0], q * part[:, :, 1]).sum(-1)
                    out[b, h, r:min(blocks, r + 256)] = x.max(-1).values
        return out
    if op == "gather":
        n = case["count"]
        k, v = (torch.zeros(B, n, hkv, dim, dtype=torch.float64, device=DEV) for _ in "kv")
        w = torch.zeros(B, hkv, n, dtype=torch.float64, device=DEV)
        for b, c in enumerate(s["counts"].tolist()):
            for h in range(hkv):
                j = s["index"][b, h, :c].long()
                k[b, :c, h], v[b, :c, h] = _held(s, b, h, j, 0), _held(s, b, h, j, 1)
                w[b, h, :c] = s["weights"][b, h, j].double()
        return k.view(B * n, hkv, dim), v.view(B * n, hkv, dim), w
    M, G = case["tokens"], case["hq"] // hkv
    if op == "weights":
        out = s["after"].double()
        lse = s["lse"].double().view(B, M, hkv, G)
        for b, n in enumerate(lens):
            if n == 0:
                continue
            j = torch.arange(n, device=DEV)
            for h in range(hkv):
                q, i = _rows(s, b, h)
                x = q @ _held(s, b, h, j, 0).T / math.sqrt(dim)
                p = n - M + i[:, None]
                seen = (j <= p) & (j > p - case["window"]) if case["window"] else j <= p
                x = (x - lse[b, :, h].reshape(-1, 1)).masked_fill(~seen, -math.inf)
                out[b, h, :n] = torch.exp(x).sum(0)
                out[b, h, :max(0, n - M)] += DECAY * s["before"][b, h, :max(0, n - M)].double()
        return out
    out = torch.zeros(B, M, case["hq"], dim, dtype=torch.float64, device=DEV)
    lse = torch.full((B, M, case["hq"]), -math.inf, dtype=torch.float64, device=DEV)
    for b, c in enumerate(s["counts"].tolist()):
        for h in range(hkv):
            blocks = s["blocks"][b, h, :c].long()
            j = (blocks[:, None] * page + torch.arange(page, device=DEV)).flatten()
            j = j[j < lens[b]]
            if not len(j):
                continue
            q, i = _rows(s, b, h)
            x = q @ _held(s, b, h, j, 0).T / math.sqrt(dim)
            x = x.masked_fill(j > (lens[b] - M + i)[:, None], -math.inf)
            total = torch.logsumexp(x, -1)
            p = torch.exp(x - total.masked_fill(total == -math.inf, 0.0)[:, None])
            out[b, :, h * G:(h + 1) * G] = (p @ _held(s, b, h, j, 1)).view(M, G, dim)
            lse[b, :, h * G:(h + 1) * G] = total.view(M, G)
    return out.view(B * M, case["hq"], dim), lse.view(B * M, case["hq"])
