"""The operators between the qkv and the o product of a decoder layer, as
cases to be measured: rotary positions, a paged key-value cache that is
quantised as it is written and read back, and the attention of new tokens over
that cache.

``run`` computes a case in its plain form (elementary torch operations in
fp32) or, where ``own`` is true, with this library's calls.  Both work on the
same state: the cache is held in the library's documented record layout
(include/w4.h, "Paged key-value cache"), which the plain form packs and unpacks
with reshapes.

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


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # The 8 token rows of a speculative-verify batch: q and k of the fused
        # qkv row rotated in one call; latency only.
        dict(name="rope.verify8", op="rope", tokens=8, heads=32, dim=128, rot=128,
             layout="half", base=1e6, factor=1.0, start=4000),
        # A prompt chunk far into a long context: half of each head rotated,
        # neighbouring pairs, frequencies stretched by parts.
        dict(name="rope.prompt", op="rope", tokens=8192, heads=32, dim=128, rot=64,
             layout="interleaved", base=1e4, factor=4.0, start=100001),
        # One decode step of 64 requests, written in 4 bits.
        dict(name="kv.decode64.int4", op="kv", fmt="int4", seqs=64, tokens=1, hq=28, hkv=4,
             dim=128, page=16, start=3000, layout="half"),
        # A prompt of 4096 tokens written in 8 bits.
        dict(name="kv.prompt4096.int8", op="kv", fmt="int8", seqs=1, tokens=4096, hq=28, hkv=4,
             dim=128, page=64, start=0, layout="half"),
        # Chunks of five prompts, starting inside a page, kept in bf16.
        dict(name="kv.chunks.bf16", op="kv", fmt="bf16", seqs=5, tokens=333, hq=14, hkv=2,
             dim=64, page=32, start=1001, layout="interleaved"),
        # A long prompt written in 4 bits.
        dict(name="kv.prompt16k.int4", op="kv", fmt="int4", seqs=1, tokens=16384, hq=28, hkv=4,
             dim=128, page=16, start=0, layout="half"),
        # Decode at a short context of the small shape: latency only.
        dict(name="attn.short.bf16", op="attn", fmt="bf16", seqs=1, tokens=1, hq=14, hkv=2,
             dim=64, page=16, longest=201, ragged=False, window=0),
        # A single request at 64 k tokens: the length has to be split.
        dict(name="attn.single64k.bf16", op="attn", fmt="bf16", seqs=1, tokens=1, hq=28, hkv=4,
             dim=128, page=16, longest=65536, ragged=False, window=0),
        # 64 requests of very different lengths, some empty.
        dict(name="attn.batch64.int8", op="attn", fmt="int8", seqs=64, tokens=1, hq=28, hkv=4,
             dim=128, page=64, longest=8192, ragged=True, window=0),
        # Four requests at 128 k tokens in 4 bits.
        dict(name="attn.long4.int4", op="attn", fmt="int4", seqs=4, tokens=1, hq=28, hkv=4,
             dim=128, page=16, longest=131072, ragged=False, window=0),
        # Speculative verification: 8 new tokens a request.
        dict(name="attn.verify8.bf16", op="attn", fmt="bf16", seqs=8, tokens=8, hq=28, hkv=4,
             dim=128, page=16, longest=8192, ragged=True, window=0),
        # A sliding window over 4-bit caches, 3 draft tokens, small shape.
        dict(name="attn.window.int4", op="attn", fmt="int4", seqs=48, tokens=3, hq=14, hkv=2,
             dim=64, page=32, longest=20000, ragged=True, window=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "kv", "attn", "attn"])
    dim, hkv, ratio = rng.choice([(128, 4, 7), (128, 4, 7), (64, 2, 7), (128, 8, 4), (64, 8, 1),
                                  (128, 2, 8), (64, 3, 5)])
    if op == "rope":
        return dict(op="rope", tokens=_log(rng, 1, 8000), heads=hkv * (ratio + 1), dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, dim // 4]),
                    layout=rng.choice(["half", "interleaved"]),
                    base=rng.choice([1e4, 5e5, 1e6]), factor=rng.choice([1.0, 2.0, 4.0, 8.0]),
                    start=rng.randrange(0, 120000))
    fmt = rng.choice(["bf16", "int8", "int4"])
    page = rng.choice([16, 16, 32, 64, 128])
    if op == "kv":
        seqs = _log(rng, 1, 64)
        return dict(op="kv", fmt=fmt, seqs=seqs, tokens=_log(rng, 1, 9000 // seqs), hq=hkv * ratio,
                    hkv=hkv, dim=dim, page=page, start=rng.randrange(0, 4000),
                    layout=rng.choice(["half", "interleaved"]))
    seqs, tokens = _log(rng, 1, 96), rng.choice([1, 1, 1, 2, 3, 5, 8])
    # as many keys as the largest listed case may cost, by bytes and by products
    cost = max(_record_bytes(fmt, dim) / 16 * hkv, 4 * tokens * hkv * ratio * dim / 50)
    most = min(131072, int(2.8e8 / cost) // seqs)
    return dict(op="attn", fmt=fmt, seqs=seqs, tokens=tokens, hq=hkv * ratio, hkv=hkv, dim=dim,
                page=page, longest=_log(rng, 30, most), ragged=rng.random() < 0.6,
                window=rng.choice([0, 0, 0, 1000]))


# ---- inputs ------------------------------------------------------------------

def _frequencies(rot, base, factor):
    """Angles per position of the rot/2 pairs (fp64, on the host): f = base^(-2i/rot),
    stretched by `factor` where fewer than one turn fits 4096 positions, kept
    where more than 32 do, and mixed linearly in the number of turns between."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    turns = 4096.0 * f / (2 * math.pi)
    keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    return f * (keep + (1.0 - keep) / factor)


def _rope_table(rot, base, factor, rows):
    """(cos, sin) of every position and pair, fp32 [rows, rot/2, 2]."""
    f = _frequencies(rot, base, factor).to(DEV)
    angle = torch.arange(rows, dtype=torch.float64, device=DEV)[:, None] * f
    amplitude = 1.0 if factor == 1.0 else 0.1 * math.log(factor) + 1.0
    return torch.stack([angle.cos() * amplitude, angle.sin() * amplitude], -1).float()


def _record_bytes(fmt, dim):
    return 64 * dim if fmt == "bf16" else 16 * dim * 2 * BITS[fmt] // 8 + 128


def _normal(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _channels(gen, heads, dim):
    """Some channels of keys carry larger values than the rest."""
    wide = torch.rand(heads, dim, generator=gen, device=DEV) < 1 / 16
    return torch.where(wide, 4.0, 1.0)


def _block_table(gen, seqs, pages_each):
    """Every sequence's pages, in a random order of the pool's."""
    order = torch.randperm(seqs * pages_each, generator=gen, device=DEV)
    return order.view(seqs, pages_each).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, dim = case["op"], case["dim"]
    if op == "rope":
        T, H = case["tokens"], case["heads"]
        v_heads = 4
        rows = _normal(gen, T, (H + v_heads) * dim)             # the fused qkv product's output
        return dict(case=case, x=rows.view(T, H + v_heads, dim)[:, :H],
                    positions=torch.arange(case["start"], case["start"] + T, device=DEV,
                                           dtype=torch.int32),
                    rope=_rope_table(case["rot"], case["base"], case["factor"],
                                     case["start"] + T),
                    out=torch.empty(T, H, dim, device=DEV, dtype=torch.bfloat16))
    hq, hkv, page, fmt = case["hq"], case["hkv"], case["page"], case["fmt"]
    rec = _record_bytes(fmt, dim)
    if op == "kv":
        B, M, start = case["seqs"], case["tokens"], case["start"]
        T, pages_each = B * M, -(-(start + M + 7 * B) // page)
        rows = _normal(gen, T, hq + 2 * hkv, dim, dtype=torch.float32)
        rows[:, hq:hq + hkv] *= _channels(gen, hkv, dim)
        rows = rows.to(torch.bfloat16)
        first = start + 7 * torch.arange(B, device=DEV)         # each sequence at its own length
        positions = (first[:, None] + torch.arange(M, device=DEV)).reshape(-1).to(torch.int32)
        buf = lambda h: torch.empty(T, h, dim, device=DEV, dtype=torch.bfloat16)  # noqa: E731
        return dict(case=case, q=rows[:, :hq], k=rows[:, hq:hq + hkv], v=rows[:, hq + hkv:],
                    positions=positions,
                    rope=_rope_table(dim, 1e6, 1.0, start + M + 7 * B),
                    table=_block_table(gen, B, pages_each),
                    pool=torch.zeros(B * pages_each * hkv * (page // 16) * rec, device=DEV,
                                     dtype=torch.uint8),
                    q_out=buf(hq), k_out=buf(hkv), v_out=buf(hkv))
    B, M, longest = case["seqs"], case["tokens"], case["longest"]
    pages_each = -(-longest // page)
    lens = torch.full((B,), longest, device=DEV, dtype=torch.int32)
    if case["ragged"]:
        lens = torch.randint(0, longest + 1, (B,), generator=gen, device=DEV, dtype=torch.int32)
        lens[B // 2] = longest
        if B > 3:
            lens[0] = 0                                         # a slot without a request
    pool = torch.empty(B * pages_each, hkv, page // 16, rec, device=DEV, dtype=torch.uint8)
    chan = _channels(gen, hkv, dim)[:, None, None]
    step = max(1, (1 << 27) // (hkv * page * dim))
    for p in range(0, B * pages_each, step):                    # a part of the pool at a time
        n = min(step, B * pages_each - p)
        k = _normal(gen, n, hkv, page // 16, 16, dim, dtype=torch.float32) * chan
        v = _normal(gen, n, hkv, page // 16, 16, dim, dtype=torch.float32)
        pool[p:p + n] = _pack(k.to(torch.bfloat16).float(), v.to(torch.bfloat16).float(), fmt)
    return dict(case=case, q=_normal(gen, B * M, hq, dim), lens=lens, pool=pool.view(-1),
                table=_block_table(gen, B, pages_each),
                out=torch.empty(B * M, hq, dim, device=DEV, dtype=torch.bfloat16),
                lse=torch.empty(B * M, hq, device=DEV))


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
    return q.to(torch.uint8), s16.squeeze(-1), z.squeeze(-1)


def _meta(s16, z):
    both = torch.stack([s16.view(torch.int16), z.to(torch.int16)], -1)
    return both.contiguous().view(torch.uint8).flatten(-2)


def _pack(k, v, fmt):
    """fp32 [..., 16, dim] keys and values -> records [..., bytes]."""
    lead, dim = k.shape[:-2], k.shape[-1]
    if fmt == "bf16":
        parts = [_swap_pieces(x.to(torch.bfloat16).view(torch.uint8), fmt, dim).flatten(-2)
                 for x in (k, v)]
        return torch.cat(parts, -1)
    kq, ks, kz = _quantise(k, fmt)
    vq, vs, vz = _quantise(v, fmt)
    if fmt == "int8":
        kb = _swap_pieces(kq, fmt, dim).flatten(-2)
        w = vq.view(*lead, 2, 4, 2, dim // 32, 4, 8)             # h, t, r, i, e, g
        vb = w.permute(*range(len(lead)), *(len(lead) + a for a in (3, 5, 1, 4, 2, 0)))
    else:
        kb = (kq[..., 0::2] | (kq[..., 1::2] << 4)).flatten(-2)
        w = vq.view(*lead, 2, 4, 2, dim // 64, 4, 2, 8)          # h, t, r, i, e, high, g
        w = w[..., 0, :] | (w[..., 1, :] << 4)
        vb = w.permute(*range(len(lead)), *(len(lead) + a for a in (3, 5, 1, 4, 2, 0)))
    return torch.cat([kb, vb.reshape(*lead, -1), _meta(ks, kz), _meta(vs, vz)], -1)


def _unpack(rec, fmt, dim):
    """Records [..., bytes] -> fp32 keys and values [..., 16, dim]."""
    lead = rec.shape[:-1]
    size = 16 * dim * BITS[fmt] // 8
    kb, vb = rec[..., :size], rec[..., size:2 * size]
    if fmt == "bf16":
        k, v = (_swap_pieces(x.reshape(*lead, 16, 2 * dim), fmt, dim).view(torch.bfloat16).float()
                for x in (kb, vb))
        return k, v
    meta = rec[..., 2 * size:].contiguous().view(torch.int16).view(*lead, 2, 16, 2)
    s, z = meta[..., 0].contiguous().view(torch.float16).float(), meta[..., 1].float()
    if fmt == "int8":
        kq = _swap_pieces(kb.reshape(*lead, 16, dim), fmt, dim)
        vq = vb.reshape(*lead, dim // 32, 8, 4, 4, 2, 2)         # i, g, t, e, r, h
        order = (5, 2, 4, 0, 3, 1)
    else:
        kq = torch.stack([kb & 15, kb >> 4], -1).reshape(*lead, 16, dim)
        vq = vb.reshape(*lead, dim // 64, 8, 4, 4, 2, 2)
        vq = torch.stack([vq & 15, vq >> 4], -1)                 # i, g, t, e, r, h, high
        order = (5, 2, 4, 0, 3, 6, 1)
    vq = vq.permute(*range(len(lead)), *(len(lead) + a for a in order)).reshape(*lead, 16, dim)
    k = (kq.float() - z[..., 0, :, None]) * s[..., 0, :, None]
    v = (vq.float() - z[..., 1, :, None]) * s[..., 1, :, None]
    return k, v


# ---- plain forms ----------------------------------------------------------------

def _plain_rope(x, positions, table, layout):
    """fp32 rotation of the first 2 * table.shape[1] values of every head."""
    n = table.shape[1]
    cs = table[positions.long()][:, None]
    c, s = cs[..., 0], cs[..., 1]
    x = x.float()
    if layout == "half":
        a, b = x[..., :n], x[..., n:2 * n]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([y, x[..., 2 * n:]], -1)


def _plain_kv(s):
    """The new tokens packed into their records, and read back out of them.
    Tokens of a record that are not written keep what they hold."""
    case = s["case"]
    fmt, dim, hkv, page, B = case["fmt"], case["dim"], case["hkv"], case["page"], case["seqs"]
    q = _plain_rope(s["q"], s["positions"], s["rope"], case["layout"])
    k = _plain_rope(s["k"], s["positions"], s["rope"], case["layout"])
    T, M = k.shape[0], case["tokens"]
    pos = s["positions"].long()
    seq = torch.arange(B, device=pos.device).repeat_interleave(M)
    # the runs of 16-token records that the tokens of each sequence touch
    pool = s["pool"].view(-1, hkv, page // 16, _record_bytes(fmt, dim))
    first = pos.view(B, M)[:, 0] // 16
    n = (M + 14) // 16 + 1
    blk = (first[:, None] + torch.arange(n, device=pos.device)).clamp(
        max=s["table"].shape[1] * (page // 16) - 1)
    pg = s["table"].long().gather(1, blk // (page // 16))
    rec = pool[pg, :, blk % (page // 16)]                       # [B, n, hkv, bytes]
    kk, vv = _unpack(rec, fmt, dim)                             # [B, n, hkv, 16, dim]
    at = pos // 16 - first[seq]
    kk[seq, at, :, pos % 16] = k
    vv[seq, at, :, pos % 16] = s["v"].float()
    new = torch.zeros(*kk.shape[:2], 16, dtype=torch.bool, device=pos.device)
    new[seq, at, pos % 16] = True
    packed = _pack(kk, vv, fmt)
    kk, vv = _unpack(packed, fmt, dim)
    touched = new.any(-1)
    pool[pg[touched], :, (blk % (page // 16))[touched]] = packed[touched]
    s["q_out"].copy_(q)
    s["k_out"].copy_(kk[seq, at, :, pos % 16])
    s["v_out"].copy_(vv[seq, at, :, pos % 16])
    return s["q_out"], s["k_out"], s["v_out"]


def _plain_attn(s):
    case = s["case"]
    fmt, dim, hkv, page = case["fmt"], case["dim"], case["hkv"], case["page"]
    B, M, R = case["seqs"], case["tokens"], case["hq"] // case["hkv"]
    pool = s["pool"].view(-1, hkv, page // 16, _record_bytes(fmt, dim))
    rec = pool[s["table"].long()].permute(0, 2, 1, 3, 4).flatten(2, 3)
    k, v = _unpack(rec, fmt, dim)                               # [B, hkv, records, 16, dim]
    k, v = k.flatten(2, 3), v.flatten(2, 3)
    q = s["q"].float().view(B, M, hkv, R, dim).transpose(1, 2).flatten(2, 3)
    score = torch.matmul(q, k.transpose(-1, -2)) * dim ** -0.5  # [B, hkv, M * R, keys]
    key = torch.arange(k.shape[2], device=q.device)
    last = s["lens"].long()[:, None] - M + torch.arange(M, device=q.device)
    seen = key <= last[..., None]
    if case["window"]:
        seen &= key > last[..., None] - case["window"]
    seen = seen.repeat_interleave(R, 1)[:, None]                # [B, 1, M * R, keys]
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / total.masked_fill(total == 0, 1.0)
    lse = top + torch.log(total)
    back = lambda x: x.view(B, hkv, M, R, -1).transpose(1, 2).reshape(B * M, hkv * R, -1)  # noqa: E731
    s["out"].copy_(back(out))
    s["lse"].copy_(back(lse).squeeze(-1))
    return s["out"], s["lse"]


# ---- the library's calls ----------------------------------------------------------

def _handle(s):
    """What a program keeps beside its tensors: the cache and the rotation."""
    from int4_weight_only_w4_gb300 import w4
    case = s["case"]
    layout = {"half": w4.ROPE_HALF, "interleaved": w4.ROPE_INTERLEAVED}
    h = {}
    if "rope" in s:
        h["rope"] = w4.RopeTable(s["rope"], layout[case["layout"]])
    if "pool" in s:
        fmt = {"bf16": w4.KV_BF16, "int8": w4.KV_INT8, "int4": w4.KV_INT4}[case["fmt"]]
        h["cache"] = w4.PagedCache(s["pool"], fmt, case["hkv"], case["dim"], case["page"])
    return h


def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "rope":
            s["out"].copy_(_plain_rope(s["x"], s["positions"], s["rope"], s["case"]["layout"]))
            return s["out"]
        return _plain_kv(s) if op == "kv" else _plain_attn(s)
    h = s.get("handle")
    if h is None:
        h = s["handle"] = _handle(s)
    if op == "rope":
        return h["rope"].apply(s["x"], s["positions"], out=s["out"])
    if op == "kv":
        h["cache"].append(s["k"], s["v"], s["positions"], s["table"], q=s["q"], q_out=s["q_out"],
                          rope=h["rope"])
        k, v = h["cache"].read(s["positions"], s["table"], k=s["k_out"], v=s["v_out"])
        return s["q_out"], k, v
    return h["cache"].attend(s["q"], s["lens"], s["table"], window=s["case"]["window"],
                             out=s["out"], lse=s["lse"])


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    op, dim = case["op"], case["dim"]
    if op == "rope":
        n = case["tokens"] * case["heads"] * dim
        return dict(bytes=4 * n + case["tokens"] * (4 * case["rot"] + 4), flops=3 * n)
    per_token = _record_bytes(case["fmt"], dim) / 16 * case["hkv"]
    if op == "kv":
        T, row = case["seqs"] * case["tokens"], 2 * dim
        # q, k, v and a table row in; q out; the records out, and in again; k, v out
        heads_in, heads_out = case["hq"] + 2 * case["hkv"], case["hq"] + 2 * case["hkv"]
        return dict(bytes=T * (row * (heads_in + heads_out) + 2 * per_token + 4 * dim),
                    flops=3 * T * dim * heads_in)
    B, M = case["seqs"], case["tokens"]
    mean = case["longest"] * (0.5 if case["ragged"] else 1.0)
    if case["window"]:
        # lengths are uniform up to the longest: the mean of min(length, window)
        w, top = min(case["window"], case["longest"]), case["longest"]
        mean = w - w * w / (2 * top) if case["ragged"] else w
    if case["ragged"] and B > 3 and not case["window"]:
        # one sequence is empty and one has the full length
        mean = (mean * (B - 2) + case["longest"]) / B
    keys = B * mean
    return dict(bytes=keys * per_token + 4 * B * M * case["hq"] * (dim + 1),
                flops=4 * keys * M * case["hq"] * dim)


# ---- 64 bits ------------------------------------------------------------------------

def _exact_turn(x, positions, table, layout):
    x = x.double().clone()
    n = table.shape[1]
    i = torch.arange(n, device=x.device)
    a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
    z = torch.view_as_complex(torch.stack([x[..., a], x[..., b]], -1))
    z = z * torch.view_as_complex(table.double())[positions.long()][:, None]
    x[..., a], x[..., b] = z.real, z.imag
    return x


def _exact_round_trip(x, bits):
    """Values that `bits`-bit codes of the rows of x stand for."""
    if bits == 16:
        return x.to(torch.bfloat16).double()
    top = 2.0 ** bits - 1
    lo, hi = x.min(-1, True).values.clamp_max(0), x.max(-1, True).values.clamp_min(0)
    s = ((hi - lo) / top).half().double()
    z = (-lo / s).round().clamp(0, top)
    return ((x / s).round() + z).clamp(0, top).sub(z) * s


def _exact_values(pool, record, token, fmt, dim):
    """fp64 keys and values [n, dim] of the given tokens of the given records
    (record, token: [n]), byte by byte from the layout's formulas."""
    nb = _record_bytes(fmt, dim)
    r, d = token[:, None], torch.arange(dim, device=pool.device)
    base = record[:, None] * nb
    u16 = lambda at: pool[at].long() | (pool[at + 1].long() << 8)  # noqa: E731
    if fmt == "bf16":
        at = r * 2 * dim + (((d // 8) ^ (r % 8)) * 16) + d % 8 * 2
        val = lambda a: (u16(a) << 16).to(torch.int32).view(torch.float32).double()  # noqa: E731
        return val(base + at), val(base + 32 * dim + at)
    half = 16 * dim * BITS[fmt] // 8
    out = []
    for which in (0, 1):
        if which == 0 and fmt == "int8":
            at = r * dim + (((d // 16) ^ (4 * (r % 2) if dim == 128 else 0)) * 16) + d % 16
            code = pool[base + at].double()
        elif which == 0:
            code = ((pool[base + r * (dim // 2) + d // 2] >> (4 * (d % 2)).to(torch.uint8)) & 15).double()
        else:
            lane = 4 * (d % 8) + (r % 8) // 2
            byte = 2 * (r % 2) + r // 8
            if fmt == "int8":
                code = pool[base + half + d // 32 * 512 + lane * 16 + d // 8 % 4 * 4 + byte].double()
            else:
                raw = pool[base + half + d // 64 * 512 + lane * 16 + d // 16 % 4 * 4 + byte]
                code = ((raw >> (4 * (d // 8 % 2)).to(torch.uint8)) & 15).double()
        m = base + 2 * half + 64 * which + 4 * r
        s = u16(m).to(torch.int16).view(torch.float16).double()
        out.append((code - u16(m + 2).double()) * s)
    return out[0], out[1]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_turn(s["x"], s["positions"], s["rope"], case["layout"])
    if case["op"] == "kv":
        bits = BITS[case["fmt"]]
        q, k = (_exact_turn(s[n], s["positions"], s["rope"], case["layout"]) for n in "qk")
        return q, _exact_round_trip(k, bits), _exact_round_trip(s["v"].double(), bits)
    B, M, hq, hkv, dim, page = (case[n] for n in ("seqs", "tokens", "hq", "hkv", "dim", "page"))
    out = torch.zeros(B, M, hq, dim, dtype=torch.float64, device=DEV)
    lse = torch.full((B, M, hq), -math.inf, dtype=torch.float64, device=DEV)
    q = s["q"].double().view(B, M, hq, dim)
    R, lens = hq // hkv, s["lens"].tolist()
    for b in range(B):
        n = lens[b]
        lo = max(0, n - M + 1 - case["window"]) if case["window"] else 0
        j = torch.arange(lo, n, device=DEV)
        if not len(j):
            continue
        pg = s["table"][b].long()[j // page]
        for h in range(hkv):
            record = (pg * hkv + h) * (page // 16) + j % page // 16
            k, v = _exact_values(s["pool"], record, j % 16, case["fmt"], dim)
            for i in range(M):
                last = n - M + i
                a = max(0, last + 1 - case["window"]) - lo if case["window"] else 0
                e = last + 1 - lo
                if e <= a:
                    continue
                heads = slice(h * R, (h + 1) * R)
                x = q[b, i, heads] @ k[a:e].T / math.sqrt(dim)
                lse[b, i, heads] = torch.logsumexp(x, -1)
                out[b, i, heads] = torch.softmax(x, -1) @ v[a:e]
    return out.view(B * M, hq, dim), lse.view(B * M, hq)
