"""The operators that extend a paged K/V cache by new tokens: cases, plain forms and what each has to move.

extend   block tables, slot map and per-token indices from request lengths (kara_extend_tables)
append   per-head norms of q and k, rotary positions, K/V written into the pages, queries into the
         window-query ring (kara_append_kv)
chunk    causal attention of the new tokens over the paged cache (kara_chunk_attention)

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits; with ``own`` true it
calls the library.  ``exact`` gives the same outputs in 64 bits.  A case's lengths follow from the case alone;
its values and block ids follow from the seed.
"""
import math
import random

import torch

own = False

BS = 16          # tokens per cache block
EPS = 1e-6
NPOS = 40960     # rows of the rotation table


def listed():
    return [
        # one short conversation grows by one token: the latency of a single-user decode step
        dict(name="extend_one", op="extend", n=1, len_lo=256, len_hi=256, new_lo=1, new_hi=1, pad=0, lseed=0),
        # one decode step of a full serving batch, every table at its own fill
        dict(name="extend_decode", op="extend", n=128, len_lo=2048, len_hi=16383, new_lo=1, new_hi=1, pad=0, lseed=1),
        # admission: prompts and continued chunks of very different lengths, some waiting (0 new), padded buffers
        dict(name="extend_prompts", op="extend", n=256, len_lo=0, len_hi=2048, new_lo=0, new_hi=1024, pad=1000, lseed=2),
        # one token of the smallest model shape
        dict(name="append_one", op="append", n=1, len_lo=255, len_hi=255, new_lo=1, new_hi=1, hq=4, hkv=2, d=64,
             norm=True, W=64, rot=64, inter=False, lseed=3),
        # a decode step of 128 sequences, with the query ring
        dict(name="append_decode", op="append", n=128, len_lo=2048, len_hi=16383, new_lo=1, new_hi=1, hq=40, hkv=8,
             d=128, norm=True, W=1024, rot=128, inter=False, lseed=4),
        # prefill chunks: 4 prompts of 2048 tokens, the last window's queries kept
        dict(name="append_prefill", op="append", n=4, len_lo=0, len_hi=6000, new_lo=2048, new_hi=2048, hq=40, hkv=8,
             d=128, norm=True, W=1024, rot=128, inter=False, lseed=5),
        # a ragged mix of decodes and chunks, rotation without norms, no ring
        dict(name="append_mixed", op="append", n=64, len_lo=1024, len_hi=8192, new_lo=1, new_hi=257, hq=32, hkv=8,
             d=128, norm=False, W=0, rot=128, inter=False, lseed=6),
        # the smallest model shape, one prompt chunk
        dict(name="chunk_tiny", op="chunk", n=1, len_lo=192, len_hi=192, new_lo=64, new_hi=64, hq=4, hkv=2, d=64,
             lseed=7),
        # four drafted tokens per sequence over long caches: bound by the cache's bytes
        dict(name="chunk_drafts", op="chunk", n=128, len_lo=2048, len_hi=16380, new_lo=4, new_hi=4, hq=40, hkv=8,
             d=128, lseed=8),
        # a serving step that mixes decodes with prompt chunks
        dict(name="chunk_mixed", op="chunk", n=64, len_lo=1024, len_hi=8064, new_lo=1, new_hi=128, hq=32, hkv=8,
             d=128, lseed=9),
        # chunked prefill of a batch at 4096 cached tokens
        dict(name="chunk_batch", op="chunk", n=32, len_lo=3584, len_hi=3584, new_lo=512, new_hi=512, hq=32, hkv=8,
             d=128, lseed=10),
        # the second half of one long prompt
        dict(name="chunk_prefill", op="chunk", n=1, len_lo=8192, len_hi=8192, new_lo=8192, new_hi=8192, hq=40, hkv=8,
             d=128, lseed=11),
    ]


def _log(rng, lo, hi):
    return min(hi, int(lo * math.exp(rng.random() * math.log((hi + 1) / lo))))


def draw(rng):
    op = rng.choice(["extend", "append", "chunk"])
    c = dict(op=op, lseed=rng.randrange(1 << 30))
    if op == "extend":
        c["n"] = _log(rng, 1, 256)
        c["len_lo"] = rng.randrange(0, 2048)
        c["len_hi"] = c["len_lo"] + rng.randrange(0, 8192)
        c["new_lo"] = rng.randrange(0, 2)
        c["new_hi"] = max(1, c["new_lo"], min(1024, _log(rng, 1, 131072) // c["n"] + rng.randrange(0, 3)))
        c["pad"] = rng.choice([0, rng.randrange(1, 999)])
        return c
    c["hq"], c["hkv"] = rng.choice([(4, 2), (32, 8), (40, 8), (8, 8), (16, 2), (18, 3), (14, 2)])
    c["d"] = rng.choice([64, 128])
    c["n"] = _log(rng, 1, 128 if op == "append" else 64)
    c["len_lo"] = rng.randrange(0, 2000)
    c["len_hi"] = c["len_lo"] + rng.randrange(0, 6000)
    if op == "append":
        c["new_lo"] = 1
        c["new_hi"] = max(1, _log(rng, 1, 8192) // c["n"])
        c["norm"] = rng.random() < 0.7
        c["W"] = rng.choice([0, 64, 512, 1024])
        c["rot"] = rng.choice([c["d"], c["d"], c["d"] // 2])
        c["inter"] = rng.random() < 0.3
    else:
        c["new_lo"] = 1
        c["new_hi"] = max(1, _log(rng, 1, 8192) // c["n"])
    return c


def _lengths(case):
    """Cached lengths and new tokens of each sequence: of the case, not of the seed."""
    r = random.Random(case["lseed"] * 7919 + 1)
    old = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["n"])]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["n"])]
    if sum(new) == 0:
        new[0] = 1
    return old, new


def _blocks(x):
    return (x + BS - 1) // BS


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + case["lseed"])
    old, new = _lengths(case)
    n, total = case["n"], sum(new)
    s = dict(case=case, n=n, total=total, old=_i32(old), new=_i32(new))
    lens = [a + b for a, b in zip(old, new)]
    width = max(_blocks(x) for x in lens) + 1
    have = [_blocks(x) for x in old]
    want = [_blocks(x) for x in lens]
    if case["op"] == "extend":
        # each table lists its cached blocks, the unused entries are -1; the fresh list is longer than the need
        used, spare = sum(have), sum(want) - sum(have) + 17
        ids = torch.randperm(used + spare, generator=g, device="cuda").to(torch.int32)
        col = torch.arange(width, device="cuda")
        first = torch.cumsum(_i32(have), 0) - _i32(have)
        bt = torch.where(col < _i32(have)[:, None], ids[(first[:, None] + col).clamp(max=used + spare - 1)], -1)
        s.update(table=bt.to(torch.int32).contiguous(), fresh=ids[used:].contiguous(), nblocks=used + spare,
                 rows=total + case["pad"], width=width)
        return s
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    nb = sum(want)
    ids = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    first = torch.cumsum(_i32(want), 0) - _i32(want)
    bt = torch.where(col < _i32(want)[:, None], ids[(first[:, None] + col).clamp(max=nb - 1)], -1)
    s.update(table=bt.to(torch.int32).contiguous(), nblocks=nb, width=width, max_new=max(new), max_len=max(lens))
    # the per-token indices that extending the tables gave
    starts = [0]
    for m in new:
        starts.append(starts[-1] + m)
    s["q_start"], s["len"] = _i32(starts), _i32(lens)
    t = torch.arange(total, device="cuda")
    seq = torch.searchsorted(s["q_start"][1:].contiguous(), t, right=True)
    pos = s["old"][seq] + (t - s["q_start"][seq])
    s["seq"], s["pos"] = seq.to(torch.int32), pos.to(torch.int32)
    s["slot"] = s["table"][seq, pos // BS].to(torch.int64) * BS + pos % BS
    if case["op"] == "append":
        # a fused projection's output: q, k and v of a token side by side
        qkv = torch.randn(total, (hq + 2 * hkv) * d, generator=g, device="cuda").to(torch.bfloat16)
        s["q"] = qkv[:, :hq * d].view(total, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(total, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(total, hkv, d)
        s["kpool"] = torch.zeros(1, nb, hkv, BS, d, dtype=torch.bfloat16, device="cuda")
        s["vpool"] = torch.zeros_like(s["kpool"])
        s["qw"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) if case["norm"] else None
        s["kw"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) if case["norm"] else None
        half = case["rot"] // 2
        freq = 1e6 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        ang = torch.arange(NPOS, device="cuda", dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        # tokens that earlier compressions dropped: the rotary position runs ahead of the cached one
        s["shift"] = torch.randint(0, 8192, (n,), generator=g, device="cuda", dtype=torch.int32)
        W = case["W"]
        s["ring"] = torch.zeros(n, 1, hq, W, d, dtype=torch.bfloat16, device="cuda") if W else None
        s["q_out"] = torch.empty(total, hq, d, dtype=torch.bfloat16, device="cuda")
        return s
    # queries and keys after their norms: logits with a standard deviation of 2
    s["q"] = (2 * torch.randn(total, hq, d, generator=g, device="cuda")).to(torch.bfloat16)
    s["kpool"] = torch.randn(1, nb, hkv, BS, d, generator=g, device="cuda", dtype=torch.bfloat16)
    s["vpool"] = torch.randn(1, nb, hkv, BS, d, generator=g, device="cuda", dtype=torch.bfloat16)
    s["out"] = torch.empty(total, hq, d, dtype=torch.bfloat16, device="cuda")
    return s


# ---- plain forms -----------------------------------------------------------------

def _plain_extend(s):
    old, new, table, rows = s["old"], s["new"], s["table"], s["rows"]
    have = (old + BS - 1) // BS
    length = old + new
    need = (length + BS - 1) // BS - have
    off = torch.cumsum(need, 0) - need
    col = torch.arange(s["width"], device=old.device)
    i = col - have[:, None]
    table = torch.where((i >= 0) & (i < need[:, None]),
                        s["fresh"][(off[:, None] + i).clamp(0, s["fresh"].numel() - 1)], table)
    q_start = torch.zeros(s["n"] + 1, dtype=torch.int32, device=old.device)
    q_start[1:] = torch.cumsum(new, 0)
    t = torch.arange(rows, device=old.device)
    seq = torch.searchsorted(q_start[1:].contiguous(), t, right=True)
    live = seq < s["n"]
    at = seq.clamp(max=s["n"] - 1)
    pos = old[at] + (t - q_start[at])
    slot = table[at, (pos // BS).clamp(max=s["width"] - 1)].to(torch.int64) * BS + pos % BS
    return dict(table=table, q_start=q_start, length=length, slot=torch.where(live, slot, -1),
                seq=torch.where(live, at, -1).to(torch.int32), pos=torch.where(live, pos, -1).to(torch.int32),
                used=need.sum().to(torch.int32).reshape(1))


def _pairs(x, rot, inter):
    """The two members of each rotated pair, and the dims that pass through."""
    y, rest = x[..., :rot], x[..., rot:]
    if inter:
        return y[..., 0::2], y[..., 1::2], rest
    return y[..., :rot // 2], y[..., rot // 2:], rest


def _join(a, b, rest, inter):
    y = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([y, rest], -1)


def _plain_append(s):
    case = s["case"]
    rot, inter, W = case["rot"], case["inter"], case["W"]
    row = s["cos_sin"][(s["pos"] + s["shift"][s["seq"]]).long()]
    cos, sin = row[:, None, :rot // 2], row[:, None, rot // 2:]

    def turn(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        a, b, rest = _pairs(x, rot, inter)
        return _join(a * cos - b * sin, b * cos + a * sin, rest, inter).to(torch.bfloat16)

    q, k = turn(s["q"], s["qw"]), turn(s["k"], s["kw"])
    blk, at = s["slot"] // BS, s["slot"] % BS
    s["kpool"][0, blk, :, at] = k
    s["vpool"][0, blk, :, at] = s["v"]
    if W:
        s["ring"][:, 0] = torch.where(_ring_live(s)[:, None, :, None],
                                      q[_ring_token(s)].permute(0, 2, 1, 3), s["ring"][:, 0])
    return dict(q=q, k=s["kpool"], v=s["vpool"], ring=s["ring"])


def _ring_pos(s):
    """The last position of each sequence that falls on each ring row."""
    W = s["case"]["W"]
    last = s["len"][:, None] - 1
    return last - (last - torch.arange(W, device=last.device)) % W


def _ring_live(s):
    return _ring_pos(s) >= s["old"][:, None]


def _ring_token(s):
    return (s["q_start"][:-1, None] + _ring_pos(s) - s["old"][:, None]).clamp(0, s["total"] - 1)


def _plain_chunk(s):
    case = s["case"]
    n, hq, hkv, d, m = s["n"], case["hq"], case["hkv"], case["d"], s["max_new"]
    nb = _blocks(s["max_len"])
    ids = s["table"][:, :nb].clamp(min=0).long()
    live = torch.arange(nb * BS, device=ids.device) < s["len"][:, None]

    def dense(pool):
        x = pool[0][ids].float().permute(0, 2, 1, 3, 4).reshape(n, hkv, nb * BS, d)
        return torch.where(live[:, None, :, None], x, 0.0)

    tok = (s["q_start"][:-1, None] + torch.arange(m, device=ids.device)).clamp(max=s["total"] - 1)
    q = s["q"][tok].float().reshape(n, m, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    p = torch.matmul(q, dense(s["kpool"]).transpose(-1, -2)).mul_(1 / math.sqrt(d))
    seen = (torch.arange(nb * BS, device=ids.device) <= s["old"][:, None, None]
            + torch.arange(m, device=ids.device)[:, None])
    p = p.view(n, hq, m, -1).masked_fill_(~seen[:, None], float("-inf"))
    p = p.sub_(p.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, hkv, -1, nb * BS), dense(s["vpool"])).view(n, hq, m, d) / total
    return o.permute(0, 2, 1, 3)[s["seq"].long(), (s["pos"] - s["old"][s["seq"]]).long()].to(torch.bfloat16)


# ---- the library -----------------------------------------------------------------

def _handle(s):
    """Descriptors, buffers and workspaces that a serving program keeps for its cache and its step."""
    from decode_kv_cache_03_gb300 import kara
    case, n = s["case"], s["n"]
    h = dict(kara=kara, err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["op"] == "extend":
        new = lambda k, t: torch.empty(k, dtype=t, device="cuda")  # noqa: E731
        h["used"] = new(1, torch.int32)
        h["q_start"], h["length"] = new(n + 1, torch.int32), new(n, torch.int32)
        h["slot"], h["seq"], h["pos"] = (new(s["rows"], torch.int64), new(s["rows"], torch.int32),
                                         new(s["rows"], torch.int32))
        h["tokens"] = kara.tokens(h["q_start"], h["length"], h["slot"], h["seq"], h["pos"])
        return h
    h["cache"] = kara.cache(s["kpool"], s["vpool"], case["hq"])
    h["tokens"] = kara.tokens(s["q_start"], s["len"], s["slot"], s["seq"], s["pos"])
    if case["op"] == "append":
        h["rope"] = kara.rope(s["cos_sin"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS, interleaved=case["inter"],
                              pos_offset=s["shift"])
    else:
        h["ws"] = torch.empty(kara.kara_chunk_workspace_size(h["cache"], n, s["total"]), dtype=torch.uint8,
                              device="cuda")
    return h


def _own(s):
    h = s.get("handle")
    if h is None:
        h = s["handle"] = _handle(s)
    kara, op = h["kara"], s["case"]["op"]
    if op == "extend":
        kara.kara_extend_tables(s["nblocks"], BS, s["old"], s["new"], s["table"], s["fresh"], h["tokens"], h["used"],
                                h["err"])
        return dict(table=s["table"], q_start=h["q_start"], length=h["length"], slot=h["slot"], seq=h["seq"],
                    pos=h["pos"], used=h["used"])
    if op == "append":
        kara.kara_append_kv(h["cache"], 0, h["tokens"], h["rope"], s["q"], s["k"], s["v"], s["q_out"], h["err"],
                            ring=s["ring"])
        return dict(q=s["q_out"], k=s["kpool"], v=s["vpool"], ring=s["ring"])
    kara.kara_chunk_attention(h["cache"], 0, h["tokens"], s["table"], s["q"], s["out"], h["ws"], h["err"])
    return s["out"]


def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    return _plain_extend(s) if op == "extend" else _plain_append(s) if op == "append" else _plain_chunk(s)


def work(case):
    old, new = _lengths(case)
    n, total = case["n"], sum(new)
    if case["op"] == "extend":
        opened = sum(_blocks(a + b) - _blocks(a) for a, b in zip(old, new))
        part = sum(1 for a, b in zip(old, new) if a % BS and b)
        return dict(bytes=4 * n * 2 + 4 * (2 * n + 1) + 8 * opened + 4 * part + 16 * (total + case["pad"]) + 4, flops=0)
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    if case["op"] == "append":
        ring = sum(min(m, case["W"]) for m in new) * hq * d * 2
        return dict(bytes=2 * total * (hq + 2 * hkv) * d * 2 + ring + total * (case["rot"] * 4 + 16) + 4 * n
                    + (4 * d if case["norm"] else 0), flops=total * (hq + hkv) * d * (7 if case["norm"] else 3))
    pairs = sum(m * a + m * (m + 1) // 2 for a, m in zip(old, new))
    return dict(bytes=sum(a + m for a, m in zip(old, new)) * hkv * d * 4 + 2 * total * hq * d * 2,
                flops=4 * d * hq * pairs)


# ---- the definition in 64 bits ----------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    old, new = _lengths(case)
    if case["op"] == "extend":
        return None   # whole numbers only
    if case["op"] == "append":
        return _exact_append(s, old, new)
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    G = hq // hkv
    out = torch.empty(s["total"], hq, d, dtype=torch.float64, device="cuda")
    t0 = 0
    for i, (a, m) in enumerate(zip(old, new)):
        length = a + m
        ids = s["table"][i, :_blocks(length)].long()
        for g in range(hkv):
            k = s["kpool"][0, ids, g].reshape(-1, d)[:length].double()
            v = s["vpool"][0, ids, g].reshape(-1, d)[:length].double()
            for lo in range(0, m, 2048):
                hi = min(m, lo + 2048)
                top = a + hi
                q = s["q"][t0 + lo:t0 + hi, g * G:(g + 1) * G].double()
                z = torch.einsum("thd,xd->htx", q, k[:top]) * d ** -0.5
                late = torch.arange(top, device="cuda")[None] > torch.arange(a + lo, a + hi, device="cuda")[:, None]
                w = torch.softmax(z.masked_fill(late, -math.inf), -1)
                out[t0 + lo:t0 + hi, g * G:(g + 1) * G] = torch.einsum("htx,xd->thd", w, v[:top])
        t0 += m
    return out


def _exact_append(s, old, new):
    case = s["case"]
    rot, W, d = case["rot"], case["W"], case["d"]
    r = (s["pos"] + s["shift"][s["seq"].long()]).long()
    cs = s["cos_sin"][r].double()
    # each pair (x_a, x_b) as a complex number times cos + i sin
    turn = torch.complex(cs[:, :rot // 2], cs[:, rot // 2:])
    a = torch.arange(0, rot, 2, device="cuda") if case["inter"] else torch.arange(rot // 2, device="cuda")
    b = a + 1 if case["inter"] else a + rot // 2

    def make(x, w):
        y = x.double().clone()
        if w is not None:
            y = y / (y.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * w.double()
        z = torch.complex(y[..., a], y[..., b]) * turn[:, None]
        y[..., a], y[..., b] = z.real, z.imag
        return y

    q, k = make(s["q"], s["qw"]), make(s["k"], s["kw"])
    flat = torch.zeros(s["nblocks"] * BS, case["hkv"], d, dtype=torch.float64, device="cuda")

    def paged(x):
        rows = flat.clone()
        rows[s["slot"]] = x.double()
        return rows.view(1, s["nblocks"], BS, case["hkv"], d).transpose(2, 3)

    ring = None
    if W:
        ring = torch.zeros(s["n"], 1, case["hq"], W, d, dtype=torch.float64, device="cuda")
        t0 = 0
        for i, (o, m) in enumerate(zip(old, new)):
            keep = min(m, W)
            at = torch.arange(o + m - keep, o + m, device="cuda") % W
            ring[i, 0, :, at] = q[t0 + m - keep:t0 + m].transpose(0, 1)
            t0 += m
    return dict(q=q, k=paged(k), v=paged(s["v"]), ring=ring)
