"""The operators of a paged K/V cache held in 8 bits: cases, plain forms and what each has to move.

append8   per-head norms, rotary positions, K/V rounded to e4m3 with a power-of-two scale for each block and
          head and written into the pages, queries into the window-query ring (kara_append_kv8)
decode8   attention of one token a sequence over the 8-bit cache (kara_decode_attention8)
chunk8    causal attention of several new tokens a sequence over it (kara_chunk_attention8)
expand8   the keys of the windows that a compression scores, back in bf16 (kara_expand8)
compact8  the gather-compaction with new scales for the rebuilt blocks, tables rewritten (kara_compact8)

A value of the cache is its code times the scale of its block and head; the scale is the smallest power of two
with which the block's largest value stays within 448.  With ``own`` false, ``run`` computes the operators with
elementary torch operations in 32 bits; with ``own`` true it calls the library.  ``exact`` gives the same outputs
in 64 bits.  A case's lengths follow from the case alone; its values and block ids follow from the seed.
"""
import math
import random

import torch

own = False

BS = 16          # tokens per cache block
TOP = 448.0      # largest finite e4m3 value
E_MIN, E_MAX = -63, 63   # exponents of a block's scale
EPS = 1e-6
NPOS = 40960     # rows of the rotation table
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # a decode step of 128 sequences with the query ring: partly filled blocks, some of which get a new scale
        dict(name="append8_decode", op="append8", n=128, len_lo=2048, len_hi=16383, new_lo=1, new_hi=1, hq=40, hkv=8,
             d=128, norm=True, W=1024, rot=128, inter=False, lseed=1),
        # prefill chunks: 4 prompts of 2048 tokens, the last window's queries kept
        dict(name="append8_prefill", op="append8", n=4, len_lo=0, len_hi=6000, new_lo=2048, new_hi=2048, hq=40, hkv=8,
             d=128, norm=True, W=1024, rot=128, inter=False, lseed=2),
        # one user of the smallest model shape: the latency of a step
        dict(name="decode8_one", op="decode8", n=1, len_lo=256, len_hi=256, hq=4, hkv=2, d=64, lseed=3),
        # a full serving batch over long caches: bound by the cache's bytes
        dict(name="decode8_batch", op="decode8", n=128, len_lo=2048, len_hi=16384, hq=40, hkv=8, d=128, lseed=4),
        # the smallest model shape, one prompt chunk
        dict(name="chunk8_tiny", op="chunk8", n=1, len_lo=192, len_hi=192, new_lo=64, new_hi=64, hq=4, hkv=2, d=64,
             lseed=5),
        # four drafted tokens per sequence over long caches: bound by the cache's bytes
        dict(name="chunk8_drafts", op="chunk8", n=128, len_lo=2048, len_hi=16380, new_lo=4, new_hi=4, hq=40, hkv=8,
             d=128, lseed=6),
        # a serving step that mixes decodes with prompt chunks
        dict(name="chunk8_mixed", op="chunk8", n=64, len_lo=1024, len_hi=8064, new_lo=1, new_hi=128, hq=32, hkv=8,
             d=128, lseed=7),
        # the second half of one long prompt
        dict(name="chunk8_prefill", op="chunk8", n=1, len_lo=8192, len_hi=8192, new_lo=8192, new_hi=8192, hq=40,
             hkv=8, d=128, lseed=8),
        # the window of the smallest model shape, ahead of its scoring
        dict(name="expand8_one", op="expand8", n=1, layers=1, len_lo=250, len_hi=256, hq=4, hkv=2, d=64, W=64, lseed=9),
        # the windows of 16 sequences in all layers of a 36-layer model
        dict(name="expand8_batch", op="expand8", n=16, layers=36, len_lo=4096, len_hi=4111, hq=32, hkv=8, d=128, W=512,
             lseed=10),
        # one compressed window of the smallest model shape
        dict(name="compact8_one", op="compact8", n=1, layers=1, len_lo=250, len_hi=256, hq=4, hkv=2, d=64, W=64, B=16,
             R=16, lseed=11),
        # 8 sequences of the largest serving shape, all layers
        dict(name="compact8_batch", op="compact8", n=8, layers=40, len_lo=2048, len_hi=16384, hq=40, hkv=8, d=128,
             W=1024, B=128, R=268, lseed=12),
    ]


def _log(rng, lo, hi):
    return min(hi, int(lo * math.exp(rng.random() * math.log((hi + 1) / lo))))


def draw(rng):
    op = rng.choice(["append8", "decode8", "chunk8", "expand8", "compact8"])
    c = dict(op=op, lseed=rng.randrange(1 << 30))
    c["hq"], c["hkv"] = rng.choice([(4, 2), (32, 8), (40, 8), (8, 8), (16, 2), (18, 3), (14, 2)])
    c["d"] = rng.choice([64, 128])
    if op in ("expand8", "compact8"):
        c["n"], c["layers"] = _log(rng, 1, 16), _log(rng, 1, 8)
        c["W"] = 64 * rng.choice([1, 2, 3, 5, 8, 13, 16])
        if op == "compact8":
            c["B"] = rng.choice([0, c["W"] // 8, rng.randrange(1, c["W"] // 2)])
            c["R"] = rng.randrange(1, (c["W"] - c["B"]) // 2 + 1)
        c["len_lo"] = c["W"] + rng.randrange(0, 100)
        c["len_hi"] = c["len_lo"] + rng.randrange(0, 6000)
        return c
    c["n"] = _log(rng, 1, 64 if op == "chunk8" else 128)
    c["len_lo"] = rng.randrange(0, 2000)
    c["len_hi"] = c["len_lo"] + rng.randrange(0, 6000)
    if op == "decode8":
        if rng.random() < 0.3:
            c["len_lo"] = 0     # some sequences of the batch are empty
        c["len_hi"] = max(1, c["len_hi"])
        return c
    c["new_lo"] = 1
    c["new_hi"] = max(1, _log(rng, 1, 8192) // c["n"])
    if op == "append8":
        c["norm"] = rng.random() < 0.7
        c["W"] = rng.choice([0, 64, 512, 1024])
        c["rot"] = rng.choice([c["d"], c["d"], c["d"] // 2])
        c["inter"] = rng.random() < 0.3
    return c


def _lengths(case):
    """Cached lengths and new tokens of each sequence: of the case, not of the seed."""
    r = random.Random(case["lseed"] * 7919 + 1)
    old = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["n"])]
    if case["op"] == "decode8" and max(old) == 0:
        old[0] = 1
    new = [r.randint(case["new_lo"], case["new_hi"]) if "new_lo" in case else 0 for _ in range(case["n"])]
    return old, new


def _blocks(x):
    return (x + BS - 1) // BS


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---- the 8-bit form --------------------------------------------------------------

def _scale(amax):
    """The smallest power of two with which amax is within 448 (0 for 0)."""
    m, e = torch.frexp(amax)            # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(E_MIN, E_MAX)
    return torch.where(amax > 0, (e + 127 << 23).view(torch.float32), 0.0)   # (torch's powers may be an ulp off)


def _inverse(scale):
    return torch.where(scale > 0, 1 / scale, 0.0)


def _codes(x, scale):
    """x / scale as e4m3, its bits."""
    return (x * _inverse(scale)).clamp(-TOP, TOP).to(E4M3).view(torch.uint8)


def _value(codes):
    return codes.view(E4M3).float()


def _pool(g, shape, lo, hi):
    """A pool of random values in 8 bits, the blocks' magnitudes 2^lo to 2^hi."""
    codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
    scale = torch.empty(shape[:3], dtype=torch.float32, device="cuda")
    for layer in range(shape[0]):
        for b in range(0, shape[1], 16384):
            part = codes[layer, b:b + 16384]
            x = torch.randn(part.shape, generator=g, device="cuda", dtype=torch.bfloat16).float()
            x *= 2.0 ** torch.randint(lo, hi + 1, part.shape[:2], generator=g, device="cuda")[..., None, None]
            s = _scale(x.abs().amax((-1, -2)))
            scale[layer, b:b + 16384] = s
            part.copy_(_codes(x, s[..., None, None]))
    return codes, scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + case["lseed"])
    old, new = _lengths(case)
    s = dict(case=case, n=case["n"], total=sum(new), old=_i32(old))
    if case["op"] in ("expand8", "compact8"):
        return _prepare_windows(s, g, case, old)
    if case["op"] == "append8":
        return _prepare_append(s, g, case, old, new)
    n, total, d, hq, hkv = s["n"], s["total"], case["d"], case["hq"], case["hkv"]
    lens = [a + b for a, b in zip(old, new)]
    want = [_blocks(x) for x in lens]
    nb, width = sum(want), max(want) + 1
    ids = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    first = torch.cumsum(_i32(want), 0) - _i32(want)
    bt = torch.where(col < _i32(want)[:, None], ids[(first[:, None] + col).clamp(max=nb - 1)], -1)
    s.update(table=bt.to(torch.int32).contiguous(), max_len=max(lens), len=_i32(lens))
    s["k"], s["k_scale"] = _pool(g, (1, nb, hkv, BS, d), -1, 0)
    s["v"], s["v_scale"] = _pool(g, (1, nb, hkv, BS, d), -2, 2)
    rows = total if case["op"] == "chunk8" else n
    # queries after their norms: logits with a standard deviation of 1 to 2
    s["q"] = (2 * torch.randn(rows, hq, d, generator=g, device="cuda")).to(torch.bfloat16)
    s["out"] = torch.empty(rows, hq, d, dtype=torch.bfloat16, device="cuda")
    if case["op"] == "chunk8":
        s["max_new"] = max(new)
        _tokens(s, old, new)
    return s


def _tokens(s, old, new):
    """The per-token indices that extending the tables gave."""
    starts = [0]
    for m in new:
        starts.append(starts[-1] + m)
    s["q_start"] = _i32(starts)
    t = torch.arange(s["total"], device="cuda")
    seq = torch.searchsorted(s["q_start"][1:].contiguous(), t, right=True)
    pos = s["old"][seq] + (t - s["q_start"][seq])
    s["seq"], s["pos"] = seq.to(torch.int32), pos.to(torch.int32)
    if "first" in s:
        s["slot"] = s["ids"][s["first"][seq] + pos // BS].to(torch.int64) * BS + pos % BS
    else:
        s["slot"] = s["table"][seq, pos // BS].to(torch.int64) * BS + pos % BS


def _prepare_append(s, g, case, old, new):
    n, total, d, hq, hkv = s["n"], s["total"], case["d"], case["hq"], case["hkv"]
    # a pool of the blocks that get tokens: each sequence's from the one that its first new token falls into
    have = [a // BS for a in old]
    want = [_blocks(a + m) - h for a, m, h in zip(old, new, have)]
    nb = sum(want)
    s["ids"] = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    s["first"] = torch.cumsum(_i32(want), 0) - _i32(want) - _i32(have)
    s["len"] = _i32([a + m for a, m in zip(old, new)])
    _tokens(s, old, new)
    s["k"], s["k_scale"] = _pool(g, (1, nb, hkv, BS, d), -2, 0)
    s["v"], s["v_scale"] = _pool(g, (1, nb, hkv, BS, d), -2, 0)
    # a fused projection's output: q, k and v of a token side by side
    qkv = torch.randn(total, (hq + 2 * hkv) * d, generator=g, device="cuda").to(torch.bfloat16)
    s["q_new"] = qkv[:, :hq * d].view(total, hq, d)
    s["k_new"] = qkv[:, hq * d:(hq + hkv) * d].view(total, hkv, d)
    s["v_new"] = qkv[:, (hq + hkv) * d:].view(total, hkv, d)
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


def _prepare_windows(s, g, case, lens):
    n, W, d, hkv, layers = s["n"], case["W"], case["d"], case["hkv"], case["layers"]
    # the windows' blocks are their own; earlier ones, which nothing reads, come from a few that all share
    p0 = [(L - W) // BS for L in lens]
    win = [_blocks(L) - p for L, p in zip(lens, p0)]
    shared, width = 16, max(_blocks(L) for L in lens) + 1
    if case["op"] == "compact8":
        after = [L - W + case["R"] + case["B"] for L in lens]
        take = [_blocks(x) - p for x, p in zip(after, p0)]
    else:
        take = [0] * n
    nb = shared + sum(win) + sum(take) + 3
    ids = shared + torch.randperm(nb - shared, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    first = torch.cumsum(_i32(win), 0) - _i32(win)
    at = col - _i32(p0)[:, None]
    own_ids = ids[(first[:, None] + at).clamp(0, nb - shared - 1)]
    bt = torch.where(at < 0, (col % shared).to(torch.int32), torch.where(at < _i32(win)[:, None], own_ids, -1))
    s.update(len=s["old"], table=bt.to(torch.int32).contiguous(), p0=_i32(p0), win=_i32(win), width=width)
    s["k"], s["k_scale"] = _pool(g, (layers, nb, hkv, BS, d), -2, 1)
    if case["op"] == "expand8":
        nw = W // BS + 1
        s["out"] = torch.zeros(layers, n * nw, hkv, BS, d, dtype=torch.bfloat16, device="cuda")
        s["out_table"] = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
        return s
    s["v"], s["v_scale"] = _pool(g, (layers, nb, hkv, BS, d), -2, 1)
    C, R = W - case["B"], case["R"]
    pick = torch.rand(n, layers, hkv, C, generator=g, device="cuda").topk(R, -1).indices
    s["kept"] = pick.sort(-1).values.to(torch.int32).contiguous()
    s["fresh"] = ids[sum(win):].contiguous()
    s["take"], s["after"], s["max_take"] = _i32(take), _i32(after), max(take)
    s["max_win"], s["total_old"], s["total_new"] = max(win), sum(win), sum(take)
    s["table0"] = s["table"].clone()
    s["freed"] = torch.empty(sum(win), dtype=torch.int32, device="cuda")
    s["new_len"] = torch.empty(n, dtype=torch.int32, device="cuda")
    return s


# ---- plain forms -----------------------------------------------------------------

def _pairs(x, rot, inter):
    """The two members of each rotated pair, and the dims that pass through."""
    y, rest = x[..., :rot], x[..., rot:]
    if inter:
        return y[..., 0::2], y[..., 1::2], rest
    return y[..., :rot // 2], y[..., rot // 2:], rest


def _join(a, b, rest, inter):
    y = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([y, rest], -1)


def _store(s, pool, scales, x):
    """New rows x [rows][hkv][d] into a pool: each touched block's scale covers them and the rows ahead of them."""
    codes, scale, blk, at = s[pool][0], s[scales][0], s["slot"] // BS, s["slot"] % BS
    amax = torch.zeros_like(scale).scatter_reduce_(0, blk[:, None].expand(-1, scale.shape[1]), x.abs().amax(-1), "amax")
    first = torch.full((codes.shape[0],), BS, dtype=torch.int64, device=x.device).scatter_reduce_(0, blk, at, "amin")
    before = torch.where((first > 0)[:, None], scale, 0.0)
    after = torch.maximum(before, _scale(amax))
    ahead = torch.arange(BS, device=x.device) < torch.where(first < BS, first, 0)[:, None]
    ratio = (before * _inverse(after))[:, :, None, None]
    moved = (_value(codes) * ratio).to(E4M3).view(torch.uint8)
    codes.copy_(torch.where(ahead[:, None, :, None] & (ratio < 1), moved, codes))
    scale.copy_(torch.where((first < BS)[:, None], after, scale))
    codes[blk, :, at] = _codes(x, scale[blk][..., None])


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
        return _join(a * cos - b * sin, b * cos + a * sin, rest, inter)

    q = turn(s["q_new"], s["qw"]).to(torch.bfloat16)
    _store(s, "k", "k_scale", turn(s["k_new"], s["kw"]))
    _store(s, "v", "v_scale", s["v_new"].float())
    if W:
        s["ring"][:, 0] = torch.where(_ring_live(s)[:, None, :, None],
                                      q[_ring_token(s)].permute(0, 2, 1, 3), s["ring"][:, 0])
    return _append_outputs(s, q)


def _append_outputs(s, q):
    return dict(q=q, k=s["k"].view(E4M3), k_scale=s["k_scale"], v=s["v"].view(E4M3), v_scale=s["v_scale"],
                ring=s["ring"])


def _ring_pos(s):
    """The last position of each sequence that falls on each ring row."""
    W = s["case"]["W"]
    last = s["len"][:, None] - 1
    return last - (last - torch.arange(W, device=last.device)) % W


def _ring_live(s):
    return _ring_pos(s) >= s["old"][:, None]


def _ring_token(s):
    return (s["q_start"][:-1, None] + _ring_pos(s) - s["old"][:, None]).clamp(0, s["total"] - 1)


def _dense(s, pool, scales):
    """[n][hkv][keys][d] of every sequence, zeros past its end."""
    nb, d = _blocks(s["max_len"]), s["case"]["d"]
    ids = s["table"][:, :nb].clamp(min=0).long()
    x = _value(s[pool][0][ids]) * s[scales][0][ids][..., None, None]
    x = x.permute(0, 2, 1, 3, 4).reshape(s["n"], -1, nb * BS, d)
    live = torch.arange(nb * BS, device=ids.device) < s["len"][:, None]
    return torch.where(live[:, None, :, None], x, 0.0)


def _weighted(s, q, seen):
    """Softmax attention of q [n][hkv][rows][d] over the cache, seen broadcastable to [n][hkv][rows][keys]."""
    p = torch.matmul(q, _dense(s, "k", "k_scale").transpose(-1, -2)).mul_(1 / math.sqrt(s["case"]["d"]))
    p = p.masked_fill_(~seen, float("-inf"))
    top = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(top > float("-inf"), top, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, _dense(s, "v", "v_scale")) / torch.where(total > 0, total, 1.0)


def _plain_decode(s):
    hkv, d = s["case"]["hkv"], s["case"]["d"]
    keys = torch.arange(_blocks(s["max_len"]) * BS, device="cuda")
    o = _weighted(s, s["q"].float().view(s["n"], hkv, -1, d), (keys < s["len"][:, None])[:, None, None])
    return o.reshape(s["n"], -1, d).to(torch.bfloat16)


def _plain_chunk(s):
    n, m, hq, hkv, d = s["n"], s["max_new"], s["case"]["hq"], s["case"]["hkv"], s["case"]["d"]
    tok = (s["q_start"][:-1, None] + torch.arange(m, device="cuda")).clamp(max=s["total"] - 1)
    q = s["q"][tok].float().reshape(n, m, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    keys = torch.arange(_blocks(s["max_len"]) * BS, device="cuda")
    seen = keys <= s["old"][:, None, None] + torch.arange(m, device="cuda")[:, None]
    o = _weighted(s, q, seen.repeat(1, hq // hkv, 1)[:, None]).view(n, hq, m, d)
    return o.permute(0, 2, 1, 3)[s["seq"].long(), (s["pos"] - s["old"][s["seq"]]).long()].to(torch.bfloat16)


def _plain_expand(s):
    case, n = s["case"], s["n"]
    nw = case["W"] // BS + 1
    i = torch.arange(nw, device="cuda")
    col = s["p0"][:, None] + i
    live = i < s["win"][:, None]
    ids = torch.where(live, s["table"].gather(1, col.clamp(max=s["width"] - 1).long()), 0).long()
    x = _value(s["k"][:, ids]) * s["k_scale"][:, ids][..., None, None]
    row = col[..., None] * BS + torch.arange(BS, device="cuda")
    x = torch.where((row < s["len"][:, None, None])[:, :, None, :, None], x, 0.0).to(torch.bfloat16)
    out = s["out"].view(case["layers"], n, nw, *s["out"].shape[2:])
    out.copy_(torch.where(live[:, :, None, None, None], x, out))
    new = torch.arange(n * nw, dtype=torch.int32, device="cuda").view(n, nw)
    keep = s["out_table"].gather(1, col.clamp(max=s["width"] - 1).long())
    s["out_table"].scatter_(1, col.clamp(max=s["width"] - 1).long(), torch.where(live, new, keep))
    return dict(k=s["out"], table=s["out_table"])


def _plain_compact(s):
    case, n, hkv, layers = s["case"], s["n"], s["case"]["hkv"], s["case"]["layers"]
    W, B, R, d = case["W"], case["B"], case["R"], case["d"]
    s["table"].copy_(s["table0"])
    # old position of each new row
    r = torch.arange(s["max_take"] * BS, device="cuda")
    ws = (s["len"] - W)[:, None]
    new = s["p0"][:, None] * BS + r
    j = new - ws
    kept = s["kept"].gather(-1, j.clamp(0, R - 1).long()[:, None, None, :].expand(-1, layers, hkv, -1))
    src = torch.where(j < 0, new, s["len"][:, None] - B + j - R)[:, None, None]
    src = torch.where(((j >= 0) & (j < R))[:, None, None], ws[:, None, None] + kept, src)
    live = new < s["after"][:, None]
    src = torch.where(live[:, None, None], src, ws[:, None, None]).long()
    blk = s["table"][torch.arange(n, device="cuda")[:, None, None, None], src // BS].long()
    layer = torch.arange(layers, device="cuda")[None, :, None, None]
    head = torch.arange(hkv, device="cuda")[None, None, :, None]
    # where the new blocks go
    i = torch.arange(s["max_take"], device="cuda")
    mine = i < s["take"][:, None]
    off = torch.cumsum(s["take"], 0) - s["take"]
    to = s["fresh"][(off[:, None] + i)[mine].long()].long()
    rows = live.view(n, 1, 1, -1, BS, 1)
    for pool, scales in (("k", "k_scale"), ("v", "v_scale")):
        x = _value(s[pool][layer, blk, head, src % BS]) * s[scales][layer, blk, head][..., None]
        x = x.view(n, layers, hkv, -1, BS, d)
        scale = _scale(torch.where(rows, x, 0.0).abs().amax((-1, -2)))
        codes = _codes(x, scale[..., None, None]).permute(0, 3, 1, 2, 4, 5)[mine]
        there = s[pool][:, to].transpose(0, 1)
        there = torch.where(live.view(n, -1, 1, 1, BS, 1)[mine], codes, there)
        s[pool][:, to] = there.transpose(0, 1)
        s[scales][:, to] = scale.permute(0, 3, 1, 2)[mine].transpose(0, 1)
    # released ids, new entries, new lengths
    i = torch.arange(s["max_win"], device="cuda")
    had = i < s["win"][:, None]
    col = (s["p0"][:, None] + i).clamp(max=s["width"] - 1).long()
    s["freed"].copy_(s["table"].gather(1, col)[had])
    entry = torch.where(i < s["take"][:, None], s["fresh"][(off[:, None] + i).clamp(max=s["fresh"].numel() - 1).long()],
                        -1)
    at = torch.arange(n, device="cuda")[:, None].expand_as(col)
    s["table"][at[had], col[had]] = entry[had]
    s["new_len"].copy_(s["after"])
    return _compact_outputs(s)


def _compact_outputs(s):
    return dict(k=s["k"].view(E4M3), k_scale=s["k_scale"], v=s["v"].view(E4M3), v_scale=s["v_scale"], table=s["table"],
                freed=s["freed"], new_len=s["new_len"])


# ---- the library -----------------------------------------------------------------

def _handle(s):
    """Descriptors, buffers and workspaces that a serving program keeps for its cache and its step."""
    from decode_kv_cache_03_gb300 import kara
    case, n, op = s["case"], s["n"], s["case"]["op"]
    h = dict(kara=kara, err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    v, v_scale = s.get("v", s["k"]), s.get("v_scale", s["k_scale"])
    c = h["cache"] = kara.cache8(s["k"], v, s["k_scale"], v_scale, case["hq"])
    if op in ("append8", "chunk8"):
        h["tokens"] = kara.tokens(s["q_start"], s["len"], s["slot"], s["seq"], s["pos"])
    new = lambda size: torch.empty(size, dtype=torch.uint8, device="cuda")  # noqa: E731
    if op == "append8":
        h["rope"] = kara.rope(s["cos_sin"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS, interleaved=case["inter"],
                              pos_offset=s["shift"])
    elif op == "decode8":
        h["ws"] = new(kara.kara_decode8_workspace_size(c, n, s["table"].shape[1]))
    elif op == "chunk8":
        h["ws"] = new(kara.kara_chunk8_workspace_size(c, n, s["total"]))
    elif op == "expand8":
        h["out"] = kara.cache(s["out"], s["out"], case["hq"])
    else:
        h["params"] = kara.params(case["W"], case["B"], 1, case["R"], 0.1)
        h["ws"] = new(kara.kara_compact8_workspace_size(c, h["params"], n))
    return h


def _own(s):
    h = s.get("handle")
    if h is None:
        h = s["handle"] = _handle(s)
    kara, op, c, err = h["kara"], s["case"]["op"], h["cache"], h["err"]
    if op == "append8":
        kara.kara_append_kv8(c, 0, h["tokens"], h["rope"], s["q_new"], s["k_new"], s["v_new"], s["q_out"], err,
                             ring=s["ring"])
        return _append_outputs(s, s["q_out"])
    if op == "decode8":
        kara.kara_decode_attention8(c, 0, s["len"], s["table"], s["q"], s["out"], h["ws"], err)
        return s["out"]
    if op == "chunk8":
        kara.kara_chunk_attention8(c, 0, h["tokens"], s["table"], s["q"], s["out"], h["ws"], err)
        return s["out"]
    if op == "expand8":
        kara.kara_expand8(c, h["out"], s["case"]["W"], s["len"], s["table"], s["out_table"], err)
        return dict(k=s["out"], table=s["out_table"])
    s["table"].copy_(s["table0"])
    kara.kara_compact8(c, h["params"], s["len"], s["table"], s["kept"], s["fresh"], s["freed"], s["new_len"], h["ws"],
                       err)
    return _compact_outputs(s)


def run(s):
    if own:
        return _own(s)
    plain = dict(append8=_plain_append, decode8=_plain_decode, chunk8=_plain_chunk, expand8=_plain_expand,
                 compact8=_plain_compact)
    return plain[s["case"]["op"]](s)


def work(case):
    old, new = _lengths(case)
    n, total, op = case["n"], sum(new), case["op"]
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    slice8 = BS * d + 4     # codes and scale of a block and head
    if op == "append8":
        ring = sum(min(m, case["W"]) for m in new) * hq * d * 2
        touched = sum(_blocks(a + m) - a // BS for a, m in zip(old, new))
        return dict(bytes=total * (hq + 2 * hkv) * d * 2 + total * hq * d * 2 + total * 2 * hkv * d + ring
                    + touched * hkv * 8 + total * (case["rot"] * 4 + 16) + 4 * n + (4 * d if case["norm"] else 0),
                    flops=total * (hq + hkv) * d * (7 if case["norm"] else 3) + total * 2 * hkv * d * 2)
    if op == "decode8":
        return dict(bytes=sum(a * 2 * d + _blocks(a) * 8 for a in old) * hkv + 2 * n * hq * d * 2
                    + 4 * sum(_blocks(a) for a in old), flops=4 * d * hq * sum(old))
    if op == "chunk8":
        pairs = sum(m * a + m * (m + 1) // 2 for a, m in zip(old, new))
        return dict(bytes=sum((a + m) * 2 * d + _blocks(a + m) * 8 for a, m in zip(old, new)) * hkv
                    + 2 * total * hq * d * 2 + 4 * sum(_blocks(a + m) for a, m in zip(old, new)),
                    flops=4 * d * hq * pairs)
    heads = case["layers"] * hkv
    win = sum(_blocks(a) - (a - case["W"]) // BS for a in old)
    if op == "expand8":
        return dict(bytes=win * (heads * (slice8 + BS * d * 2) + 8), flops=win * heads * BS * d)
    rows = sum((a - case["W"]) % BS + case["R"] + case["B"] for a in old)
    take = sum(_blocks(a - case["W"] + case["R"] + case["B"]) - (a - case["W"]) // BS for a in old)
    return dict(bytes=heads * (2 * rows * 2 * d + (win + take) * 8 + n * case["R"] * 4) + 4 * (2 * win + 2 * take + n),
                flops=2 * rows * heads * d * 2)


# ---- the definition in 64 bits ----------------------------------------------------

def _e4m3_values(codes):
    """Sign, exponent and mantissa of the bits, in 64 bits."""
    b = codes.long()
    e, m = b >> 3 & 15, (b & 7).double()
    power = torch.tensor([2.0 ** (i - 10) for i in range(16)], dtype=torch.float64, device=codes.device)
    size = torch.where(e > 0, (8 + m) * power[e], m * 2.0 ** -9)
    return torch.where(b > 127, -size, size)


def _power_of_two(amax):
    all_of_them = torch.tensor([2.0 ** e for e in range(E_MIN, E_MAX + 1)], dtype=torch.float64, device=amax.device)
    i = torch.searchsorted(all_of_them * TOP, amax).clamp(max=len(all_of_them) - 1)
    return torch.where(amax > 0, all_of_them[i], 0.0)


def exact(case, seed):
    s = prepare(case, seed)
    old, new = _lengths(case)
    op = case["op"]
    if op == "append8":
        return _exact_append(s, old, new)
    if op == "expand8":
        return _exact_expand(s, old)
    if op == "compact8":
        return _exact_compact(s, old)
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    G = hq // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    t0 = 0
    for i, (a, m) in enumerate(zip(old, new)):
        length = a + m
        ids = s["table"][i, :_blocks(length)].long()
        rows = m if op == "chunk8" else 1
        for h in range(hkv if length else 0):
            k = (_e4m3_values(s["k"][0, ids, h]) * s["k_scale"][0, ids, h, None, None]).reshape(-1, d)[:length]
            v = (_e4m3_values(s["v"][0, ids, h]) * s["v_scale"][0, ids, h, None, None]).reshape(-1, d)[:length]
            for lo in range(0, rows, 2048):
                hi = min(rows, lo + 2048)
                top = a + hi if m else a
                q = s["q"][t0 + lo:t0 + hi, h * G:(h + 1) * G].double()
                z = torch.einsum("thd,xd->htx", q, k[:top]) * d ** -0.5
                if m:
                    late = torch.arange(top, device="cuda")[None] > torch.arange(a + lo, a + hi, device="cuda")[:, None]
                    z = z.masked_fill(late, -math.inf)
                out[t0 + lo:t0 + hi, h * G:(h + 1) * G] = torch.einsum("htx,xd->thd", torch.softmax(z, -1), v[:top])
        t0 += rows
    return out


def _exact_rows(s, pool, scales, x, old, new):
    """A pool's unrounded codes and its scales once rows x [rows][hkv][d] are in: block by block."""
    codes, scale = _e4m3_values(s[pool][0]), s[scales][0].double()
    t0, slot = 0, s["slot"].tolist()
    for a, m in zip(old, new):
        t = 0
        while t < m:
            at = (a + t) % BS
            take, blk = min(BS - at, m - t), slot[t0 + t] // BS
            rows = x[t0 + t:t0 + t + take].transpose(0, 1)
            after = _power_of_two(rows.abs().amax((-1, -2)))
            if at:
                after = torch.maximum(after, scale[blk])
                codes[blk, :, :at] *= (scale[blk] / after.clamp(min=2.0 ** E_MIN))[:, None, None]
            codes[blk, :, at:at + take] = rows / after.clamp(min=2.0 ** E_MIN)[:, None, None]
            scale[blk] = after
            t += take
        t0 += m
    return codes[None], scale[None]


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

    q = make(s["q_new"], s["qw"])
    k, k_scale = _exact_rows(s, "k", "k_scale", make(s["k_new"], s["kw"]), old, new)
    v, v_scale = _exact_rows(s, "v", "v_scale", s["v_new"].double(), old, new)
    ring = None
    if W:
        ring = torch.zeros(s["n"], 1, case["hq"], W, d, dtype=torch.float64, device="cuda")
        t0 = 0
        for i, (o, m) in enumerate(zip(old, new)):
            keep = min(m, W)
            at = torch.arange(o + m - keep, o + m, device="cuda") % W
            ring[i, 0, :, at] = q[t0 + m - keep:t0 + m].transpose(0, 1)
            t0 += m
    return dict(q=q, k=k, k_scale=k_scale, v=v, v_scale=v_scale, ring=ring)


def _exact_expand(s, lens):
    W = s["case"]["W"]
    nw = W // BS + 1
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for i, L in enumerate(lens):
        p0 = (L - W) // BS
        for j, blk in enumerate(s["table"][i, p0:_blocks(L)].tolist()):
            rows = min(BS, L - (p0 + j) * BS)
            out[:, i * nw + j, :, :rows] = (_e4m3_values(s["k"][:, blk, :, :rows])
                                            * s["k_scale"][:, blk, :, None, None].double())
    return dict(k=out, table=None)


def _exact_compact(s, lens):
    case = s["case"]
    W, B, R, layers, hkv = case["W"], case["B"], case["R"], case["layers"], case["hkv"]
    found = {}
    li = torch.arange(layers, device="cuda")[:, None, None]
    hi = torch.arange(hkv, device="cuda")[None, :, None]
    for pool, scales in (("k", "k_scale"), ("v", "v_scale")):
        codes, scale = s[pool].clone(), s[scales].double()
        values = _e4m3_values(codes)
        used = 0
        for i, L in enumerate(lens):
            p0, ws = (L - W) // BS, L - W
            head = torch.arange(p0 * BS, ws, device="cuda").expand(layers, hkv, -1)
            tail = torch.arange(L - B, L, device="cuda").expand(layers, hkv, -1)
            src = torch.cat([head, ws + s["kept"][i].long(), tail], -1)
            blk = s["table"][i].long()[src // BS]
            x = _e4m3_values(codes[li, blk, hi, src % BS]) * s[scales][li, blk, hi].double()[..., None]
            for j in range(_blocks(src.shape[-1])):
                rows = x[:, :, j * BS:(j + 1) * BS]
                to = int(s["fresh"][used])
                scale[:, to] = _power_of_two(rows.abs().amax((-1, -2)))
                values[:, to, :, :rows.shape[2]] = rows / scale[:, to].clamp(min=2.0 ** E_MIN)[..., None, None]
                used += 1
        found[pool], found[scales] = values, scale
    return dict(found, table=None, freed=None, new_len=None)
