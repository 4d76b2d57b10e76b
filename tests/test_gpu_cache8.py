"""GPU tests of the 8-bit cache's operators against their plain forms in 64 bits.

Tolerances, before the first run (a rounding is off by at most half a step: e4m3 2^-4 of the value, or half a
subnormal step, 2^-10 of the scale; bf16 2^-8; f16 2^-11):
append   fp32 sums and products of one row (about 20 roundings of 2^-24, against the larger member of the
         rotated pair), then one rounding: |got - ref| <= 2^-4 |ref| + 2^-10 s + 2^-19 max|row|.  A scale may
         be the next one only where the block's largest value is within 2^-19 of the border.  Values, and keys
         without norm and rotation, are not computed with: their codes and scales are equal.
decode   logits: fp32 sums of exact products and two multiplications; with |logit| <= 40 and 128 terms below
         2^-11 of a weight.  A weight is rounded to f16 once (2^-11 of it, or 2^-40 of the split's largest).  One
         rounding of the output: |got - ref| <= 2^-8 |ref| + 2^-10 sum_x w_x |v_x| + 2^-30 max|v|.
chunk    that of kara_chunk_attention, whose arithmetic it is but for 2^-17 of a query's largest element in the small
         ones: 2^-8 |ref| + (2^-8 + 2^-10) sum_x w_x |v_x| against 64 bits; twice that against kara_chunk_attention
         over a bf16 cache of the same values, which holds them exactly (and whose output stands for the sums, 2 % off).
expand, compact   equal: code times scale is exact, and a code is rounded once from an exact quotient."""

import numpy as np
import pytest
import torch

from _cache8 import (BS, dense, divide, plain_compact, plain_decode, quantise, random_pool, round_code, runs, scale_of,
                     source_rows, value)
from _gpu import lib
from _newtokens import blocks, make_tables, plain_chunk, plain_extend, plain_turn

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).to(DEV).contiguous()


def error_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def status(kara, err):
    return kara.kara_get_error(err)


# ---- append ---------------------------------------------------------------------

class Append:
    """Random inputs of an append: n sequences, `new` tokens each after `old` cached ones."""

    def __init__(self, seed, old, new, hq, hkv, d, norm=True, rot=None, inter=False, W=0, pad=0, layers=2, fused=True):
        self.kara = lib()
        g = torch.Generator().manual_seed(seed)
        old, new = np.asarray(old, np.int32), np.asarray(new, np.int32)
        n, rows = len(old), int(new.sum()) + pad
        self.n, self.rows, self.hq, self.hkv, self.d, self.norm, self.inter, self.W = n, rows, hq, hkv, d, norm, inter, W
        self.old, self.new = old, new
        self.rot = d if rot is None else rot
        nb = int(blocks(old + new).sum()) + 3
        bt, fresh = make_tables(old, int(blocks(old + new).max()) + 1, nb, seed)
        _, q_start, ln, self.slot, self.seq, self.pos, _ = plain_extend(old, new, bt, fresh, rows)
        self.q_start, self.len = q_start, ln
        shape = (layers, nb, hkv, BS, d)
        self.k0, self.ks0 = random_pool(shape, seed + 1)
        self.v0, self.vs0 = random_pool(shape, seed + 2)
        width = (hq + 2 * hkv) * d + (8 if fused else 0)
        mag = 2.0 ** torch.randint(-3, 4, (rows, 1), generator=g)
        self.qkv = (torch.randn(rows, width, generator=g) * mag).bfloat16()
        self.qw = (1 + 0.2 * torch.randn(d, generator=g)).bfloat16() if norm else None
        self.kw = (1 + 0.2 * torch.randn(d, generator=g)).bfloat16() if norm else None
        self.shift = torch.randint(0, 100, (n,), generator=g).int()
        npos = int(self.len.max()) + 200
        if self.rot:
            ang = torch.arange(npos, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(self.rot // 2) / (self.rot / 2))
            self.cs = torch.cat([ang.cos(), ang.sin()], 1).float()
        else:
            self.cs = None

    def split(self, x):
        hq, hkv, d = self.hq, self.hkv, self.d
        return (x[:, :hq * d].unflatten(1, (hq, d)), x[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
                x[:, (hq + hkv) * d:(hq + 2 * hkv) * d].unflatten(1, (hkv, d)))

    def buffers(self):
        dev = lambda x: None if x is None else x.to(DEV)  # noqa: E731
        b = dict(k=dev(self.k0).clone(), v=dev(self.v0).clone(), ks=dev(self.ks0).clone(), vs=dev(self.vs0).clone(),
                 qkv=dev(self.qkv), q_out=torch.full((self.rows, self.hq, self.d), 7.0, dtype=torch.bfloat16, device=DEV),
                 ring=torch.full((self.n, 2, self.hq, self.W, self.d), 9.0, dtype=torch.bfloat16, device=DEV)
                 if self.W else None, err=error_word())
        kara = self.kara
        b["rope"] = kara.rope(dev(self.cs), dev(self.qw), dev(self.kw), 1e-6, self.inter, dev(self.shift))
        b["t"] = kara.tokens(i32(self.q_start), i32(self.len), torch.as_tensor(self.slot).to(DEV), i32(self.seq),
                             i32(self.pos))
        b["c"] = kara.cache8(b["k"], b["v"], b["ks"], b["vs"], self.hq)
        return b

    def run(self, layer=1, stream=None):
        b = self.buffers()
        q, k, v = self.split(b["qkv"])
        self.kara.kara_append_kv8(b["c"], layer, b["t"], b["rope"], q, k, v, b["q_out"], b["err"], b["ring"], stream)
        st = status(self.kara, b["err"])
        return st, {x: None if b[x] is None else b[x].cpu() for x in ("k", "v", "ks", "vs", "q_out", "ring")}

    def turned(self):
        """Keys in float64, and each row's largest magnitude before the rotation."""
        _, k, _ = self.split(self.qkv)
        r = torch.as_tensor(self.pos).long() + self.shift[torch.as_tensor(self.seq).clamp(min=0).long()].long()
        return plain_turn(k, self.kw, 1e-6, self.cs, r.clamp(min=0), self.inter)


def check_store(codes, scale, codes0, scale0, x, slot, exact, ok=None):
    """One layer's pool after rows x [rows][hkv][d] went to `slot`: scales, rounded rows, rows ahead, the rest."""
    want, want_s = codes0.clone(), scale0.clone()
    fine = torch.isfinite(x)
    x = torch.where(fine, x, float("nan"))
    for t, m, blk, at in runs(slot, ok):
        rows = x[t:t + m].transpose(0, 1)                      # [hkv][m][d]
        top = torch.nan_to_num(rows, nan=0.0).abs().amax((-1, -2))
        old = scale0[blk].double().abs() if at else torch.zeros_like(top)
        got_s = scale[blk].double().abs()
        s = torch.maximum(old, scale_of(top))
        if not exact:   # at the border either neighbour will do
            lo, hi = (torch.maximum(old, scale_of(top * (1 + e))) for e in (-2.0 ** -19, 2.0 ** -19))
            assert ((got_s == lo) | (got_s == hi)).all(), (blk, got_s, lo, hi)
            s = got_s
        nan = torch.isnan(rows).any(-1).any(-1) | (torch.signbit(scale0[blk]) if at else False)
        want_s[blk] = torch.where(nan, -s, s).float()
        if at:
            ratio = torch.where(s > 0, old / torch.where(s > 0, s, 1.0), 1.0)
            moved = round_code(value(codes0[blk, :, :at]) * ratio[:, None, None])
            want[blk, :, :at] = torch.where((ratio < 1)[:, None, None], moved, codes0[blk, :, :at])
        if exact:
            want[blk, :, at:at + m] = divide(rows, s[:, None, None])
        else:
            got = value(codes[blk, :, at:at + m]) * s[:, None, None]
            tol = 2.0 ** -4 * rows.abs() + 2.0 ** -10 * s[:, None, None] + 2.0 ** -19 * rows.abs().amax(-1, keepdim=True)
            assert torch.equal(torch.isnan(got), torch.isnan(rows))
            assert torch.nan_to_num((got - rows).abs() - tol, nan=-1.0).max() <= 0, blk
            want[blk, :, at:at + m] = codes[blk, :, at:at + m]
    assert torch.equal(scale, want_s) and torch.equal(torch.signbit(scale), torch.signbit(want_s))
    assert torch.equal(codes, want)


APPENDS = [
    # old, new, heads, D, norm, rot, interleaved, ring, padding
    ([0], [1], 4, 2, 64, True, None, False, 0, 0),
    ([255], [1], 4, 2, 64, True, None, False, 64, 3),
    ([3, 15, 16, 0, 40], [1, 1, 1, 1, 1], 40, 8, 128, True, None, False, 128, 0),
    ([3, 15, 16, 0, 40], [14, 1, 33, 17, 0], 14, 2, 128, True, 64, True, 64, 5),
    ([5, 0, 31], [100, 16, 2], 8, 8, 64, False, 32, False, 0, 0),
    ([0, 7], [700, 41], 18, 3, 128, True, None, True, 64, 9),
    ([1] * 90, [7] * 90, 4, 2, 64, False, 16, False, 0, 0),
    ([9, 100], [300, 333], 5, 1, 128, True, 0, False, 0, 1),
    # long calls, of every kind of rotation
    ([3, 0], [600, 90], 8, 2, 64, True, None, True, 64, 2),
    ([3, 0], [600, 90], 8, 2, 128, True, 64, True, 0, 0),
    ([2] * 80, [9] * 80, 8, 2, 128, True, 32, False, 64, 0),
    ([0, 33], [500, 300], 6, 3, 64, True, 32, False, 0, 0),
    ([0, 33], [500, 300], 40, 8, 128, True, None, False, 64, 0),
    ([0, 33], [500, 300], 40, 8, 128, False, None, False, 0, 0),
]


@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append_matches_plain(case):
    """Runs of one to sixteen rows, short and long calls, norms, both pairings, partial rotations, padding."""
    old, new, hq, hkv, d, norm, rot, inter, W, pad = APPENDS[case]
    a = Append(case + 10, old, new, hq, hkv, d, norm, rot, inter, W, pad)
    st, got = a.run()
    assert st == 0
    assert torch.equal(got["k"][0], a.k0[0]) and torch.equal(got["vs"][0], a.vs0[0])   # the other layer
    _, _, v = a.split(a.qkv)
    check_store(got["v"][1], got["vs"][1], a.v0[1], a.vs0[1], v.double(), a.slot, True)
    check_store(got["k"][1], got["ks"][1], a.k0[1], a.ks0[1], a.turned(), a.slot, not norm and a.rot == 0)


@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append_queries_like_the_bf16_append(case):
    """Queries and ring have the bits that kara_append_kv gives them; padding rows stay."""
    old, new, hq, hkv, d, norm, rot, inter, W, pad = APPENDS[case]
    a = Append(case + 10, old, new, hq, hkv, d, norm, rot, inter, W, pad)
    st, got = a.run()
    b = a.buffers()
    q, k, v = a.split(b["qkv"])
    pool = torch.zeros(a.k0.shape, dtype=torch.bfloat16, device=DEV)
    a.kara.kara_append_kv(a.kara.cache(pool, pool.clone(), hq), 1, b["t"], b["rope"], q, k, v, b["q_out"], b["err"],
                          b["ring"])
    assert st == status(a.kara, b["err"]) == 0
    assert torch.equal(got["q_out"], b["q_out"].cpu())
    assert (got["ring"] is None and b["ring"] is None) or torch.equal(got["ring"], b["ring"].cpu())


def test_append_grows_a_block_token_by_token():
    """Sixteen single tokens of growing magnitude: the scale follows, the rows ahead are rounded anew each time."""
    kara = lib()
    g = torch.Generator().manual_seed(3)
    x = torch.randn(16, 2, 64, generator=g).bfloat16() * 2.0 ** torch.arange(-20, 12, 2)[:, None, None]
    x = x.bfloat16()
    k = torch.full((1, 1, 2, BS, 64), 0x55, dtype=torch.uint8, device=DEV)
    v, err = k.clone(), error_word()
    ks, vs = (torch.full((1, 1, 2), float("nan"), device=DEV) for _ in range(2))   # never read
    c = kara.cache8(k, v, ks, vs, 2)
    codes, scale = torch.full((2, BS, 64), 0x55, dtype=torch.uint8), torch.zeros(2, dtype=torch.float64)
    for i in range(16):
        t = kara.tokens(i32([0, 1]), i32([i + 1]), torch.tensor([i], device=DEV), i32([0]), i32([i]))
        row = x[i:i + 1].to(DEV)
        kara.kara_append_kv8(c, 0, t, kara.rope(None), row, row, row, torch.empty_like(row), err)
        s = torch.maximum(scale, scale_of(x[i].double().abs().amax(-1)))
        ratio = (scale / s)[:, None, None]
        codes[:, :i] = torch.where(ratio < 1, round_code(value(codes[:, :i]) * ratio), codes[:, :i])
        codes[:, i] = divide(x[i].double(), s[:, None])
        scale = s
        assert torch.equal(k[0, 0].cpu(), codes) and torch.equal(v[0, 0].cpu(), codes), i
        assert torch.equal(ks[0, 0].cpu().double(), scale) and torch.equal(vs[0, 0].cpu().double(), scale), i
    assert status(kara, err) == 0


@pytest.mark.parametrize("what", ["nan", "inf", "all nan", "zero", "tiny", "huge", "border"])
@pytest.mark.parametrize("d", [64, 128])
def test_append_special_values(what, d):
    """Values that are not finite become NaN and mark the block; zeros, subnormals, the largest and 448 2^e."""
    a = Append(5, [4, 0], [3, 30], 4, 2, d, norm=False, rot=0)
    _, k, v = a.split(a.qkv)
    for x in (k, v):
        if what == "nan":
            x[1, 0, 5] = float("nan")
            x[20, 1, 7] = -float("nan")
        elif what == "inf":
            x[1, 0, 5], x[9, 1, 0] = float("inf"), -float("inf")
        elif what == "all nan":
            x[3:19] = float("nan")
        elif what == "zero":
            x[:] = 0.0
            x[5, 0] = -0.0
        elif what == "tiny":
            x[:] = (x.float() * 2.0 ** -128).bfloat16()
        elif what == "huge":
            x[2] = torch.finfo(torch.bfloat16).max
            x[12] = (x[12].float() * 2.0 ** 80).bfloat16()
        else:
            x[:] = x.clamp(-1, 1)
            x[0, 0, 0], x[4, 1, 3], x[25, 0, 2] = 7.0, 7.03125, -448.0
    st, got = a.run()
    assert st == 0
    check_store(got["v"][1], got["vs"][1], a.v0[1], a.vs0[1], v.double(), a.slot, True)
    check_store(got["k"][1], got["ks"][1], a.k0[1], a.ks0[1], k.double(), a.slot, True)
    if what in ("nan", "inf", "all nan"):
        assert torch.signbit(got["ks"][1]).any()


def test_append_keeps_a_mark_and_continues_an_empty_scale():
    """A block marked as holding a NaN stays so; one whose rows ahead are all zeros takes the new rows' scale."""
    a = Append(6, [4, 4], [2, 2], 4, 2, 64, norm=False, rot=0)
    b0, b1 = (int(a.slot[t]) // BS for t in (0, 2))
    a.k0[1, b0, 0, 1, 3] = 0x7f
    a.ks0[1, b0, 0] *= -1
    a.k0[1, b1, :, :4] = 0
    a.ks0[1, b1] = 0.0
    st, got = a.run()
    _, k, v = a.split(a.qkv)
    assert st == 0
    check_store(got["k"][1], got["ks"][1], a.k0[1], a.ks0[1], k.double(), a.slot, True)
    assert got["ks"][1, b0, 0] < 0 and got["k"][1, b0, 0, 1, 3] == 0x7f and (got["ks"][1, b1] > 0).all()


@pytest.mark.parametrize("what", ["slot past the pool", "slot negative", "sequence", "position", "past the table"])
@pytest.mark.parametrize("long", [False, True])
def test_append_skips_bad_rows(what, long):
    """A bad row, the last of its sequence, is recorded and skipped; everything else is as without it."""
    kara = lib()
    a = Append(7, [20, 3], [600, 9] if long else [6, 9], 8, 2, 128, norm=False, rot=0 if what != "past the table" else 16)
    bad = int(a.new[0]) - 1
    want = kara.EBADBLOCK if "slot" in what else kara.EINVAL
    if what == "slot past the pool":
        a.slot[bad] = a.k0.shape[1] * BS
    elif what == "slot negative":
        a.slot[bad] = -5
    elif what == "sequence":
        a.seq[bad] = 2
    elif what == "position":
        a.pos[bad] = -1
    else:
        a.shift[1] = 10 ** 6
    ok = np.ones(a.rows, bool)
    if what == "past the table":
        ok[a.q_start[1]:] = False
    else:
        ok[bad] = False
    st, got = a.run()
    assert st == want
    _, k, v = a.split(a.qkv)
    check_store(got["v"][1], got["vs"][1], a.v0[1], a.vs0[1], v.double(), a.slot, True, ok)
    assert (got["q_out"][~torch.as_tensor(ok)] == 7.0).all() and not (got["q_out"][torch.as_tensor(ok)] == 7.0).all()


def test_append_into_strided_pools():
    """Pools that are views of larger ones: what lies between is not touched."""
    kara = lib()
    a = Append(8, [5, 30], [40, 3], 8, 2, 128, norm=False, rot=0)
    big = [torch.full((3, a.k0.shape[1] + 2, 4, BS, 128), 0xa5, dtype=torch.uint8, device=DEV) for _ in range(2)]
    k, v = (x[:2, 1:-1, 1:3] for x in big)
    k.copy_(a.k0.to(DEV)), v.copy_(a.v0.to(DEV))
    b = a.buffers()
    q, kn, vn = a.split(b["qkv"])
    kara.kara_append_kv8(kara.cache8(k, v, b["ks"], b["vs"], 8), 1, b["t"], b["rope"], q, kn, vn, b["q_out"], b["err"])
    assert status(kara, b["err"]) == 0
    _, _, x = a.split(a.qkv)
    check_store(v[1].cpu(), b["vs"][1].cpu(), a.v0[1], a.vs0[1], x.double(), a.slot, True)
    for y in big:
        y[:2, 1:-1, 1:3] = 0xa5
        assert (y == 0xa5).all()


# ---- decode ---------------------------------------------------------------------

def decode_case(seed, lengths, hq, hkv, d, layers=2, spread=2, qmag=1.5):
    g = torch.Generator().manual_seed(seed)
    lengths = np.asarray(lengths, np.int32)
    nb = int(blocks(lengths).sum()) + 2
    bt, _ = make_tables(lengths, max(1, int(blocks(lengths).max())) + 1, nb, seed)
    k, ks = random_pool((layers, nb, hkv, BS, d), seed + 1, min(spread, 1))
    v, vs = random_pool((layers, nb, hkv, BS, d), seed + 2, spread)
    q = (qmag * torch.randn(len(lengths), hq, d, generator=g)).bfloat16()
    return lengths, bt, k, ks, v, vs, q


def run_decode(lengths, bt, k, ks, v, vs, q, layer=1, stream=None):
    kara = lib()
    keep = [x.to(DEV) for x in (k, v, ks, vs)]
    c = kara.cache8(*keep, q.shape[1])
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(kara.kara_decode8_workspace_size(c, len(lengths), bt.shape[1]), dtype=torch.uint8, device=DEV)
    err = error_word()
    kara.kara_decode_attention8(c, layer, i32(lengths), i32(bt), q.to(DEV), out, ws, err, stream)
    return status(kara, err), out.cpu()


def check_decode(out, lengths, bt, k, ks, v, vs, q, layer=1):
    kv = dense(k, ks), dense(v, vs)
    ref = plain_decode(q, kv, layer, bt, lengths)
    tol = (2.0 ** -8 * ref.abs() + 2.0 ** -10 * plain_decode(q, kv, layer, bt, lengths, True)
           + 2.0 ** -30 * torch.nan_to_num(kv[1], nan=0.0).abs().max())
    bad = (out.double() - ref).abs() > tol
    assert not bad.any(), ((out.double() - ref).abs() / tol).max()


@pytest.mark.parametrize("hq,hkv", [(8, 8), (4, 2), (6, 2), (32, 8), (40, 8), (12, 2), (14, 2), (8, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_matches_plain(hq, hkv, d):
    """Every group size; lengths of zero, one, around blocks, stages and splits."""
    c = decode_case(hq * 7 + d, [0, 1, 15, 16, 17, 31, 33, 64, 65, 1023, 1024, 1025, 2500, 0, 700], hq, hkv, d)
    st, out = run_decode(*c)
    assert st == 0
    assert (out[[0, 13]] == 0).all()
    check_decode(out, *c)


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (40, 8, 128), (8, 1, 128)])
@pytest.mark.parametrize("lengths", [[0, 1, 17, 255, 256], [1024, 0, 257, 3, 2048], [1], [5000],
                                     [700, 511, 512, 513, 2049, 255, 256, 257, 1], [1008] * 45, [1024, 1025] * 22])
def test_decode_splits(lengths, hq, hkv, d):
    """Splits of 256, 512 and 1024 keys: sequences of one, which write their outputs at once, alone (a table that
    holds no more) and beside longer ones."""
    case = decode_case(len(lengths) + hq, lengths, hq, hkv, d)
    st, out = run_decode(*case)
    assert st == 0
    check_decode(out, *case)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_far_apart_scales(d):
    """Blocks whose magnitudes differ by up to 2^24, and queries with a few large elements."""
    lengths, bt, k, ks, v, vs, q = decode_case(5, [1500, 40, 300], 8, 2, d, spread=12)
    q[:, :, 3] *= 64
    st, out = run_decode(lengths, bt, k, ks, v, vs, q)
    assert st == 0
    check_decode(out, lengths, bt, k, ks, v, vs, q)


def test_decode_one_key_takes_nearly_all():
    """A first key with nearly all the weight and a value of zero: the others' shares, 2^-20 and less, keep their digits."""
    d, hkv = 128, 2
    lengths, bt, k, ks, v, vs, q = decode_case(6, [1000, 2000], 4, hkv, d, qmag=0.05)
    for s in range(2):
        b = int(bt[s, 0])
        x = dense(k[1, b], ks[1, b])
        x[:, 0] = 0.0
        x[:, 0, 0] = 64.0
        k[1, b], ks[1, b] = quantise(x)
        v[1, b, :, 0] = 0
    q[:, :, 0] = 3.0    # logit 17 for the first key, about 0 for the others
    st, out = run_decode(lengths, bt, k, ks, v, vs, q)
    assert st == 0
    check_decode(out, lengths, bt, k, ks, v, vs, q)
    assert (out != 0).all()


def test_decode_ignores_what_lies_past_the_end():
    """NaN codes and marks in the rows past a sequence's end, and in blocks it does not list, do not count."""
    lengths, bt, k, ks, v, vs, q = decode_case(8, [5, 37, 1029], 10, 2, 128)
    want = run_decode(lengths, bt, k, ks, v, vs, q)[1]
    for s, L in enumerate(lengths):
        b = int(bt[s, blocks(L) - 1])
        k[:, b, :, L % BS:] = 0x7f
        v[:, b, :, L % BS:] = 0xff
        ks[:, b] *= -1
        vs[:, b] *= -1
    spare = [b for b in range(k.shape[1]) if b not in bt]
    k[:, spare], v[:, spare], vs[:, spare] = 0x7f, 0x7f, float("nan")
    st, out = run_decode(lengths, bt, k, ks, v, vs, q)
    assert st == 0 and torch.equal(out, want)


def test_decode_shows_a_nan():
    """A cached NaN reaches the rows that see it, of its own KV head and sequence only."""
    lengths, bt, k, ks, v, vs, q = decode_case(9, [40, 40], 4, 2, 64)
    want = run_decode(lengths, bt, k, ks, v, vs, q)[1]
    b = int(bt[0, 1])
    v[1, b, 1, 3, 7] = 0x7f
    vs[1, b, 1] *= -1
    st, out = run_decode(lengths, bt, k, ks, v, vs, q)
    assert st == 0 and torch.isnan(out[0, 2:, 7]).all()
    out[0, 2:, 7] = want[0, 2:, 7]
    assert torch.equal(out, want)


def test_decode_bad_blocks_and_lengths():
    """A block outside the pool counts as zeros; a length out of range gives zeros and an error."""
    kara = lib()
    lengths, bt, k, ks, v, vs, q = decode_case(10, [100, 300, 50, 20], 8, 2, 128)
    bt[1, 3], bt[1, 18] = -7, k.shape[1]
    st, out = run_decode(lengths, bt, k, ks, v, vs, q)
    assert st == kara.EBADBLOCK
    check_decode(out, lengths, bt, k, ks, v, vs, q)
    bt2 = np.where(bt < 0, 0, np.minimum(bt, k.shape[1] - 1))
    for L in (-1, bt.shape[1] * BS + 1):
        bad = lengths.copy()
        bad[2] = L
        st, out = run_decode(bad, bt2, k, ks, v, vs, q)
        assert st == kara.EINVAL and (out[2] == 0).all()
        bad[2] = 0
        check_decode(out, bad, bt2, k, ks, v, vs, q)


def test_decode_strided_pools_and_long_table():
    """Pools that are views of larger ones, and a table far wider than the lengths."""
    lengths, bt, k, ks, v, vs, q = decode_case(11, [70, 1100], 10, 2, 64)
    wide = np.full((2, 4000), -1, np.int32)
    wide[:, :bt.shape[1]] = bt
    kara = lib()
    big = [torch.full((2, k.shape[1] + 3, 5, BS, 64), 0x7f, dtype=torch.uint8, device=DEV) for _ in range(2)]
    kk, vv = (x[:, 2:-1, 1:3] for x in big)
    kk.copy_(k.to(DEV)), vv.copy_(v.to(DEV))
    sc = ks.to(DEV), vs.to(DEV)
    c = kara.cache8(kk, vv, *sc, 10)
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(kara.kara_decode8_workspace_size(c, 2, 4000), dtype=torch.uint8, device=DEV)
    err = error_word()
    kara.kara_decode_attention8(c, 1, i32(lengths), i32(wide), q.to(DEV), out, ws, err)
    # (the width decides on the splits, whose partial sums are added in fp32: not the bits of a narrow table)
    assert status(kara, err) == 0
    check_decode(out.cpu(), lengths, bt, k, ks, v, vs, q)


# ---- chunk attention ------------------------------------------------------------

def chunk_case(seed, lengths, n_new, hq, hkv, d, layers=1, pad=0, qmag=1.5):
    """Lengths include the new tokens; rows of a block where no token lives hold NaN, in marked blocks."""
    g = torch.Generator().manual_seed(seed)
    lengths, bt, k, ks, v, vs, _ = decode_case(seed, lengths, 1, 1, 64)
    nb = k.shape[1]
    k, ks = random_pool((layers, nb, hkv, BS, d), seed + 1, 1)
    v, vs = random_pool((layers, nb, hkv, BS, d), seed + 2)
    used = np.zeros((nb, BS), bool)
    for s, L in enumerate(lengths):
        for x in range(int(L)):
            used[bt[s, x // BS], x % BS] = True
    for codes, scale in ((k, ks), (v, vs)):
        codes.permute(1, 3, 0, 2, 4)[torch.from_numpy(~used)] = 0xff
        scale[:, torch.from_numpy(~used.all(1))] *= -1
    q_start = np.concatenate([[0], np.cumsum(n_new)]).astype(np.int32)
    q = (qmag * torch.randn(int(q_start[-1]) + pad, hq, d, generator=g)).bfloat16()
    return dict(q=q, k=k, v=v, ks=ks, vs=vs, bt=bt, q_start=q_start, lengths=lengths)


def chunk_descriptor(kara, d):
    rows = d["q"].shape[0]
    z, z4 = (torch.empty(rows, dtype=t, device=DEV) for t in (torch.int64, torch.int32))
    return kara.tokens(i32(d["q_start"]), i32(d["lengths"]), z, z4, z4)


def run_chunk(d, layer=0, bf16=False, pools=None, fill=77.0):
    """The output over the 8-bit cache, or over a bf16 cache of its values."""
    kara, hq = lib(), d["q"].shape[1]
    t, out, err = chunk_descriptor(kara, d), torch.full(d["q"].shape, fill, dtype=torch.bfloat16, device=DEV), error_word()
    if bf16:
        keep = [dense(d[x], d[x + "s"]).bfloat16().to(DEV) for x in "kv"]
        c, size, call = kara.cache(*keep, hq), kara.kara_chunk_workspace_size, kara.kara_chunk_attention
    else:
        keep = [d[x].to(DEV) for x in ("k", "v", "ks", "vs")] if pools is None else pools
        c, size, call = kara.cache8(*keep, hq), kara.kara_chunk8_workspace_size, kara.kara_chunk_attention8
    ws = torch.empty(size(c, t.n, t.rows), dtype=torch.uint8, device=DEV)
    call(c, layer, t, i32(d["bt"]), d["q"].to(DEV), out, ws, err)
    return status(kara, err), out.cpu()


def near_bf16(c, layer, got):
    """Whether the output is as near to the bf16 cache's as two results within the tolerance are."""
    st, want = run_chunk(c, layer, bf16=True)
    _, size = run_chunk(dict(c, v=c["v"] & 0x7f), layer, bf16=True)
    want, size = want.double(), size.double()
    off = (got.double() - want).abs() - 1.02 * (2.0 ** -7 * want.abs() + (2.0 ** -7 + 2.0 ** -9) * size)
    pad = want == 77.0
    assert st == 0 and torch.equal(got.double()[pad], want[pad])
    assert off[~pad].max() <= 0, off[~pad].max()


def same_bits(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


CHUNKS = [([1, 17, 128, 129, 300, 64, 513, 255, 700], [1, 17, 1, 129, 4, 0, 140, 255, 33]),
          ([2500], [1]), ([5000, 3], [3, 3]), ([900] * 40, [1] * 40), ([1500], [1500]), ([16] * 130, [16] * 130)]


@pytest.mark.parametrize("case", range(len(CHUNKS)))
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (4, 2, 128), (6, 2, 64), (8, 2, 128), (10, 2, 128), (7, 1, 128),
                                      (16, 2, 64)])
def test_chunk_is_near_the_bf16_cache(case, hq, hkv, d):
    """Every group size and head dim, single tokens to whole prompts, on both caches."""
    lengths, n_new = CHUNKS[case]
    c = chunk_case(case * 31 + hq, lengths, n_new, hq, hkv, d, layers=2, pad=3)
    for layer in (0, 1):
        st, got = run_chunk(c, layer)
        assert st == 0 and torch.isfinite(got).all() and (got[-3:] == 77.0).all()
        near_bf16(c, layer, got)


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (10, 2, 128)])
def test_chunk_matches_plain(hq, hkv, d):
    """Against 64 bits: the weights' rounding to bf16 and the output's."""
    c = chunk_case(hq, CHUNKS[0][0], CHUNKS[0][1], hq, hkv, d, pad=2)
    st, got = run_chunk(c)
    kv = [dense(c[x], c[x + "s"]) for x in "kv"]
    ref = plain_chunk(c["q"], *kv, 0, c["bt"], c["q_start"], c["lengths"])
    size = plain_chunk(c["q"], *kv, 0, c["bt"], c["q_start"], c["lengths"], absolute=True)
    n = int(c["q_start"][-1])
    lim = (ref.abs() * 2.0 ** -8 + size * (2.0 ** -8 + 2.0 ** -10))[:n]
    assert st == 0 and ((got.double() - ref).abs()[:n] <= lim).all()


def test_chunk_scales_at_their_limits():
    """Scales of 2^-63, 2^63 and 0, above the range of one product too; queries of zeros and tiny ones."""
    c = chunk_case(4, [200, 333, 100], [60, 200, 1], 8, 2, 128, qmag=0.01)
    for i, e in enumerate((-63, -40, 5, 7, 8, 9, 30)):
        c["ks"][0, int(c["bt"][0, i])] = 2.0 ** e if e < 9 else 2.0 ** -20
        c["vs"][0, int(c["bt"][1, i])] = 2.0 ** e
    c["vs"][0, int(c["bt"][2, 1])] = 2.0 ** 63
    c["vs"][0, int(c["bt"][2, 2])] = 0.0
    c["v"][0, int(c["bt"][2, 2])] = 0
    c["ks"][0, int(c["bt"][0, 9])] = 0.0
    c["k"][0, int(c["bt"][0, 9])] = 0
    c["q"][5] = 0.0
    c["q"][6] *= 2.0 ** -60
    st, got = run_chunk(c)
    assert st == 0 and torch.isfinite(got).all()
    near_bf16(c, 0, got)


@pytest.mark.parametrize("pool", ["k", "v"])
@pytest.mark.parametrize("at", [3, 55, 120])
def test_chunk_nan_reaches_those_who_see_it(pool, at):
    """A NaN among the earlier tokens, or among the chunk's own: rows before it keep their bits, rows behind it
    show it, in its dim (a value) or altogether (a key), of its KV head."""
    c = chunk_case(9, [150, 300], [100, 290], 4, 2, 128)
    want = run_chunk(c)[1]
    b = int(c["bt"][0, at // BS])
    c[pool][0, b, 1, at % BS, 7] = 0x7f
    c[pool + "s"][0, b, 1] = -c[pool + "s"][0, b, 1].abs()
    st, got = run_chunk(c)
    assert st == 0
    first = max(0, at - 50)     # the row of the first token that sees it
    if pool == "v":
        assert torch.isnan(got[first:100, 2:, 7]).all()
        got[first:100, 2:, 7] = want[first:100, 2:, 7]
    else:
        assert torch.isnan(got[first:100, 2:]).all()
        got[first:100, 2:] = want[first:100, 2:]
    assert same_bits(got, want)


def test_chunk_bad_lengths_and_blocks():
    """The refusals on the device of kara_chunk_attention."""
    kara = lib()
    c = chunk_case(61, [100, 90, 80, 70], [10, 20, 30, 5], 4, 2, 64)
    want = run_chunk(c)[1]
    for L in (19, BS * c["bt"].shape[1] + 1):
        bad = dict(c, lengths=c["lengths"].copy())
        bad["lengths"][1] = L
        st, got = run_chunk(bad)
        assert st == kara.EINVAL and (got[10:30] == 0).all()
        assert same_bits(got[:10], want[:10]) and same_bits(got[30:], want[30:])
    for bid in (-1, c["k"].shape[1]):
        bad = dict(c, bt=c["bt"].copy())
        bad["bt"][2, 1] = bid
        st, got = run_chunk(bad)
        assert st == kara.EBADBLOCK and same_bits(got[:30], want[:30]) and same_bits(got[60:], want[60:])
        pools = [torch.cat([bad[x], torch.zeros_like(bad[x][:, :1])], 1) for x in ("k", "v", "ks", "vs")]
        bad["bt"][2, 1] = c["k"].shape[1]       # a block of zeros
        assert same_bits(got, run_chunk(dict(bad, **dict(zip(("k", "v", "ks", "vs"), pools))))[1])
    for qs in ([0, 10, 5, 60, 65], [0, 10, 30, 60, 900], [-3, 10, 30, 60, 65]):
        assert run_chunk(dict(c, q_start=np.array(qs, np.int32)))[0] == kara.EINVAL


def test_chunk_nothing_to_do_and_strided_pools():
    c = chunk_case(71, [50, 60], [0, 0], 4, 2, 64, pad=4)
    st, got = run_chunk(c)
    assert st == 0 and (got == 77.0).all()
    c = chunk_case(41, [300, 77], [50, 77], 8, 2, 128, layers=2)
    L, nb, hkv, _, D = c["k"].shape
    big = [torch.full((L + 1, nb, hkv + 3, BS, D), 0x7f, dtype=torch.uint8, device=DEV) for _ in range(2)]
    k, v = (x[:L, :, 1:1 + hkv] for x in big)
    k.copy_(c["k"]), v.copy_(c["v"])
    for layer in (0, 1):
        st, got = run_chunk(c, layer, pools=[k, v, c["ks"].to(DEV), c["vs"].to(DEV)])
        assert st == 0 and same_bits(got, run_chunk(c, layer)[1])


@pytest.mark.parametrize("lengths,n_new,hq,hkv,d", [
    ([4096 + 512] * 12, [512] * 12, 8, 4, 128), ([700 + 3 * i for i in range(200)], [1 + i % 5 for i in range(200)], 4, 2, 64),
    ([3000, 20, 9000], [2900, 20, 40], 8, 2, 128), ([40] * 1500, [2] * 1500, 4, 2, 128)])
def test_chunk_large_calls(lengths, n_new, hq, hkv, d):
    """Whole items dealt round, many sequences, partials that are joined, several times over."""
    c = chunk_case(len(lengths), lengths, n_new, hq, hkv, d)
    want = run_chunk(c)[1]
    near_bf16(c, 0, want)
    for _ in range(3):
        st, got = run_chunk(c)
        assert st == 0 and same_bits(got, want)


# ---- bounded waits --------------------------------------------------------------

def test_stalled_attention_times_out(monkeypatch):
    """With copies that are never issued both attentions report KARA_ETIMEOUT, and the next call is right."""
    kara = lib()
    dc = decode_case(3, [600, 40], 8, 2, 128)
    cc = chunk_case(5, [300, 500], [200, 3], 8, 2, 128)
    want = run_chunk(cc)[1]
    monkeypatch.setenv("KARA_DEBUG_STALL", "1")
    assert run_decode(*dc)[0] == kara.ETIMEOUT
    assert run_chunk(cc)[0] == kara.ETIMEOUT
    monkeypatch.delenv("KARA_DEBUG_STALL")
    st, out = run_decode(*dc)
    assert st == 0
    check_decode(out, *dc)
    st, got = run_chunk(cc)
    assert st == 0 and same_bits(got, want)


# ---- expand and compact ---------------------------------------------------------

def window_case(seed, lengths, W, hkv, d, layers, extra=0):
    lengths = np.asarray(lengths, np.int32)
    nb = int(blocks(lengths).sum()) + extra
    bt, left = make_tables(lengths, int(blocks(lengths).max()) + 1, nb, seed)
    k, ks = random_pool((layers, nb, hkv, BS, d), seed + 1)
    v, vs = random_pool((layers, nb, hkv, BS, d), seed + 2)
    return lengths, bt, left, k, ks, v, vs


@pytest.mark.parametrize("W,hkv,d,layers,lengths", [
    (64, 2, 64, 1, [64]), (64, 2, 128, 3, [65, 79, 80, 300]), (512, 8, 128, 2, [512, 700, 1000]),
    (16, 1, 64, 5, [16, 17, 31, 32]), (192, 3, 64, 40, [200, 333])])
@pytest.mark.parametrize("values", [False, True])
def test_expand_matches_plain(W, hkv, d, layers, lengths, values):
    """The windows' rows in bf16, zeros past the end; other blocks and entries stay."""
    kara = lib()
    lengths, bt, _, k, ks, v, vs = window_case(W + d, lengths, W, hkv, d, layers)
    n, nw = len(lengths), W // BS + 1
    k[0, int(bt[0, blocks(lengths[0]) - 1]), 0, 0, 0] = 0x7f
    shape = (layers, n * nw + 1, hkv, BS, d)
    ko, vo = (torch.full(shape, 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    keep = [x.to(DEV) for x in (k, v, ks, vs)]
    table, err = torch.full(bt.shape, -9, dtype=torch.int32, device=DEV), error_word()
    out = kara.cache(ko, vo if values else ko, hkv)
    kara.kara_expand8(kara.cache8(*keep, hkv), out, W, i32(lengths), i32(bt), table, err)
    assert status(kara, err) == 0
    want_t = np.full(bt.shape, -9, np.int32)
    want = [torch.full(shape, 3.0, dtype=torch.float64) for _ in range(2)]
    for s, L in enumerate(lengths):
        p0 = (L - W) // BS
        for j in range(blocks(L) - p0):
            want_t[s, p0 + j] = s * nw + j
            rows = min(BS, L - (p0 + j) * BS)
            for w, c, sc in ((want[0], k, ks), (want[1], v, vs)):
                w[:, s * nw + j] = 0.0
                w[:, s * nw + j, :, :rows] = dense(c[:, int(bt[s, p0 + j])], sc[:, int(bt[s, p0 + j])])[:, :, :rows]
    assert np.array_equal(table.cpu().numpy(), want_t)
    torch.testing.assert_close(ko.cpu().double(), want[0], rtol=0, atol=0, equal_nan=True)
    torch.testing.assert_close(vo.cpu().double(), want[1] if values else torch.full_like(want[1], 3.0), rtol=0, atol=0)


def test_expand_bad_inputs():
    """A short or long sequence is left out, a block outside the pool gives zeros."""
    kara = lib()
    W, d = 64, 64
    lengths, bt, _, k, ks, v, vs = window_case(4, [100, 90, 130, 70], W, 2, d, 2)
    keep = [x.to(DEV) for x in (k, v, ks, vs)]
    ko = torch.full((2, 20, 2, BS, d), 3.0, dtype=torch.bfloat16, device=DEV)
    for bad, want in ((63, kara.EINVAL), (bt.shape[1] * BS + 1, kara.EINVAL), (None, kara.EBADBLOCK)):
        ln, b, err = lengths.copy(), bt.copy(), error_word()
        if bad is None:
            b[1, 3] = k.shape[1]
        else:
            ln[1] = bad
        table = torch.full(bt.shape, -9, dtype=torch.int32, device=DEV)
        ko.fill_(3.0)
        kara.kara_expand8(kara.cache8(*keep, 2), kara.cache(ko, ko, 2), W, i32(ln), i32(b), table, err)
        assert status(kara, err) == want
        if bad is not None:
            assert (table[1] == -9).all() and (ko[:, 5:10] == 3.0).all()
        else:
            assert (ko[:, 5 + 3 - (90 - W) // BS] == 0.0).all() and table[1, 3] == 7
        assert (ko[:, :5] != 3.0).any() and (table[2] >= 0).sum() == blocks(130) - (130 - W) // BS


def run_compact(lengths, bt, fresh, k, ks, v, vs, kept, W, B, R, err=None):
    kara = lib()
    n = len(lengths)
    keep = [x.to(DEV) for x in (k, v, ks, vs)]
    c, p = kara.cache8(*keep, k.shape[2]), kara.params(W, B, 1, R, 0.1)
    table, new_len = i32(bt), torch.full((n,), -7, dtype=torch.int32, device=DEV)
    freed = torch.full((sum(blocks(int(L)) for L in lengths),), -7, dtype=torch.int32, device=DEV)
    ws = torch.empty(kara.kara_compact8_workspace_size(c, p, n), dtype=torch.uint8, device=DEV)
    err = error_word() if err is None else err
    kara.kara_compact8(c, p, i32(lengths), table, i32(kept), i32(fresh), freed, new_len, ws, err)
    st = status(kara, err)
    return st, [x.cpu() for x in keep], table.cpu().numpy(), freed.cpu().numpy(), new_len.cpu().numpy()


@pytest.mark.parametrize("W,B,R,hkv,d,layers,lengths", [
    (64, 16, 16, 2, 64, 1, [250]), (64, 0, 1, 2, 128, 2, [64, 79, 300]), (128, 63, 30, 3, 64, 2, [128, 143, 144, 500]),
    (512, 64, 89, 8, 128, 2, [512, 1000]), (192, 16, 176, 1, 128, 3, [200, 333]),
    (64, 16, 16, 8, 64, 40, [70, 64, 1000, 255])])   # the last: more than one block compares
def test_compact_matches_plain(W, B, R, hkv, d, layers, lengths):
    """Rebuilt blocks, their scales, tables, freed ids and lengths; NaN codes mark their new block."""
    r = np.random.default_rng(W + B)
    lengths, bt, fresh, k, ks, v, vs = window_case(W + R, lengths, W, hkv, d, layers, extra=200)
    n, C = len(lengths), W - B
    kept = np.stack([np.sort(r.choice(C, R, replace=False)) for _ in range(n * layers * hkv)])
    kept = kept.reshape(n, layers, hkv, R).astype(np.int32)
    L0 = int(lengths[0])
    pos = L0 - W + int(kept[0, 0, 0, 0])
    b = int(bt[0, pos // BS])
    k[0, b, 0, pos % BS, 1] = 0xff
    ks[0, b, 0] *= -1
    st, got, table, freed, new_len = run_compact(lengths, bt, fresh, k, ks, v, vs, kept, W, B, R)
    assert st == 0
    want_bt, want_freed, used = bt.copy(), [], 0
    want = [x.clone() for x in (k, v, ks, vs)]
    for s, L in enumerate(lengths.tolist()):
        p0, after = (L - W) // BS, L - W + R + B
        n_old, n_new = blocks(L) - p0, blocks(after) - p0
        want_freed += bt[s, p0:p0 + n_old].tolist()
        want_bt[s, p0:p0 + n_old] = -1
        ids = fresh[used:used + n_new]
        used += n_new
        want_bt[s, p0:p0 + n_new] = ids
        assert new_len[s] == after
        for layer in range(layers):
            for g in range(hkv):
                src = source_rows(L, W, B, R, kept[s, layer, g])
                blk = torch.as_tensor(bt[s, src // BS]).long()
                for codes, scale, wc, wsc in ((k, ks, want[0], want[2]), (v, vs, want[1], want[3])):
                    x = value(codes[layer, blk, g, torch.as_tensor(src % BS)]) * scale[layer, blk, g].double().abs()[:, None]
                    for j, (cc, sc) in enumerate(plain_compact(codes, scale, x)):
                        wc[layer, ids[j], g, :len(cc)] = cc
                        wsc[layer, ids[j], g] = sc.float()
    assert np.array_equal(table, want_bt) and freed[:len(want_freed)].tolist() == want_freed
    assert (freed[len(want_freed):] == -7).all()
    nan_same = lambda a, b: bool(((a == b) | ((a & 127 == 127) & (b & 127 == 127))).all())  # noqa: E731
    assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3]) and (got[2] < 0).sum() == (want[2] < 0).sum()
    assert nan_same(got[0], want[0]) and nan_same(got[1], want[1])


@pytest.mark.parametrize("what", ["fresh twice", "fresh listed", "fresh outside", "few", "kept order", "kept range",
                                  "short", "earlier", "old outside", "old -2"])
@pytest.mark.parametrize("layers,width", [(2, 0), (160, 0), (2, 80000)])
def test_compact_refuses_on_the_device(what, layers, width):
    """The statuses of kara_compact, and no block of the pools written (but for an old block met while copying);
    checked by one block, kept rows by several, or everything by several (a wide table)."""
    kara = lib()
    W, B, R = 64, 16, 20
    lengths, bt, fresh, k, ks, v, vs = window_case(3, [100, 200, 300], W, 2, 64, layers, extra=40)
    bt = np.concatenate([bt, np.full((3, width), -1, np.int32)], 1)
    kept = np.broadcast_to(np.arange(R, dtype=np.int32), (3, layers, 2, R)).copy()
    err = None
    if what == "fresh twice":
        fresh[4], want = fresh[1], kara.EDUPBLOCK
    elif what == "fresh listed":
        fresh[0], want = bt[1, 0], kara.EDUPBLOCK
    elif what == "fresh outside":
        fresh[2], want = k.shape[1], kara.EBADBLOCK
    elif what == "few":
        fresh, want = fresh[:2], kara.ENOBLOCKS
    elif what == "kept order":
        kept[1, 1, 0, 3], want = 2, kara.EINVAL
    elif what == "kept range":
        kept[2, 1, 1, R - 1], want = W - B, kara.EINVAL
    elif what == "short":
        lengths[1], want = W - 1, kara.EINVAL
    elif what == "earlier":
        err, want = torch.full((1,), kara.ETIMEOUT, dtype=torch.int32, device=DEV), kara.ETIMEOUT
    else:
        bt[1, 9], want = -2 if what == "old -2" else -3, kara.EBADBLOCK
    st, got, table, freed, new_len = run_compact(lengths, bt, fresh, k, ks, v, vs, kept, W, B, R, err)
    assert st == want
    assert np.array_equal(table, bt) and (freed == -7).all() and np.array_equal(new_len, lengths)
    if what.startswith("old"):   # live blocks are never written
        old = [int(b) for b in bt.ravel() if 0 <= b < k.shape[1]]
        assert torch.equal(got[0][:, old], k[:, old]) and torch.equal(got[3][:, old], vs[:, old])
    else:
        assert torch.equal(got[0], k) and torch.equal(got[1], v) and torch.equal(got[2], ks) and torch.equal(got[3], vs)


def test_compact_compares_more_ids_than_a_tile():
    """2600 fresh ids: none twice, one twice far apart, one that the last table lists."""
    W, B, R, n = 256, 40, 200, 160
    lengths, bt, fresh, k, ks, v, vs = window_case(8, [W + 5] * n, W, 1, 64, 1, extra=2800)
    kept = np.broadcast_to(np.arange(R, dtype=np.int32), (n, 1, 1, R)).copy()
    used = n * blocks(5 + R + B)
    assert used > 2048 and len(fresh) > used
    st, _, table, freed, new_len = run_compact(lengths, bt, fresh, k, ks, v, vs, kept, W, B, R)
    assert st == 0 and (new_len == 5 + R + B).all() and table[-1, 0] == fresh[used - blocks(5 + R + B)]
    again, listed = fresh.copy(), fresh.copy()
    again[used - 1], listed[3] = fresh[1], bt[n - 1, 2]
    for ids in (again, listed):
        st, got, table, freed, new_len = run_compact(lengths, bt, ids, k, ks, v, vs, kept, W, B, R)
        assert st == lib().EDUPBLOCK and np.array_equal(table, bt) and (freed == -7).all()
        assert torch.equal(got[0], k) and torch.equal(got[3], vs)
    again = fresh.copy()
    again[used] = fresh[0]   # behind the ids that the call takes
    assert run_compact(lengths, bt, again, k, ks, v, vs, kept, W, B, R)[0] == 0
