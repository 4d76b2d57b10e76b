"""GPU tests of the 8-bit cache's calls where blocks' scales lie far apart, against 64 bits.

Chunk attention's tolerance, before the first run, from what include/kara.h states (a rounding is off by at most half a
step: bf16 2^-8, f16 2^-11).  With p_x a row's weights, s_x the scale of the block that key x lies in, in V, and P the
row's largest p_x s_x:
    output   2^-8 |ref|
    weights  sum_x max(2^-11 p_x, 2^-24 P / s_x) |v_x|: an f16 rounding, or half of f16's smallest step, 2^-25, where the
             largest weight times scale is 2^-1 at least (2^7, but for scales of a tile that are up to 2^8 apart)
    logits   a weight is off by its logit's error, and the sum of all by as much: twice 2^-17 of the query's largest
             element times the keys' dims whose query element is below 2^-9 of it; 2^-20 of the sum of the products'
             magnitudes (256 fp32 additions of exact products, at 2^-28 to 2^-22 of the largest partial sum); 2^-15 for
             the logit's scaling, the subtraction of the row's reference (up to 2^7 in log2: 2^-17) and the exponential.
Decode attention's is the same but for weights, sum_x max(2^-11 p_x, 2^-39 P / s_x) |v_x|, and queries, 2^-39 of the head's
largest element for those below 2^-29 of it."""

import numpy as np
import pytest
import torch

from _cache8 import BS, dense, plain_compact, quantise, source_rows, value
from _newtokens import blocks
from test_gpu_cache8 import CHUNKS, chunk_case, decode_case, run_chunk, run_compact, run_decode, window_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("apart", [17, 30, 31, 32, 60, 126])
def test_compact_zero_rows_of_a_large_block(d, apart):
    """Rows of zeros from a block whose scale is 2^apart that of the others: code 0 (either sign), not NaN, whatever
    the rebuilt block's scale, which the others' rows set.  Where nothing but the smallest codes of the large block
    is kept, they move by 2^17.  Exact: a code is rounded once."""
    W, B, R, hkv, lo = 64, 16, 32, 2, -63
    lengths, bt, fresh, k, ks, v, vs = window_case(apart + d, [W], W, hkv, d, 1, extra=9)
    large = int(bt[0, 1])                 # positions 16 to 31
    for codes, scale in ((k, ks), (v, vs)):
        scale[0] = 2.0 ** lo
        scale[0, large] = 2.0 ** (lo + apart)
        codes[0, large] = 0
        codes[0, large, :, 1::2] = 0x80   # -0
        codes[0, large, :, 15] = 0x7e     # the row that set the scale: not kept
    v[0, large, 1] = 0x01                 # head 1 of V: the smallest code alone
    # head 0 keeps rows of the large block beside others', head 1 all of it
    kept = np.stack([np.r_[np.arange(8, 24), np.arange(32, 48)], np.arange(16, 48)])
    kept = kept.reshape(1, 1, hkv, R).astype(np.int32)
    st, got, *_ = run_compact(lengths, bt, fresh, k, ks, v, vs, kept, W, B, R)
    assert st == 0
    n_new = blocks(R + B)
    for pool, (codes, scale) in enumerate(((k, ks), (v, vs))):
        for g in range(hkv):
            src = source_rows(W, W, B, R, kept[0, 0, g])
            blk = torch.as_tensor(bt[0, src // BS]).long()
            x = value(codes[0, blk, g, torch.as_tensor(src % BS)]) * scale[0, blk, g].double()[:, None]
            want = plain_compact(codes, scale, x)
            assert len(want) == n_new
            for j, (wc, ws) in enumerate(want):
                assert torch.equal(got[2 + pool][0, fresh[j], g], ws.float())
                assert torch.equal(got[pool][0, fresh[j], g, :len(wc)], wc)


# ---- chunk attention ------------------------------------------------------------

def bound(q, k, v, sv, chunk=True):
    """Output and tolerance of queries [G][D] over keys and values [n][D] with V's scales sv [n]."""
    D = q.shape[-1]
    near, query, weight = (2.0 ** -9, 2.0 ** -17, 2.0 ** -24) if chunk else (2.0 ** -29, 2.0 ** -39, 2.0 ** -39)
    p = torch.softmax(q @ k.T / D ** 0.5, -1)
    top = q.abs().amax(-1, keepdim=True)
    small = torch.where(q.abs() < near * top, top, 0.0)
    logit = query * small @ k.abs().T + 2.0 ** -20 * (q.abs() @ k.abs().T)
    most = (p * sv).amax(-1, keepdim=True)
    w = torch.maximum(2.0 ** -11 * p, weight * most / torch.where(sv > 0, sv, torch.inf))
    w = w + p * 2 * (logit.amax(-1, keepdim=True) / D ** 0.5 + 2.0 ** -15)
    ref = p @ v
    return ref, ref.abs() * 2.0 ** -8 + w @ v.abs()


def check_chunk(c, got, rows=None):
    """Rows of a chunk's output (all, or those of the given numbers) within the tolerance above."""
    hq, D = c["q"].shape[1:]
    hkv = c["k"].shape[2]
    G = hq // hkv
    k_all, v_all = (dense(c[x], c[x + "s"])[0] for x in "kv")
    for s, L in enumerate(int(x) for x in c["lengths"]):
        t0, t1 = int(c["q_start"][s]), int(c["q_start"][s + 1])
        ids = torch.as_tensor(c["bt"][s, :blocks(L)]).long()
        for g in range(hkv):
            k, v = (x[ids, g].reshape(-1, D)[:L] for x in (k_all, v_all))
            sv = c["vs"][0, ids, g].double().abs().repeat_interleave(BS)[:L]
            for t in range(t0, t1):
                if rows is None or t in rows:
                    n = L - (t1 - t) + 1
                    ref, lim = bound(c["q"][t, g * G:(g + 1) * G].double(), k[:n], v[:n], sv[:n])
                    off = ((got[t, g * G:(g + 1) * G].double() - ref).abs() / lim).max()
                    assert (lim > 0).all() and off <= 1, (s, g, t, float(off))


SHAPES = [(8, 2, 128), (4, 2, 64), (5, 1, 128)]


@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("n_new", [100, 5])
@pytest.mark.parametrize("up", [9, 20, 40, 60])
def test_chunk_rows_before_a_large_value(hq, hkv, d, n_new, up):
    """Blocks of V that hold later tokens only, 2^up above the others: rows that do not see them are what they are
    without them, within the tolerance of their own values."""
    L = 300
    c = chunk_case(up + d, [L, L - 7], [n_new, n_new], hq, hkv, d)
    for s in range(2):
        c["vs"][0, int(c["bt"][s, (L - 1 - 7 * s) // BS])] *= 2.0 ** up
    st, got = run_chunk(c)
    assert st == 0
    check_chunk(c, got)


@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("n_new", [60, 1])
@pytest.mark.parametrize("up,down", [(9, 5), (20, 15), (30, 30), (40, 60), (60, 60), (60, 90), (-60, 0), (-40, -20)])
def test_chunk_large_values_of_small_weight(hq, hkv, d, n_new, up, down):
    """A block that every row sees, with V 2^up above (below) the others and logits about 2^down times less (more)
    likely: what it adds counts, and takes nothing from the rest."""
    L = 400
    c = chunk_case(1000 + up + 2 * down + d, [L], [n_new], hq, hkv, d)
    g = torch.Generator().manual_seed(up + 107)
    lean = 1.0 + torch.randint(0, 2, (d,), generator=g).double()     # what all queries have in common
    c["q"] = (lean + 0.1 * torch.randn(c["q"].shape, generator=g)).bfloat16()
    at = int(c["bt"][0, 20])                                         # positions 320 to 335, in the same tile as the end
    far = -down * np.log(2.0) * d ** 0.5 * lean / (lean * lean).sum() * torch.ones(hkv, BS, 1)
    c["k"][0, at], c["ks"][0, at] = quantise(far + 0.01 * torch.randn(hkv, BS, d, generator=g))
    c["vs"][0, at] *= 2.0 ** up
    st, got = run_chunk(c)
    assert st == 0
    check_chunk(c, got)


@pytest.mark.parametrize("n_new", [1, 3, 150])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("up", [63, 60, 50, 30])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_chunk_tiles_of_far_apart_scales(n_new, zeros, up, where):
    """One tile of V at 2^up, all others zeros or at 2^-63, each key with its part of the weight: more than a
    thousandth of it to about half of it in the one tile."""
    tiles, d, hq, hkv = 36, 64, 4, 2
    L = tiles * 128
    c = chunk_case(7 + up, [L, 700], [n_new, 2], hq, hkv, d, qmag=1.0)
    g = torch.Generator().manual_seed(up)
    lean = 1.0 + torch.randint(0, 2, (d,), generator=g).double()
    c["q"] = (lean + 0.3 * torch.randn(c["q"].shape, generator=g)).bfloat16()
    one = {"first": 0, "middle": 17, "last": tiles - 2}[where]
    ids = torch.as_tensor(c["bt"][0, :blocks(L)]).long()
    big = ids[8 * one:8 * one + 8]
    c["vs"][0, ids] = 0.0 if zeros else 2.0 ** -63
    if zeros:
        c["v"][0, ids] = 0
    c["v"][0, big], c["vs"][0, big] = quantise(torch.randn(8, hkv, BS, d, generator=g))
    c["vs"][0, big] = 2.0 ** up
    for i, bits in enumerate([0, 3, 6]):     # of a third of the tile: its keys' weight over the others', log2
        blk = big[i::3]
        up_by = bits * np.log(2.0) * d ** 0.5 * lean / (lean * lean).sum() * torch.ones(len(blk), hkv, BS, 1)
        c["k"][0, blk], c["ks"][0, blk] = quantise(up_by + 0.01 * torch.randn(up_by.shape, generator=g))
    far = torch.ones(len(ids), dtype=torch.bool)
    far[8 * one:8 * one + 8] = False
    c["k"][0, ids[far]], c["ks"][0, ids[far]] = quantise(0.05 * torch.randn(int(far.sum()), hkv, BS, d, generator=g))
    st, got = run_chunk(c)
    assert st == 0
    check_chunk(c, got, rows=None if n_new < 100 else list(range(0, n_new, 13)) + [n_new, n_new + 1])


@pytest.mark.parametrize("lo,hi", [(-63, 63), (-63, 0), (0, 63), (-20, 20)])
def test_chunk_scales_at_random(lo, hi):
    """Every block of V with a scale of its own, and of K too; one call in one tile, one cut into many pieces."""
    for L, n_new, hq, hkv, d in ((100, 40, 8, 2, 64), (5000, 7, 4, 2, 128)):
        c = chunk_case(L + lo + hi + 200, [L, 33], [n_new, 5], hq, hkv, d, qmag=1.0)
        g = torch.Generator().manual_seed(L + hi)
        shape = c["vs"][0].shape
        c["vs"][0] = c["vs"][0].sign() * 2.0 ** torch.randint(lo, hi + 1, shape, generator=g).float()
        c["ks"][0] = c["ks"][0].sign() * 2.0 ** torch.randint(-9, -6, shape, generator=g).float()
        st, got = run_chunk(c)
        assert st == 0
        check_chunk(c, got)


@pytest.mark.parametrize("outliers", [False, True])
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_chunk_within_its_stated_errors(hq, hkv, d, outliers):
    """Lengths around blocks and tiles; V's scales within a tile's one exponent.  With outliers, three dims of each query
    2^12 and more above the rest, which then are where the queries' two terms lose digits."""
    c = chunk_case(hq + 5, CHUNKS[0][0], CHUNKS[0][1], hq, hkv, d, pad=2)
    if outliers:
        c["q"][:, :, 3:] *= 2.0 ** -7
        c["q"][:, :, :3] *= 2.0 ** 4
        c["k"][..., :3] = 0x20       # 2^-4 times the scale: the large dims do not decide alone
    st, got = run_chunk(c)
    assert st == 0
    check_chunk(c, got)


@pytest.mark.parametrize("hq,hkv,d", SHAPES)
@pytest.mark.parametrize("lo,hi", [(0, 0), (-63, 63), (-63, 0), (0, 63)])
def test_decode_scales_at_random(hq, hkv, d, lo, hi):
    """Every block of V with a scale of its own; sequences of one split and of several."""
    lengths, bt, k, ks, v, vs, q = decode_case(hq + 70, [1, 40, 1000, 2500], hq, hkv, d)
    g = torch.Generator().manual_seed(d + hi)
    if lo < hi:
        vs = vs.sign() * 2.0 ** torch.randint(lo, hi + 1, vs.shape, generator=g).float()
    q[:, :, 5] *= 2.0 ** 10
    k[..., 5] = 0x08                 # 2^-6 times the scale
    st, out = run_decode(lengths, bt, k, ks, v, vs, q)
    assert st == 0
    kd, vd = dense(k, ks)[1], dense(v, vs)[1]
    for s, L in enumerate(lengths):
        ids = torch.as_tensor(bt[s, :blocks(L)]).long()
        for g in range(hkv):
            kk, vv = (x[ids, g].reshape(-1, d)[:L] for x in (kd, vd))
            sv = vs[1, ids, g].double().abs().repeat_interleave(BS)[:L]
            h = slice(g * (hq // hkv), (g + 1) * (hq // hkv))
            ref, lim = bound(q[s, h].double(), kk, vv, sv, chunk=False)
            off = ((out[s, h].double() - ref).abs() / lim).max()
            assert off <= 1, (s, g, float(off))
