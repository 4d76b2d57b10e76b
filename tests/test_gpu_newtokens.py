"""GPU tests of the new-token operators against their plain forms in 64 bits.

Tolerances, before the first run (a bf16 rounding is off by at most 2^-8 of the value):
append   fp32 sums and products of one row (about 20 roundings of 2^-24, against the larger member of
         the rotated pair), then one rounding: |got - ref| <= 2^-8 |ref| + 2^-19 max|row|.
chunk    each softmax weight is rounded to bf16 (2^-8 of itself), logits and sums are fp32 (together
         below 2^-10 of a weight at these lengths and logits), then one rounding of the output:
         |got - ref| <= 2^-8 |ref| + (2^-8 + 2^-10) sum_x w_x |v_x|."""

import numpy as np
import pytest
import torch

from _gpu import lib
from _newtokens import blocks, make_tables, plain_chunk, plain_extend, plain_turn

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).to(DEV).contiguous()


def error_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def new_tokens(kara, n, rows, fill=-77):
    f = lambda k, t: torch.full((k,), fill, dtype=t, device=DEV)  # noqa: E731
    b = dict(q_start=f(n + 1, torch.int32), length=f(n, torch.int32), slot=f(rows, torch.int64),
             seq=f(rows, torch.int32), pos=f(rows, torch.int32))
    return b, kara.tokens(*b.values())


# ---- tables ---------------------------------------------------------------------

def run_extend(kara, lengths, n_new, bt, fresh, rows, num_blocks, in_place=False, err=None):
    b, t = new_tokens(kara, len(lengths), rows)
    ln = i32(lengths)
    if in_place:
        t = kara.tokens(b["q_start"], ln, b["slot"], b["seq"], b["pos"])
        b["length"] = ln
    table, used = i32(bt), torch.full((1,), -77, dtype=torch.int32, device=DEV)
    err = error_word() if err is None else err
    kara.kara_extend_tables(num_blocks, 16, ln, i32(n_new), table, i32(fresh), t, used, err)
    st = kara.kara_get_error(err)
    return st, [x.cpu().numpy() for x in (table, b["q_start"], b["length"], b["slot"], b["seq"], b["pos"], used)]


def extend_case(seed, n, len_hi, new_hi, extra_width=1):
    r = np.random.default_rng(seed)
    lengths = r.integers(0, len_hi + 1, n).astype(np.int32)
    n_new = r.integers(0, new_hi + 1, n).astype(np.int32)
    width = max(1, int(blocks(lengths + n_new).max()) + extra_width)
    need = int((blocks(lengths + n_new) - blocks(lengths)).sum())
    num_blocks = int(blocks(lengths).sum()) + need + 5
    bt, left = make_tables(lengths, width, num_blocks, seed)
    return lengths, n_new, bt, left, num_blocks


@pytest.mark.parametrize("n,len_hi,new_hi,pad", [
    (1, 300, 1, 0), (1, 0, 1, 3), (3, 40, 33, 5), (128, 2000, 1, 0), (31, 5000, 700, 77), (1024, 64, 3, 0),
    (1025, 50, 2, 9), (2500, 30, 1, 100), (1, 100, 9000, 1), (20000, 20, 2, 3)])
def test_extend_matches_plain(n, len_hi, new_hi, pad):
    """One cluster CTA and eight, lists below, at and past one pass of the scan, zero new tokens, padding."""
    kara = lib()
    lengths, n_new, bt, fresh, nb = extend_case(n + new_hi, n, len_hi, new_hi)
    rows = int(n_new.sum()) + pad
    want = plain_extend(lengths, n_new, bt, fresh, rows)
    for in_place in (False, True):
        st, got = run_extend(kara, lengths, n_new, bt, fresh, rows, nb, in_place)
        assert st == 0
        for name, g, w in zip(("table", "q_start", "len", "slot", "seq", "pos", "used"), got, want):
            assert np.array_equal(g, w), (name, in_place)


def test_extend_of_nothing():
    """No new tokens at all, no sequences at all, and no rows."""
    kara = lib()
    lengths, n_new, bt, fresh, nb = extend_case(3, 5, 100, 0)
    st, got = run_extend(kara, lengths, n_new, bt, fresh, 4, nb)
    assert st == 0 and np.array_equal(got[0], bt) and np.array_equal(got[2], lengths)
    assert got[1].tolist() == [0] * 6 and (got[3] == -1).all() and got[6][0] == 0
    st, got = run_extend(kara, lengths, n_new, bt, fresh, 0, nb)
    assert st == 0 and got[1].tolist() == [0] * 6
    st, got = run_extend(kara, lengths[:0], n_new[:0], bt[:0], fresh, 4, nb)
    assert st == 0 and got[1].tolist() == [0] and (got[3] == -1).all() and (got[4] == -1).all()


def assert_nothing_done(got, lengths, bt):
    table, q_start, ln, slot, seq, pos, used = got
    assert np.array_equal(table, bt) and np.array_equal(ln, lengths) and used[0] == 0
    assert (q_start == 0).all() and (slot == -1).all() and (seq == -1).all() and (pos == -1).all()


@pytest.mark.parametrize("n", [3, 200])
@pytest.mark.parametrize("what", ["negative length", "negative count", "table full", "rows short", "few blocks",
                                  "id twice", "id still listed", "id past the pool", "id negative", "open block bad",
                                  "earlier error"])
def test_extend_refuses_on_the_device(what, n):
    """Every check leaves the call without effect; small batches (one CTA) and large ones (a cluster)."""
    kara = lib()
    r = np.random.default_rng(n)
    lengths = r.integers(20, 900, n).astype(np.int32)
    lengths[1] = 40 * 16 + 5
    n_new = r.integers(17, 60, n).astype(np.int32)
    width = int(blocks(lengths + n_new).max())
    need = int((blocks(lengths + n_new) - blocks(lengths)).sum())
    nb = int(blocks(lengths).sum()) + need + 5
    bt, fresh = make_tables(lengths, width, nb, 5)
    rows, err, want = int(n_new.sum()) + 2, None, None
    if what == "negative length":
        lengths[n - 1], want = -1, kara.EINVAL
    elif what == "negative count":
        n_new[0], want = -1, kara.EINVAL
    elif what == "table full":
        n_new[int(lengths.argmax())], want = width * 16, kara.EINVAL
    elif what == "rows short":
        rows, want = int(n_new.sum()) - 1, kara.EINVAL
    elif what == "few blocks":
        fresh, want = fresh[:need - 1], kara.ENOBLOCKS
    elif what == "id twice":
        fresh[need - 1], want = fresh[0], kara.EDUPBLOCK
    elif what == "id still listed":
        fresh[1], want = bt[n - 1, 0], kara.EDUPBLOCK
    elif what == "id past the pool":
        fresh[2], want = nb, kara.EBADBLOCK
    elif what == "id negative":
        fresh[0], want = -1, kara.EBADBLOCK
    elif what == "open block bad":
        bt[1, 40], want = nb + 3, kara.EBADBLOCK
    else:
        err, want = torch.full((1,), kara.ETIMEOUT, dtype=torch.int32, device=DEV), kara.ETIMEOUT
    st, got = run_extend(kara, lengths, n_new, bt, fresh, rows, nb, err=err)
    assert st == want
    assert_nothing_done(got, lengths, bt)


def test_extend_ids_past_the_need_are_not_looked_at():
    kara = lib()
    lengths, n_new, bt, fresh, nb = extend_case(8, 6, 200, 50)
    need = int((blocks(lengths + n_new) - blocks(lengths)).sum())
    fresh = np.concatenate([fresh[:need], np.array([-5, nb + 9, fresh[0], bt[0, 0]], np.int32)])
    st, got = run_extend(kara, lengths, n_new, bt, fresh, int(n_new.sum()), nb)
    assert st == 0 and np.array_equal(got[0], plain_extend(lengths, n_new, bt, fresh, int(n_new.sum()))[0])


def test_extend_pool_of_several_bitmap_windows():
    """More than 2^20 blocks: ids, repeats and listed ids in each window."""
    kara = lib()
    nb = (1 << 21) + 100
    lengths, n_new = np.array([33, 16, 0], np.int32), np.array([16, 16, 40], np.int32)
    bt = np.array([[5, (1 << 20) + 7, (1 << 21) + 50, -1, -1], [9, -1, -1, -1, -1], [-1] * 5], np.int32)
    fresh = np.array([1 << 20, (1 << 21) + 99, 3, (1 << 20) - 1, 77], np.int32)
    rows = int(n_new.sum())
    st, got = run_extend(kara, lengths, n_new, bt, fresh, rows, nb)
    want = plain_extend(lengths, n_new, bt, fresh, rows)
    assert st == 0 and all(np.array_equal(g, w) for g, w in zip(got, want))
    for at, bad in ((1, (1 << 20)), (2, (1 << 20) + 7), (0, (1 << 21) + 50), (3, 9)):
        f = fresh.copy()
        f[at] = bad
        st, got = run_extend(kara, lengths, n_new, bt, f, rows, nb)
        assert st == kara.EDUPBLOCK, (at, bad)
        assert_nothing_done(got, lengths, bt)


# ---- norms, rotation, append -----------------------------------------------------

def angles(n_pos, rot, seed=0):
    a = torch.arange(n_pos, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(rot // 2, dtype=torch.float64)
                                                                    / max(1, rot // 2))
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def append_inputs(seed, hq, hkv, D, rows, fused=True):
    g = torch.Generator().manual_seed(seed)
    if fused:
        x = torch.randn(rows, (hq + 2 * hkv) * D + 8, generator=g).bfloat16()
        q = x[:, :hq * D].view(rows, hq, D)
        k = x[:, hq * D:(hq + hkv) * D].view(rows, hkv, D)
        v = x[:, (hq + hkv) * D:(hq + 2 * hkv) * D].view(rows, hkv, D)
        return q, k, v
    return tuple(torch.randn(rows, h, D, generator=g).bfloat16() for h in (hq, hkv, hkv))


def on_gpu(q, k, v):
    """q, k, v on the GPU with the strides that they have here (views of one buffer stay views)."""
    if q.is_contiguous():
        return q.to(DEV), k.to(DEV), v.to(DEV)
    base = q._base.to(DEV)
    return tuple(torch.as_strided(base, x.shape, x.stride(), x.storage_offset()) for x in (q, k, v))


def close_rows(got, ref, scale):
    """|got - ref| <= 2^-8 |ref| + 2^-19 max|row|."""
    lim = ref.abs() * 2.0 ** -8 + scale.abs().amax(-1, keepdim=True) * 2.0 ** -19
    bad = (got.double() - ref).abs() > lim
    assert not bad.any(), ((got.double() - ref).abs() - lim).max()


@pytest.mark.parametrize("hq,hkv,D,rot,inter,norm,W,fused", [
    (4, 2, 64, 64, False, True, 64, True), (40, 8, 128, 128, False, True, 128, True),
    (32, 8, 128, 128, False, False, 0, True), (8, 1, 128, 64, False, True, 64, False),
    (3, 3, 64, 32, False, True, 0, True), (14, 2, 64, 64, True, True, 64, True),
    (5, 1, 128, 128, True, False, 0, False), (6, 2, 128, 48, True, True, 64, True),
    (7, 1, 64, 16, False, False, 64, True), (2, 2, 128, 0, False, True, 0, True), (2, 2, 64, 0, False, False, 0, False),
    (18, 3, 128, 96, False, True, 0, True)])
def test_append_matches_plain(hq, hkv, D, rot, inter, norm, W, fused):
    """Norm on or off, both pairings, partial rotations (halves that are no power of two among them),
    fused or separate inputs, padding rows, the ring with chunks longer and shorter than its window,
    rotary positions that run ahead of the cached ones."""
    kara = lib()
    r = np.random.default_rng(hq * D + rot)
    lengths = np.array([0, 100, 47, 31, 250], np.int32)
    n_new = np.array([70, 1, 0, 150, 17], np.int32)
    width = int(blocks(lengths + n_new).max())
    nb = int(blocks(lengths + n_new).sum()) + 3
    bt, fresh = make_tables(lengths, width, nb, 1)
    total, rows = int(n_new.sum()), int(n_new.sum()) + 5
    table, q_start, ln, slot, seq, pos, _ = plain_extend(lengths, n_new, bt, fresh, rows)
    shift = r.integers(0, 300, 5).astype(np.int32)
    layers, layer, eps = 2, 1, 1e-5
    q, k, v = append_inputs(hq + rot, hq, hkv, D, rows, fused)
    g = torch.Generator().manual_seed(9)
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g)).bfloat16() for _ in range(2)) if norm else (None, None)
    cs = angles(800, rot) if rot else None

    pool = torch.randn(2, layers, nb, hkv, 16, D, generator=g).bfloat16()
    kp, vp = pool[0].to(DEV), pool[1].to(DEV)
    ring0 = torch.randn(5, layers, hq, W, D, generator=g).bfloat16() if W else None
    ring = ring0.to(DEV) if W else None
    dq, dk, dv = on_gpu(q, k, v)
    q_out = torch.full((rows, hq, D), 77.0, dtype=torch.bfloat16, device=DEV)
    t = kara.tokens(i32(q_start), i32(ln), torch.from_numpy(slot).to(DEV), i32(seq), i32(pos))
    keep = [x.to(DEV) if x is not None else None for x in (cs, qw, kw)]
    sh = i32(shift)
    c = kara.cache(kp, vp, hq)
    err = error_word()
    kara.kara_append_kv(c, layer, t, kara.rope(keep[0], keep[1], keep[2], eps, inter, sh), dq, dk, dv, q_out, err,
                        ring=ring)
    assert kara.kara_get_error(err) == 0

    at = torch.from_numpy(pos[:total] + shift[seq[:total]]).long()
    zq = plain_turn(q[:total], qw, eps, cs, at, inter)
    zk = plain_turn(k[:total], kw, eps, cs, at, inter)
    nq, nk = plain_turn(q[:total], qw, eps, None, None, inter), plain_turn(k[:total], kw, eps, None, None, inter)
    got = q_out.cpu()
    close_rows(got[:total], zq, nq)
    assert (got[total:] == 77.0).all()                       # padding rows are left alone
    sl = torch.from_numpy(slot[:total])
    kr = kp.cpu()[layer].permute(0, 2, 1, 3).reshape(-1, hkv, D)
    vr = vp.cpu()[layer].permute(0, 2, 1, 3).reshape(-1, hkv, D)
    close_rows(kr[sl], zk, nk)
    assert torch.equal(vr[sl], v[:total])
    # every other pool row, and the other layer, is as it was
    rest = torch.ones(nb * 16, dtype=torch.bool)
    rest[sl] = False
    for now, was in ((kp, pool[0]), (vp, pool[1])):
        a, b = (x.cpu()[layer].permute(0, 2, 1, 3).reshape(-1, hkv, D)[rest] for x in (now, was))
        assert torch.equal(a, b) and torch.equal(now.cpu()[0], was[0])
    if W:
        rg = ring.cpu()
        want = ring0.clone()
        for i in range(total):
            s, x = int(seq[i]), int(pos[i])
            if x >= int(ln[s]) - W:
                want[s, layer, :, x % W] = got[i]
        assert torch.equal(rg, want)


def test_append_in_place_and_strided_pool():
    """q_out = q, and pools that are views with padded strides."""
    kara = lib()
    hq, hkv, D, rows = 4, 2, 128, 33
    q, k, v = append_inputs(5, hq, hkv, D, rows, fused=False)
    big = torch.zeros(3, 6, 4, 16, D, dtype=torch.bfloat16, device=DEV)
    kp, vp = big[:2, :, :2], torch.zeros_like(big)[:2, :, :2]
    bt = np.array([[4, 0, 5]], np.int32)
    _, q_start, ln, slot, seq, pos, _ = plain_extend(np.array([0], np.int32), np.array([rows], np.int32), bt,
                                                     np.array([4, 0, 5], np.int32), rows)
    t = kara.tokens(i32(q_start), i32(ln), torch.from_numpy(slot).to(DEV), i32(seq), i32(pos))
    cs = angles(64, D).to(DEV)
    dq, dk, dv = q.to(DEV), k.to(DEV), v.to(DEV)
    err = error_word()
    kara.kara_append_kv(kara.cache(kp, vp, hq), 1, t, kara.rope(cs), dq, dk, dv, dq, err)
    assert kara.kara_get_error(err) == 0
    at = torch.from_numpy(pos).long()
    close_rows(dq.cpu(), plain_turn(q, None, 0, cs.cpu(), at, False), q.double())
    rowsk = kp[1].cpu().permute(0, 2, 1, 3).reshape(-1, hkv, D)[torch.from_numpy(slot)]
    close_rows(rowsk, plain_turn(k, None, 0, cs.cpu(), at, False), k.double())
    assert (big[:, :, 2:] == 0).all() and (big[0] == 0).all() and (big[2] == 0).all()


def test_append_zero_rows_and_large_values():
    """Rows of zeros (the norm's eps alone), and rows whose squares pass bf16's and near fp32's range."""
    kara = lib()
    hq, hkv, D, rows = 2, 1, 64, 4
    q, k, v = append_inputs(6, hq, hkv, D, rows, fused=False)
    q[0], k[1] = 0.0, 0.0
    q[2] *= 1e16
    k[3] *= 1e-18
    kp = torch.zeros(1, 1, hkv, 16, D, dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    t = kara.tokens(i32([0, rows]), i32([rows]), torch.arange(rows, device=DEV), i32([0] * rows), i32(range(rows)))
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    cs = angles(8, D).to(DEV)
    out = torch.empty(rows, hq, D, dtype=torch.bfloat16, device=DEV)
    err = error_word()
    kara.kara_append_kv(kara.cache(kp, vp, hq), 0, t, kara.rope(cs, w, w, 1e-6), q.to(DEV), k.to(DEV), v.to(DEV), out,
                        err)
    assert kara.kara_get_error(err) == 0
    at = torch.arange(rows)
    close_rows(out.cpu(), plain_turn(q, w.cpu(), 1e-6, cs.cpu(), at, False),
               plain_turn(q, w.cpu(), 1e-6, None, None, False))
    close_rows(kp.cpu()[0, 0].permute(1, 0, 2)[:rows], plain_turn(k, w.cpu(), 1e-6, cs.cpu(), at, False),
               plain_turn(k, w.cpu(), 1e-6, None, None, False))
    assert (out[0] == 0).all()


@pytest.mark.parametrize("what,row", [("slot past the pool", 2), ("slot below -1", 1), ("sequence past n", 3),
                                      ("sequence negative", 0), ("position negative", 2),
                                      ("rotary position past the table", 3)])
def test_append_skips_and_reports_bad_rows(what, row):
    kara = lib()
    hq, hkv, D, rows = 2, 1, 64, 4
    q, k, v = append_inputs(7, hq, hkv, D, rows, fused=False)
    kp = torch.zeros(1, 2, hkv, 16, D, dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    slot, seq, pos = np.arange(rows), np.zeros(rows, np.int32), np.arange(rows)
    want = kara.EINVAL
    if what.startswith("slot"):
        slot[row], want = (32 if "past" in what else -2), kara.EBADBLOCK
    elif what.startswith("sequence"):
        seq[row] = 1 if "past" in what else -1
    elif what == "position negative":
        pos[row] = -3
    else:
        pos[row] = 8
    t = kara.tokens(i32([0, rows]), i32([rows]), torch.from_numpy(slot).to(DEV), i32(seq), i32(pos))
    out = torch.full((rows, hq, D), 5.0, dtype=torch.bfloat16, device=DEV)
    err = error_word()
    ring = torch.zeros(1, 1, hq, 64, D, dtype=torch.bfloat16, device=DEV)
    kara.kara_append_kv(kara.cache(kp, vp, hq), 0, t, kara.rope(angles(8, D).to(DEV)), q.to(DEV), k.to(DEV), v.to(DEV),
                        out, err, ring=ring)
    assert kara.kara_get_error(err) == want
    good = [i for i in range(rows) if i != row]
    assert (out[row] == 5.0).all() and (out[good] != 5.0).any()
    assert (kp[0, 0, 0, row] == 0).all() and torch.equal(vp.cpu()[0, 0, 0, good], v[good, 0])
    assert (vp[0, 0, 0, row] == 0).all() and (kp[0, 1] == 0).all() and (ring[0, 0, :, row] == 0).all()


# ---- chunk attention -------------------------------------------------------------

def chunk_inputs(seed, lengths, n_new, hq, hkv, D, layers=1, qscale=2.0, extra=0):
    """Lengths include the new tokens; pools are filled with NaN where no token of a table lives."""
    g = torch.Generator().manual_seed(seed)
    lengths, n_new = np.asarray(lengths, np.int32), np.asarray(n_new, np.int32)
    nb = max(1, int(blocks(lengths).sum())) + 2
    width = max(1, int(blocks(lengths).max())) + 1
    bt, _ = make_tables(lengths, width, nb, seed)
    k, v = (torch.randn(layers, nb, hkv, 16, D, generator=g).bfloat16() for _ in range(2))
    used = np.zeros((nb, 16), bool)
    for s, L in enumerate(lengths):
        for x in range(int(L)):
            used[bt[s, x // 16], x % 16] = True
    stale = torch.from_numpy(~used)
    for pool in (k, v):
        pool.permute(1, 3, 0, 2, 4)[stale] = float("nan")
    q_start = np.concatenate([[0], np.cumsum(n_new)]).astype(np.int32)
    rows = int(q_start[-1]) + extra
    q = (qscale * torch.randn(rows, hq, D, generator=g)).bfloat16()
    return dict(q=q, k=k, v=v, bt=bt, q_start=q_start, lengths=lengths, hq=hq, rows=rows)


def chunk_tokens(kara, d):
    z = torch.empty(d["rows"], dtype=torch.int64, device=DEV)
    z4 = torch.empty(d["rows"], dtype=torch.int32, device=DEV)
    return kara.tokens(i32(d["q_start"]), i32(d["lengths"]), z, z4, z4)


def run_chunk(kara, d, layer=0, k=None, v=None, fill=77.0):
    k = d["k"].to(DEV) if k is None else k
    v = d["v"].to(DEV) if v is None else v
    c = kara.cache(k, v, d["hq"])
    t = chunk_tokens(kara, d)
    ws = torch.empty(kara.kara_chunk_workspace_size(c, t.n, t.rows), dtype=torch.uint8, device=DEV)
    out = torch.full(d["q"].shape, fill, dtype=torch.bfloat16, device=DEV)
    err = error_word()
    kara.kara_chunk_attention(c, layer, t, i32(d["bt"]), d["q"].to(DEV), out, ws, err)
    return out.cpu(), kara.kara_get_error(err)


def check_chunk(d, got, layer=0, rows=None):
    ref = plain_chunk(d["q"], d["k"], d["v"], layer, d["bt"], d["q_start"], d["lengths"])
    scale = plain_chunk(d["q"], d["k"], d["v"], layer, d["bt"], d["q_start"], d["lengths"], absolute=True)
    n = int(d["q_start"][-1])
    pick = torch.arange(n) if rows is None else torch.tensor(rows)
    lim = ref.abs() * 2.0 ** -8 + scale * (2.0 ** -8 + 2.0 ** -10)
    off = (got.double() - ref).abs()[pick]
    assert not (off > lim[pick]).any() and torch.isfinite(got[pick]).all(), (off - lim[pick]).max()
    assert (got[n:] == 77.0).all()


@pytest.mark.parametrize("G,D", [(1, 64), (1, 128), (2, 128), (3, 64), (4, 128), (5, 128), (6, 64), (7, 128), (8, 128),
                                 (8, 64)])
def test_chunk_matches_plain(G, D):
    """Every group size and head dim, on lengths at and around tile and block borders: single tokens,
    chunks of a few, one and several query tiles, sequences without new tokens, whole prompts."""
    kara = lib()
    lengths = [1, 17, 128, 129, 300, 64, 513, 255, 700]
    n_new = [1, 17, 1, 129, 4, 0, 140, 255, 33]
    d = chunk_inputs(G * D, lengths, n_new, 2 * G, 2, D, layers=2, extra=3)
    for layer in (0, 1):
        got, st = run_chunk(kara, d, layer)
        assert st == 0
        check_chunk(d, got, layer)


@pytest.mark.parametrize("lengths,n_new,hq,hkv,D", [
    ([2500], [1], 8, 1, 128), ([5000], [3], 5, 1, 128), ([3333, 40], [2, 40], 4, 2, 64), ([4097], [300], 2, 1, 128),
    ([1], [1], 1, 1, 64), ([900] * 40, [1] * 40, 8, 2, 128), ([1500], [1500], 4, 2, 128),
    ([16] * 130, [16] * 130, 2, 2, 64)])
def test_chunk_long_caches_and_many_sequences(lengths, n_new, hq, hkv, D):
    """Few rows over long caches (the key axis is split), one token, many sequences, a whole prompt."""
    kara = lib()
    d = chunk_inputs(len(lengths) + hq, lengths, n_new, hq, hkv, D)
    got, st = run_chunk(kara, d)
    assert st == 0
    check_chunk(d, got)


def test_chunk_of_one_token_is_decode():
    """A chunk of one token per sequence agrees with kara_decode_attention (fp32 weights, fp32 out)."""
    kara = lib()
    d = chunk_inputs(77, [1, 40, 1025, 333], [1] * 4, 10, 2, 128)
    got, st = run_chunk(kara, d)
    assert st == 0
    check_chunk(d, got)
    k, v = d["k"].to(DEV), d["v"].to(DEV)
    c = kara.cache(k, v, 10)
    bt = i32(d["bt"])
    ws = torch.empty(kara.kara_decode_workspace_size(c, 4, bt.shape[1]), dtype=torch.uint8, device=DEV)
    out = torch.empty(4, 10, 128, device=DEV)
    err = error_word()
    kara.kara_decode_attention(c, 0, i32(d["lengths"]), bt, d["q"].to(DEV), out, ws, err)
    assert kara.kara_get_error(err) == 0
    scale = plain_chunk(d["q"], d["k"], d["v"], 0, d["bt"], d["q_start"], d["lengths"], absolute=True)
    off = (got.double() - out.cpu().double()).abs()
    assert (off <= out.cpu().double().abs() * 2.0 ** -8 + scale * (2.0 ** -8 + 2.0 ** -10) + 2e-4).all()


@pytest.mark.parametrize("qscale", [0.0, 30.0, 300.0])
def test_chunk_flat_and_peaked_logits(qscale):
    """Equal logits, and logits whose maxima keep rising along the keys by far more than a power of two."""
    kara = lib()
    d = chunk_inputs(31, [600, 520], [40, 300], 4, 2, 128, qscale=qscale)
    if qscale:   # keys that grow along the sequence: the running maximum moves in every tile
        for s in range(2):
            for b in range(int(blocks(d["lengths"])[s])):
                d["k"][0, d["bt"][s, b]] = (d["k"][0, d["bt"][s, b]].float() * (b + 1) / 40).bfloat16()
    got, st = run_chunk(kara, d)
    assert st == 0
    ref = plain_chunk(d["q"], d["k"], d["v"], 0, d["bt"], d["q_start"], d["lengths"])
    scale = plain_chunk(d["q"], d["k"], d["v"], 0, d["bt"], d["q_start"], d["lengths"], absolute=True)
    # logits of magnitude |l| carry an absolute fp32 error of at most D 2^-24 sum|q k| / sqrt(D): here a
    # row's |q||k| / sqrt(D) is below qscale * 128 / 11.3 * 1.3, which enters a weight as a relative error
    err = 2 * 128 * 2.0 ** -24 * (qscale * 128 / 11.3 * 1.3)
    lim = ref.abs() * 2.0 ** -8 + scale * (2.0 ** -8 + 2.0 ** -10 + err) + err * 6
    assert ((got.double() - ref).abs() <= lim).all(), ((got.double() - ref).abs() - lim).max()


def test_chunk_strided_pool_views():
    kara = lib()
    d = chunk_inputs(41, [300, 77], [50, 77], 8, 2, 128, layers=2)
    L, nb, hkv, _, D = d["k"].shape
    big = torch.full((L + 1, nb, hkv + 3, 16, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    big2 = big.clone()
    kv, vv = big[:L, :, 1:1 + hkv], big2[:L, :, 1:1 + hkv]
    kv.copy_(d["k"])
    vv.copy_(d["v"])
    for layer in (0, 1):
        got, st = run_chunk(kara, d, layer, kv, vv)
        assert st == 0
        check_chunk(d, got, layer)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_chunk_earlier_tokens_do_not_see_later_values(value):
    """A token whose K or V is not finite (and every token after it) may give anything that its own sums
    give; the tokens before it are exact."""
    kara = lib()
    for pool in ("k", "v"):
        d = chunk_inputs(51, [200, 400], [150, 300], 4, 2, 128)
        bad = {0: 120, 1: 350}
        for s, x in bad.items():
            d[pool][0, d["bt"][s, x // 16], :, x % 16, 3] = value
        got, st = run_chunk(kara, d)
        assert st == 0
        rows = [t for s in (0, 1) for t in range(d["q_start"][s], d["q_start"][s + 1])
                if d["lengths"][s] - (d["q_start"][s + 1] - t) < bad[s]]
        check_chunk(d, got, rows=rows)
        if pool == "v":   # a seen value of infinity or NaN shows, in its dim and nowhere else
            seen = [t for s in (0, 1) for t in range(d["q_start"][s], d["q_start"][s + 1])
                    if d["lengths"][s] - (d["q_start"][s + 1] - t) >= bad[s]]
            ref = plain_chunk(d["q"], d["k"], d["v"], 0, d["bt"], d["q_start"], d["lengths"])
            assert torch.equal(torch.isfinite(got[seen]), torch.isfinite(ref[seen]))


def test_chunk_reports_bad_lengths_and_blocks():
    kara = lib()
    d = chunk_inputs(61, [100, 90, 80, 70], [10, 20, 30, 5], 4, 2, 64)
    bad = dict(d, lengths=d["lengths"].copy())
    bad["lengths"][1] = 19                                   # fewer cached than new
    got, st = run_chunk(kara, bad)
    assert st == kara.EINVAL and (got[10:30] == 0).all()
    ref, _ = run_chunk(kara, d)
    assert torch.equal(got[:10], ref[:10]) and torch.equal(got[30:], ref[30:])
    bad["lengths"][1] = 16 * d["bt"].shape[1] + 1            # past the table
    got, st = run_chunk(kara, bad)
    assert st == kara.EINVAL and (got[10:30] == 0).all() and torch.equal(got[:10], ref[:10])
    for bid in (-1, d["k"].shape[1]):                        # a bad id reads as zeros
        b2 = dict(d, bt=d["bt"].copy())
        b2["bt"][2, 1] = bid
        got, st = run_chunk(kara, b2)
        assert st == kara.EBADBLOCK
        check_chunk(b2, got)
    # rows out of order: the sequences whose rows are wrong give nothing outside [0, rows)
    for qs in ([0, 10, 5, 60, 65], [0, 10, 30, 60, 900], [-3, 10, 30, 60, 65]):
        got, st = run_chunk(kara, dict(d, q_start=np.array(qs, np.int32)))
        assert st == kara.EINVAL


def test_chunk_nothing_to_do():
    kara = lib()
    d = chunk_inputs(71, [50, 60], [0, 0], 4, 2, 64, extra=4)
    got, st = run_chunk(kara, d)
    assert st == 0 and (got == 77.0).all()


# ---- together --------------------------------------------------------------------

class Model:
    """Two layers' projections and a Compressor: what a serving loop keeps."""

    def __init__(self, kara, n, hq, hkv, D, W, nb, width, seed):
        from decode_kv_cache_03_gb300.compressor import Compressor
        g = torch.Generator().manual_seed(seed)
        self.kara, self.n, self.hq, self.hkv, self.D, self.W, self.layers = kara, n, hq, hkv, D, W, 2
        self.k = torch.full((2, nb, hkv, 16, D), float("nan"), dtype=torch.bfloat16, device=DEV)
        self.v = self.k.clone()
        self.B, self.K, self.R = 16, 8, 16
        self.comp = Compressor(self.k, self.v, hq, W, self.B, self.K, self.R)
        self.qw = (1 + 0.2 * torch.randn(D, generator=g)).bfloat16().to(DEV)
        self.kw = (1 + 0.2 * torch.randn(D, generator=g)).bfloat16().to(DEV)
        self.cs = angles(2000, D).to(DEV)
        self.shift = torch.zeros(n, dtype=torch.int32, device=DEV)
        self.rope = kara.rope(self.cs, self.qw, self.kw, 1e-6, False, self.shift)
        self.ring = torch.zeros(n, 2, hq, W, D, dtype=torch.bfloat16, device=DEV)
        self.bt = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
        self.len = torch.zeros(n, dtype=torch.int32, device=DEV)

    def step(self, n_new, fresh, rows, qkv):
        """One step over both layers; qkv [layers][rows][(hq + 2 hkv) D].  Returns (outputs, used)."""
        kara, hq, hkv, D = self.kara, self.hq, self.hkv, self.D
        b, _ = new_tokens(kara, self.n, rows)
        t = kara.tokens(b["q_start"], self.len, b["slot"], b["seq"], b["pos"])
        used = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.comp.extend(self.len, n_new, self.bt, fresh, t, used)
        outs = []
        for layer in range(2):
            x = qkv[layer]
            q = x[:, :hq * D].view(rows, hq, D)
            k = x[:, hq * D:(hq + hkv) * D].view(rows, hkv, D)
            v = x[:, (hq + hkv) * D:].view(rows, hkv, D)
            qo = torch.zeros(rows, hq, D, dtype=torch.bfloat16, device=DEV)
            o = torch.zeros_like(qo)
            self.comp.append(layer, t, self.rope, q, k, v, qo, ring=self.ring)
            self.comp.chunk(layer, t, self.bt, qo, o)
            outs.append((qo, o, b))
        return outs, used


def test_prefill_decode_compress_and_go_on():
    """Prompts in two chunks, decode steps, a compression of the window whose queries the appends kept in
    the ring, then more tokens with their rotary positions running on: outputs against a plain model that
    keeps each sequence's keys and values in lists, and the step's scores against the oracle."""
    kara = lib()
    n, hq, hkv, D, W = 3, 4, 2, 64, 64
    m = Model(kara, n, hq, hkv, D, W, 60, 16, 3)
    free = list(np.random.default_rng(0).permutation(60))
    g = torch.Generator().manual_seed(4)
    hist = [[[[], []] for _ in range(2)] for _ in range(n)]     # [seq][layer] -> keys, values
    true_pos = [0] * n
    cs, qw, kw = m.cs.cpu(), m.qw.cpu(), m.kw.cpu()

    def step(counts, pad):
        rows = sum(counts) + pad
        qkv = torch.randn(2, rows, (hq + 2 * hkv) * D, generator=g).bfloat16()
        fresh = i32(free[:20])
        outs, used = m.step(i32(counts), fresh, rows, qkv.to(DEV))
        assert m.comp.error() == 0
        del free[:int(used)]
        for layer in range(2):
            qo, o, _ = (x.cpu() if torch.is_tensor(x) else x for x in outs[layer])
            t = 0
            for s in range(n):
                for _ in range(counts[s]):
                    at = torch.tensor([true_pos[s] + _])
                    x = qkv[layer, t]
                    q, k = x[:hq * D].view(1, hq, D), x[hq * D:(hq + hkv) * D].view(1, hkv, D)
                    close_rows(qo[t][None], plain_turn(q, qw, 1e-6, cs, at, False),
                               plain_turn(q, qw, 1e-6, None, None, False))
                    # the cache holds the rounded keys: take them as the library rounded them
                    slot = int(outs[layer][2]["slot"][t])
                    kk = m.k[layer, slot // 16, :, slot % 16].cpu()
                    close_rows(kk[None], plain_turn(k, kw, 1e-6, cs, at, False),
                               plain_turn(k, kw, 1e-6, None, None, False))
                    hist[s][layer][0].append(kk)
                    hist[s][layer][1].append(x[(hq + hkv) * D:].view(hkv, D))
                    K, V = (torch.stack(h, 1).double() for h in hist[s][layer])
                    qq = qo[t].view(hkv, hq // hkv, D).double()
                    w = torch.softmax(qq @ K.transpose(1, 2) / D ** 0.5, -1)
                    ref, scale = (w @ V).view(hq, D), (w @ V.abs()).view(hq, D)
                    off = (o[t].double() - ref).abs()
                    assert (off <= ref.abs() * 2.0 ** -8 + scale * (2.0 ** -8 + 2.0 ** -10)).all(), (layer, s, t)
                    t += 1
            assert (o[t:] == 0).all() and (qo[t:] == 0).all()
        for s in range(n):
            true_pos[s] += counts[s]

    step([50, 0, 33], 2)
    step([40, 90, 47], 0)
    for _ in range(3):
        step([1, 1, 1], 1)
    # compress every sequence's window with the queries that the appends left in the ring
    lengths = m.len.cpu()
    _, _, tn, to = m.comp.plan(lengths, m.bt.shape[1])
    fresh, freed = i32(free[:tn]), torch.empty(to, dtype=torch.int32, device=DEV)
    del free[:tn]
    new_len = torch.empty(n, dtype=torch.int32, device=DEV)
    C = W - m.B
    scores = torch.empty(n, 2, hkv, C, device=DEV)
    kept = torch.empty(n, 2, hkv, m.R, dtype=torch.int32, device=DEV)
    k0, bt0 = m.k.cpu(), m.bt.cpu()
    m.comp.compress(m.len, m.bt, m.ring, fresh, freed, new_len, scores=scores, kept=kept)
    assert m.comp.error() == 0
    for s in range(n):
        L = int(lengths[s])
        for layer in range(2):
            kw_ = torch.stack(hist[s][layer][0], 1)[:, L - W:].double()
            for h in range(hkv):
                q = m.ring[s, layer, 2 * h:2 * h + 2].cpu().double()
                ref = torch.softmax(q @ kw_[h].T / D ** 0.5, -1).sum((0, 1))[:C]
                torch.testing.assert_close(scores[s, layer, h].cpu().double(), ref, rtol=1e-3, atol=0)
    kara.kara_compact_queries(m.comp.cache, m.comp.params, kara.batch(m.len, m.bt, m.ring), kept, m.comp.err)
    assert m.comp.error() == 0
    free.extend(freed.cpu().tolist())
    kc = kept.cpu()
    for s in range(n):
        L = int(lengths[s])
        for layer in range(2):
            for side in range(2):
                h = hist[s][layer][side]
                rows = torch.stack(h)                                     # [L][hkv][D]
                new = list(rows[:L - W])
                for j in range(m.R):
                    new.append(torch.stack([rows[L - W + kc[s, layer, gk, j], gk] for gk in range(hkv)]))
                hist[s][layer][side] = new + list(rows[L - m.B:])
    m.len.copy_(new_len)
    m.shift += C - m.R
    step([1, 30, 1], 0)
    step([20, 1, 70], 5)


def test_captured_step_replays():
    """extend, append and chunk attention of a decode step captured once and replayed: each replay
    advances the lengths in place and continues where the last one stopped."""
    kara = lib()
    n, hq, hkv, D = 4, 8, 2, 128
    m = Model(kara, n, hq, hkv, D, 64, 80, 20, 5)
    g = torch.Generator().manual_seed(6)
    mk = lambda: torch.randn(2, n, (hq + 2 * hkv) * D, generator=g).bfloat16().to(DEV)  # noqa: E731
    ids = np.random.default_rng(1).permutation(80)
    qkv, fresh = mk(), i32(ids[:n])
    n_new = i32([1] * n)
    m.step(n_new, fresh, n, qkv)                    # the workspace and kernels exist before the capture
    assert m.comp.error() == 0
    m.bt.fill_(-1)
    m.len.zero_()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        outs, used = m.step(n_new, fresh, n, qkv)
    keys = []
    at = 0
    for i in range(40):
        fresh.copy_(i32(ids[at:at + n]))
        qkv.copy_(mk())
        graph.replay()
        assert m.comp.error() == 0
        at += int(used)
        assert int(used) == (n if i % 16 == 0 else 0) and m.len.tolist() == [i + 1] * n
        keys.append((qkv[1].cpu(), outs[1][1].cpu(), outs[1][0].cpu()))
    d = dict(q=keys[-1][2], k=m.k.cpu(), v=m.v.cpu(), bt=m.bt.cpu().numpy(), q_start=np.arange(n + 1), hq=hq,
             lengths=np.full(n, 40, np.int32), rows=n)
    check_chunk(d, keys[-1][1], layer=1)


def test_two_streams_with_their_own_workspaces():
    """Two calls in flight at once, each with its own workspace, and one on a side stream."""
    kara = lib()
    ds = [chunk_inputs(80 + i, [3000 - 700 * i], [200 + 50 * i], 8, 2, 128) for i in range(2)]
    want = [run_chunk(kara, d)[0] for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    keep = []
    for d in ds:
        k, v, q = (d[x].to(DEV) for x in ("k", "v", "q"))
        c = kara.cache(k, v, 8)
        t, b = chunk_tokens(kara, d), i32(d["bt"])
        ws = torch.empty(kara.kara_chunk_workspace_size(c, t.n, t.rows), dtype=torch.uint8, device=DEV)
        keep.append((c, t, b, q, torch.zeros_like(q), ws, error_word(), k, v))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (c, t, b, q, o, ws, err, _, _) in zip(streams, keep):
            kara.kara_chunk_attention(c, 0, t, b, q, o, ws, err, stream=s)
    torch.cuda.synchronize()
    for w, (_, _, _, _, o, _, err, _, _) in zip(want, keep):
        assert torch.equal(o.cpu(), w) and int(err) == 0


def test_chunk_workspace_too_small_is_refused():
    kara = lib()
    d = chunk_inputs(91, [40], [4], 4, 2, 64)
    k, v = d["k"].to(DEV), d["v"].to(DEV)
    c = kara.cache(k, v, 4)
    t = chunk_tokens(kara, d)
    need = kara.kara_chunk_workspace_size(c, 1, 4)
    q = d["q"].to(DEV)
    with pytest.raises(kara.KaraError) as e:
        kara.kara_chunk_attention(c, 0, t, i32(d["bt"]), q, torch.empty_like(q),
                                  torch.empty(need - 1, dtype=torch.uint8, device=DEV), error_word())
    assert e.value.status == kara.EWORKSPACE


def test_stalled_chunk_attention_times_out(monkeypatch):
    """With KARA_DEBUG_STALL=1 no copy is issued: the bounded waits run out, the call reports it and the
    next call on the same context is right."""
    kara = lib()
    d = chunk_inputs(95, [300, 900, 40], [10, 200, 1], 8, 2, 128)
    monkeypatch.setenv("KARA_DEBUG_STALL", "1")
    _, st = run_chunk(kara, d)
    assert st == kara.ETIMEOUT
    monkeypatch.delenv("KARA_DEBUG_STALL")
    got, st = run_chunk(kara, d)
    assert st == 0
    check_chunk(d, got)


@pytest.mark.parametrize("hq,hkv,D,rot,inter,norm,W,rows,pad", [
    (40, 8, 128, 128, False, True, 128, 700, 3), (32, 8, 128, 64, True, False, 0, 801, 0),
    (4, 2, 64, 64, False, True, 64, 3000, 40), (8, 8, 64, 32, False, True, 0, 1001, 7),
    (18, 3, 128, 96, False, True, 64, 999, 1), (2, 2, 128, 0, False, True, 0, 5000, 0),
    (160, 20, 128, 128, False, True, 0, 150, 2), (320, 40, 128, 128, True, True, 0, 70, 1),
    (512, 256, 128, 128, False, True, 0, 30, 0)])
def test_append_long_calls(hq, hkv, D, rot, inter, norm, W, rows, pad):
    """Calls past the short kernel's limit: tokens staged with four, two and one CTAs per SM, and heads
    that fit no stage; padding in the middle as well as at the end."""
    kara = lib()
    r = np.random.default_rng(rows)
    m = rows // 2
    bt, fresh = make_tables(np.array([m, rows - m]), int(blocks(rows)) + 1, int(blocks(m) + blocks(rows - m)) + 2, 3)
    lengths, n_new = np.array([0, 0], np.int32), np.array([m, rows - m], np.int32)
    table, q_start, ln, slot, seq, pos, _ = plain_extend(lengths, n_new, np.full_like(bt, -1), np.concatenate(
        [bt[0][bt[0] >= 0], bt[1][bt[1] >= 0], fresh]), rows + pad)
    hole = r.integers(0, rows, 5)
    slot[hole] = -1
    q, k, v = append_inputs(rows, hq, hkv, D, rows + pad)
    g = torch.Generator().manual_seed(9)
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g)).bfloat16() for _ in range(2)) if norm else (None, None)
    cs = angles(6000, rot) if rot else None
    nb = int(table.max()) + 3
    kp = torch.zeros(1, nb, hkv, 16, D, dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    ring = torch.zeros(2, 1, hq, W, D, dtype=torch.bfloat16, device=DEV) if W else None
    q_out = torch.full((rows + pad, hq, D), 77.0, dtype=torch.bfloat16, device=DEV)
    t = kara.tokens(i32(q_start), i32(ln), torch.from_numpy(slot).to(DEV), i32(seq), i32(pos))
    keep = [x.to(DEV) if x is not None else None for x in (cs, qw, kw)]
    err = error_word()
    kara.kara_append_kv(kara.cache(kp, vp, hq), 0, t, kara.rope(keep[0], keep[1], keep[2], 1e-5, inter), *on_gpu(q, k, v),
                        q_out, err, ring=ring)
    assert kara.kara_get_error(err) == 0
    live = np.flatnonzero(slot >= 0)
    at = torch.from_numpy(pos[live]).long()
    got = q_out.cpu()
    gone = np.setdiff1d(np.arange(rows + pad), live)
    assert (got[gone] == 77.0).all()
    close_rows(got[live], plain_turn(q[live], qw, 1e-5, cs, at, inter), plain_turn(q[live], qw, 1e-5, None, None, inter))
    sl = torch.from_numpy(slot[live])
    kr = kp.cpu()[0].permute(0, 2, 1, 3).reshape(-1, hkv, D)
    vr = vp.cpu()[0].permute(0, 2, 1, 3).reshape(-1, hkv, D)
    close_rows(kr[sl], plain_turn(k[live], kw, 1e-5, cs, at, inter), plain_turn(k[live], kw, 1e-5, None, None, inter))
    assert torch.equal(vr[sl], v[live])
    rest = torch.ones(nb * 16, dtype=torch.bool)
    rest[sl] = False
    assert (kr[rest] == 0).all() and (vr[rest] == 0).all()
    if W:
        want = torch.zeros(2, 1, hq, W, D, dtype=torch.bfloat16)
        for i in live:
            if pos[i] >= ln[seq[i]] - W:
                want[seq[i], 0, :, pos[i] % W] = got[i]
        assert torch.equal(ring.cpu(), want)


def test_append_long_call_reports_bad_rows_and_stalls(monkeypatch):
    """Bad rows among the staged tokens are skipped and reported; with KARA_DEBUG_STALL=1 the waits run
    out; the next call is right."""
    kara = lib()
    hq, hkv, D, rows = 4, 2, 64, 4000
    q, k, v = append_inputs(8, hq, hkv, D, rows, fused=False)
    kp = torch.zeros(1, 250, hkv, 16, D, dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    dq, dk, dv, cs = q.to(DEV), k.to(DEV), v.to(DEV), angles(rows, D).to(DEV)

    def call(slot, seq, pos):
        t = kara.tokens(i32([0, rows]), i32([rows]), torch.from_numpy(slot).to(DEV), i32(seq), i32(pos))
        out = torch.full((rows, hq, D), 5.0, dtype=torch.bfloat16, device=DEV)
        err = error_word()
        kara.kara_append_kv(kara.cache(kp, vp, hq), 0, t, kara.rope(cs), dq, dk, dv, out, err)
        return kara.kara_get_error(err), out.cpu()

    slot, seq, pos = np.arange(rows), np.zeros(rows, np.int32), np.arange(rows)
    monkeypatch.setenv("KARA_DEBUG_STALL", "1")
    assert call(slot, seq, pos)[0] == kara.ETIMEOUT
    monkeypatch.delenv("KARA_DEBUG_STALL")
    st, good = call(slot, seq, pos)
    assert st == 0 and torch.equal(vp.cpu()[0].permute(0, 2, 1, 3).reshape(-1, hkv, D), v)
    for what in ("slot", "seq", "pos"):
        s2, q2, p2 = slot.copy(), seq.copy(), pos.copy()
        {"slot": s2, "seq": q2, "pos": p2}[what][1234] = 4000 if what != "pos" else -1
        st, got = call(s2, q2, p2)
        assert st == (kara.EBADBLOCK if what == "slot" else kara.EINVAL)
        assert (got[1234] == 5.0).all()
        keep = np.arange(rows) != 1234
        assert torch.equal(got[keep], good[keep])


def test_chunk_edge_tiles_again_and_again():
    """Many items with two and three edge tiles in a row (ragged ends, chunks across tile borders): the
    warps that clear them may be a tile apart."""
    kara = lib()
    r = np.random.default_rng(5)
    n_new = r.integers(100, 400, 12).astype(np.int32)
    lengths = n_new + r.integers(0, 200, 12).astype(np.int32)
    d = chunk_inputs(96, lengths, n_new, 8, 2, 128)
    first, st = run_chunk(kara, d)
    assert st == 0
    check_chunk(d, first)
    for _ in range(30):
        got, st = run_chunk(kara, d)
        assert st == 0 and torch.equal(got, first)


@pytest.mark.parametrize("n", [513, 1500])
def test_chunk_more_sequences_than_one_pass(n):
    """Batches past one pass of the prefix sums (512 sequences): single tokens, short chunks, sequences
    without new tokens, and some that are refused in between."""
    kara = lib()
    r = np.random.default_rng(n)
    n_new = r.integers(0, 4, n).astype(np.int32)
    n_new[r.integers(0, n, 5)] = r.integers(30, 150, 5)
    lengths = n_new + r.integers(0, 90, n).astype(np.int32)
    d = chunk_inputs(n, lengths, n_new, 4, 2, 64, extra=2)
    got, st = run_chunk(kara, d)
    assert st == 0
    check_chunk(d, got)
    bad = dict(d, lengths=d["lengths"].copy())
    refused = [i for i in (3, n // 2, n - 2) if n_new[i] > 0]
    for i in refused:
        bad["lengths"][i] = n_new[i] - 1
    again, st = run_chunk(kara, bad)
    assert st == (kara.EINVAL if refused else 0)
    for s in range(n):
        rows = slice(d["q_start"][s], d["q_start"][s + 1])
        assert s not in refused or (again[rows] == 0).all()
    pick = [t for s in range(n) if s not in refused for t in range(d["q_start"][s], d["q_start"][s + 1])]
    check_chunk(d, again, rows=pick)


@pytest.mark.parametrize("lengths, n_new, hq, hkv, D", [
    ([9000, 8300, 900, 2600], [1200, 800, 0, 5], 40, 8, 128),   # whole items ahead of the ranges
    ([2000] * 80, [300] * 80, 8, 8, 64),                        # two costs, in turn
    ([9000, 400, 300], [1, 400, 290], 16, 4, 64),               # too little work for whole items
    ([8000], [4000], 32, 4, 128),                               # one sequence, each pair sees more than the last
    ([2100, 17, 2100, 40], [2100, 1, 1500, 40], 2, 2, 128),
])
def test_chunk_items_of_shared_keys(lengths, n_new, hq, hkv, D):
    """Batches whose pairs of query tiles share keys: CTAs take whole items ahead of their ranges."""
    kara = lib()
    d = chunk_inputs(61, lengths, n_new, hq, hkv, D, extra=3)
    got, st = run_chunk(kara, d)
    assert st == 0
    check_chunk(d, got)
    again, st = run_chunk(kara, d)
    assert st == 0 and torch.equal(got, again)


def test_chunk_more_items_than_shared_memory_holds():
    """Long calls whose items are too many to be dealt round keep equal ranges."""
    kara = lib()
    n = 21000
    r = np.random.default_rng(5)
    n_new = r.integers(0, 3, n).astype(np.int32)
    n_new[[0, 7, 20481, n - 1]] = [300, 0, 513, 700]
    lengths = n_new + r.integers(0, 3, n).astype(np.int32)
    lengths[[0, n - 1]] += 900
    d = chunk_inputs(62, lengths, n_new, 4, 4, 64)
    got, st = run_chunk(kara, d)
    assert st == 0
    check_chunk(d, got)


def test_chunk_captured_call_follows_the_lengths():
    """One captured call, replayed over lengths that are shared out differently: long chunks that share
    keys, single tokens, nothing, and the long ones again, on a workspace that nobody clears."""
    kara = lib()
    n = 20
    d = chunk_inputs(63, [4000] * n, [400] * n, 16, 8, 128)
    k, v, q, bt = d["k"].to(DEV), d["v"].to(DEV), d["q"].to(DEV), i32(d["bt"])
    c, t = kara.cache(k, v, 16), chunk_tokens(kara, d)
    q_start = t.keep[0]
    ws = torch.full((kara.kara_chunk_workspace_size(c, n, t.rows),), 0xff, dtype=torch.uint8, device=DEV)
    out = torch.full(d["q"].shape, 77.0, dtype=torch.bfloat16, device=DEV)
    err = error_word()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    kara.kara_chunk_attention(c, 0, t, bt, q, out, ws, err)   # the kernels are loaded before the capture
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        kara.kara_chunk_attention(c, 0, t, bt, q, out, ws, err, torch.cuda.current_stream())
    first = None
    for new in ([400] * n, [1] * n, [0] * n, [400] * n, [0] * (n - 1) + [300]):
        at = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        q_start.copy_(i32(at))
        out.fill_(77.0)
        graph.replay()
        torch.cuda.synchronize()
        assert kara.kara_get_error(err) == 0
        got = out.cpu()
        if first is not None and new[0] == 400:
            assert torch.equal(got, first)
            continue
        first = got if new[0] == 400 else first
        check_chunk(dict(d, q_start=at), got)


def test_stalled_long_chunk_attention_times_out(monkeypatch):
    """The same for a call that deals whole items round."""
    kara = lib()
    d = chunk_inputs(64, [4000] * 20, [400] * 20, 16, 8, 128)
    monkeypatch.setenv("KARA_DEBUG_STALL", "1")
    _, st = run_chunk(kara, d)
    assert st == kara.ETIMEOUT
    monkeypatch.delenv("KARA_DEBUG_STALL")
    got, st = run_chunk(kara, d)
    assert st == 0
    check_chunk(d, got, rows=list(range(0, 8000, 7)))


def test_chunk_results_repeat_bit_for_bit():
    """Cuts and merges follow the lengths, not the timing."""
    kara = lib()
    d = chunk_inputs(98, [4000, 700, 33, 2048], [3, 400, 33, 1], 8, 2, 128)
    first, st = run_chunk(kara, d)
    assert st == 0
    for _ in range(20):
        assert torch.equal(run_chunk(kara, d)[0], first)


def test_chunk_output_alignment():
    """Outputs on a 16-byte boundary that is no 32-byte one."""
    kara = lib()
    d = chunk_inputs(99, [300, 40], [100, 3], 8, 2, 128)
    want, _ = run_chunk(kara, d)
    k, v, q = (d[x].to(DEV) for x in ("k", "v", "q"))
    c, t = kara.cache(k, v, 8), chunk_tokens(kara, d)
    flat = torch.full((q.numel() + 8,), 77.0, dtype=torch.bfloat16, device=DEV)
    out = flat[8:].view(q.shape)
    assert out.data_ptr() % 32 == 16
    ws = torch.empty(kara.kara_chunk_workspace_size(c, t.n, t.rows), dtype=torch.uint8, device=DEV)
    err = error_word()
    kara.kara_chunk_attention(c, 0, t, i32(d["bt"]), q, out, ws, err)
    assert kara.kara_get_error(err) == 0 and torch.equal(out.cpu(), want) and (flat[:8] == 77.0).all()


@pytest.mark.parametrize("rows", [3, 3000])
@pytest.mark.parametrize("rot,inter", [(0, False), (32, False), (32, True)])
def test_append_passes_dims_through_bit_for_bit(rows, rot, inter):
    """Without a norm, dims past rot_dim (all of them without a rotation) keep their bits, infinities, NaN
    and the sign of zero among them, in short calls and in staged ones."""
    kara = lib()
    hq, hkv, D = 4, 2, 64
    q, k, v = append_inputs(rows + rot, hq, hkv, D, rows, fused=False)
    for x in (q, k, v):
        x[0, 0, rot:rot + 5] = torch.tensor([float("inf"), -float("inf"), float("nan"), -0.0, 0.0])
        x[rows - 1, 1, 40:43] = torch.tensor([-0.0, float("inf"), 3e38])
    nb = rows // 16 + 1
    kp = torch.zeros(1, nb, hkv, 16, D, dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    t = kara.tokens(i32([0, rows]), i32([rows]), torch.arange(rows, device=DEV), i32([0] * rows), i32(range(rows)))
    out = torch.empty(rows, hq, D, dtype=torch.bfloat16, device=DEV)
    err = error_word()
    cs = angles(rows, rot).to(DEV) if rot else None
    kara.kara_append_kv(kara.cache(kp, vp, hq), 0, t, kara.rope(cs, interleaved=inter), q.to(DEV), k.to(DEV),
                        v.to(DEV), out, err)
    assert kara.kara_get_error(err) == 0
    rows_of = lambda p: p.cpu()[0].permute(0, 2, 1, 3).reshape(-1, hkv, D)[:rows]  # noqa: E731
    for got, want in ((out.cpu(), q), (rows_of(kp), k)):
        a, b = got[..., rot:].contiguous().view(torch.int16), want[..., rot:].contiguous().view(torch.int16)
        nan = torch.isnan(want[..., rot:])
        assert torch.equal(a[~nan], b[~nan]) and torch.isnan(got[..., rot:][nan]).all()
        assert torch.isfinite(got[1:-1, :, :rot]).all()
    assert torch.equal(rows_of(vp).contiguous().view(torch.int16), v.view(torch.int16))
