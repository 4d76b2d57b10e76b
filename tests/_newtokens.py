"""Inputs and 64-bit plain forms of the new-token operators (tables, append, chunk attention).

Everything here is numpy / torch on the CPU, written from the formulas in include/kara.h."""
import numpy as np
import torch

BS = 16


def blocks(x):
    return (x + BS - 1) // BS


def make_tables(lengths, width, num_blocks, seed):
    """Distinct shuffled ids for ceil(len/16) blocks of each sequence; the other entries are -1.
    Returns (table, the ids left over)."""
    ids = np.random.default_rng(seed).permutation(num_blocks).astype(np.int32)
    bt = np.full((len(lengths), width), -1, np.int32)
    at = 0
    for s, L in enumerate(lengths):
        nb = blocks(int(L))
        bt[s, :nb] = ids[at:at + nb]
        at += nb
    assert at <= num_blocks
    return bt, ids[at:].copy()


def plain_extend(lengths, n_new, table, fresh, rows):
    """(table, q_start, len, slot, seq, pos, used) of a call without errors."""
    table = table.copy()
    q_start, at, used = [0], 0, 0
    slot, seq, pos = (np.full(rows, -1, np.int64), np.full(rows, -1, np.int32), np.full(rows, -1, np.int32))
    for s, (L, m) in enumerate(zip(lengths.tolist(), n_new.tolist())):
        for b in range(blocks(L), blocks(L + m)):
            table[s, b] = fresh[used]
            used += 1
        for x in range(L, L + m):
            slot[at], seq[at], pos[at] = int(table[s, x // BS]) * BS + x % BS, s, x
            at += 1
        q_start.append(at)
    return (table, np.array(q_start, np.int32), (lengths + n_new).astype(np.int32), slot, seq, pos,
            np.array([used], np.int32))


def plain_turn(x, w, eps, cos_sin, r, inter):
    """Norm (weight w or None) and rotation at table rows r of x [rows][heads][D], in float64."""
    y = x.double().clone()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    if cos_sin is None:
        return y
    rot = cos_sin.shape[1]
    z = y.clone()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        c, s = cos_sin[r, i].double()[:, None], cos_sin[r, rot // 2 + i].double()[:, None]
        z[..., a] = y[..., a] * c - y[..., b] * s
        z[..., b] = y[..., b] * c + y[..., a] * s
    return z


def plain_chunk(q, kpool, vpool, layer, table, q_start, lengths, absolute=False):
    """Causal attention in float64: q [rows][hq][D], pools [layers][blocks][hkv][16][D].  A block id
    outside the pool counts as zeros.  With `absolute` the weights sum |v| (the scale of a weight's
    rounding in the output)."""
    rows, hq, D = q.shape
    nb_all, hkv = kpool.shape[1], kpool.shape[2]
    G = hq // hkv
    out = torch.zeros(rows, hq, D, dtype=torch.float64)
    for s in range(len(lengths)):
        t0, t1, L = int(q_start[s]), int(q_start[s + 1]), int(lengths[s])
        if t1 == t0:
            continue
        ids = torch.tensor([int(b) for b in table[s, :blocks(L)]])
        inside = (ids >= 0) & (ids < nb_all)

        def rows_of(pool):
            x = pool[layer, torch.where(inside, ids, 0)].double()
            x[~inside] = 0.0
            return x.permute(1, 0, 2, 3).reshape(hkv, -1, D)[:, :L]

        k, v = rows_of(kpool), rows_of(vpool)
        v = v.abs() if absolute else v
        if torch.isfinite(k).all() and torch.isfinite(v).all():
            late = torch.arange(L)[None] > torch.arange(L - (t1 - t0), L)[:, None]
            for g in range(hkv):
                z = torch.einsum("thd,xd->htx", q[t0:t1, g * G:(g + 1) * G].double(), k[g]) / D ** 0.5
                w = torch.softmax(z.masked_fill(late, -float("inf")), -1)
                out[t0:t1, g * G:(g + 1) * G] = (w @ v[g]).transpose(0, 1)
            continue
        for t in range(t0, t1):   # a token's sums hold its own keys only: nothing of later ones enters
            p = L - (t1 - t)
            for g in range(hkv):
                w = torch.softmax(q[t, g * G:(g + 1) * G].double() @ k[g, :p + 1].T / D ** 0.5, -1)
                out[t, g * G:(g + 1) * G] = w @ v[g, :p + 1]
    return out
