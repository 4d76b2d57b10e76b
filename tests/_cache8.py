"""The 8-bit cache in 64 bits: codes, scales and the plain forms of its operators.

Everything here is torch / numpy on the CPU, written from the formulas in include/kara.h."""
import numpy as np
import torch

from _newtokens import BS, blocks

# value of each code: s eeee mmm, bias 7; exponent 0: subnormals; 0x7f and 0xff: NaN
VALUE = torch.tensor([(-1.0 if b > 127 else 1.0) * (float("nan") if b & 127 == 127 else
                      (b & 7) * 2.0 ** -9 if (b >> 3 & 15) == 0 else (8 + (b & 7)) * 2.0 ** ((b >> 3 & 15) - 10))
                      for b in range(256)], dtype=torch.float64)
E_MIN, E_MAX = -63, 63


def value(codes):
    return VALUE[codes.long()]


def round_code(x):
    """The nearest code of each float64 (ties to the even one), 448 above it, NaN for NaN."""
    grid = VALUE[:127].contiguous()
    a = x.abs().clamp(max=448.0)
    hi = torch.searchsorted(grid, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    to_hi, to_lo = grid[hi] - a, a - grid[lo]
    code = torch.where((to_hi < to_lo) | ((to_hi == to_lo) & (hi % 2 == 0)), hi, lo)
    code = torch.where(torch.isnan(x), 127, code)
    return (code + torch.where(torch.signbit(x), 128, 0)).to(torch.uint8)


def scale_of(amax):
    """The smallest power of two s with amax <= 448 s (float64; 0 for 0)."""
    powers = torch.tensor([2.0 ** e for e in range(E_MIN, E_MAX + 1)], dtype=torch.float64)
    i = torch.searchsorted(powers * 448.0, amax.double().contiguous()).clamp(max=len(powers) - 1)
    return torch.where(amax > 0, powers[i], 0.0)


def quantise(x):
    """Codes and scales of whole blocks x [..., 16, D]; a negative scale where a value is not finite."""
    x = x.double()
    fine = torch.isfinite(x)
    s = scale_of(torch.where(fine, x, 0.0).abs().amax((-1, -2)))
    codes = divide(torch.where(fine, x, float("nan")), s[..., None, None])
    return codes, torch.where(fine.all(-1).all(-1), s, -s).float()


def divide(x, s):
    """Codes of x / s, 0 for s = 0 (NaN stays)."""
    return round_code(torch.where(s > 0, x / torch.where(s > 0, s, 1.0), x * 0.0))


def dense(codes, scale):
    """Stored values in float64, codes [..., 16, D], scale [...]."""
    return value(codes) * scale.double().abs()[..., None, None]


def random_pool(shape, seed, spread=2, device="cpu"):
    """Codes and scales of random values whose blocks differ in magnitude by powers of two."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * 2.0 ** torch.randint(-spread, spread + 1, shape[:3], generator=g)[..., None, None]
    codes, scale = quantise(x)
    return codes.to(device), scale.to(device)


def runs(slot, ok=None):
    """(first row, rows, block, first row of the block) of each run of consecutive slots in one block."""
    found, t, n = [], 0, len(slot)
    while t < n:
        if slot[t] < 0 or (ok is not None and not ok[t]):
            t += 1
            continue
        m = 1
        while t + m < n and slot[t + m] == slot[t] + m and slot[t + m] % BS and (ok is None or ok[t + m]):
            m += 1
        found.append((t, m, int(slot[t]) // BS, int(slot[t]) % BS))
        t += m
    return found


def plain_decode(q, kv, layer, table, lengths, absolute=False):
    """Decode attention in float64: q [n][hq][D], kv = (k, v) values [layers][blocks][hkv][16][D]."""
    n, hq, D = q.shape
    k_all, v_all = kv
    nb_all, hkv = k_all.shape[1], k_all.shape[2]
    G = hq // hkv
    out = torch.zeros(n, hq, D, dtype=torch.float64)
    for s in range(n):
        L = int(lengths[s])
        if L <= 0:
            continue
        ids = torch.tensor([int(b) for b in table[s, :blocks(L)]])
        inside = (ids >= 0) & (ids < nb_all)

        def rows_of(pool):
            x = pool[layer, torch.where(inside, ids, 0)].clone()
            x[~inside] = 0.0
            return x.permute(1, 0, 2, 3).reshape(hkv, -1, D)[:, :L]

        k, v = rows_of(k_all), rows_of(v_all)
        v = v.abs() if absolute else v
        for g in range(hkv):
            w = torch.softmax(q[s, g * G:(g + 1) * G].double() @ k[g].T / D ** 0.5, -1)
            out[s, g * G:(g + 1) * G] = w @ v[g]
    return out


def plain_compact(codes, scale, layer_rows):
    """Codes and scales of rebuilt blocks: layer_rows [..., rows, D] stored values in order, 16 to a block
    (the last one may have fewer).  Returns lists over the blocks."""
    found = []
    for b in range(blocks(layer_rows.shape[-2])):
        x = layer_rows[..., b * BS:(b + 1) * BS, :]
        odd = torch.isnan(x)
        s = scale_of(torch.where(odd, 0.0, x).abs().amax((-1, -2)))
        found.append((divide(x, s[..., None, None]), torch.where(odd.any(-1).any(-1), -s, s)))
    return found


def source_rows(L, W, B, R, kept):
    """Old positions of the rows from the first rebuilt block on: prefix head, kept rows, buffer."""
    ws = L - W
    return np.concatenate([np.arange(ws // BS * BS, ws), ws + np.asarray(kept), np.arange(L - B, L)])
