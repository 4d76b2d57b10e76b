"""Chunk attention over the bf16 cache keeps its bits: the order of its fp32 sums is part of what it returns."""

import hashlib

import numpy as np
import pytest
import torch

from _gpu import lib

pytestmark = pytest.mark.gpu

DEV = "cuda"
# (heads, D, cached tokens, new tokens): the first 16 digits of sha256 over the outputs' bytes, on 152 SMs
GOLDEN = {(40, 8, 128, (3000,) * 4, (300,) * 4): "b9787ea0d627aadb",
          (32, 8, 128, (2000,) * 48, (4,) * 48): "73edc2cc446a256b",
          (16, 4, 64, (900, 3000, 20, 1500), (700, 300, 900, 1)): "1674d1921ca4f59d"}


def numbers(n, seed, scale):
    """n bf16 values, multiples of 2^-6 / scale, from integers alone."""
    x = (np.arange(n, dtype=np.uint64) + np.uint64(seed << 32)) * np.uint64(0x9e3779b97f4a7c15)
    x = (x ^ (x >> np.uint64(29))) * np.uint64(0xbf58476d1ce4e5b9)
    x = ((x >> np.uint64(40)) & np.uint64(255)).astype(np.int64) - 128
    return torch.from_numpy((x / 64.0 / scale).astype(np.float32)).bfloat16()


def run(hq, hkv, d, old, new):
    kara = lib()
    lengths = [a + b for a, b in zip(old, new)]
    want = [(x + 15) // 16 for x in lengths]
    nb, rows, width = sum(want), sum(new), max(want)
    k, v = (numbers(nb * hkv * 16 * d, i, 1).view(1, nb, hkv, 16, d).to(DEV) for i in (1, 2))
    q = numbers(rows * hq * d, 3, 1).view(rows, hq, d).to(DEV)
    table = torch.full((len(old), width), -1, dtype=torch.int32)
    at = 0
    for s, w in enumerate(want):
        table[s, :w] = torch.arange(at, at + w)
        at += w
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    z4 = torch.zeros(rows, dtype=torch.int32, device=DEV)
    t = kara.tokens(i32([0, *np.cumsum(new).tolist()]), i32(lengths), torch.zeros(rows, dtype=torch.int64, device=DEV), z4,
                    z4.clone())
    c, err, out = kara.cache(k, v, hq), i32([0]), torch.zeros_like(q)
    ws = torch.empty(kara.kara_chunk_workspace_size(c, t.n, t.rows), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    kara.kara_chunk_attention(c, 0, t, table.to(DEV), q, out, ws, err)
    assert kara.kara_get_error(err) == 0
    return out.cpu()


@pytest.mark.parametrize("case", range(len(GOLDEN)))
def test_chunk_attention_keeps_its_bits(case):
    args = list(GOLDEN)[case]
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("where a call is cut follows the number of SMs")
    out = run(*args)
    assert hashlib.sha256(out.view(torch.int16).numpy().tobytes()).hexdigest()[:16] == GOLDEN[args]
