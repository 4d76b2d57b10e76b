"""GPU tests of the 8-bit cache's calls where blocks' scales lie far apart, against 64 bits."""

import numpy as np
import pytest
import torch

from _cache8 import BS, plain_compact, source_rows, value
from _newtokens import blocks
from test_gpu_cache8 import run_compact, window_case

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
