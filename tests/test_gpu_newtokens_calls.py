"""New-token calls as a program makes them: empty steps, several host threads, streams, other lengths."""
import numpy as np
import pytest
import torch

from _gpu import lib
from _newtokens import plain_chunk, plain_extend
from test_gpu_newtokens import DEV, assert_nothing_done, chunk_inputs, i32, new_tokens, run_chunk, run_extend

pytestmark = pytest.mark.gpu


def test_extend_of_no_sequences_and_no_rows():
    """A step without sequences and rows still says that it took nothing: buffers that the last step filled
    are not read again as this one's, eagerly, captured, on a side stream and after an earlier error."""
    kara = lib()
    for earlier in (0, kara.EBADBLOCK):
        b, t = new_tokens(kara, 0, 0)
        used = torch.full((1,), 41, dtype=torch.int32, device=DEV)
        err = torch.full((1,), earlier, dtype=torch.int32, device=DEV)
        none, table, fresh = i32([]), i32(np.zeros((0, 3))), i32([5, 6])
        call = lambda s=None: kara.kara_extend_tables(9, 16, none, none, table, fresh, t, used, err, s)  # noqa: E731
        call()
        assert used.item() == 0 and b["q_start"].tolist() == [0] and err.item() == earlier
        side = torch.cuda.Stream()
        used.fill_(41)
        side.wait_stream(torch.cuda.current_stream())
        call(side)
        side.synchronize()
        assert used.item() == 0
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for _ in range(2):
            used.fill_(41)
            b["q_start"].fill_(-77)
            graph.replay()
            assert used.item() == 0 and b["q_start"].tolist() == [0]
        assert fresh.tolist() == [5, 6]


def test_extend_takes_the_largest_pool():
    """Ids up to 2^31 - 2: every window of the bitmap is looked at, once."""
    kara = lib()
    nb = (1 << 31) - 1
    lengths, n_new = np.array([20, 0], np.int32), np.array([30, 17], np.int32)
    bt = np.array([[7, nb - 3, -1, -1], [-1, -1, -1, -1]], np.int32)
    fresh = np.array([nb - 1, 0, (1 << 30) + 5, nb - 2], np.int32)
    want = plain_extend(lengths, n_new, bt, fresh, 50)
    st, got = run_extend(kara, lengths, n_new, bt, fresh, 50, nb)
    assert st == 0 and all(np.array_equal(g, w) for g, w in zip(got, want))
    for at, bad, code in ((2, nb - 1, kara.EDUPBLOCK), (0, nb - 3, kara.EDUPBLOCK), (1, nb, kara.EBADBLOCK)):
        f = fresh.copy().astype(np.int64)
        f[at] = bad
        st, got = run_extend(kara, lengths, n_new, bt, f.astype(np.int32), 50, nb)
        assert st == code
        assert_nothing_done(got, lengths, bt)


def test_chunk_values_of_short_items_that_follow_each_other():
    """Every sequence has new values that are not finite: items of two query tiles, each followed by four of
    one query tile and one key tile, whose values are cleared while the first is still being finished."""
    kara = lib()
    n_new = [64, 3, 1, 32, 2] * 130
    lengths = [m + (s * 7) % 50 * (m < 64) for s, m in enumerate(n_new)]
    d = chunk_inputs(73, lengths, n_new, 8, 2, 128, extra=1)
    for s, (L, m) in enumerate(zip(lengths, n_new)):
        x = L - m + (s * 5) % m
        d["v"][0, d["bt"][s, x // 16], :, x % 16, s % 128] = [float("inf"), -float("inf"), float("nan")][s % 3]
    want = plain_chunk(d["q"], d["k"], d["v"], 0, d["bt"], d["q_start"], d["lengths"])
    first = None
    for _ in range(20):
        got, st = run_chunk(kara, d)
        assert st == 0
        n = want.shape[0] - 1
        if first is None:
            ok = torch.isfinite(want[:n])
            assert torch.equal(torch.isfinite(got[:n]), ok)
            assert torch.equal(torch.isnan(got[:n]), torch.isnan(want[:n]))
            assert torch.equal(got[:n].double()[torch.isinf(want[:n])], want[:n][torch.isinf(want[:n])])
            # every finite value: the dims that hold none of those, against values without them
            clean = dict(d, v=torch.nan_to_num(d["v"], 0.0, 0.0, 0.0))
            ref = plain_chunk(d["q"], d["k"], clean["v"], 0, d["bt"], d["q_start"], d["lengths"])
            scale = plain_chunk(d["q"], d["k"], clean["v"], 0, d["bt"], d["q_start"], d["lengths"], absolute=True)
            lim = ref.abs() * 2.0 ** -8 + scale * (2.0 ** -8 + 2.0 ** -10)
            assert ((got.double() - ref).abs()[:n][ok] <= lim[:n][ok]).all()
            first = got.view(torch.int16)
        assert torch.equal(got.view(torch.int16), first)
