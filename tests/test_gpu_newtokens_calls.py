"""New-token calls as a program makes them: empty steps, several host threads, streams, other lengths."""
import numpy as np
import pytest
import torch

from _gpu import lib
from _newtokens import plain_extend
from test_gpu_newtokens import DEV, assert_nothing_done, i32, new_tokens, run_extend

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
