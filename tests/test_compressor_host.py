"""The workspaces of Compressor and Compressor8, without a GPU: the pools lie in host memory and no call is made."""

import pytest
import torch


def make8(layers=2, nb=9, hkv=2, d=64, hq=4, W=64):
    from decode_kv_cache_03_gb300 import Compressor8, build
    build.build()
    codes = [torch.zeros(layers, nb, hkv, 16, d, dtype=torch.uint8) for _ in range(2)]
    scales = [torch.zeros(layers, nb, hkv) for _ in range(2)]
    return Compressor8(*codes, *scales, hq, W, 16, 8, 16)


def test_workspace_needs_the_width_of_the_tables():
    """A compression over the 8-bit cache has a table of its own in its workspace: reserved without the tables'
    width it would be too small, and allocated anew inside the first call, a captured one too."""
    comp = make8()
    with pytest.raises(TypeError):
        comp.workspace(3)
    ws = comp.workspace(3, bt_stride=40)
    assert comp.workspace(3, None, bt_stride=40).data_ptr() == ws.data_ptr()
    for n, width in ((3, 40), (3, 7), (1, 40)):
        sizes = comp._compress_sizes(n, width)
        assert sizes[1] == 4 * n * width and comp._space("_xws", sum(sizes), None).data_ptr() == ws.data_ptr()


def test_windows_keep_their_memory():
    """What `windows` describes stays allocated while it is held, also when the workspace grew since."""
    comp = make8()
    windows = comp._window_cache(comp.workspace(1, bt_stride=4), 1)
    comp.workspace(3, bt_stride=40)
    where = windows.keep.untyped_storage()
    assert where.data_ptr() <= windows.k < where.data_ptr() + where.nbytes()


@pytest.mark.parametrize("name", ["_dws", "_cws", "_xws", "_ws"])
def test_captured_workspaces_outlive_their_growth(name, monkeypatch):
    """A workspace that a captured call uses is not given back when a later call needs a larger one: the graph
    writes to it whenever it is replayed.  One that no graph uses is."""
    comp = make8()
    capturing = False
    monkeypatch.setattr(comp, "_capturing", lambda stream: capturing, raising=False)
    for capturing, size in ((False, 100), (True, 200), (True, 150), (False, 300), (False, 400)):
        comp._space(name, size, None)
    kept = [getattr(comp, name), *getattr(comp, "_in_graphs", [])]
    assert sorted(x.numel() for x in kept) == [200, 400]
