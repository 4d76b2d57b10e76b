"""GPU tests of the workspaces that Compressor and Compressor8 hold, over graphs and larger calls."""

import pytest
import torch

from _cache8 import dense
from _gpu import lib
from test_gpu_cache8 import DEV, decode_case, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("given", [False, True])
def test_a_larger_call_leaves_a_graph_its_workspace(bits, given):
    """Decode attention of one sequence captured, then called for many: the graph's workspace is not given back,
    replays give the same bits and write to nothing else's memory."""
    from decode_kv_cache_03_gb300 import Compressor, Compressor8
    lib()
    lengths, bt, k, ks, v, vs, q = decode_case(8, [2500] + [600 + 9 * i for i in range(40)], 8, 2, 128)
    if bits == 8:
        pools = [x.to(DEV) for x in (k, v, ks, vs)]
        comp, dtype = Compressor8(*pools, 8, 64, 16, 8, 16), torch.bfloat16
    else:
        pools = [dense(k, ks).bfloat16().to(DEV), dense(v, vs).bfloat16().to(DEV)]
        comp, dtype = Compressor(*pools, 8, 64, 16, 8, 16), torch.float32
    ln, table, qd = i32(lengths), i32(bt), q.to(DEV)
    one, out = torch.zeros_like(qd[:1], dtype=dtype), torch.zeros_like(qd, dtype=dtype)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream = side if given else None
    small = lambda: comp.decode(1, ln[:1], table[:1], qd[:1], one, stream=stream)  # noqa: E731
    with torch.cuda.stream(side):
        small()
    torch.cuda.synchronize()
    want, at, size = one.clone(), comp._dws.data_ptr(), comp._dws.numel()
    with torch.cuda.graph(graph, stream=side):
        small()
    with torch.cuda.stream(side):
        comp.decode(1, ln, table, qd, out, stream=stream)
        assert comp._dws.data_ptr() != at
        others = [torch.full((size,), 7, dtype=torch.uint8, device=DEV) for _ in range(8)]
        assert all(not at <= x.data_ptr() < at + size for x in others)
    for _ in range(3):
        one.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert comp.error() == 0 and torch.equal(one, want) and all((x == 7).all() for x in others)
