"""New-token calls as a program makes them: empty steps, several host threads, streams, other lengths."""
import ctypes
import threading

import numpy as np
import pytest
import torch

from _gpu import lib
from _newtokens import blocks, make_tables, plain_chunk, plain_extend, plain_turn
from test_gpu_newtokens import (DEV, angles, append_inputs, assert_nothing_done, check_chunk, chunk_inputs,
                                chunk_tokens, close_rows, error_word, i32, new_tokens, on_gpu, run_chunk, run_extend)

pytestmark = pytest.mark.gpu


class NodeParams(ctypes.Structure):   # CUDA_KERNEL_NODE_PARAMS_v2
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("smem", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def launches(call):
    """The kernels that call(stream) would launch, captured and not run: (grid, dynamic shared memory, the
    limit of that which the function has now)."""
    cu = ctypes.CDLL("libcuda.so.1")
    s = torch.cuda.Stream()
    handle, graph, n = ctypes.c_void_p(s.cuda_stream), ctypes.c_void_p(), ctypes.c_size_t(0)

    def do(f, *args):
        assert getattr(cu, f)(*args) == 0, f

    do("cuStreamBeginCapture_v2", handle, 1)   # of this thread alone
    try:
        call(s)
    finally:
        ended = cu.cuStreamEndCapture(handle, ctypes.byref(graph))
    assert ended == 0
    do("cuGraphGetNodes", graph, None, ctypes.byref(n))
    nodes = (ctypes.c_void_p * n.value)()
    do("cuGraphGetNodes", graph, nodes, ctypes.byref(n))
    out = []
    for node in nodes:
        kind = ctypes.c_int(-1)
        do("cuGraphNodeGetType", ctypes.c_void_p(node), ctypes.byref(kind))
        if kind.value != 0:
            continue
        p, limit = NodeParams(), ctypes.c_int(0)
        do("cuGraphKernelNodeGetParams_v2", ctypes.c_void_p(node), ctypes.byref(p))
        func = ctypes.c_void_p(p.func)
        if not p.func:
            do("cuKernelGetFunction", ctypes.byref(func), ctypes.c_void_p(p.kern))
        do("cuFuncGetAttribute", ctypes.byref(limit), 8, func)   # the most dynamic shared memory
        out.append((tuple(p.grid), p.smem, limit.value))
    do("cuGraphDestroy", graph)
    return out


def append_call(kara, hq, hkv, D, rows, rot=0, inter=False):
    """An append of `rows` tokens of one sequence, as a function of the stream; q_out, the pools, the error word."""
    q, k, v = (x.to(DEV) for x in append_inputs(hq + rows, hq, hkv, D, rows, fused=False))
    nb = (rows + 15) // 16
    kp = torch.zeros(1, nb, hkv, 16, D, dtype=torch.bfloat16, device=DEV)
    vp, out, err = torch.zeros_like(kp), torch.zeros_like(q), error_word()
    t = kara.tokens(i32([0, rows]), i32([rows]), torch.arange(rows, device=DEV), i32([0] * rows), i32(range(rows)))
    c, r = kara.cache(kp, vp, hq), kara.rope(angles(rows, rot).to(DEV) if rot else None, interleaved=inter)
    torch.cuda.synchronize()
    return (lambda s=None: kara.kara_append_kv(c, 0, t, r, q, k, v, out, err, stream=s)), out, (kp, vp), err


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


def test_calls_of_other_shapes_keep_the_shared_memory_limit():
    """A kernel's limit of dynamic shared memory is one value for all host threads: a call of another shape
    does not lower it between a larger call's setting of it and its launch."""
    kara = lib()
    big, small = append_call(kara, 160, 20, 128, 600), append_call(kara, 4, 2, 128, 3000)
    (_, need, had), = launches(big[0])
    (_, less, now), = launches(small[0])
    assert less < need <= had and now >= need
    b, t = new_tokens(kara, 1, 4)
    err, used, table, fresh = error_word(), i32([0]), i32([[1, -1]]), i32([2])
    lengths, n_new = i32([16]), i32([4])
    ext = lambda nb: lambda s: kara.kara_extend_tables(  # noqa: E731
        nb, 16, lengths, n_new, table, fresh, t, used, err, s)
    torch.cuda.synchronize()
    (_, need, had), = launches(ext(1 << 20))
    (_, less, now), = launches(ext(500000))
    assert less < need <= had and now >= need


def test_two_host_threads_with_other_shapes():
    """A wide and a narrow model append from two threads, each on a stream of its own."""
    kara = lib()
    calls = [append_call(kara, 160, 20, 128, 300), append_call(kara, 4, 2, 128, 3000)]
    for call, *_ in calls:
        call()
    torch.cuda.synchronize()
    want = [(out.clone(), kp.clone(), vp.clone()) for _, out, (kp, vp), _ in calls]
    failed = []

    def work(call):
        s = torch.cuda.Stream()
        try:
            for _ in range(2000):
                call(s)
        except Exception as e:   # noqa: BLE001 (told to the test's thread)
            failed.append(e)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(call,)) for call, *_ in calls]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not failed
    for (_, out, (kp, vp), err), now in zip(calls, want):
        assert err.item() == 0 and all(torch.equal(a, b) for a, b in zip((out, kp, vp), now))


@pytest.mark.parametrize("what", ["chunk", "decode", "workspace"])
def test_compressor_workspace_belongs_to_its_stream(what):
    """The workspace of a call on a given stream is that stream's memory: not a block that the current stream
    has just given back, and may still be using."""
    from decode_kv_cache_03_gb300 import Compressor
    kara = lib()
    d = chunk_inputs(71, [300, 90], [1, 1], 8, 2, 128)
    k, v, q, bt, ln = d["k"].to(DEV), d["v"].to(DEV), d["q"].to(DEV), i32(d["bt"]), i32(d["lengths"])
    t = chunk_tokens(kara, d)
    comp = Compressor(k, v, 8, 64, 16, 8, 20)
    side, out = torch.cuda.Stream(), torch.empty_like(q)
    out32 = torch.empty(q.shape, dtype=torch.float32, device=DEV)
    size = {"chunk": kara.kara_chunk_workspace_size(comp.cache, t.n, t.rows),
            "decode": kara.kara_decode_workspace_size(comp.cache, *bt.shape),
            "workspace": kara.kara_workspace_size(comp.cache, comp.params, 2)}[what]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    given_back = torch.empty(size, dtype=torch.uint8, device=DEV)
    at = given_back.data_ptr()
    del given_back
    if what == "chunk":
        comp.chunk(0, t, bt, q, out, stream=side)
        ws = comp._cws
    elif what == "decode":
        comp.decode(0, ln, bt, q, out32, stream=side)
        ws = comp._dws
    else:
        ws = comp.workspace(2, stream=side)
    assert ws.numel() >= size and ws.data_ptr() != at
    again = torch.empty(size, dtype=torch.uint8, device=DEV)   # (the current stream still has its block)
    assert again.data_ptr() == at
    side.synchronize()
    if what == "chunk":
        check_chunk(d, out.cpu())
    assert comp.error() == 0


def test_compressor_workspace_outlives_calls_on_other_streams():
    """Dropped while a call on another stream than its own may still run, a workspace is not handed out
    until that call has run, and the error word is not."""
    from decode_kv_cache_03_gb300 import Compressor
    kara = lib()
    d = chunk_inputs(72, [300, 90], [1, 1], 8, 2, 128)
    k, v, q, bt = d["k"].to(DEV), d["v"].to(DEV), d["q"].to(DEV), i32(d["bt"])
    t, side, out = chunk_tokens(kara, d), torch.cuda.Stream(), torch.empty_like(q)
    comp = Compressor(k, v, 8, 64, 16, 8, 20)
    comp.chunk(0, t, bt, q, out)              # the workspace is the current stream's
    at, size, word = comp._cws.data_ptr(), comp._cws.numel(), comp.err.data_ptr()
    busy, dump = torch.randn(8192, 8192, device=DEV), torch.empty(8192, 8192, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(10):                    # milliseconds ahead of the call
            torch.mm(busy, busy, out=dump)
    comp.chunk(0, t, bt, q, out, stream=side)
    held = not side.query()
    del comp
    again = torch.empty(size, dtype=torch.uint8, device=DEV)
    words = [torch.empty(1, dtype=torch.int32, device=DEV) for _ in range(50)]
    assert held and not side.query() and again.data_ptr() != at
    assert all(w.data_ptr() != word for w in words)
    side.synchronize()
    check_chunk(d, out.cpu())


@pytest.mark.parametrize("hq,hkv,rot,ctas,stages", [
    (4, 2, 64, 4, 8), (40, 8, 128, 4, 3), (64, 16, 128, 4, 2), (64, 32, 128, 4, 1), (64, 64, 128, 4, 1),
    (128, 32, 128, 4, 1), (128, 16, 128, 4, 1), (160, 20, 128, 4, 1), (192, 24, 128, 3, 1), (256, 64, 128, 2, 1),
    (320, 80, 128, 0, 0)])
def test_append_has_as_many_ctas_as_hold_a_token(hq, hkv, rot, ctas, stages):
    """Long calls: four CTAs per SM, three or two, whatever tokens then fit in each; none with the widest."""
    kara = lib()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = 20480 // (hq + 2 * hkv) + 4 * sms
    held = append_call(kara, hq, hkv, 128, rows, rot)
    (grid, smem, _), = launches(held[0])
    assert smem // ((hq + 2 * hkv) * 256 + rot * 4) == stages
    assert grid == (sms * ctas, 1, 1) if ctas else grid == ((rows + 7) // 8, (hq + 2 * hkv) // 2, 1)


@pytest.mark.parametrize("hq,hkv,D,rot,inter,W,rows", [
    (64, 64, 128, 128, False, 64, 700), (160, 20, 128, 64, True, 0, 701), (192, 24, 128, 128, False, 0, 650),
    (256, 64, 128, 32, True, 64, 333), (320, 80, 128, 128, False, 0, 211), (128, 128, 64, 64, False, 64, 800)])
def test_append_long_calls_of_wide_shapes(hq, hkv, D, rot, inter, W, rows):
    """Values of long calls whose CTAs hold one token or few, four, three and two CTAs per SM, and none."""
    kara = lib()
    lengths, n_new = np.array([31, 300]), np.array([rows // 3, rows - rows // 3])
    width = int(blocks(lengths + n_new).max())
    nb = int(blocks(lengths + n_new).sum()) + 1
    bt, fresh = make_tables(lengths, width, nb, 4)
    _, q_start, ln, slot, seq, pos, _ = plain_extend(lengths, n_new, bt, fresh, rows + 2)
    q, k, v = append_inputs(hq, hq, hkv, D, rows + 2)
    g = torch.Generator().manual_seed(2)
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g)).bfloat16() for _ in range(2))
    cs = angles(1200, rot)
    kp = torch.zeros(1, nb, hkv, 16, D, dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    ring = torch.zeros(2, 1, hq, W, D, dtype=torch.bfloat16, device=DEV) if W else None
    out, err = torch.full((rows + 2, hq, D), 77.0, dtype=torch.bfloat16, device=DEV), error_word()
    t = kara.tokens(i32(q_start), i32(ln), torch.from_numpy(slot).to(DEV), i32(seq), i32(pos))
    r = kara.rope(cs.to(DEV), qw.to(DEV), kw.to(DEV), 1e-5, inter)
    kara.kara_append_kv(kara.cache(kp, vp, hq), 0, t, r, *on_gpu(q, k, v), out, err, ring=ring)
    assert kara.kara_get_error(err) == 0
    at, got = torch.from_numpy(pos[:rows]).long(), out.cpu()
    turned = lambda x, w: (plain_turn(x[:rows], w, 1e-5, cs, at, inter),  # noqa: E731
                           plain_turn(x[:rows], w, 1e-5, None, None, inter))
    close_rows(got[:rows], *turned(q, qw))
    assert (got[rows:] == 77.0).all()
    flat = lambda p: p.cpu()[0].permute(0, 2, 1, 3).reshape(-1, hkv, D)[torch.from_numpy(slot[:rows])]  # noqa: E731
    close_rows(flat(kp), *turned(k, kw))
    assert torch.equal(flat(vp), v[:rows])
    if W:
        rg = ring.cpu()[:, 0].permute(0, 2, 1, 3)   # [sequence][row][head][D]
        for s in (0, 1):
            last = torch.arange(int(ln[s]) - W, int(ln[s]))
            assert torch.equal(rg[s, last % W], got[int(q_start[s]) + last - int(lengths[s])])


@pytest.mark.parametrize("hq,hkv,D,rot,inter,norms", [
    (40, 8, 128, 128, False, "qk"), (32, 8, 128, 128, False, ""), (4, 2, 64, 64, True, "qk"),
    (6, 2, 128, 48, True, "k"), (7, 1, 64, 32, False, "q"), (18, 3, 128, 96, False, "qk"), (2, 2, 128, 0, False, "qk")])
def test_append_bits_do_not_depend_on_the_calls_length(hq, hkv, D, rot, inter, norms):
    """A token's stored bits are the same whether it comes alone, with a few, or in a long call."""
    kara = lib()
    rows = 20480 // (hq + 2 * hkv) + 100
    q, k, v = (x.to(DEV) for x in append_inputs(hq + D, hq, hkv, D, rows, fused=False))
    g = torch.Generator().manual_seed(3)
    w = [(1 + 0.3 * torch.randn(D, generator=g)).bfloat16().to(DEV) for _ in "qk"]
    cs = angles(rows, rot).to(DEV) if rot else None
    r = kara.rope(cs, w[0] if "q" in norms else None, w[1] if "k" in norms else None, interleaved=inter)
    nb, got = (rows + 15) // 16, []
    slot, pos, zero = torch.arange(rows, device=DEV), i32(range(rows)), i32([0] * rows)
    for step in (rows, 37):
        kp = torch.zeros(1, nb, hkv, 16, D, dtype=torch.bfloat16, device=DEV)
        vp, out, err = torch.zeros_like(kp), torch.zeros_like(q), error_word()
        c = kara.cache(kp, vp, hq)
        for a in range(0, rows, step):
            b = min(rows, a + step)
            t = kara.tokens(i32([0, b - a]), i32([b]), slot[a:b], zero[a:b], pos[a:b])
            kara.kara_append_kv(c, 0, t, r, q[a:b], k[a:b], v[a:b], out[a:b], err)
        assert kara.kara_get_error(err) == 0
        got.append([x.view(torch.int16) for x in (out, kp, vp)])
    for one, other in zip(*got):
        assert torch.equal(one, other)


def test_chunk_items_may_take_longer_than_a_wait(monkeypatch):
    """Warps with nothing to do while an item's key tiles go by do not take that for a stall: here an item's
    share of a CTA takes several times the limit.  Equal keys: the values' mean, exact in fp32."""
    kara = lib()
    L, m, hq, D = 12_000_000, 32, 8, 64
    nb = L // 16
    k = torch.zeros(1, nb, 1, 16, D, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    v[:] = 2.0 ** (torch.arange(D, device=DEV) % 5 - 2)
    q = torch.randn(m, hq, D, device=DEV).bfloat16()
    z, z4 = torch.empty(m, dtype=torch.int64, device=DEV), torch.empty(m, dtype=torch.int32, device=DEV)
    t, c = kara.tokens(i32([0, m]), i32([L]), z, z4, z4), kara.cache(k, v, hq)
    bt = torch.arange(nb, dtype=torch.int32, device=DEV)[None]
    ws = torch.empty(kara.kara_chunk_workspace_size(c, 1, m), dtype=torch.uint8, device=DEV)
    out, err = torch.empty_like(q), error_word()
    call = lambda: kara.kara_chunk_attention(c, 0, t, bt, q, out, ws, err)  # noqa: E731
    call()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    call()
    end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) > 0.5
    out.fill_(77.0)
    monkeypatch.setenv("KARA_DEBUG_WAIT_NS", "150000")
    call()
    assert kara.kara_get_error(err) == 0
    assert (out == v[0, 0, 0, 0]).all()
