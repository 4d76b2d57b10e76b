"""GPU tests of the 8-bit cache's calls together and in the ways that programs make them: a serving loop with
compressions, captured steps, streams, workspaces.

Tolerance of an attention output against 64 bits over the stored values: 2^-8 |ref| (its rounding) and
(2^-8 + 2^-10) sum_x w_x |v_x| (the weights' rounding, the logits'); scores 1e-3, the scorer's own."""

import threading

import numpy as np
import pytest
import torch

from _cache8 import BS, dense, divide, plain_decode, random_pool, scale_of
from _gpu import lib
from _newtokens import blocks, make_tables, plain_chunk, plain_turn
from test_gpu_cache8 import (DEV, Append, chunk_case, chunk_descriptor, decode_case, error_word, i32, run_chunk, run_decode,
                             same_bits, status)

pytestmark = pytest.mark.gpu


class Model:
    """Two layers' projections and a Compressor8: what a serving loop keeps."""

    def __init__(self, n, hq, hkv, D, W, nb, width, seed):
        from decode_kv_cache_03_gb300 import Compressor8
        self.kara = lib()
        g = torch.Generator().manual_seed(seed)
        self.n, self.hq, self.hkv, self.D, self.W = n, hq, hkv, D, W
        self.k = torch.full((2, nb, hkv, BS, D), 0x7f, dtype=torch.uint8, device=DEV)
        self.v = self.k.clone()
        self.ks = torch.full((2, nb, hkv), float("nan"), device=DEV)
        self.vs = self.ks.clone()
        self.B, self.K, self.R = 16, 8, 16
        self.comp = Compressor8(self.k, self.v, self.ks, self.vs, hq, W, self.B, self.K, self.R)
        self.qw, self.kw = ((1 + 0.2 * torch.randn(D, generator=g)).bfloat16().to(DEV) for _ in range(2))
        ang = torch.arange(2000, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(D // 2) / (D / 2))
        self.cs = torch.cat([ang.cos(), ang.sin()], 1).float().to(DEV)
        self.shift = torch.zeros(n, dtype=torch.int32, device=DEV)
        self.rope = self.kara.rope(self.cs, self.qw, self.kw, 1e-6, False, self.shift)
        self.ring = torch.zeros(n, 2, hq, W, D, dtype=torch.bfloat16, device=DEV)
        self.bt = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
        self.len = torch.zeros(n, dtype=torch.int32, device=DEV)

    def step(self, n_new, fresh, rows, qkv):
        """One step over both layers; qkv [layers][rows][(hq + 2 hkv) D].  Returns (outputs, blocks used)."""
        hq, hkv, D = self.hq, self.hkv, self.D
        f = lambda k, t: torch.full((k,), -77, dtype=t, device=DEV)  # noqa: E731
        b = dict(q_start=f(self.n + 1, torch.int32), slot=f(rows, torch.int64), seq=f(rows, torch.int32),
                 pos=f(rows, torch.int32))
        t = self.kara.tokens(b["q_start"], self.len, b["slot"], b["seq"], b["pos"])
        used = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.comp.extend(self.len, n_new, self.bt, fresh, t, used)
        outs = []
        for layer in range(2):
            x = qkv[layer]
            q, k, v = (y.view(rows, -1, D) for y in x.split([hq * D, hkv * D, hkv * D], 1))
            qo = torch.zeros(rows, hq, D, dtype=torch.bfloat16, device=DEV)
            o = torch.zeros_like(qo)
            self.comp.append(layer, t, self.rope, q, k, v, qo, ring=self.ring)
            self.comp.chunk(layer, t, self.bt, qo, o)
            outs.append((qo, o, b))
        return outs, used

    def values(self):
        """Stored values of both pools in float64; zeros where no scale was written."""
        return [torch.nan_to_num(dense(c.cpu(), torch.nan_to_num(s.cpu(), nan=0.0)), nan=0.0)
                for c, s in ((self.k, self.ks), (self.v, self.vs))]


def near(out, ref, size):
    off = (out.double() - ref).abs() - (2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -10) * size)
    assert off.max() <= 0, off.max()


def test_prefill_decode_compress_and_go_on():
    """Prompts in two chunks, decode steps, a compression with the ring that the appends filled, then more tokens:
    every attention against 64 bits over the stored values, those against the tokens that came, the scores
    against the expanded keys, the compacted rows against the kept ones."""
    kara = lib()
    n, hq, hkv, D, W = 3, 4, 2, 64, 64
    m = Model(n, hq, hkv, D, W, 60, 16, 3)
    free = list(np.random.default_rng(0).permutation(60))
    g = torch.Generator().manual_seed(4)
    true_pos = [0] * n
    came = [[[] for _ in range(2)] for _ in range(n)]       # [seq][layer]: each token's (key, value) in float64

    def step(counts, pad):
        rows, old = sum(counts) + pad, m.len.tolist()
        qkv = torch.randn(2, rows, (hq + 2 * hkv) * D, generator=g).bfloat16()
        outs, used = m.step(i32(counts), i32(free[:20]), rows, qkv.to(DEV))
        assert m.comp.error() == 0
        del free[:int(used)]
        kv, bt, ln = m.values(), m.bt.cpu().numpy(), m.len.cpu().numpy()
        q_start = np.concatenate([[0], np.cumsum(counts)])
        total = int(q_start[-1])
        for layer in range(2):
            qo, o, b = outs[layer]
            args = (qo.cpu(), *kv, layer, bt, q_start, ln)
            near(o.cpu()[:total], plain_chunk(*args)[:total], plain_chunk(*args, absolute=True)[:total])
            assert (o[total:] == 0).all() and (qo[total:] == 0).all()
            _, k, v = (y.view(rows, -1, D) for y in qkv[layer].split([hq * D, hkv * D, hkv * D], 1))
            for s in range(n):
                at = torch.arange(true_pos[s], true_pos[s] + counts[s])
                sl = slice(int(q_start[s]), int(q_start[s + 1]))
                turned = plain_turn(k[sl], m.kw.cpu(), 1e-6, m.cs.cpu(), at, False)
                came[s][layer] += list(zip(turned, v[sl].double()))
                # what is stored of all tokens: off by one rounding, and by half a subnormal step of the scale
                for x in range(int(ln[s])):
                    blk = int(bt[s, x // BS])
                    for side, scale in ((0, m.ks), (1, m.vs)):
                        want = came[s][layer][x][side]
                        step_ = scale[layer, blk].cpu().double().abs()[:, None] * 2.0 ** -9
                        off = (kv[side][layer, blk, :, x % BS] - want).abs()
                        assert (off <= 2.0 ** -4 * want.abs() + step_ + 2.0 ** -16).all(), (s, layer, x, side)
        for s in range(n):
            true_pos[s] += counts[s]
        assert [a + c for a, c in zip(old, counts)] == m.len.tolist()

    step([50, 0, 33], 2)
    step([40, 90, 47], 0)
    for _ in range(3):
        step([1, 1, 1], 1)
    lengths, bt0, kv0 = m.len.cpu(), m.bt.cpu().numpy(), m.values()
    _, _, tn, to = m.comp.plan(lengths, m.bt.shape[1])
    fresh, freed = i32(free[:tn]), torch.empty(to, dtype=torch.int32, device=DEV)
    del free[:tn]
    new_len = torch.empty(n, dtype=torch.int32, device=DEV)
    C = W - m.B
    scores = torch.empty(n, 2, hkv, C, device=DEV)
    kept = torch.empty(n, 2, hkv, m.R, dtype=torch.int32, device=DEV)
    m.comp.err.fill_(kara.ETIMEOUT)                           # a compression starts from a clear error word
    m.comp.compress(m.len, m.bt, m.ring, fresh, freed, new_len, scores=scores, kept=kept)
    assert m.comp.error() == 0
    rows_of = lambda kv, bt, s, layer, x: torch.stack(  # noqa: E731
        [kv[layer, int(bt[s, y // BS]), :, y % BS] for y in x], 1)    # [hkv][rows][D]
    for s in range(n):
        L = int(lengths[s])
        for layer in range(2):
            k = rows_of(kv0[0], bt0, s, layer, range(L - W, L))
            for h in range(hkv):
                q = m.ring[s, layer, 2 * h:2 * h + 2].cpu().double()
                ref = torch.softmax(q @ k[h].T / D ** 0.5, -1).sum((0, 1))[:C]
                torch.testing.assert_close(scores[s, layer, h].cpu().double(), ref, rtol=1e-3, atol=0)
    again = torch.empty_like(kept)
    kara.kara_select(m.comp.params, n * 2 * hkv, scores, None, again)
    assert torch.equal(again, kept)
    kara.kara_compact_queries(m.comp.windows, m.comp.params, kara.batch(m.len, m.bt, m.ring), kept, m.comp.err)
    assert m.comp.error() == 0
    free.extend(freed.cpu().tolist())
    kv1, bt1, kc = m.values(), m.bt.cpu().numpy(), kept.cpu()
    for s in range(n):
        L = int(lengths[s])
        for layer in range(2):
            new = came[s][layer][:L - W]
            for j in range(m.R):
                new.append(tuple(torch.stack([came[s][layer][L - W + kc[s, layer, h, j]][side][h] for h in range(hkv)])
                                 for side in range(2)))
            came[s][layer] = new + came[s][layer][L - m.B:]
            src = [np.concatenate([np.arange(L - W), L - W + kc[s, layer, h].numpy(), np.arange(L - m.B, L)])
                   for h in range(hkv)]
            for side, scale in ((0, m.ks), (1, m.vs)):        # a row keeps its values but for the subnormals
                for h in range(hkv):
                    was = rows_of(kv0[side], bt0, s, layer, src[h])[h]
                    now = rows_of(kv1[side], bt1, s, layer, range(int(new_len[s])))[h]
                    top = scale[layer].cpu().double()[torch.as_tensor(bt1[s, :blocks(int(new_len[s]))]).long(), h].abs()
                    step_ = top.repeat_interleave(BS)[:len(was), None] * 2.0 ** -10
                    assert ((was - now).abs() <= step_).all()
    m.len.copy_(new_len)
    m.shift += C - m.R
    step([1, 30, 1], 0)
    step([20, 1, 70], 5)
    # a decode call of the last tokens' queries over what is there now
    q, out = torch.randn(n, hq, D, generator=g).bfloat16().to(DEV), torch.empty(n, hq, D, dtype=torch.bfloat16, device=DEV)
    m.comp.decode(1, m.len, m.bt, q, out)
    assert m.comp.error() == 0
    args = (q.cpu(), m.values(), 1, m.bt.cpu().numpy(), m.len.cpu().numpy())
    near(out.cpu(), plain_decode(*args), plain_decode(*args, absolute=True))


def test_failed_compression_changes_nothing():
    """A sequence shorter than the window: the status, and tables, lengths, codes and scales as they were."""
    kara = lib()
    m = Model(2, 4, 2, 64, 64, 30, 8, 5)
    g = torch.Generator().manual_seed(1)
    m.step(i32([40, 80]), i32(range(20)), 120, torch.randn(2, 120, 8 * 64, generator=g).bfloat16().to(DEV))
    was = [x.clone() for x in (m.bt, m.k, m.v, m.ks, m.vs)]
    freed, new_len = torch.full((20,), -7, dtype=torch.int32, device=DEV), i32([0, 0])
    m.comp.compress(m.len, m.bt, m.ring, i32(range(20, 30)), freed, new_len)
    assert m.comp.error() == kara.EINVAL
    assert new_len.tolist() == [40, 80] and (freed == -7).all()
    for a, b in zip(was, (m.bt, m.k, m.v, m.ks, m.vs)):
        assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def test_captured_step_replays():
    """extend, append8 and chunk8 of a decode step captured once and replayed: lengths advance in place, blocks
    grow token by token and their scales with them."""
    n, hq, hkv, D = 4, 8, 2, 128
    m = Model(n, hq, hkv, D, 64, 80, 20, 5)
    g = torch.Generator().manual_seed(6)
    mk = lambda: torch.randn(2, n, (hq + 2 * hkv) * D, generator=g).bfloat16().to(DEV)  # noqa: E731
    ids = np.random.default_rng(1).permutation(80)
    qkv, fresh, n_new = mk(), i32(ids[:n]), i32([1] * n)
    m.step(n_new, fresh, n, qkv)                    # the workspace and kernels exist before the capture
    assert m.comp.error() == 0
    m.bt.fill_(-1)
    m.len.zero_()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        outs, used = m.step(n_new, fresh, n, qkv)
    at, came = 0, []
    for i in range(40):
        fresh.copy_(i32(ids[at:at + n]))
        qkv.copy_(mk())
        graph.replay()
        assert m.comp.error() == 0
        came.append(qkv[1, :, (hq + hkv) * D:].view(n, hkv, D).cpu().double())
        at += int(used)
        assert int(used) == (n if i % BS == 0 else 0) and m.len.tolist() == [i + 1] * n
    q_start, ln, bt = np.arange(n + 1), np.full(n, 40, np.int32), m.bt.cpu().numpy()
    args = (outs[1][0].cpu(), *m.values(), 1, bt, q_start, ln)
    near(outs[1][1].cpu(), plain_chunk(*args), plain_chunk(*args, absolute=True))
    for seq in range(n):                            # a block's scale is that of its largest value
        for b in range(blocks(40)):
            rows = torch.stack([came[x][seq] for x in range(b * BS, min(40, b * BS + BS))], 1)
            s_ = m.vs[1, int(bt[seq, b])].cpu().double()
            assert torch.equal(s_, scale_of(rows.abs().amax((-1, -2))))
            last = divide(rows[:, -1], s_[:, None])
            assert torch.equal(m.v[1, int(bt[seq, b]), :, rows.shape[1] - 1].cpu(), last)


def test_captured_decode_and_compression_replay():
    """decode8 and the four calls of a compression captured together: every replay gives the eager bytes."""
    kara = lib()
    from decode_kv_cache_03_gb300 import Compressor8
    lengths, bt, k, ks, v, vs, q = decode_case(21, [300, 90, 257], 8, 2, 128)
    spare = torch.zeros(2, 40, 2, BS, 128, dtype=torch.uint8)
    pools = [torch.cat([x, spare], 1).to(DEV) for x in (k, v)] + [
        torch.cat([x, torch.ones(2, 40, 2)], 1).to(DEV) for x in (ks, vs)]
    first = [x.clone() for x in pools]
    comp = Compressor8(*pools, 8, 64, 16, 8, 20)
    g = torch.Generator().manual_seed(2)
    ring = torch.randn(3, 2, 8, 64, 128, generator=g).bfloat16().to(DEV)
    table0, ln, fresh = i32(bt), i32(lengths), i32(range(k.shape[1], k.shape[1] + 30))
    table, freed, new_len = table0.clone(), torch.zeros(60, dtype=torch.int32, device=DEV), i32([0, 0, 0])
    out, qd = torch.empty(2, 3, 8, 128, dtype=torch.bfloat16, device=DEV), q.to(DEV)

    def step():
        for x, y in zip(pools, first):
            x.copy_(y)
        table.copy_(table0)
        comp.compress(ln, table, ring, fresh, freed, new_len)
        for layer in range(2):
            comp.decode(layer, new_len, table, qd, out[layer])

    step()
    assert comp.error() == 0
    want = [x.clone() for x in (*pools, table, freed, new_len, out)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(3):
        for x in (*pools, table, freed, new_len, out):
            x.zero_()
        graph.replay()
        assert comp.error() == 0
        for a, b in zip(want, (*pools, table, freed, new_len, out)):
            assert torch.equal(a, b)
    assert kara.kara_get_error(comp.err) == 0


def test_streams_with_their_own_workspaces():
    """Decode and chunk calls in flight at once on two streams, neither of them the current one."""
    kara = lib()
    dc = [decode_case(30 + i, [3000 - 700 * i, 40], 10, 2, 128) for i in range(2)]
    cc = [chunk_case(40 + i, [3000 - 700 * i], [200 + 50 * i], 8, 2, 128) for i in range(2)]
    want_d, want_c = [run_decode(*d)[1] for d in dc], [run_chunk(c)[1] for c in cc]
    keep = []
    for d, c in zip(dc, cc):
        lengths, bt, k, ks, v, vs, q = d
        pd, pc = [x.to(DEV) for x in (k, v, ks, vs)], [c[x].to(DEV) for x in ("k", "v", "ks", "vs")]
        cd, cp = kara.cache8(*pd, 10), kara.cache8(*pc, 8)
        t = chunk_descriptor(kara, c)
        ws = [torch.empty(kara.kara_decode8_workspace_size(cd, *bt.shape), dtype=torch.uint8, device=DEV),
              torch.empty(kara.kara_chunk8_workspace_size(cp, t.n, t.rows), dtype=torch.uint8, device=DEV)]
        keep.append((cd, cp, t, i32(lengths), i32(bt), i32(c["bt"]), q.to(DEV), c["q"].to(DEV), ws, error_word(),
                     torch.zeros(q.shape, dtype=torch.bfloat16, device=DEV),
                     torch.full(c["q"].shape, 77.0, dtype=torch.bfloat16, device=DEV), pd, pc))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in keep]
    for _ in range(5):
        for s, (cd, cp, t, ln, bt, cbt, q, cq, ws, err, od, oc, _, _) in zip(streams, keep):
            kara.kara_decode_attention8(cd, 1, ln, bt, q, od, ws[0], err, stream=s)
            kara.kara_chunk_attention8(cp, 0, t, cbt, cq, oc, ws[1], err, stream=s)
    torch.cuda.synchronize()
    for a, b, x in zip(want_d, want_c, keep):
        assert same_bits(x[10].cpu(), a) and same_bits(x[11].cpu(), b) and int(x[9]) == 0


def test_two_host_threads():
    """The same calls from two host threads on streams of their own."""
    cases = [Append(50 + i, [5, 300], [700, 60 + i], 8, 2, 128, W=64) for i in range(2)]
    want = [a.run()[1] for a in cases]
    failed = []

    def work(a, w):
        try:
            s = torch.cuda.Stream()
            for _ in range(5):
                with torch.cuda.stream(s):
                    st, got = a.run(stream=s)
                assert st == 0 and all(torch.equal(got[x].view(torch.uint8), w[x].view(torch.uint8)) for x in w)
        except Exception as e:   # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip(cases, want)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not failed, failed


def test_append_bits_do_not_depend_on_the_calls_length():
    """Values and queries of a token, and whole blocks of keys, whether tokens come in one long call or in calls
    that end with a block."""
    kara = lib()
    hq, hkv, D, rows = 40, 8, 128, 720
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(rows, h, D, generator=g).bfloat16().to(DEV) for h in (hq, hkv, hkv))
    kw = (1 + 0.2 * torch.randn(D, generator=g)).bfloat16().to(DEV)
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(64) / 64)
    r = kara.rope(torch.cat([ang.cos(), ang.sin()], 1).float().to(DEV), kw, kw)
    slot, pos, zero, got = torch.arange(rows, device=DEV), i32(range(rows)), i32([0] * rows), []
    for step in (rows, 48, 16):
        pools = [torch.zeros(1, rows // BS, hkv, BS, D, dtype=torch.uint8, device=DEV) for _ in range(2)]
        scales = [torch.zeros(1, rows // BS, hkv, device=DEV) for _ in range(2)]
        c, out, err = kara.cache8(*pools, *scales, hq), torch.zeros_like(q), error_word()
        for a in range(0, rows, step):
            b = min(rows, a + step)
            t = kara.tokens(i32([0, b - a]), i32([b]), slot[a:b], zero[a:b], pos[a:b])
            kara.kara_append_kv8(c, 0, t, r, q[a:b], k[a:b], v[a:b], out[a:b], err)
        assert status(kara, err) == 0
        got.append([out.view(torch.int16), *pools, *scales])
    for other in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(got[0], other))


def test_offsets_past_two_to_the_31st():
    """A pool of more than 2^31 codes, a table that names its far end: append, decode, chunk, expand, compact."""
    kara = lib()
    hq, hkv, D, nb = 8, 4, 128, 300000              # 2.46e9 codes a pool
    k = torch.zeros(1, nb, hkv, BS, D, dtype=torch.uint8, device=DEV)
    v = torch.zeros_like(k)
    ks, vs = (torch.zeros(1, nb, hkv, device=DEV) for _ in range(2))
    c = kara.cache8(k, v, ks, vs, hq)
    ids = list(range(nb - 1, nb - 13, -1))
    bt, L = np.array([ids[:8] + [-1] * 2], np.int32), 120
    g = torch.Generator().manual_seed(1)
    x = torch.randn(L, hq + 2 * hkv, D, generator=g).bfloat16().to(DEV)
    q, kn, vn = x.split([hq, hkv, hkv], 1)
    q = q.contiguous()
    slot = torch.tensor([ids[p // BS] * BS + p % BS for p in range(L)], device=DEV)
    t = kara.tokens(i32([0, L]), i32([L]), slot, i32([0] * L), i32(range(L)))
    err, out = error_word(), torch.empty_like(q)
    kara.kara_append_kv8(c, 0, t, kara.rope(None), q, kn, vn, torch.empty_like(q), err)
    kv = [dense(p[:, nb - 16:].cpu(), s[:, nb - 16:].cpu()) for p, s in ((k, ks), (v, vs))]
    near_bt = np.where(bt >= 0, bt - (nb - 16), -1)
    assert (kv[1][0, near_bt[0, 0], :, 3] - vn[3].cpu().double()).abs().max() < 0.3
    ws = torch.empty(kara.kara_chunk8_workspace_size(c, 1, L), dtype=torch.uint8, device=DEV)
    kara.kara_chunk_attention8(c, 0, t, i32(bt), q, out, ws, err)
    args = (q.cpu(), *kv, 0, near_bt, [0, L], [L])
    near(out.cpu(), plain_chunk(*args), plain_chunk(*args, absolute=True))
    one = torch.empty(1, hq, D, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(kara.kara_decode8_workspace_size(c, 1, bt.shape[1]), dtype=torch.uint8, device=DEV)
    kara.kara_decode_attention8(c, 0, i32([L]), i32(bt), q[-1:].contiguous(), one, ws, err)
    args = (q[-1:].cpu(), kv, 0, near_bt, [L])
    near(one.cpu(), plain_decode(*args), plain_decode(*args, absolute=True))
    wide = torch.zeros(1, 5, hkv, BS, D, dtype=torch.bfloat16, device=DEV)
    table = i32(np.full(bt.shape, -9))
    kara.kara_expand8(c, kara.cache(wide, wide, hq), 64, i32([L]), i32(bt), table, err)
    assert table[0].tolist() == [-9] * 3 + [0, 1, 2, 3, 4] + [-9] * 2
    assert torch.equal(wide[0, 0].cpu().double(), kv[0][0, near_bt[0, 3]])
    p, kept = kara.params(64, 16, 1, 16, 0.1), i32(np.arange(16) * 3)[None, None, None].expand(1, 1, hkv, 16).contiguous()
    ws = torch.empty(kara.kara_compact8_workspace_size(c, p, 1), dtype=torch.uint8, device=DEV)
    table, freed, new_len = i32(bt), torch.zeros(8, dtype=torch.int32, device=DEV), i32([0])
    kara.kara_compact8(c, p, i32([L]), table, kept, i32(ids[8:]), freed, new_len, ws, err)
    assert status(kara, err) == 0 and new_len.tolist() == [L - 32] and table[0, 3].item() == ids[8]
    now = dense(v[:, ids[8]].cpu(), vs[:, ids[8]].cpu())[0]
    assert torch.equal(now[:, :8], kv[1][0, near_bt[0, 3], :, :8])      # the rows ahead of the window


def test_long_table_of_one_sequence():
    """Decode and a draft over a cache of 300000 keys whose table names the same blocks again and again."""
    kara = lib()
    hq, hkv, D, many = 8, 2, 64, 18750
    k, ks = random_pool((1, 50, hkv, BS, D), 1, 1)
    v, vs = random_pool((1, 50, hkv, BS, D), 2, 1)
    bt = np.resize(np.random.default_rng(0).permutation(50), (1, many)).astype(np.int32)
    L = many * BS - 7
    g = torch.Generator().manual_seed(3)
    q = torch.randn(1, hq, D, generator=g).bfloat16()
    st, out = run_decode(np.array([L], np.int32), bt, k, ks, v, vs, q, layer=0)
    kv = dense(k, ks), dense(v, vs)
    args = (q, kv, 0, bt, [L])
    assert st == 0
    near(out, plain_decode(*args), plain_decode(*args, absolute=True))
    q3 = torch.randn(3, hq, D, generator=g).bfloat16()
    st, out = run_chunk(dict(q=q3, k=k, v=v, ks=ks, vs=vs, bt=bt, q_start=np.array([0, 3]), lengths=np.array([L])))
    args = (q3, *kv, 0, bt, [0, 3], [L])
    assert st == 0
    near(out, plain_chunk(*args), plain_chunk(*args, absolute=True))


def test_compress_selected_with_an_8_bit_compressor():
    """The periodic policy's helper takes either compressor."""
    from decode_kv_cache_03_gb300 import Compressor8
    from decode_kv_cache_03_gb300.periodic import BlockPool, compress_selected
    lib()
    lengths, nb = torch.tensor([200, 90, 300], dtype=torch.int32), 90
    bt, left = make_tables(lengths.numpy(), 20, nb, 3)
    k, ks = random_pool((2, nb, 2, BS, 64), 1)
    v, vs = random_pool((2, nb, 2, BS, 64), 2)
    comp = Compressor8(*(x.to(DEV) for x in (k, v, ks, vs)), 8, 64, 16, 8, 20)
    pool, table = BlockPool(left.tolist()), torch.from_numpy(bt)
    ring = torch.randn(2, 2, 8, 64, 64).bfloat16().to(DEV)
    freed, st = compress_selected(comp, [0, 2], lengths, table, ring, pool)
    assert st == 0 and lengths.tolist() == [200 - 48 + 20, 90, 300 - 48 + 20] and len(freed) > 0
    live = [int(b) for s in range(3) for b in table[s, :blocks(int(lengths[s]))]]
    assert len(set(live)) == len(live) and not set(live) & set(freed)
