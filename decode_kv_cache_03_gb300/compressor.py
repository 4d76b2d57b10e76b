"""Convenience wrapper around the C ABI for one paged cache."""
from __future__ import annotations

import torch

from . import kara


class Compressor:
    """Periodic compression of the trailing windows of selected sequences.

    Holds the device workspaces and error word; the cache, tables and fresh
    block ids stay owned by the caller.  A workspace is memory of the stream that
    first used it; dropped, it and the error word are given back once every stream
    that used them has run its calls.  What calls captured into a graph use stays as
    long as this object does, which must outlive the graph.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, num_q_heads: int, W: int, B: int, K: int, R: int,
                 lam: float = 0.1, score_mode: int = 0, select_mode: int = 0, chunk: int = 0):
        self._keep(k, v, kara.cache(k, v, num_q_heads),
                   kara.params(W, B, K, R, lam, score_mode, select_mode, chunk))

    def _keep(self, k, v, cache, params):
        self.k, self.v, self.cache, self.params = k, v, cache, params
        self._ws = torch.empty(0, dtype=torch.uint8, device=k.device)
        self._dws = torch.empty(0, dtype=torch.uint8, device=k.device)
        self._cws = torch.empty(0, dtype=torch.uint8, device=k.device)
        self.err = torch.zeros(1, dtype=torch.int32, device=k.device)
        self._users = {"err": {self._handle(None)}}   # handles of the streams that the allocator knows to use each
        self._captured, self._in_graphs = set(), []   # workspaces that a graph uses; those of them since replaced

    def _handle(self, stream):
        if stream is not None:
            return stream.cuda_stream
        device = self.k.device
        return torch._C._cuda_getCurrentRawStream(device.index) if device.type == "cuda" else None

    def _capturing(self, stream) -> bool:
        if self.k.device.type != "cuda":
            return False
        if stream is None:
            return torch._C._cuda_isCurrentStreamCapturing()
        # (what torch.cuda.stream does, in a third of its 10 microseconds of host time)
        current = torch._C._cuda_getCurrentStream(stream.device_index)
        torch._C._cuda_setStream(stream_id=stream.stream_id, device_index=stream.device_index,
                                 device_type=stream.device_type)
        try:
            return torch._C._cuda_isCurrentStreamCapturing()
        finally:
            torch._C._cuda_setStream(stream_id=current[0], device_index=current[1], device_type=current[2])

    def _used(self, name: str, stream) -> torch.Tensor:
        """A buffer of this object's that a call on `stream` (None: the current one) uses: once dropped it is
        not handed out again before that call has run."""
        x, handle = getattr(self, name), self._handle(stream)
        if handle not in self._users[name]:
            x.record_stream(torch.cuda.current_stream(x.device) if stream is None else stream)
            self._users[name].add(handle)
        return x

    def _space(self, name: str, need: int, stream) -> torch.Tensor:
        """Workspace `name` of at least `need` bytes, for a call on `stream`."""
        if getattr(self, name).numel() < need or name not in self._users:
            if name in self._captured:
                self._in_graphs.append(getattr(self, name))
                self._captured.remove(name)
            with torch.cuda.stream(stream):   # of that stream's memory: what others gave back may be in use yet
                setattr(self, name, torch.empty(need, dtype=torch.uint8, device=self.k.device))
            self._users[name] = {self._handle(stream)}
        if name not in self._captured and self._capturing(stream):
            self._captured.add(name)
        return self._used(name, stream)

    def workspace(self, n: int, stream=None) -> torch.Tensor:
        return self._space("_ws", kara.kara_workspace_size(self.cache, self.params, n), stream)

    def plan(self, lengths_host: torch.Tensor, bt_stride: int):
        return kara.kara_plan(self.params, self.cache.block_size, lengths_host, bt_stride)

    def compress(self, lengths, block_table, q, fresh, freed, new_len, scores=None, cand=None, kept=None,
                 stream=None):
        """Enqueue the whole step; block_table is rewritten in place on success."""
        b = kara.batch(lengths, block_table, q)
        ws = self.workspace(b.n, stream)
        kara.kara_compress_batch(self.cache, self.params, b, fresh, freed, new_len, ws, self._used("err", stream),
                                 scores, cand, kept, stream)

    def decode(self, layer: int, lengths, block_table, q, out, stream=None):
        """Enqueue decode attention for one layer over the paged cache.  Called on
        the same stream right after compress() with its new_len and the table it
        rewrote in place, it reads the compacted cache with no host round trip."""
        n, bt_stride = block_table.shape
        ws = self._space("_dws", kara.kara_decode_workspace_size(self.cache, n, bt_stride), stream)
        kara.kara_decode_attention(self.cache, layer, lengths, block_table, q, out, ws, self._used("err", stream),
                                   stream)

    def extend(self, lengths, n_new, block_table, fresh, t, n_used, stream=None):
        """Enqueue opening blocks for n_new[s] tokens per sequence: block_table gets ids from
        `fresh` and the descriptor t (kara.tokens) is filled for append() and chunk()."""
        kara.kara_extend_tables(self.cache.num_blocks, self.cache.block_size, lengths, n_new, block_table, fresh, t,
                                n_used, self._used("err", stream), stream)

    def append(self, layer: int, t, rope, q, k, v, q_out, ring=None, stream=None):
        """Enqueue norms, rotation and the cache write of the new tokens for one layer;
        with `ring` (the q that compress() takes) the window queries are kept too."""
        kara.kara_append_kv(self.cache, layer, t, rope, q, k, v, q_out, self._used("err", stream), ring,
                            stream)

    def chunk(self, layer: int, t, block_table, q, out, stream=None):
        """Enqueue causal attention of the new tokens for one layer over the paged cache,
        after append() wrote their K and V.  The calls of one Compressor share a workspace:
        they run one after another, on one stream or ordered by events."""
        ws = self._space("_cws", kara.kara_chunk_workspace_size(self.cache, t.n, t.rows), stream)
        kara.kara_chunk_attention(self.cache, layer, t, block_table, q, out, ws, self._used("err", stream), stream)

    def error(self, stream=None) -> int:
        return kara.kara_get_error(self.err, stream)


def _pieces(sizes):
    """Offsets of pieces of these byte sizes, each on 256 bytes, and the bytes of all."""
    at, offsets = 0, []
    for size in sizes:
        offsets.append(at)
        at += (size + 255) // 256 * 256
    return offsets, at


class Compressor8(Compressor):
    """The same over an 8-bit cache (kara.cache8): pools of e4m3 codes, float scales for each block and head.

    compress() brings the windows' keys back to bf16 in a workspace, scores them there and compacts the codes;
    `windows` then describes those keys (what kara_compact_queries takes for the ring).  decode() and chunk()
    give bf16.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                 num_q_heads: int, W: int, B: int, K: int, R: int, lam: float = 0.1, score_mode: int = 0,
                 select_mode: int = 0, chunk: int = 0):
        self._keep(k, v, kara.cache8(k, v, k_scale, v_scale, num_q_heads),
                   kara.params(W, B, K, R, lam, score_mode, select_mode, chunk))
        self.k_scale, self.v_scale, self.windows = k_scale, v_scale, None
        self._xws = torch.empty(0, dtype=torch.uint8, device=k.device)

    def _window_cache(self, ws: torch.Tensor, n: int):
        """The bf16 keys of n windows as a cache at the start of `ws`."""
        c = self.cache
        blocks = n * (self.params.W // c.block_size + 1)
        shape = (c.num_layers, blocks, c.num_kv_heads, c.block_size, c.head_dim)
        keys = ws[:2 * torch.Size(shape).numel()].view(torch.bfloat16).view(shape)
        windows = kara.cache(keys, keys, c.num_q_heads)
        windows.keep = keys   # the workspace may be replaced by a larger one while `windows` is in use
        return windows

    def _compress_sizes(self, n: int, bt_stride: int):
        """Bytes of a compression's window keys, their table, the scorer's workspace, scores, candidates, kept
        rows and the compaction's workspace."""
        c, p = self.cache, self.params
        windows, slice_ = n * c.num_layers * c.num_kv_heads, c.block_size * c.head_dim * 2
        cache16 = kara.Cache(c.k, c.v, 0, 0, 0, c.num_layers, c.num_blocks, c.num_kv_heads, c.num_q_heads, c.head_dim,
                             c.block_size)
        return (windows * (p.W // c.block_size + 1) * slice_, n * bt_stride * 4,
                kara.kara_workspace_size(cache16, p, n), windows * (p.W - p.B) * 4, windows * p.K * 4,
                windows * p.R * 4, kara.kara_compact8_workspace_size(c, p, n))

    def workspace(self, n: int, stream=None, *, bt_stride: int) -> torch.Tensor:
        """What compress() of n sequences uses, with block tables of bt_stride columns: the windows have a table too."""
        return self._space("_xws", _pieces(self._compress_sizes(n, bt_stride))[1], stream)

    def compress(self, lengths, block_table, q, fresh, freed, new_len, scores=None, cand=None, kept=None,
                 stream=None):
        """Enqueue the whole step: expand, score, select, compact; block_table is rewritten in place on success."""
        n, bt_stride = block_table.shape
        if n == 0:
            return
        sizes = self._compress_sizes(n, bt_stride)
        at, total = _pieces(sizes)
        ws, err = self._space("_xws", total, stream), self._used("err", stream)
        piece = [ws[a:a + size] for a, size in zip(at, sizes)]
        c, p = self.cache, self.params
        windows = (n, c.num_layers, c.num_kv_heads)
        shaped = lambda x, i, t, last: piece[i].view(t).view(*windows, last) if x is None else x  # noqa: E731
        table = piece[1].view(torch.int32).view(n, bt_stride)
        scores, cand, kept = (shaped(scores, 3, torch.float32, p.W - p.B), shaped(cand, 4, torch.int32, p.K),
                              shaped(kept, 5, torch.int32, p.R))
        self.windows = self._window_cache(piece[0], n)
        with torch.cuda.stream(stream):
            err.zero_()
        kara.kara_expand8(c, self.windows, p.W, lengths, block_table, table, err, stream)
        kara.kara_score(self.windows, p, kara.batch(lengths, table, q), scores, piece[2], err, stream)
        kara.kara_select(p, n * c.num_layers * c.num_kv_heads, scores, cand, kept, stream)
        kara.kara_compact8(c, p, lengths, block_table, kept, fresh, freed, new_len, piece[6], err, stream)

    def decode(self, layer: int, lengths, block_table, q, out, stream=None):
        """Enqueue decode attention for one layer over the paged cache; out is bf16, zeros for an empty sequence."""
        n, bt_stride = block_table.shape
        ws = self._space("_dws", kara.kara_decode8_workspace_size(self.cache, n, bt_stride), stream)
        kara.kara_decode_attention8(self.cache, layer, lengths, block_table, q, out, ws, self._used("err", stream),
                                    stream)

    def append(self, layer: int, t, rope, q, k, v, q_out, ring=None, stream=None):
        """Enqueue norms, rotation, rounding to codes and the cache write of the new tokens for one layer;
        with `ring` (the q that compress() takes) the window queries are kept too."""
        kara.kara_append_kv8(self.cache, layer, t, rope, q, k, v, q_out, self._used("err", stream), ring, stream)

    def chunk(self, layer: int, t, block_table, q, out, stream=None):
        """Enqueue causal attention of the new tokens for one layer over the paged cache, after append() wrote
        their K and V.  The calls of one Compressor8 share a workspace, as those of a Compressor do."""
        ws = self._space("_cws", kara.kara_chunk8_workspace_size(self.cache, t.n, t.rows), stream)
        kara.kara_chunk_attention8(self.cache, layer, t, block_table, q, out, ws, self._used("err", stream), stream)
