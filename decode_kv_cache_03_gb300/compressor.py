"""Convenience wrapper around the C ABI for one paged cache."""
from __future__ import annotations

import torch

from . import kara


class Compressor:
    """Periodic compression of the trailing windows of selected sequences.

    Holds the device workspaces and error word; the cache, tables and fresh
    block ids stay owned by the caller.  A workspace is memory of the stream that
    first used it; dropped, it and the error word are given back once every stream
    that used them has run its calls.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, num_q_heads: int, W: int, B: int, K: int, R: int,
                 lam: float = 0.1, score_mode: int = 0, select_mode: int = 0, chunk: int = 0):
        self.k, self.v = k, v
        self.cache = kara.cache(k, v, num_q_heads)
        self.params = kara.params(W, B, K, R, lam, score_mode, select_mode, chunk)
        self._ws = torch.empty(0, dtype=torch.uint8, device=k.device)
        self._dws = torch.empty(0, dtype=torch.uint8, device=k.device)
        self._cws = torch.empty(0, dtype=torch.uint8, device=k.device)
        self.err = torch.zeros(1, dtype=torch.int32, device=k.device)
        self._users = {"err": {self._handle(None)}}   # handles of the streams that the allocator knows to use each

    def _handle(self, stream):
        if stream is not None:
            return stream.cuda_stream
        device = self.k.device
        return torch._C._cuda_getCurrentRawStream(device.index) if device.type == "cuda" else None

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
            with torch.cuda.stream(stream):   # of that stream's memory: what others gave back may be in use yet
                setattr(self, name, torch.empty(need, dtype=torch.uint8, device=self.k.device))
            self._users[name] = {self._handle(stream)}
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
