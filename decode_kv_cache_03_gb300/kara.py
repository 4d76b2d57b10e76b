"""ctypes binding of libkara.so: the C entry points under the same names.

Marshalling only: every step of the compression runs in the library's CUDA
kernels.  Tensors are torch tensors on the GPU (host tensors only where the C
signature takes h_* pointers); the library never allocates.  If libkara.so is
missing or cannot be loaded this module raises at import, so no code path can
silently fall back to anything else.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkara.so")

OK, EINVAL, EUNSUPPORTED, ENOBLOCKS, EDUPBLOCK, ECUDA, EBADBLOCK, ETIMEOUT, EWORKSPACE = (
    0, -1, -2, -3, -4, -5, -6, -7, -8)


class KaraError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


class Params(ctypes.Structure):
    _fields_ = [("W", ctypes.c_int32), ("B", ctypes.c_int32), ("K", ctypes.c_int32),
                ("R", ctypes.c_int32), ("lam", ctypes.c_float), ("score_mode", ctypes.c_int32),
                ("select_mode", ctypes.c_int32), ("chunk", ctypes.c_int32)]


# kara_score_mode / kara_select_mode
SCORE_BIDIRECTIONAL, SCORE_CAUSAL = 0, 1
SELECT_TOKEN2CHUNK, SELECT_TOP_R, SELECT_FIXED_CHUNK = 0, 1, 2


class Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("layer_stride", ctypes.c_int64),
                ("block_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("num_layers", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32)]


class Cache8(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("layer_stride", ctypes.c_int64),
                ("block_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("num_layers", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32)]


class Batch(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("len", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("bt_stride", ctypes.c_int32), ("q", ctypes.c_void_p)]


class Tokens(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("rows", ctypes.c_int32), ("q_start", ctypes.c_void_p),
                ("len", ctypes.c_void_p), ("slot", ctypes.c_void_p), ("seq", ctypes.c_void_p),
                ("pos", ctypes.c_void_p)]


class Rope(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("cos_sin", ctypes.c_void_p), ("n_pos", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("pos_offset", ctypes.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libkara.so is not built ({LIB_PATH}); run decode_kv_cache_03_gb300.build.build()")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    PP, PC, PB = ctypes.POINTER(Params), ctypes.POINTER(Cache), ctypes.POINTER(Batch)
    PT, PR, PC8 = ctypes.POINTER(Tokens), ctypes.POINTER(Rope), ctypes.POINTER(Cache8)
    I32, I64, SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    sig = {
        "kara_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "kara_version": ([], ctypes.c_int),
        "kara_plan": ([PP, I32, I32, P, I32, P, P, P, P], ctypes.c_int),
        "kara_workspace_size": ([PC, PP, I32], SZ),
        "kara_score": ([PC, PP, PB, P, P, SZ, P, P], ctypes.c_int),
        "kara_select": ([PP, I64, P, P, P, P], ctypes.c_int),
        "kara_compact": ([PC, PP, PB, P, P, I64, P, P, P, P, SZ, P], ctypes.c_int),
        "kara_compress_batch": ([PC, PP, PB, P, I64, P, P, P, P, P, P, SZ, P, P, P], ctypes.c_int),
        "kara_get_error": ([P, P], ctypes.c_int),
        "kara_batch_groups": ([PC, PP, PB], I32),
        "kara_compact_static": ([PC, PP, PB, P, P, I64, P, P, P, P], ctypes.c_int),
        "kara_decode_workspace_size": ([PC, I32, I32], SZ),
        "kara_compact_queries": ([PC, PP, PB, P, P, P], ctypes.c_int),
        "kara_append_queries": ([PC, PP, PB, P, P], ctypes.c_int),
        "kara_decode_attention": ([PC, I32, I32, P, P, I32, P, P, P, SZ, P, P], ctypes.c_int),
        "kara_extend_tables": ([I32, I32, P, P, P, I32, P, I64, PT, P, P, P], ctypes.c_int),
        "kara_append_kv": ([PC, I32, PT, PR, P, I64, P, I64, P, I64, P, P, I32, P, P], ctypes.c_int),
        "kara_append_kv8": ([PC8, I32, PT, PR, P, I64, P, I64, P, I64, P, P, I32, P, P], ctypes.c_int),
        "kara_decode8_workspace_size": ([PC8, I32, I32], SZ),
        "kara_decode_attention8": ([PC8, I32, I32, P, P, I32, P, P, P, SZ, P, P], ctypes.c_int),
        "kara_chunk8_workspace_size": ([PC8, I32, I32], SZ),
        "kara_chunk_attention8": ([PC8, I32, PT, P, I32, P, P, P, SZ, P, P], ctypes.c_int),
        "kara_expand8": ([PC8, PC, I32, I32, P, P, I32, P, P, P], ctypes.c_int),
        "kara_compact8_workspace_size": ([PC8, PP, I32], SZ),
        "kara_compact8": ([PC8, PP, I32, P, P, I32, P, P, I64, P, P, P, SZ, P, P], ctypes.c_int),
        "kara_chunk_workspace_size": ([PC, I32, I32], SZ),
        "kara_chunk_attention": ([PC, I32, PT, P, I32, P, P, P, SZ, P, P], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return lib


_lib = _load()
EXPORTED = ("kara_status_string", "kara_version", "kara_plan", "kara_workspace_size", "kara_score",
            "kara_select", "kara_compact", "kara_compress_batch", "kara_get_error", "kara_compact_static",
            "kara_decode_workspace_size", "kara_decode_attention", "kara_compact_queries", "kara_append_queries",
            "kara_batch_groups", "kara_extend_tables", "kara_append_kv", "kara_chunk_workspace_size",
            "kara_chunk_attention", "kara_append_kv8", "kara_decode8_workspace_size", "kara_decode_attention8",
            "kara_chunk8_workspace_size", "kara_chunk_attention8", "kara_expand8", "kara_compact8_workspace_size", "kara_compact8")
STATIC_MAX_SEQS = 8192     # KARA_STATIC_MAX_SEQS


def status_string(status: int) -> str:
    return _lib.kara_status_string(int(status)).decode()


def version() -> int:
    return int(_lib.kara_version())


def _check(status: int, where: str):
    if status != OK:
        raise KaraError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def params(W, B, K, R, lam, score_mode=SCORE_BIDIRECTIONAL, select_mode=SELECT_TOKEN2CHUNK, chunk=0) -> Params:
    return Params(int(W), int(B), int(K), int(R), float(lam), int(score_mode), int(select_mode), int(chunk))


def cache(k: torch.Tensor, v: torch.Tensor, num_q_heads: int) -> Cache:
    """Describe bf16 pools laid out [layers][num_blocks][hkv][block][d] (rows contiguous)."""
    assert k.dtype == v.dtype == torch.bfloat16 and v.shape == k.shape and v.stride() == k.stride()
    assert v.device == k.device
    Lyr, nb, hkv, bs, d = k.shape
    assert k.stride(4) == 1 and k.stride(3) == d
    c = Cache(k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), k.stride(2), Lyr, nb, hkv,
              int(num_q_heads), d, bs)
    c.device = k.device
    return c


def cache8(k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor, num_q_heads: int) -> Cache8:
    """Describe pools of e4m3 codes (torch.float8_e4m3fn, or their bits as torch.uint8) laid out
    [layers][num_blocks][hkv][block][d] (rows contiguous), with scales float [layers][num_blocks][hkv]."""
    assert k.dtype == v.dtype and k.dtype in (torch.float8_e4m3fn, torch.uint8)
    assert v.shape == k.shape and v.stride() == k.stride()
    Lyr, nb, hkv, bs, d = k.shape
    assert k.stride(4) == 1 and k.stride(3) == d
    for s in (k_scale, v_scale):
        assert s.dtype == torch.float32 and s.shape == (Lyr, nb, hkv) and s.is_contiguous()
    assert v.device == k_scale.device == v_scale.device == k.device
    c = Cache8(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k.stride(0), k.stride(1),
               k.stride(2), Lyr, nb, hkv, int(num_q_heads), d, bs)
    c.device = k.device
    return c


def batch(lengths: torch.Tensor, block_table: torch.Tensor, q: torch.Tensor) -> Batch:
    assert lengths.dtype == torch.int32 and block_table.dtype == torch.int32
    assert block_table.is_contiguous() and q.is_contiguous() and q.dtype == torch.bfloat16
    return Batch(int(lengths.shape[0]), lengths.data_ptr(), block_table.data_ptr(),
                 int(block_table.shape[1]), q.data_ptr())


def kara_plan(p: Params, block_size: int, h_len: torch.Tensor, bt_stride: int):
    """Host plan: (n_new[n], n_old[n], total_new, total_old) as CPU tensors / ints."""
    h_len = h_len.cpu().to(torch.int32).contiguous()
    n = h_len.shape[0]
    nn = torch.zeros(n, dtype=torch.int32)
    no = torch.zeros(n, dtype=torch.int32)
    tn, to = ctypes.c_int64(0), ctypes.c_int64(0)
    _check(_lib.kara_plan(ctypes.byref(p), block_size, n, _ptr(h_len), bt_stride, _ptr(nn), _ptr(no),
                          ctypes.byref(tn), ctypes.byref(to)), "kara_plan")
    return nn, no, tn.value, to.value


def kara_workspace_size(c: Cache, p: Params, n: int) -> int:
    return int(_lib.kara_workspace_size(ctypes.byref(c), ctypes.byref(p), int(n)))


def kara_score(c: Cache, p: Params, b: Batch, scores: torch.Tensor, ws: torch.Tensor, err: torch.Tensor,
               stream=None):
    _check(_lib.kara_score(ctypes.byref(c), ctypes.byref(p), ctypes.byref(b), _ptr(scores), _ptr(ws),
                           ws.numel() * ws.element_size(), _ptr(err), _stream(stream)), "kara_score")


def kara_compact_queries(c: Cache, p: Params, b: Batch, kept: torch.Tensor, err: torch.Tensor, stream=None):
    """Move the kept and buffer queries of the ring b.q with the step's K/V compaction."""
    _check(_lib.kara_compact_queries(ctypes.byref(c), ctypes.byref(p), ctypes.byref(b), _ptr(kept), _ptr(err),
                                     _stream(stream)), "kara_compact_queries")


def kara_append_queries(c: Cache, p: Params, b: Batch, q_new: torch.Tensor, stream=None):
    """Write one decode step's queries [n][layers][hq][D] into row len mod W of each ring."""
    assert q_new.dtype == torch.bfloat16 and q_new.is_contiguous()
    _check(_lib.kara_append_queries(ctypes.byref(c), ctypes.byref(p), ctypes.byref(b), _ptr(q_new),
                                    _stream(stream)), "kara_append_queries")


def kara_decode_workspace_size(c: Cache, n: int, bt_stride: int) -> int:
    return int(_lib.kara_decode_workspace_size(ctypes.byref(c), int(n), int(bt_stride)))


def kara_decode_attention(c: Cache, layer: int, lengths: torch.Tensor, block_table: torch.Tensor,
                          q: torch.Tensor, out: torch.Tensor, ws: torch.Tensor, err: torch.Tensor, stream=None):
    """Decode attention of q [n][num_q_heads][head_dim] (bf16) over layer `layer`
    of the paged cache, read through block_table [n][bt_stride]; out is float."""
    assert lengths.dtype == torch.int32 and block_table.dtype == torch.int32 and block_table.is_contiguous()
    assert q.dtype == torch.bfloat16 and q.is_contiguous() and out.dtype == torch.float32
    n, bt_stride = block_table.shape
    _check(_lib.kara_decode_attention(ctypes.byref(c), int(layer), int(n), _ptr(lengths), _ptr(block_table),
                                      int(bt_stride), _ptr(q), _ptr(out), _ptr(ws),
                                      ws.numel() * ws.element_size(), _ptr(err), _stream(stream)),
           "kara_decode_attention")


def _raw_stream(err: torch.Tensor, stream):
    """The stream's handle, the current one of err's device if None (torch.cuda.current_stream costs
    several microseconds of host time, as much as a whole small call)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(err.get_device())
    return stream.cuda_stream


def _same_device(err: torch.Tensor, where: str, *tensors):
    """Refuses tensors that are not on the current CUDA device: the launch goes there."""
    d = err.device
    if d.type != "cuda" or d.index != torch.cuda.current_device():
        raise KaraError(EINVAL, f"{where}: tensors on {d}, not on the current CUDA device")
    for t in tensors:
        if t is not None and t.device != d:
            raise KaraError(EINVAL, f"{where}: tensors on {t.device} and on {d}")


def tokens(q_start: torch.Tensor, length: torch.Tensor, slot: torch.Tensor, seq: torch.Tensor,
           pos: torch.Tensor) -> Tokens:
    """Describe the new tokens of a step: q_start [n + 1], length [n] (int32), slot (int64), seq, pos
    (int32) [rows].  kara_extend_tables fills the arrays; the descriptor keeps them alive."""
    n, rows = int(length.shape[0]), int(slot.shape[0])
    assert q_start.shape == (n + 1,) and seq.shape == pos.shape == (rows,) and slot.dtype == torch.int64
    for t in (q_start, length, seq, pos):
        assert t.dtype == torch.int32 and t.device == slot.device
    for t in (q_start, length, slot, seq, pos):
        assert t.is_contiguous()
    t = Tokens(n, rows, q_start.data_ptr(), length.data_ptr(), slot.data_ptr(), seq.data_ptr(), pos.data_ptr())
    t.device = slot.device
    t.keep = (q_start, length, slot, seq, pos)
    return t


def rope(cos_sin, q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
         pos_offset=None) -> Rope:
    """Describe norms and rotation: cos_sin float [n_pos][rot_dim] (None: no rotation), weights bf16
    [head_dim] or None, pos_offset int32 [n] or None.  The descriptor keeps the tensors alive."""
    n_pos = rot = 0
    if cos_sin is not None:
        assert cos_sin.dtype == torch.float32 and cos_sin.is_contiguous()
        n_pos, rot = cos_sin.shape
    for w in (q_weight, k_weight):
        assert w is None or (w.dtype == torch.bfloat16 and w.is_contiguous() and w.dim() == 1)
    assert pos_offset is None or (pos_offset.dtype == torch.int32 and pos_offset.is_contiguous())
    p = [None if t is None else t.data_ptr() for t in (q_weight, k_weight, cos_sin, pos_offset)]
    r = Rope(p[0], p[1], float(eps), p[2], int(n_pos), int(rot), int(bool(interleaved)), p[3])
    r.head_dim = {int(w.shape[0]) for w in (q_weight, k_weight) if w is not None}
    r.n = None if pos_offset is None else int(pos_offset.shape[0])
    r.keep = [t for t in (q_weight, k_weight, cos_sin, pos_offset) if t is not None]
    r.on = r.keep[:1]
    assert all(t.device == r.on[0].device for t in r.keep)
    return r


def kara_extend_tables(num_blocks: int, block_size: int, lengths: torch.Tensor, n_new: torch.Tensor,
                       block_table: torch.Tensor, fresh: torch.Tensor, t: Tokens, n_used: torch.Tensor,
                       err: torch.Tensor, stream=None):
    """Open blocks for n_new[s] tokens after lengths[s] cached ones (ids from `fresh`, table rewritten
    in place) and fill the descriptor t; t's lengths may be `lengths` itself."""
    _same_device(err, "kara_extend_tables", lengths, n_new, block_table, fresh, n_used, t)
    assert lengths.dtype == n_new.dtype == block_table.dtype == fresh.dtype == n_used.dtype == torch.int32
    assert lengths.shape == n_new.shape == (t.n,) and block_table.shape[0] == t.n and n_used.numel() == 1
    assert (lengths.is_contiguous() and n_new.is_contiguous() and block_table.is_contiguous()
            and fresh.is_contiguous())
    _check(_lib.kara_extend_tables(num_blocks, block_size, lengths.data_ptr(), n_new.data_ptr(),
                                   block_table.data_ptr(), block_table.shape[1], fresh.data_ptr(), fresh.numel(),
                                   t, n_used.data_ptr(), err.data_ptr(), _raw_stream(err, stream)), "kara_extend_tables")


def _append(entry, where: str, c, layer: int, t: Tokens, r: Rope, q, k, v, q_out, err, ring, stream):
    """The checks and the call of an append into a cache of either type."""
    _same_device(err, where, q, k, v, q_out, ring, c, t, *r.on)
    hq, hkv, d, rows, W = c.num_q_heads, c.num_kv_heads, c.head_dim, t.rows, 0
    assert q.dtype == k.dtype == v.dtype == q_out.dtype == torch.bfloat16
    assert q.shape == q_out.shape == (rows, hq, d) and k.shape == v.shape == (rows, hkv, d)
    strides = []
    for x, heads in ((q, hq), (k, hkv), (v, hkv)):   # rows apart as they like, their heads contiguous
        a, b, e = x.stride()
        assert e == 1 and (b == d or heads == 1)
        strides.append(a if rows > 1 else heads * d)
    assert q_out.is_contiguous()
    assert r.head_dim <= {d} and (r.n is None or r.n == t.n)
    if ring is not None:
        W = ring.shape[3]
        assert ring.dtype == torch.bfloat16 and ring.is_contiguous()
        assert ring.shape == (t.n, c.num_layers, hq, W, d)
    _check(entry(c, layer, t, r, q.data_ptr(), strides[0], k.data_ptr(), strides[1], v.data_ptr(), strides[2],
                 q_out.data_ptr(), None if ring is None else ring.data_ptr(), W, err.data_ptr(),
                 _raw_stream(err, stream)), where)


def kara_append_kv(c: Cache, layer: int, t: Tokens, r: Rope, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                   q_out: torch.Tensor, err: torch.Tensor, ring=None, stream=None):
    """Norm and rotate q [rows][num_q_heads][D] and k [rows][num_kv_heads][D] and write k, v into layer
    `layer` of the cache at t's slots, queries to q_out (and to ring [n][layers][num_q_heads][W][D])."""
    _append(_lib.kara_append_kv, "kara_append_kv", c, layer, t, r, q, k, v, q_out, err, ring, stream)


def kara_append_kv8(c: Cache8, layer: int, t: Tokens, r: Rope, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                    q_out: torch.Tensor, err: torch.Tensor, ring=None, stream=None):
    """kara_append_kv into an 8-bit cache: k and v rounded to e4m3, a scale for each block and head."""
    _append(_lib.kara_append_kv8, "kara_append_kv8", c, layer, t, r, q, k, v, q_out, err, ring, stream)


def kara_chunk_workspace_size(c: Cache, n: int, rows: int) -> int:
    return int(_lib.kara_chunk_workspace_size(ctypes.byref(c), int(n), int(rows)))


def _chunk(entry, where: str, c, layer: int, t: Tokens, block_table, q, out, ws, err, stream):
    """The checks and the call of a chunk's attention over a cache of either type."""
    _same_device(err, where, block_table, q, out, ws, c, t)
    assert block_table.dtype == torch.int32 and block_table.is_contiguous() and block_table.shape[0] == t.n
    assert q.dtype == out.dtype == torch.bfloat16 and q.is_contiguous() and out.is_contiguous()
    assert q.shape == out.shape == (t.rows, c.num_q_heads, c.head_dim)
    _check(entry(c, layer, t, block_table.data_ptr(), block_table.shape[1], q.data_ptr(), out.data_ptr(), ws.data_ptr(),
                 ws.numel() * ws.element_size(), err.data_ptr(), _raw_stream(err, stream)), where)


def kara_chunk_attention(c: Cache, layer: int, t: Tokens, block_table: torch.Tensor, q: torch.Tensor,
                         out: torch.Tensor, ws: torch.Tensor, err: torch.Tensor, stream=None):
    """Causal attention of the new tokens q [rows][num_q_heads][head_dim] (bf16) over layer `layer` of
    the paged cache, read through block_table [n][bt_stride]; out like q, padding rows untouched."""
    _chunk(_lib.kara_chunk_attention, "kara_chunk_attention", c, layer, t, block_table, q, out, ws, err, stream)


def kara_chunk8_workspace_size(c: Cache8, n: int, rows: int) -> int:
    return int(_lib.kara_chunk8_workspace_size(ctypes.byref(c), int(n), int(rows)))


def kara_chunk_attention8(c: Cache8, layer: int, t: Tokens, block_table: torch.Tensor, q: torch.Tensor,
                          out: torch.Tensor, ws: torch.Tensor, err: torch.Tensor, stream=None):
    """kara_chunk_attention over an 8-bit cache."""
    _chunk(_lib.kara_chunk_attention8, "kara_chunk_attention8", c, layer, t, block_table, q, out, ws, err, stream)


def kara_decode8_workspace_size(c: Cache8, n: int, bt_stride: int) -> int:
    return int(_lib.kara_decode8_workspace_size(ctypes.byref(c), int(n), int(bt_stride)))


def kara_decode_attention8(c: Cache8, layer: int, lengths: torch.Tensor, block_table: torch.Tensor,
                           q: torch.Tensor, out: torch.Tensor, ws: torch.Tensor, err: torch.Tensor, stream=None):
    """Decode attention of q [n][num_q_heads][head_dim] (bf16) over layer `layer` of an 8-bit cache, read
    through block_table [n][bt_stride]; out is bf16, zeros for a sequence of length 0."""
    _same_device(err, "kara_decode_attention8", lengths, block_table, q, out, ws, c)
    n, bt_stride = block_table.shape
    assert lengths.dtype == block_table.dtype == torch.int32 and lengths.shape == (n,)
    assert lengths.is_contiguous() and block_table.is_contiguous()
    assert q.dtype == out.dtype == torch.bfloat16 and q.is_contiguous() and out.is_contiguous()
    assert q.shape == out.shape == (n, c.num_q_heads, c.head_dim)
    _check(_lib.kara_decode_attention8(c, layer, n, lengths.data_ptr(), block_table.data_ptr(), bt_stride,
                                       q.data_ptr(), out.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(),
                                       err.data_ptr(), _raw_stream(err, stream)), "kara_decode_attention8")


def kara_expand8(c: Cache8, out: Cache, W: int, lengths: torch.Tensor, block_table: torch.Tensor,
                 out_table: torch.Tensor, err: torch.Tensor, stream=None):
    """The windows (last W tokens) of an 8-bit cache as bf16 blocks of `out`, n * (W/16 + 1) of them, their
    ids in out_table: what kara_score takes.  With out.v == out.k only the keys are written."""
    _same_device(err, "kara_expand8", lengths, block_table, out_table, c, out)
    n, bt_stride = block_table.shape
    assert lengths.dtype == block_table.dtype == out_table.dtype == torch.int32 and lengths.shape == (n,)
    assert lengths.is_contiguous() and block_table.is_contiguous()
    assert out_table.shape == block_table.shape and out_table.is_contiguous()
    _check(_lib.kara_expand8(c, out, W, n, lengths.data_ptr(), block_table.data_ptr(), bt_stride,
                             out_table.data_ptr(), err.data_ptr(), _raw_stream(err, stream)), "kara_expand8")


def kara_compact8_workspace_size(c: Cache8, p: Params, n: int) -> int:
    return int(_lib.kara_compact8_workspace_size(ctypes.byref(c), ctypes.byref(p), int(n)))


def kara_compact8(c: Cache8, p: Params, lengths: torch.Tensor, block_table: torch.Tensor, kept: torch.Tensor,
                  fresh: torch.Tensor, freed: torch.Tensor, new_len: torch.Tensor, ws: torch.Tensor,
                  err: torch.Tensor, stream=None):
    """kara_compact on an 8-bit cache: kept [n][layers][hkv][R] rows into fresh blocks with new scales."""
    _same_device(err, "kara_compact8", lengths, block_table, kept, fresh, freed, new_len, ws, c)
    n, bt_stride = block_table.shape
    for t in (lengths, block_table, kept, fresh, freed, new_len):
        assert t.dtype == torch.int32 and t.is_contiguous()
    assert lengths.shape == new_len.shape == (n,) and kept.shape == (n, c.num_layers, c.num_kv_heads, p.R)
    _check(_lib.kara_compact8(c, p, n, lengths.data_ptr(), block_table.data_ptr(), bt_stride, kept.data_ptr(),
                              fresh.data_ptr(), fresh.numel(), freed.data_ptr(), new_len.data_ptr(), ws.data_ptr(),
                              ws.numel() * ws.element_size(), err.data_ptr(), _raw_stream(err, stream)),
           "kara_compact8")


def kara_select(p: Params, n_windows: int, scores: torch.Tensor, cand, kept: torch.Tensor, stream=None):
    _check(_lib.kara_select(ctypes.byref(p), int(n_windows), _ptr(scores), _ptr(cand), _ptr(kept),
                            _stream(stream)), "kara_select")


def kara_compact(c: Cache, p: Params, b: Batch, kept, fresh, freed, new_len, err, ws, stream=None):
    _check(_lib.kara_compact(ctypes.byref(c), ctypes.byref(p), ctypes.byref(b), _ptr(kept), _ptr(fresh),
                             int(fresh.numel()), _ptr(freed), _ptr(new_len), _ptr(err), _ptr(ws),
                             ws.numel() * ws.element_size(), _stream(stream)), "kara_compact")


def kara_compact_static(c: Cache, p: Params, b: Batch, kept, fresh, freed, new_len, err, stream=None):
    """kara_compact without a workspace (plan kept in the library's fixed array)."""
    _check(_lib.kara_compact_static(ctypes.byref(c), ctypes.byref(p), ctypes.byref(b), _ptr(kept), _ptr(fresh),
                                    int(fresh.numel()), _ptr(freed), _ptr(new_len), _ptr(err), _stream(stream)),
           "kara_compact_static")


def kara_compress_batch(c: Cache, p: Params, b: Batch, fresh, freed, new_len, ws, err, scores_out=None,
                        cand_out=None, kept_out=None, stream=None, phase_events=None):
    """phase_events: None or 5 torch.cuda.Event(enable_timing=True) recorded around the phases."""
    ev = None
    if phase_events is not None:
        assert len(phase_events) == 5
        assert all(e.cuda_event for e in phase_events), "record each event once before passing it"
        ev = (ctypes.c_void_p * 5)(*[e.cuda_event for e in phase_events])
    _check(_lib.kara_compress_batch(ctypes.byref(c), ctypes.byref(p), ctypes.byref(b), _ptr(fresh),
                                    int(fresh.numel()), _ptr(freed), _ptr(new_len), _ptr(scores_out),
                                    _ptr(cand_out), _ptr(kept_out), _ptr(ws), ws.numel() * ws.element_size(),
                                    _ptr(err), _stream(stream), ev), "kara_compress_batch")


def kara_batch_groups(c: Cache, p: Params, b: Batch) -> int:
    """Sequence groups kara_compress_batch pipelines this batch into (1: none)."""
    r = int(_lib.kara_batch_groups(ctypes.byref(c), ctypes.byref(p), ctypes.byref(b)))
    _check(r if r < 0 else OK, "kara_batch_groups")
    return r


def kara_get_error(err: torch.Tensor, stream=None) -> int:
    return int(_lib.kara_get_error(_ptr(err), _stream(stream)))
