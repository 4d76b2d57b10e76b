"""Refusals of the new-token entry points, and their plain forms' own pins (no GPU needed).

None of these calls launches anything: the argument checks come first."""
import ctypes

import numpy as np
import pytest
import torch

from _newtokens import make_tables, plain_chunk, plain_extend, plain_turn
from decode_kv_cache_03_gb300 import build as kbuild

PTR = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def kara():
    kbuild.build()
    from decode_kv_cache_03_gb300 import kara as k
    return k


def fake_cache(kara, **kw):
    c = kara.Cache(4096, 4096, 8 * 16 * 64 * 2, 2 * 16 * 64, 16 * 64, 2, 8, 2, 4, 64, 16)
    for k_, v_ in kw.items():
        setattr(c, k_, v_)
    return c


def fake_tokens(kara, **kw):
    t = kara.Tokens(2, 8, 4096, 4096, 4096, 4096, 4096)
    for k_, v_ in kw.items():
        setattr(t, k_, v_)
    return t


def fake_rope(kara, **kw):
    r = kara.Rope(4096, 4096, 1e-6, 4096, 100, 64, 0, None)
    for k_, v_ in kw.items():
        setattr(r, k_, v_)
    return r


def test_extend_refuses(kara):
    def ext(nb=8, bs=16, ln=PTR, nn=PTR, bt=PTR, bts=4, fresh=PTR, nf=4, t=None, used=PTR, err=PTR):
        t = fake_tokens(kara) if t is None else t
        return kara._lib.kara_extend_tables(nb, bs, ln, nn, bt, bts, fresh, nf, t, used, err, None)

    assert ext(bs=8) == kara.EUNSUPPORTED
    assert ext(t=fake_tokens(kara, n=65536)) == kara.EUNSUPPORTED
    assert ext(bts=1 << 27) == kara.EUNSUPPORTED
    for kw in (dict(nb=0), dict(bts=0), dict(nf=-1), dict(ln=None), dict(nn=None), dict(bt=None), dict(fresh=None),
               dict(used=None), dict(err=None)):
        assert ext(**kw) == kara.EINVAL, kw
    for kw in (dict(n=-1), dict(rows=-1), dict(q_start=None), dict(len=None), dict(slot=None), dict(seq=None),
               dict(pos=None)):
        assert ext(t=fake_tokens(kara, **kw)) == kara.EINVAL, kw
    assert ext(t=fake_tokens(kara, n=0, rows=0)) == kara.OK


def test_append_refuses(kara):
    def app(c=None, layer=0, t=None, r=None, q=PTR, qs=256, k=PTR, ks=128, v=PTR, vs=128, qo=PTR, ring=None, W=0,
            err=PTR):
        return kara._lib.kara_append_kv(c or fake_cache(kara), layer, t or fake_tokens(kara), r or fake_rope(kara), q,
                                        qs, k, ks, v, vs, qo, ring, W, err, None)

    odd = ctypes.c_void_p(4098)
    assert app(c=fake_cache(kara, head_dim=96)) == kara.EUNSUPPORTED
    for kw in (dict(layer=-1), dict(layer=2), dict(q=None), dict(k=None), dict(v=None), dict(qo=None), dict(err=None),
               dict(q=odd), dict(k=odd), dict(v=odd), dict(qo=odd), dict(qs=248), dict(ks=120), dict(vs=120),
               dict(qs=257), dict(ring=PTR, W=0), dict(ring=odd, W=64), dict(q=PTR, qo=PTR, qs=512)):
        assert app(**kw) == kara.EINVAL, kw
    for kw in (dict(rot_dim=24), dict(rot_dim=-16), dict(rot_dim=80), dict(eps=-1.0), dict(eps=float("nan")),
               dict(interleaved=2), dict(cos_sin=None), dict(cos_sin=4100), dict(n_pos=0), dict(q_weight=4098),
               dict(k_weight=4098)):
        assert app(r=fake_rope(kara, **kw)) == kara.EINVAL, kw
    for kw in (dict(n=-1), dict(rows=-1), dict(slot=None), dict(seq=None), dict(pos=None)):
        assert app(t=fake_tokens(kara, **kw)) == kara.EINVAL, kw
    assert app(t=fake_tokens(kara, len=None), ring=PTR, W=64) == kara.EINVAL
    assert app(t=fake_tokens(kara, rows=0)) == kara.OK


def test_chunk_refuses(kara):
    def att(c=None, layer=0, t=None, bt=PTR, bts=4, q=PTR, out=PTR, ws=PTR, wb=1 << 40, err=PTR):
        return kara._lib.kara_chunk_attention(c or fake_cache(kara), layer, t or fake_tokens(kara), bt, bts, q, out, ws,
                                              wb, err, None)

    odd = ctypes.c_void_p(4098)
    assert att(c=fake_cache(kara, block_size=32)) == kara.EUNSUPPORTED
    assert att(c=fake_cache(kara, num_q_heads=18)) == kara.EUNSUPPORTED
    assert att(t=fake_tokens(kara, n=65536)) == kara.EUNSUPPORTED
    assert att(bts=1 << 27) == kara.EUNSUPPORTED
    for kw in (dict(layer=-1), dict(layer=2), dict(bt=None), dict(bts=0), dict(q=None), dict(out=None), dict(err=None),
               dict(q=odd), dict(out=odd)):
        assert att(**kw) == kara.EINVAL, kw
    for kw in (dict(n=-1), dict(rows=-1), dict(q_start=None), dict(len=None)):
        assert att(t=fake_tokens(kara, **kw)) == kara.EINVAL, kw
    assert att(ws=None) == kara.EWORKSPACE and att(wb=1) == kara.EWORKSPACE
    assert att(t=fake_tokens(kara, rows=0)) == kara.OK and att(t=fake_tokens(kara, n=0)) == kara.OK
    assert kara.kara_chunk_workspace_size(fake_cache(kara, head_dim=96), 1, 1) == 0
    assert kara.kara_chunk_workspace_size(fake_cache(kara), 1, 1) > 0


def test_binding_refuses_tensors_off_the_current_device(kara, monkeypatch):
    """Host tensors, or tensors of another device than the current one, never reach a launch."""
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    t = kara.tokens(i32(2), i32(1), torch.zeros(4, dtype=torch.int64), i32(4), i32(4))
    with pytest.raises(kara.KaraError) as e:
        kara.kara_extend_tables(4, 16, i32(1), i32(1), i32(1, 2), i32(2), t, i32(1), i32(1))
    assert e.value.status == kara.EINVAL
    pool = torch.zeros(1, 4, 2, 16, 64, dtype=torch.bfloat16)
    c = kara.cache(pool, pool, 4)
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: kara.kara_append_kv(c, 0, t, kara.rope(None), q, q[:, :2], q[:, 2:], q, i32(1)),
                 lambda: kara.kara_chunk_attention(c, 0, t, i32(1, 2), q, q, torch.zeros(1 << 20), i32(1))):
        with pytest.raises(kara.KaraError) as e:
            call()
        assert e.value.status == kara.EINVAL

    class Far:   # stands for a tensor on a second GPU
        device = torch.device("cuda", 1)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(kara.KaraError) as e:
        kara._same_device(Far(), "here")
    assert e.value.status == kara.EINVAL
    near = Far()
    near.device = torch.device("cuda", 0)
    kara._same_device(near, "here", None)
    with pytest.raises(kara.KaraError):
        kara._same_device(near, "here", Far())


def test_plain_extend_by_hand():
    """Two sequences: 30 cached + 3 new (one open block, one fresh), 32 + 0, 0 + 17."""
    lengths, n_new = np.array([30, 32, 0], np.int32), np.array([3, 0, 17], np.int32)
    bt, _ = make_tables(lengths, 3, 8, 0)
    fresh = np.array([70, 71, 72, 73], np.int32)
    table, q_start, ln, slot, seq, pos, used = plain_extend(lengths, n_new, bt, fresh, 22)
    assert used[0] == 3 and q_start.tolist() == [0, 3, 3, 20] and ln.tolist() == [33, 32, 17]
    assert table[0, 2] == 70 and table[2].tolist() == [71, 72, -1] and table[1].tolist() == bt[1].tolist()
    assert slot[:3].tolist() == [bt[0, 1] * 16 + 14, bt[0, 1] * 16 + 15, 70 * 16] and slot[19] == 72 * 16
    assert seq[:4].tolist() == [0, 0, 0, 2] and pos[:4].tolist() == [30, 31, 32, 0]
    assert slot[20:].tolist() == [-1, -1] and seq[21] == -1 and pos[21] == -1


def test_plain_turn_keeps_lengths_and_relative_angles():
    """A rotation keeps norms, and <R(r)q, R(s)k> depends on r - s only."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(4, 3, 64, generator=g)
    ang = torch.arange(50.0, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(32) / 32)
    cs = torch.cat([ang.cos(), ang.sin()], 1)
    for inter in (False, True):
        r = torch.tensor([0, 7, 20, 31])
        y = plain_turn(x, None, 0.0, cs, r, inter)
        torch.testing.assert_close(y.norm(dim=-1), x.double().norm(dim=-1))
        torch.testing.assert_close(y[0], x[0].double())
        z = plain_turn(x, None, 0.0, cs, r + 11, inter)
        torch.testing.assert_close((y[1] * y[2]).sum(-1), (z[1] * z[2]).sum(-1))
    w = torch.ones(64)
    n = plain_turn(x, w, 0.0, None, None, False)
    torch.testing.assert_close((n * n).mean(-1), torch.ones(4, 3, dtype=torch.float64))


def test_plain_chunk_single_key_and_causality():
    """The first token of an empty cache returns its own value; later tokens do not reach back."""
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(1, 4, 2, 16, 64, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(20, 4, 64, generator=g).bfloat16()
    bt = np.array([[3, 1]], np.int32)
    a = plain_chunk(q, k, v, 0, bt, [0, 20], [20])
    torch.testing.assert_close(a[0, :2], v[0, 3, 0, 0].double().expand(2, 64))
    v2 = v.clone()
    v2[0, 1] = 99.0
    b = plain_chunk(q, k, v2, 0, bt, [0, 20], [20])
    assert torch.equal(a[:16], b[:16]) and not torch.equal(a[16:], b[16:])


def test_chunk_refuses_a_workspace_off_its_alignment(kara):
    """Partials are stored 16 bytes at a time: a view that starts in between never reaches a launch."""
    for at in (4097, 4098, 4100, 4104):
        st = kara._lib.kara_chunk_attention(fake_cache(kara), 0, fake_tokens(kara), PTR, 4, PTR, PTR,
                                            ctypes.c_void_p(at), 1 << 40, PTR, None)
        assert st == kara.EINVAL, at


def test_cache_refuses_values_unlike_the_keys(kara):
    """The values' pool is of the keys' type and device: nothing checks them after this."""
    k = torch.zeros(1, 4, 2, 16, 64, dtype=torch.bfloat16)
    kara.cache(k, k.clone(), 4)
    for v in (k.float(), k.half(), k.to("meta"), k[:, :3], k.transpose(1, 2)):
        with pytest.raises(AssertionError):
            kara.cache(k, v, 4)
