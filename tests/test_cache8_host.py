"""The 8-bit cache without a GPU: refusals of its entry points, and pins of the tests' own plain forms.

None of these calls launches anything: the argument checks come first."""
import ctypes

import pytest
import torch

from _cache8 import VALUE, dense, divide, plain_decode, quantise, round_code, runs, scale_of, value
from decode_kv_cache_03_gb300 import build as kbuild

PTR = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4104)


@pytest.fixture(scope="module")
def kara():
    kbuild.build()
    from decode_kv_cache_03_gb300 import kara as k
    return k


def fake8(kara, **kw):
    c = kara.Cache8(4096, 4096, 4096, 4096, 8 * 2 * 16 * 64, 2 * 16 * 64, 16 * 64, 2, 8, 2, 4, 64, 16)
    for k_, v_ in kw.items():
        setattr(c, k_, v_)
    return c


def fake16(kara, **kw):
    c = kara.Cache(4096, 4096, 10 * 2 * 16 * 64, 2 * 16 * 64, 16 * 64, 2, 10, 2, 4, 64, 16)
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


BAD_CACHES = [(dict(head_dim=96), "EUNSUPPORTED"), (dict(block_size=32), "EUNSUPPORTED"),
              (dict(num_q_heads=18), "EUNSUPPORTED"), (dict(num_q_heads=3), "EINVAL"), (dict(num_kv_heads=0), "EINVAL"),
              (dict(num_layers=0), "EINVAL"), (dict(num_blocks=0), "EINVAL"), (dict(k=None), "EINVAL"),
              (dict(v=None), "EINVAL"), (dict(k_scale=None), "EINVAL"), (dict(v_scale=None), "EINVAL"),
              (dict(k=4104), "EINVAL"), (dict(v=4100), "EINVAL"), (dict(k_scale=4098), "EINVAL"),
              (dict(v_scale=4097), "EINVAL"), (dict(layer_stride=8), "EINVAL"), (dict(block_stride=1032), "EINVAL"),
              (dict(head_stride=-16), "EINVAL")]


def append(kara, c=None, layer=0, t=None, r=None, q=PTR, qs=256, k=PTR, ks=128, v=PTR, vs=128, qo=PTR, ring=None, W=0,
           err=PTR):
    return kara._lib.kara_append_kv8(c or fake8(kara), layer, t or fake_tokens(kara), r or fake_rope(kara), q, qs, k, ks, v,
                                     vs, qo, ring, W, err, None)


def decode(kara, c=None, layer=0, n=2, ln=PTR, bt=PTR, bts=4, q=PTR, out=PTR, ws=PTR, wb=1 << 40, err=PTR):
    return kara._lib.kara_decode_attention8(c or fake8(kara), layer, n, ln, bt, bts, q, out, ws, wb, err, None)


def chunk(kara, c=None, layer=0, t=None, bt=PTR, bts=4, q=PTR, out=PTR, ws=PTR, wb=1 << 40, err=PTR):
    return kara._lib.kara_chunk_attention8(c or fake8(kara), layer, t or fake_tokens(kara), bt, bts, q, out, ws, wb, err,
                                           None)


def expand(kara, c=None, o=None, W=64, n=2, ln=PTR, bt=PTR, bts=8, ot=ctypes.c_void_p(8192), err=PTR):
    return kara._lib.kara_expand8(c or fake8(kara), o or fake16(kara), W, n, ln, bt, bts, ot, err, None)


def compact(kara, c=None, p=None, n=2, ln=PTR, bt=PTR, bts=8, kept=PTR, fresh=PTR, nf=9, freed=PTR, nl=PTR, ws=PTR,
            wb=1 << 20, err=PTR):
    return kara._lib.kara_compact8(c or fake8(kara), p or kara.params(64, 16, 1, 16, 0.1), n, ln, bt, bts, kept, fresh, nf,
                                   freed, nl, ws, wb, err, None)


@pytest.mark.parametrize("call", [append, decode, chunk, expand, compact])
def test_every_call_refuses_bad_caches(kara, call):
    for kw, want in BAD_CACHES:
        assert call(kara, c=fake8(kara, **kw)) == getattr(kara, want), kw
    for kw, want in BAD_CACHES:
        assert kara.kara_decode8_workspace_size(fake8(kara, **kw), 1, 1) == 0, kw
        assert kara.kara_chunk8_workspace_size(fake8(kara, **kw), 1, 1) == 0, kw
        assert kara.kara_compact8_workspace_size(fake8(kara, **kw), kara.params(64, 16, 1, 16, 0.1), 1) == 0, kw


def test_append_refuses(kara):
    for kw in (dict(layer=-1), dict(layer=2), dict(q=None), dict(k=None), dict(v=None), dict(qo=None), dict(err=None),
               dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(qo=ODD), dict(qs=248), dict(ks=120), dict(vs=120),
               dict(qs=257), dict(ring=PTR, W=0), dict(ring=ODD, W=64), dict(q=PTR, qo=PTR, qs=512)):
        assert append(kara, **kw) == kara.EINVAL, kw
    for kw in (dict(rot_dim=24), dict(rot_dim=80), dict(eps=-1.0), dict(interleaved=2), dict(cos_sin=None),
               dict(n_pos=0), dict(k_weight=4098)):
        assert append(kara, r=fake_rope(kara, **kw)) == kara.EINVAL, kw
    for kw in (dict(n=-1), dict(rows=-1), dict(slot=None), dict(seq=None), dict(pos=None)):
        assert append(kara, t=fake_tokens(kara, **kw)) == kara.EINVAL, kw
    assert append(kara, t=fake_tokens(kara, rows=0)) == kara.OK


def test_decode_refuses(kara):
    for kw in (dict(layer=-1), dict(layer=2), dict(n=-1), dict(ln=None), dict(bt=None), dict(bts=0), dict(q=None),
               dict(out=None), dict(err=None), dict(q=ODD), dict(out=ODD), dict(ws=ODD)):
        assert decode(kara, **kw) == kara.EINVAL, kw
    for kw in (dict(n=65536), dict(bts=1 << 27), dict(bts=65536 * 64)):
        assert decode(kara, **kw) == kara.EUNSUPPORTED, kw
    assert decode(kara, ws=None) == decode(kara, wb=100) == kara.EWORKSPACE
    assert decode(kara, n=0) == kara.OK
    assert kara.kara_decode8_workspace_size(fake8(kara), 3, 65) >= 3 * 4 * 2 * (64 * 4 + 8)


def test_decode_workspace_serves_smaller_batches(kara):
    """Small batches are split further, but never need more than a larger batch over tables as wide does."""
    for hq, hkv in ((8, 1), (8, 8), (4, 2), (40, 8)):
        c = fake8(kara, num_q_heads=hq, num_kv_heads=hkv)
        for bts in (1, 17, 64, 65, 130, 500, 1000, 4000):
            sizes = [kara.kara_decode8_workspace_size(c, n, bts) for n in range(1, 80)]
            assert sizes == sorted(sizes)
            wide = [kara.kara_decode8_workspace_size(c, n, bts + 1) for n in range(1, 80)]
            assert all(a <= b for a, b in zip(sizes, wide))


def test_chunk_refuses(kara):
    for kw in (dict(layer=-1), dict(layer=2), dict(bt=None), dict(bts=0), dict(q=None), dict(out=None), dict(err=None),
               dict(q=ODD), dict(out=ODD), dict(ws=ODD)):
        assert chunk(kara, **kw) == kara.EINVAL, kw
    for kw in (dict(n=-1), dict(rows=-1), dict(q_start=None), dict(len=None)):
        assert chunk(kara, t=fake_tokens(kara, **kw)) == kara.EINVAL, kw
    assert chunk(kara, t=fake_tokens(kara, n=65536)) == chunk(kara, bts=1 << 27) == kara.EUNSUPPORTED
    assert chunk(kara, ws=None) == chunk(kara, wb=1) == kara.EWORKSPACE
    assert chunk(kara, t=fake_tokens(kara, rows=0)) == chunk(kara, t=fake_tokens(kara, n=0)) == kara.OK
    assert kara.kara_chunk8_workspace_size(fake8(kara), 1, 1) > 0


def test_expand_refuses(kara):
    for kw in (dict(W=0), dict(W=-16), dict(W=72), dict(n=-1), dict(ln=None), dict(bt=None), dict(bts=0), dict(ot=None),
               dict(ot=PTR), dict(err=None)):
        assert expand(kara, **kw) == kara.EINVAL, kw
    for kw in (dict(num_layers=3), dict(num_kv_heads=1, num_q_heads=4), dict(head_dim=128), dict(k=4100), dict(v=None)):
        assert expand(kara, o=fake16(kara, **kw)) == kara.EINVAL, kw
    assert expand(kara, o=fake16(kara, num_blocks=9)) == kara.ENOBLOCKS
    assert expand(kara, n=0) == kara.OK


def test_compact_refuses(kara):
    for kw in (dict(n=-1), dict(ln=None), dict(bt=None), dict(bts=0), dict(kept=None), dict(fresh=None), dict(nf=-1),
               dict(freed=None), dict(nl=None), dict(err=None), dict(ws=ODD), dict(p=kara.params(64, 16, 1, 49, 0.1)),
               dict(p=kara.params(64, 64, 1, 1, 0.1))):
        assert compact(kara, **kw) == kara.EINVAL, kw
    assert compact(kara, p=kara.params(96, 16, 1, 16, 0.1)) == kara.EUNSUPPORTED
    assert compact(kara, ws=None) == compact(kara, wb=63) == kara.EWORKSPACE
    assert compact(kara, n=0) == kara.OK


def test_cache8_refuses_tensors_unlike_each_other(kara):
    k = torch.zeros(1, 4, 2, 16, 64, dtype=torch.uint8)
    s = torch.ones(1, 4, 2)
    kara.cache8(k, k.clone(), s, s.clone(), 4)
    kara.cache8(k.view(torch.float8_e4m3fn), k.view(torch.float8_e4m3fn), s, s, 4)
    for v in (k.view(torch.int8), k.view(torch.float8_e4m3fn), k.to("meta"), k[:, :3], k.transpose(1, 2)):
        with pytest.raises(AssertionError):
            kara.cache8(k, v, s, s, 4)
    for t in (s.double(), s[:, :3], s.transpose(0, 2), torch.ones(1, 4, 4)[..., ::2], s.to("meta")):
        with pytest.raises(AssertionError):
            kara.cache8(k, k, s, t, 4)


def test_binding_refuses_host_tensors(kara):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    t = kara.tokens(i32(2), i32(1), torch.zeros(4, dtype=torch.int64), i32(4), i32(4))
    k, s = torch.zeros(1, 4, 2, 16, 64, dtype=torch.uint8), torch.ones(1, 4, 2)
    c, q = kara.cache8(k, k, s, s, 4), torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    pool = torch.zeros(1, 4, 2, 16, 64, dtype=torch.bfloat16)
    w = torch.zeros(1 << 16, dtype=torch.uint8)
    for call in (lambda: kara.kara_append_kv8(c, 0, t, kara.rope(None), q, q[:, :2], q[:, 2:], q, i32(1)),
                 lambda: kara.kara_decode_attention8(c, 0, i32(4), i32(4, 2), q, q, w, i32(1)),
                 lambda: kara.kara_chunk_attention8(c, 0, t, i32(1, 2), q, q, w, i32(1)),
                 lambda: kara.kara_expand8(c, kara.cache(pool, pool, 4), 16, i32(1), i32(1, 2), i32(1, 2), i32(1)),
                 lambda: kara.kara_compact8(c, kara.params(64, 16, 1, 16, 0.1), i32(1), i32(1, 2), i32(1, 1, 2, 16), i32(2),
                                            i32(2), i32(1), w, i32(1))):
        with pytest.raises(kara.KaraError) as e:
            call()
        assert e.value.status == kara.EINVAL


# ---- the tests' plain forms -------------------------------------------------------

def test_codes_are_torch_s_e4m3():
    """Every code's value and the rounding of many values are those of torch.float8_e4m3fn."""
    codes = torch.arange(256, dtype=torch.uint8)
    torch.testing.assert_close(VALUE.float(), codes.view(torch.float8_e4m3fn).float(), rtol=0, atol=0, equal_nan=True)
    g = torch.Generator().manual_seed(0)
    x = torch.cat([torch.randn(20000, generator=g) * 2.0 ** torch.randint(-12, 9, (20000,), generator=g),
                   VALUE[:127].float(), (VALUE[:126].float() + VALUE[1:127].float()) / 2, torch.tensor([0.0, -0.0])])
    x = x.clamp(-448, 448)
    assert torch.equal(round_code(x.double()), x.to(torch.float8_e4m3fn).view(torch.uint8))
    assert round_code(torch.tensor([1e9, -1e9, 460.0], dtype=torch.float64)).tolist() == [126, 254, 126]


def test_scales_by_hand():
    x = torch.tensor([448.0, 448.0001, 224.0, 224.1, 7.0, 0.0, 1e-30, 1e30], dtype=torch.float64)
    assert scale_of(x).tolist() == [1.0, 2.0, 0.5, 1.0, 2.0 ** -6, 0.0, 2.0 ** -63, 2.0 ** 63]
    c, s = quantise(torch.full((1, 16, 4), 3.5))
    assert s.tolist() == [2.0 ** -7] and value(c).unique().tolist() == [448.0]
    assert torch.equal(dense(c, s), torch.full((1, 16, 4), 3.5, dtype=torch.float64))
    c, s = quantise(torch.zeros(1, 16, 4))
    assert s.tolist() == [0.0] and (c == 0).all() and (divide(torch.ones(3, dtype=torch.float64), torch.zeros(3)) == 0).all()


def test_a_larger_power_of_two_keeps_normal_codes():
    """Re-rounding to twice the scale changes nothing but the subnormals."""
    codes = torch.arange(16, 127, dtype=torch.uint8)
    assert torch.equal(value(round_code(value(codes) / 2)) * 2, value(codes))
    assert value(round_code(VALUE[1:2] / 2)).item() == 0.0     # a tie goes to the even code


def test_runs_by_hand():
    assert runs([5, 6, 7]) == [(0, 3, 0, 5)]
    assert runs([14, 15, 48, 49, -1, 33, 34, 7]) == [(0, 2, 0, 14), (2, 2, 3, 0), (5, 2, 2, 1), (7, 1, 0, 7)]
    assert runs([15, 16, 17]) == [(0, 1, 0, 15), (1, 2, 1, 0)]


def test_plain_decode_by_hand():
    """One key returns its value; queries of zero the mean."""
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(1, 3, 2, 16, 64, generator=g).double() for _ in range(2))
    bt = [[2, 0]]
    q = torch.zeros(1, 4, 64)
    a = plain_decode(q, (k, v), 0, torch.tensor(bt), [1])
    torch.testing.assert_close(a[0, :2], v[0, 2, 0, 0].expand(2, 64))
    b = plain_decode(q, (k, v), 0, torch.tensor(bt), [20])
    torch.testing.assert_close(b[0, 3], torch.cat([v[0, 2, 1], v[0, 0, 1, :4]]).mean(0))
