"""CPU tests of the 8-bit cache and of rotary positions: the oracle's definitions
against values worked out by hand, the rotation's table against whole numbers, and
the host checks of every entry point (each call here is refused before any launch)."""
import ctypes as C
import math
from fractions import Fraction

import numpy as np
import pytest

import oracle as O
import synthetic as S
import transformer_attention_iha_gb300 as T


@pytest.fixture(scope="module")
def L():
    T.build()
    return T.lib()


# ------------------------------------------------------------------ oracle pins
def test_e4m3_by_hand():
    y = [448, 447, 432, 17, 19, 1.0625, 1.1875, 2.0 ** -6, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 0]
    r = [448, 448, 448, 16, 20, 1.0, 1.25, 2.0 ** -6, 2.0 ** -9, 0, 2.0 ** -8, 0]
    assert list(O.round_e4m3(np.array(y))) == r
    assert list(O.round_e4m3(-np.array(y))) == [-v for v in r]


def test_e4m3_agrees_with_the_cast():
    import torch
    y = np.concatenate([S.normal((4000,), 1, 0, dtype="f32") * s for s in (100, 1, 0.01, 1e-3)])
    y = np.clip(y, -448, 448).astype(np.float32)
    c = torch.from_numpy(y).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(O.round_e4m3(y), c)


def test_block_exponent_by_hand():
    x = np.zeros((3, 6, 32))
    x[1, 0, 5] = -448.0
    x[0, 1, 0] = 449.0
    x[2, 2, 0] = 1.75
    x[2, 3, 0] = 1.76
    x[2, 4, 0] = 2.0 ** -120
    assert list(O.kv8_exponent(x)) == [0, 1, -8, -7, -100, -100]


def test_a_growing_block_rounds_its_codes_again():
    a = O.Kv8Rows(1, 32).append(np.full((3, 1, 32), 1.8125, np.float32))   # 1.8125 = 232 * 2^-7
    assert a.e.tolist() == [[-7]] and a.values[0, 0, 0] == 1.75            # tie, to even
    small = np.full((1, 1, 32), 2.0 ** -14, np.float32)
    a.append(small)
    assert a.values[3, 0, 0] == 2.0 ** -14                                 # 2^-7 of the scale
    a.append(np.full((1, 1, 32), 448.0, np.float32))
    assert a.e.tolist() == [[0]] and a.values[0, 0, 0] == 1.75
    assert a.values[3, 0, 0] == 0.0 and a.values[4, 0, 0] == 448.0         # below half of 2^-9
    a.append(np.full((12, 1, 32), 1.0, np.float32))
    assert a.e.tolist() == [[0], [-8]] and len(a.values) == 17
    # a row that is not all finite is NaN and has no part in the scale
    b = O.Kv8Rows(1, 32).append(np.array([[[np.inf] + [1.0] * 31], [[1.0] * 32]], np.float32))
    assert np.isnan(b.values[0]).all() and (b.values[1] == 1.0).all() and b.e.tolist() == [[-8]]


def test_kept_positions_by_hand():
    w = np.array([[5, 1, 5, np.nan, 2, 2, 9, 0], [0, 0, 0, 0, 0, 0, 0, 0.0]], np.float32)
    assert O.kv8_kept(w, 4, 2).tolist() == [[0, 2, 6, 7], [0, 1, 6, 7]]
    assert O.kv8_kept(w, 5, 1).tolist() == [[0, 2, 4, 6, 7], [0, 1, 2, 3, 7]]
    assert O.kv8_kept(w, 3, 0).tolist() == [[0, 2, 6], [0, 1, 2]]
    assert O.kv8_kept(w, 3, 3).tolist() == [[5, 6, 7], [5, 6, 7]]
    assert O.kv8_kept(w, 8, 3).tolist() == [list(range(8))] * 2


def test_weights_of_the_oracle_sum_to_its_rows():
    q, k = S.normal((3, 4, 32), 5, 0), S.normal((9, 2, 32), 5, 1, dtype="f32").astype(np.float64)
    w = O.kv8_weights(q, k)
    np.testing.assert_allclose(w.sum(1), 6.0)           # 3 rows of 2 query heads
    assert not w[:, 9 - 3 + 1:].all(0).all() or w[0, 8] < w[0].sum()
    v = np.zeros((9, 2, 32))
    v[4] = 1.0                                          # o picks out the weight of key 4
    o, _, _ = O.kv4_attention(q, k, v)
    np.testing.assert_allclose(o[:, :2, 0].sum(), w[0, 4])
    np.testing.assert_allclose(o[:, 2:, 0].sum(), w[1, 4])


def test_rope_oracle_is_the_premix_rotation():
    """Half layout, whole head: the rotation that the premix applies (an identity mix)."""
    d = 32
    x = S.normal((1, 5, 2, d), 6, 0)
    eye = np.eye(2, dtype=np.float32).reshape(2, 1, 2)
    w, _ = O.rope_frequencies(d)
    ref = O.premix_fwd(x, eye, 1, rope=True)
    np.testing.assert_allclose(O.rotate(x, np.arange(5)[None], w), ref, atol=1e-12)
    y = O.rotate(x, np.arange(5)[None], w, 1.5, True)
    z = y.reshape(1, 5, 2, d // 2, 2)
    x2 = S.bf16_bits_to_f32(x).reshape(1, 5, 2, d // 2, 2)
    np.testing.assert_allclose((z ** 2).sum(-1), 2.25 * (x2.astype(np.float64) ** 2).sum(-1))
    back = O.rotate(y.astype(np.float32), np.arange(5)[None], w, 1.0, True, back=True)
    np.testing.assert_allclose(back, 1.5 * S.bf16_bits_to_f32(x), atol=1e-6)


# ------------------------------------------------------------------ the rotation's table
@pytest.mark.parametrize("rot,base,scaling,factor,trained", [
    (2, 10000.0, None, 1.0, 0), (64, 10000.0, None, 1.0, 0), (128, 500000.0, "linear", 4.0, 0),
    (96, 10000.0, "base", 8.0, 0), (128, 10000.0, "parts", 8.0, 4096), (256, 1e6, "parts", 40.0, 2)])
def test_rope_table(L, rot, base, scaling, factor, trained):
    """turn = w / 2 pi * 2^64 to a few bits of double precision; the gain."""
    r = T.Rope(rot, base=base, scaling=scaling, factor=factor, trained=trained)
    w, gain = O.rope_frequencies(rot, base, scaling, factor, trained)
    for i in range(rot // 2):
        want = float(w[i]) / (2 * math.pi)
        got = float(Fraction(int(r._c.turn[i]), 2 ** 64))
        assert abs(got - want) <= 2.0 ** -48 * want + 2.0 ** -64
    assert r.gain == np.float32(gain) and r.rot == rot
    assert T.Rope(rot, gain=0.75).gain == 0.75


@pytest.mark.parametrize("kw,status", [
    (dict(rot=0), 1), (dict(rot=7), 1), (dict(rot=258), 2), (dict(rot=8, base=1.0), 1),
    (dict(rot=8, base=math.nan), 1), (dict(rot=8, base=math.inf), 1),
    (dict(rot=8, gain=-1.0), 1), (dict(rot=8, gain=math.nan), 1), (dict(rot=8, gain=1e-60), 1),
    (dict(rot=8, scaling="linear", factor=0.5), 1), (dict(rot=8, scaling="base", factor=math.nan), 1),
    (dict(rot=2, scaling="base", factor=2.0), 1), (dict(rot=8, scaling="parts", factor=2.0), 1),
    (dict(rot=8, scaling="parts", factor=2.0, trained=64, fast=1.0, slow=1.0), 1),
    (dict(rot=8, scaling="parts", factor=2.0, trained=64, slow=-1.0), 1)])
def test_rope_init_refusals(L, kw, status):
    with pytest.raises(T.IHAError) as e:
        T.Rope(**kw)
    assert e.value.status == status
    assert L.iha_rope_init(None) == 1
    with pytest.raises(ValueError):
        T.Rope(8, scaling="cubic")


# ------------------------------------------------------------------ refusals
def _p(i, off=0):
    return C.c_void_p((1 << 44) + (i << 38) + off)      # apart, never dereferenced


def _st(b, n, h):
    return T.Strides(b, 0, n, h)


def _rope_args(**kw):
    r = kw.pop("rope", T.Rope(64))
    a = dict(q=_p(0), k=_p(1), pos=_p(2), yq=_p(3), yk=_p(4), rope=C.addressof(r._c) if r else None,
             B=2, N=4, Hq=8, Hk=2, d=64, sq=_st(2048, 512, 64), sk=_st(512, 128, 64),
             syq=_st(2048, 512, 64), syk=_st(512, 128, 64), dt=T.BF16, stream=None)
    a.update(kw)
    return list(a.values()), r


@pytest.mark.parametrize("fn", ["iha_rope_fwd", "iha_rope_bwd"])
def test_rope_refusals(L, fn):
    def call(**kw):
        args, keep = _rope_args(**kw)
        return getattr(L, fn)(*args)
    for kw in (dict(q=None), dict(yq=None), dict(rope=None), dict(k=None), dict(yk=None),
               dict(Hk=0), dict(B=0), dict(N=-1), dict(Hq=0), dict(d=0), dict(dt=7),
               dict(rope=T.Rope(128)), dict(sq=_st(-2048, 512, 64)), dict(syq=_st(2048, 0, 64)),
               dict(syq=_st(2048, 512, 32)), dict(syk=_st(512, 128, 0)), dict(yq=_p(1)),
               dict(yk=_p(0)), dict(yk=_p(3)), dict(yq=_p(0, 16)), dict(yq=_p(2)),
               dict(yq=_p(0), syq=_st(2048, 512, 72))):
        assert call(**kw) == 1, kw
    assert call(d=60, rope=T.Rope(32)) == 2 and "multiple of 8" in L.iha_last_error().decode()
    assert call(B=1 << 16, N=1 << 15) == 2
    for kw in (dict(q=_p(0, 8)), dict(yk=_p(4, 2)), dict(pos=_p(2, 2)),
               dict(sq=_st(2048, 516, 64)), dict(syk=_st(512, 132, 64))):
        assert call(**kw) == 3, kw
    bad = T.Rope(64)
    bad._c.mul = 0.0
    assert call(rope=bad) == 1


def test_page_bytes(L):
    assert L.kv8_page_bytes(64, 80, 128) == 4 * 80 * (32 * 128 + 16)
    assert L.kv8_page_bytes(16, 1, 32) == 32 * 32 + 128      # whole lines of 128 bytes
    assert L.kv8_page_bytes(32, 3, 64) == 6 * 32 * 64 + 128
    for a in ((0, 1, 32), (24, 1, 32), (16, 0, 32), (16, 1, 16), (16, 1, 160), (16, 1, 33)):
        assert L.kv8_page_bytes(*a) == 0
        with pytest.raises(ValueError):
            T.kv8_page_bytes(*a)


def test_append_refusals(L):
    def call(**kw):
        a = dict(k=_p(0), v=_p(1), table=_p(2), lens=_p(3), counts=None, cache=_p(4), B=2, N=3,
                 n_pages=8, page=16, width=4, H=2, d=64, sk=_st(384, 128, 64),
                 sv=_st(384, 128, 64), dt=T.BF16, stream=None)
        a.update(kw)
        return L.kv8_append(*a.values())
    for kw in (dict(k=None), dict(v=None), dict(table=None), dict(lens=None), dict(cache=None),
               dict(B=0), dict(N=0), dict(n_pages=0), dict(page=0), dict(width=0), dict(H=0),
               dict(d=0), dict(dt=5), dict(sk=_st(384, -128, 64)), dict(k=_p(4, 16)),
               dict(lens=_p(4)), dict(counts=_p(4)), dict(table=_p(4))):
        assert call(**kw) == 1, kw
    for kw in (dict(page=24), dict(d=48), dict(d=160), dict(n_pages=1 << 28), dict(width=1 << 27),
               dict(H=1 << 14, N=1 << 24, width=1 << 20, sk=_st(0, 0, 64), sv=_st(0, 0, 64))):
        assert call(**kw) == 2, kw
    for kw in (dict(k=_p(0, 8)), dict(cache=_p(4, 8)), dict(sv=_st(384, 132, 64)),
               dict(lens=_p(3, 2)), dict(counts=_p(5, 1))):
        assert call(**kw) == 3, kw


def test_load_refusals(L):
    s = T.Strides(384, 0, 128, 64)

    def call(**kw):
        a = dict(cache=_p(4), slots=_p(2), k=_p(0), v=_p(1), Bo=2, Bi=1, N=3, n_pages=8, page=16,
                 H=2, d=64, sk=s, sv=s, dt=T.BF16, stream=None)
        a.update(kw)
        return L.kv8_load(*a.values())
    for kw in (dict(cache=None), dict(slots=None), dict(k=None), dict(v=None), dict(Bo=0),
               dict(N=0), dict(dt=9), dict(k=_p(4)), dict(v=_p(2)), dict(v=_p(0)),
               dict(v=_p(0, 64)), dict(sk=T.Strides(384, 0, 0, 64)),
               dict(sk=T.Strides(384, 0, 128, 32)), dict(sv=T.Strides(-384, 0, 128, 64))):
        assert call(**kw) == 1, kw
    assert call(d=40) == 2 and call(Bo=1 << 16, N=1 << 15) == 2
    assert call(k=_p(0, 4)) == 3 and call(slots=_p(2, 2)) == 3 and call(cache=_p(4, 4)) == 3
    assert call(sk=T.Strides(384, 0, 124, 64)) == 3


def _attn(L, **kw):
    a = dict(q=_p(0), cache=_p(1), table=_p(2), lens=_p(3), o=_p(4), lse=None, w=None, wo=None,
             ws=_p(6), wsb=1 << 30, B=2, Nq=1, Hq=4, Hkv=2, d=64, n_pages=8, page=16, width=4,
             sq=_st(256, 256, 64), so=_st(256, 256, 64), scale=0.0, mask=1, window=0, dt=T.BF16,
             stream=None)
    a.update(kw)
    return L.mha_fwd_kv8(*a.values())


def test_attention_refusals(L):
    for kw in (dict(q=None), dict(cache=None), dict(table=None), dict(lens=None), dict(o=None),
               dict(ws=None), dict(B=0), dict(Nq=0), dict(Hq=0), dict(Hkv=0), dict(width=0),
               dict(dt=4), dict(mask=3), dict(mask=2), dict(Hq=5), dict(scale=2e30),
               dict(wsb=4096), dict(so=_st(256, 256, 0)), dict(so=_st(256, 256, 32)),
               dict(sq=_st(-8, 256, 64)), dict(o=_p(0)), dict(o=_p(1)), dict(lse=_p(4)),
               dict(ws=_p(1)), dict(w=_p(7)), dict(wo=_p(7)), dict(w=_p(7), wo=_p(7, 4)),
               dict(w=_p(7), wo=_p(4)), dict(w=_p(7), wo=_p(0)), dict(w=_p(7), wo=_p(1)),
               dict(w=_p(7), wo=_p(6)), dict(w=_p(6, 8192), wo=_p(7)), dict(w=_p(7), wo=_p(3)),
               dict(w=_p(7), wo=_p(8), lse=_p(8)), dict(w=_p(4), wo=_p(8))):
        assert _attn(L, **kw) == 1, kw
    for kw in (dict(dt=T.F32), dict(d=48), dict(page=20), dict(width=1 << 27),
               dict(Nq=1 << 20, so=_st(1 << 28, 256, 64)), dict(B=(1 << 30) + 1),
               dict(w=_p(7), wo=_p(8), Nq=33, so=_st(1 << 14, 256, 64), sq=_st(1 << 14, 256, 64))):
        assert _attn(L, **kw) == 2, kw
    for kw in (dict(q=_p(0, 8)), dict(o=_p(4, 8)), dict(sq=_st(256, 256, 60)), dict(ws=_p(6, 128)),
               dict(lens=_p(3, 1)), dict(w=_p(7, 2), wo=_p(8)), dict(w=_p(7), wo=_p(8, 1))):
        assert _attn(L, **kw) == 3, kw


def test_attention_workspace(L):
    f = L.mha_fwd_kv8_workspace_bytes
    base = f(2, 1, 4, 2, 64, 0)
    assert base > 4096 and f(2, 1, 4, 2, 64, 512) == base + 4 * (8 + 2 * 2 * 2 * 512)
    for a in ((0, 1, 4, 2, 64, 0), (2, 1, 5, 2, 64, 0), (2, 1, 4, 2, 64, -1), (2, 0, 4, 2, 64, 0)):
        assert f(*a) == 0
    assert f(1 << 20, 1, 1 << 10, 1 << 10, 64, 1 << 30) == 0     # past any memory
    assert _attn(L, B=1 << 20, w=_p(7), wo=_p(8), width=1 << 26) == 2
    # a workspace without room for the scores is refused
    assert _attn(L, w=_p(7), wo=_p(8), wsb=base) == 1


def test_evict_refusals(L):
    def call(**kw):
        a = dict(cache=_p(0), table=_p(1), lens=_p(2), w=_p(3), dest=_p(4), nl=_p(5), kept=_p(6),
                 wo=_p(7), B=2, n_pages=8, page=16, width=4, dwidth=2, H=2, d=64, keep=32,
                 recent=8, stream=None)
        a.update(kw)
        return L.kv8_evict(*a.values())
    for kw in (dict(cache=None), dict(table=None), dict(lens=None), dict(w=None), dict(dest=None),
               dict(nl=None), dict(kept=None), dict(B=0), dict(width=0), dict(dwidth=0),
               dict(keep=0), dict(recent=-1), dict(recent=33), dict(keep=33), dict(H=0),
               dict(wo=_p(3)), dict(kept=_p(2)), dict(nl=_p(6)), dict(wo=_p(6)), dict(w=_p(0)),
               dict(dest=_p(5)), dict(kept=_p(0, 64))):
        assert call(**kw) == 1, kw
    for kw in (dict(d=48), dict(page=8), dict(width=1 << 27), dict(dwidth=1 << 27),
               dict(B=1 << 18, H=1 << 12), dict(B=1 << 27, H=1, keep=1, recent=0)):
        assert call(**kw) == 2, kw
    for kw in (dict(cache=_p(0, 8)), dict(w=_p(3, 2)), dict(kept=_p(6, 1)), dict(wo=_p(7, 3))):
        assert call(**kw) == 3, kw
