"""CPU tests of the 4-bit cache: the oracle's quantiser against values worked
out by hand, its attention against the plain oracle attention, and the host
checks of kv4_store, kv4_load, mha_fwd_kv4 and iha_premix_fwd_qkv_at (every
call here is refused before any launch)."""
import ctypes as C
import math

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
def test_quantiser_by_hand():
    """Group maximum 7: scale 1, codes the rounded values, ties to even."""
    x = np.zeros((1, 32), np.float32)
    x[0, :8] = [7, -7, 0.5, 1.5, 2.5, -0.5, -2.5, 3.25]
    r = O.kv4_values(x)
    assert list(r[0, :8]) == [7, -7, 0, 2, 2, 0, -2, 3] and not r[0, 8:].any()


def test_quantiser_scale_is_rounded_to_bf16():
    x = np.zeros((1, 64), np.float32)
    x[0, 0], x[0, 1] = 1.0, 0.5                       # scale bf16(1 / 7) = 146 / 1024
    x[0, 32:] = 2.0 ** -101                           # below the smallest group maximum
    r = O.kv4_values(x)
    s = 146 / 1024
    assert r[0, 0] == 7 * s and r[0, 1] == 4 * s and not r[0, 32:].any()
    assert O.kv4_values(np.full((1, 32), 2.0 ** -100, np.float32)).any()


def test_quantiser_float32_counts_as_bf16_and_nonfinite_groups_are_nan():
    x = np.zeros((1, 96), np.float32)
    x[0, 0], x[0, 1] = 7.0, 2.5 + 2.0 ** -10          # rounds to 2.5 first, then to even
    x[0, 33], x[0, 64] = np.inf, np.nan
    r = O.kv4_values(x)
    assert r[0, 1] == 2.0
    assert np.isnan(r[0, 32:]).all() and not np.isnan(r[0, :32]).any()


def test_quantiser_error_is_at_most_half_a_step():
    x = S.normal((50, 4, 128), 3, 0)
    f = S.bf16_bits_to_f32(x).astype(np.float64)
    r = O.kv4_values(x)
    step = np.abs(f.reshape(50, 4, 4, 32)).max(-1, keepdims=True) / 7 * (1 + 2.0 ** -8)
    assert np.all(np.abs(r - f).reshape(50, 4, 4, 32) <= 0.5 * step + 7 * 2.0 ** -8 * step)


@pytest.mark.parametrize("mask,window", [(0, 0), (1, 0), (2, 5)])
def test_cache_attention_oracle_agrees_with_plain_attention(mask, window):
    """Nq = n: the last n positions are the whole sequence."""
    n, H, d = 23, 2, 32
    q, k, v = (S.normal((n, H, d), 5, c, dtype="f32") for c in range(3))
    o, lse, _ = O.kv4_attention(q, k.astype(np.float64), v.astype(np.float64), mask, window)
    ro, rl = O.attention(q[None, None], k[None, None], v[None, None], mask, window)
    np.testing.assert_allclose(o, ro[0, 0], atol=1e-12)
    np.testing.assert_allclose(lse, rl[0, 0], atol=1e-12)


def test_premix_at_oracle_is_the_premix_at_consecutive_positions():
    x, w = S.normal((2, 5, 4, 32), 7, 0), S.premix_weight(4, 2, 7, 1)
    pos = np.arange(5)[None].repeat(2, 0)
    np.testing.assert_allclose(O.premix_at(x, w, 2, pos), O.premix_fwd(x, w, 2, rope=True),
                               atol=1e-12)


# ------------------------------------------------------------------ host checks
A = 0x100000000  # addresses far apart, never dereferenced


def _p(i, off=0):
    return C.c_void_p(A * i + off)


def _st(*s):
    return T.Strides(*s)


def test_page_bytes(L):
    assert T.kv4_page_bytes(64, 80, 128) == 64 * 80 * 144
    assert T.kv4_page_bytes(16, 1, 32) == 16 * 36
    for bad in [(8, 1, 32), (0, 1, 32), (24, 1, 64), (16, 0, 64), (16, 1, 48), (16, 1, 160)]:
        assert L.kv4_page_bytes(*bad) == 0
        with pytest.raises(ValueError):
            T.kv4_page_bytes(*bad)


@pytest.mark.parametrize("fn", ["kv4_store", "kv4_load"])
def test_store_and_load_refusals(L, fn):
    def call(k=_p(1), v=_p(2), slots=_p(3), cache=_p(4), Bo=2, Bi=1, N=3, n_pages=4, page=16, H=2,
             d=64, sk=None, sv=None, dt=T.BF16):
        s = _st(N * H * d, N * H * d, H * d, d)
        sk, sv = sk or s, sv or s
        bufs = (k, v, slots, cache) if fn == "kv4_store" else (cache, slots, k, v)
        return getattr(L, fn)(*bufs, Bo, Bi, N, n_pages, page, H, d, sk, sv, dt, None)

    for name in ("k", "v", "slots", "cache"):
        assert call(**{name: None}) == 1
    for name in ("Bo", "Bi", "N", "n_pages", "page", "H", "d"):
        assert call(**{name: 0}) == 1
        assert call(**{name: -1}) == 1
    assert call(dt=7) == 1
    assert call(d=48) == 2 and call(d=160) == 2 and call(page=24) == 2
    assert call(n_pages=1 << 27, page=16) == 2
    assert call(Bo=1 << 20, Bi=1 << 6, N=1 << 6) == 2
    assert call(k=_p(1, 8)) == 3 and call(v=_p(2, 4)) == 3 and call(cache=_p(4, 8)) == 3
    assert call(slots=_p(3, 2)) == 3
    assert call(sk=_st(0, 0, 132, 64)) == 3
    assert call(sv=_st(384, 0, 128, -64)) == 1
    assert call(k=_p(4, 64)) == 1                       # inside the cache
    assert "overlap" in L.iha_last_error().decode()
    assert call(slots=_p(4, 64)) == 1
    if fn == "kv4_load":
        assert call(v=_p(1)) == 1                       # k and v at one address
        assert call(sk=_st(0, 0, 128, 64)) == 1         # every batch row to the same place
        assert "stride 0" in L.iha_last_error().decode()


def test_attention_refusals(L):
    def call(q=_p(1), cache=_p(2), table=_p(3), lens=_p(4), o=_p(5), lse=None, ws=_p(6),
             wsb=1 << 40, B=2, Nq=3, Hq=4, Hkv=2, d=64, n_pages=4, page=16, tw=4, sq=None, so=None,
             mask=1, window=0, dt=T.BF16):
        s = _st(Nq * Hq * d, 0, Hq * d, d)
        return L.mha_fwd_kv4(q, cache, table, lens, o, lse, ws, wsb, B, Nq, Hq, Hkv, d, n_pages,
                             page, tw, sq or s, so or s, 0.0, mask, window, dt, None)

    for name in ("q", "cache", "table", "lens", "o", "ws"):
        assert call(**{name: None}) == 1
    for name in ("B", "Nq", "Hq", "Hkv", "d", "n_pages", "page", "tw"):
        assert call(**{name: 0}) == 1
    assert call(mask=3) == 1 and call(mask=2, window=0) == 1 and call(dt=9) == 1
    assert call(dt=T.F32) == 2
    assert call(Hq=5) == 1
    assert "multiple" in L.iha_last_error().decode()
    assert call(d=80) == 2 and call(page=8) == 2 and call(tw=1 << 27) == 2
    assert call(Nq=1 << 24) == 2
    assert call(q=_p(1, 8)) == 3 and call(o=_p(5, 2)) == 3 and call(cache=_p(2, 4)) == 3
    assert call(table=_p(3, 2)) == 3 and call(lens=_p(4, 1)) == 3 and call(lse=_p(7, 2)) == 3
    assert call(ws=_p(6, 128)) == 3
    assert call(wsb=0) == 1
    assert "workspace" in L.iha_last_error().decode()
    assert call(sq=_st(768, 0, 252, 64)) == 3 and call(so=_st(768, 0, -256, 64)) == 1
    assert call(o=_p(1)) == 1 and call(o=_p(2)) == 1 and call(lse=_p(5)) == 1
    assert call(ws=_p(5)) == 1 and call(ws=_p(2)) == 1
    assert "overlap" in L.iha_last_error().decode()
    assert call(so=_st(0, 0, 256, 64)) == 1 and call(so=_st(768, 0, 256, 0)) == 1
    assert "stride 0" in L.iha_last_error().decode()
    assert L.mha_fwd_kv4(*[_p(i) for i in (1, 2, 3, 4, 5)], None, _p(6), 1 << 40, 1, 1, 1, 1, 64, 4,
                         16, 4, _st(64, 0, 64, 64), _st(64, 0, 64, 64), 2e30, 1, 0, T.BF16,
                         None) == 1
    assert call(Nq=1, Hq=4096 * 2, Hkv=2) == 2           # 4096 query heads a key head
    assert L.mha_fwd_kv4_workspace_bytes(2, 3, 4, 2, 64) > 0
    assert L.mha_fwd_kv4_workspace_bytes(2, 3, 5, 2, 64) == 0


def test_premix_at_refusals(L):
    def call(xk=_p(2), pos=_p(7), yv=_p(10), H=4, P=2, d=32, dt=T.BF16, base=1e4):
        return L.iha_premix_fwd_qkv_at(_p(1), xk, _p(3), _p(4), _p(5), _p(6), pos, _p(8), _p(9),
                                       yv, 1, 8, H, P, d, dt, base, None)
    assert call(pos=None) == 1 and call(xk=None) == 1
    assert call(pos=_p(7, 2)) == 3 and call(yv=_p(10, 8)) == 3
    assert call(H=33, P=1) == 2 and call(d=96) == 2 and call(dt=5) == 1 and call(base=0.0) == 1
    assert call(yv=_p(7)) == 1
    assert "positions" in L.iha_last_error().decode()
    assert call(yv=_p(8)) == 1
