"""GPU parity of the 4-bit cache (kv4_store, kv4_load, mha_fwd_kv4) and of the
premix at given positions with the oracle, through the Python binding.

Tolerances.  Quantising and reading back are exact: fp32 values equal the
oracle's, bf16 ones its rounding.  Attention: each term of a row's sum carries
one bf16 rounding of p * s (at most 2^-8 of it), the output one more (2^-8 of
the result), and a score is off by at most
  dx = scale * 143 * 2^-21 * sum over groups of (largest scale) * sum |q|
     + 2^-20 |x|
(fp32 sums of values up to 143 |q|, a few 2^-23 steps each), which moves p by
2 dx relative and lse by dx:
  |o - r|     <= 2^-8 |r| + (2^-8 + 2 dx + 2^-16) sum_j p_j |v_j| + 2^-11 S
  |lse - r|   <= dx + 2^-20 (1 + |r|).
S, the largest scale of the group among the keys: up to two columns the codes
enter the MMAs as n = c + 8 <= 15, and 8 sum p s leaves O every 256 tokens.
Until then O holds at most 15 S sum p (over those tokens); each of its 16 MMAs
adds 16 products with at most 17 truncations of 2^-23 of that.  Summed over all
tokens, with sum p = 1: 16 * 17 * 2^-23 * 15 S < 2^-11 S.
"""
import math

import numpy as np
import pytest

import oracle as O
import synthetic as S
from helpers import assert_bf16_close, to_dev, to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import transformer_attention_iha_gb300 as T
    T.lib()
    assert T.device_error() == 0
    return T


def cache_of(T, n_pages, page, H, d, fill=0xFF):
    """0xFF: every scale of an unwritten slot is a NaN."""
    import torch
    return torch.full((n_pages, T.kv4_page_bytes(page, H, d)), fill, dtype=torch.uint8,
                      device="cuda")


def outlier_rows(shape, seed, dtype="bf16"):
    """Rows with channels of unequal size and offset, exact ties, zero groups."""
    x = S.normal(shape, seed, 0, dtype="f32")
    ch = S.normal(shape[-2:], seed, 1, dtype="f32")
    x = x * np.exp(ch) + 0.5 * S.normal(shape[-2:], seed, 2, dtype="f32")
    x[..., 0, :32] = np.round(2 * x[..., 0, :32]) / 2        # halves: many ties
    x[..., 0, 0] = 7.0
    x[..., 0, 1:32] = np.clip(x[..., 0, 1:32], -7, 7)
    if shape[-2] > 1:
        x[..., 1, -32:] = 0.0
    x = x.astype(np.float32)
    return S.f32_to_bf16_bits(x) if dtype == "bf16" else x


def assert_held(got, ref, what):
    """kv4_load's values: exact in fp32, the rounding of the oracle in bf16."""
    import torch
    g = to_f64(got)
    r = ref if got.dtype == torch.float32 else O.round_bf16(ref)
    np.testing.assert_array_equal(g, r.reshape(g.shape), err_msg=what)


# ------------------------------------------------------------------ store and load
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,H,d,page", [
    (1, 1, 1, 32, 16), (3, 7, 5, 64, 16), (2, 33, 3, 96, 48), (1, 129, 20, 128, 64),
    (5, 1, 80, 128, 32), (4, 16, 1, 128, 16), (1, 17, 2, 32, 128)])
def test_round_trip_is_exact(T, dtype, B, N, H, d, page):
    import torch
    k, v = outlier_rows((B, N, H, d), 11, dtype), S.normal((B, N, H, d), 12, 0, dtype=dtype)
    n_pages = -(-B * N // page) + 2
    cache = cache_of(T, n_pages, page, H, d)
    slots = S.rng(13).permutation(n_pages * page)[:B * N].astype(np.int32).reshape(B, N)
    T.kv4_store(to_dev(k), to_dev(v), to_dev(slots), cache, page)
    rk, rv = O.kv4_values(k), O.kv4_values(v)
    for dt in (torch.float32, torch.bfloat16):
        gk, gv = T.kv4_load(cache, to_dev(slots), H, d, page, dtype=dt)
        assert gk.dtype == dt and gk.shape == (B, N, H, d)
        assert_held(gk, rk, "k")
        assert_held(gv, rv, "v")
    assert T.device_error() == 0


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("first", [0, 1])
def test_many_rows_in_order(T, d, first):
    """A prompt's worth of rows (the store's form of several heads a warp), slots
    in order from an even and an odd one, heads that leave a unit part empty."""
    import torch
    N, H, page = 3301, 10, 16
    k, v = S.normal((1, N, H, d), 14, 0), S.normal((1, N, H, d), 14, 1)
    cache = cache_of(T, -(-N // page) + 1, page, H, d)
    slots = np.arange(first, first + N, dtype=np.int32)[None]
    slots[0, 100:103] = -1
    T.kv4_store(to_dev(k), to_dev(v), to_dev(slots), cache, page)
    gk, gv = T.kv4_load(cache, to_dev(slots), H, d, page, dtype=torch.float32)
    for got, x in ((gk, k), (gv, v)):
        r = O.kv4_values(x)
        r[0, 100:103] = 0.0
        np.testing.assert_array_equal(to_f64(got), r)
    assert T.device_error() == 0


def test_only_named_slots_change_and_load_takes_any_slots(T):
    import torch
    H, d, page = 3, 64, 16
    cache = cache_of(T, 4, page, H, d, 0)
    k0, v0 = S.normal((1, 64, H, d), 1, 0), S.normal((1, 64, H, d), 1, 1)
    every = np.arange(64, dtype=np.int32)[None]
    T.kv4_store(to_dev(k0), to_dev(v0), to_dev(every), cache, page)
    k1, v1 = S.normal((1, 5, H, d), 2, 0), S.normal((1, 5, H, d), 2, 1)
    new = np.array([[63, 0, 17, 18, 40]], np.int32)
    T.kv4_store(to_dev(k1), to_dev(v1), to_dev(new), cache, page)
    rk, rv = O.kv4_values(k0)[0], O.kv4_values(v0)[0]
    rk[new[0]], rv[new[0]] = O.kv4_values(k1)[0], O.kv4_values(v1)[0]
    pick = np.array([[5, 63, 63, 0, -1, 17, 40, 5]], np.int32)
    gk, gv = T.kv4_load(cache, to_dev(pick), H, d, page, dtype=torch.float32)
    for got, ref in ((gk, rk), (gv, rv)):
        r = ref[pick[0]]
        r[4] = 0.0                                       # padding reads as zeros
        np.testing.assert_array_equal(to_f64(got)[0], r)
    gk, gv = T.kv4_load(cache, to_dev(every), H, d, page, dtype=torch.float32)
    np.testing.assert_array_equal(to_f64(gk)[0], rk)
    np.testing.assert_array_equal(to_f64(gv)[0], rv)


def test_padding_and_slots_outside_the_cache(T):
    import torch
    H, d, page = 2, 128, 32
    cache = cache_of(T, 2, page, H, d, 0x5A)
    before = cache.clone()
    k, v = to_dev(S.normal((2, 3, H, d), 3, 0)), to_dev(S.normal((2, 3, H, d), 3, 1))
    T.kv4_store(k, v, to_dev(np.full((2, 3), -1, np.int32)), cache, page)
    assert T.device_error() == 0 and torch.equal(cache, before)
    bad = np.array([[64, -2, 2 ** 31 - 1], [-2 ** 31, 65, 1 << 20]], np.int32)
    T.kv4_store(k, v, to_dev(bad), cache, page)
    assert T.device_error() == 8 and torch.equal(cache, before)
    gk, gv = T.kv4_load(cache, to_dev(bad), H, d, page)
    assert T.device_error() == 8 and not gk.any() and not gv.any()
    assert T.device_error() == 0


def test_nonfinite_and_tiny_groups(T):
    import torch
    d, page = 128, 16
    x = np.ones((1, 6, 1, d), np.float32)
    x[0, 0, 0, 3] = np.inf
    x[0, 1, 0, 40] = -np.inf
    x[0, 2, 0, 127] = np.nan
    x[0, 3] *= np.float32(2.0 ** -101)
    x[0, 4] *= np.float32(3.3e38)
    x[0, 5] *= np.float32(2.0 ** -99)
    for xx in (x, S.f32_to_bf16_bits(x)):
        cache = cache_of(T, 1, page, 1, d)
        slots = to_dev(np.arange(6, dtype=np.int32)[None])
        T.kv4_store(to_dev(xx), to_dev(xx), slots, cache, page)
        for got in T.kv4_load(cache, slots, 1, d, page, dtype=torch.float32):
            np.testing.assert_array_equal(to_f64(got), O.kv4_values(xx))


def test_store_and_load_strided_views(T):
    """K and V as slices of one projection's output, a broadcast row, five
    dimensions, and results written into slices; rows around them untouched."""
    import torch
    B, N, H, d, page = 2, 9, 4, 64, 16
    qkv = S.normal((B, N, 3, H, d), 21, 0)
    t = to_dev(qkv)
    cache = cache_of(T, 3, page, H, d)
    slots = np.arange(B * N, dtype=np.int32)[::-1].reshape(B, N).copy()
    T.kv4_store(t[:, :, 1], t[:, :, 2], to_dev(slots), cache, page)
    out = torch.full((B, N, 2, H + 1, d + 8), 9.0, dtype=torch.float32, device="cuda")
    T.kv4_load(cache, to_dev(slots), H, d, page,
               out=(out[:, :, 0, :H, :d], out[:, :, 1, :H, :d]))
    np.testing.assert_array_equal(to_f64(out[:, :, 0, :H, :d]), O.kv4_values(qkv[:, :, 1]))
    np.testing.assert_array_equal(to_f64(out[:, :, 1, :H, :d]), O.kv4_values(qkv[:, :, 2]))
    assert torch.all(out[..., H, :] == 9.0) and torch.all(out[..., d:] == 9.0)
    one = to_dev(S.normal((1, 1, H, d), 22, 0))
    s5 = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 2, 2)
    T.kv4_store(one.expand(4, 2, H, d).unflatten(0, (2, 2)), one.expand(2, 2, 2, H, d), s5, cache,
                page)
    gk, _ = T.kv4_load(cache, s5, H, d, page, dtype=torch.float32)
    assert gk.shape == (2, 2, 2, H, d) and torch.equal(gk, gk[:1, :1, :1].expand_as(gk))
    assert T.device_error() == 0


def test_cache_longer_than_4_gib(T):
    """Offsets past 32 bits: the last pages of a cache of 5 GiB."""
    import torch
    H, d, page = 80, 128, 128
    n_pages = (5 << 30) // T.kv4_page_bytes(page, H, d)
    cache = torch.empty((n_pages, T.kv4_page_bytes(page, H, d)), dtype=torch.uint8, device="cuda")
    cache[-2:] = 0xFF
    cache[:2] = 0xFF
    n = 130
    k, v = S.normal((1, n, H, d), 31, 0), S.normal((1, n, H, d), 31, 1)
    slots = (np.arange(n)[None] + n_pages * page - n).astype(np.int32)
    T.kv4_store(to_dev(k), to_dev(v), to_dev(slots), cache, page)
    assert bool((cache[:2] == 0xFF).all())
    gk, gv = T.kv4_load(cache, to_dev(slots), H, d, page, dtype=torch.float32)
    np.testing.assert_array_equal(to_f64(gk), O.kv4_values(k))
    table = torch.tensor([[n_pages - 2, n_pages - 1]], dtype=torch.int32, device="cuda")
    q = S.normal((1, 1, H, d), 32, 0)
    # keys 126 .. 255 of the sequence are the rows stored; a window of n sees just them
    o = T.mha_fwd_kv4(to_dev(q), cache, table, torch.tensor([256], dtype=torch.int32,
                                                            device="cuda"), H, page,
                      mask=T.MASK_CAUSAL_WINDOW, window=n)
    check_rows(T, o[0], None, q[0], O.kv4_values(k)[0], O.kv4_values(v)[0], T.MASK_CAUSAL, 0)
    assert T.device_error() == 0


# ------------------------------------------------------------------ attention
def check_rows(T, o, lse, q, kv, vv, mask, window, scale=None):
    """One sequence: o [Nq, Hq, d], lse [Hq, Nq] or None, against the oracle."""
    Nq, Hq, d = q.shape
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    n, Hkv, _ = kv.shape
    r, rl, ra = O.kv4_attention(q, kv, vv, mask, window, scale)
    qa = np.abs(S.bf16_bits_to_f32(q).astype(np.float64)).reshape(Nq, Hq, d // 32, 32).sum(-1)
    s = np.abs(kv).reshape(n, Hkv, d // 32, 32).max(-1).max(0, initial=0.0) / 7  # [Hkv, d/32]
    dx = sc * 143 * 2.0 ** -21 * (qa * np.repeat(s, Hq // Hkv, 0)).sum(-1)       # [Nq, Hq]
    dx = dx + 2.0 ** -20 * sc * 7 * (qa * np.repeat(s, Hq // Hkv, 0)).sum(-1)
    g = to_f64(o)
    sv = np.abs(vv).reshape(n, Hkv, d // 32, 32).max(-1).max(0, initial=0.0) / 7
    S_ = np.repeat(np.repeat(sv, Hq // Hkv, 0), 32, -1)[None]                    # [1, Hq, d]
    bound = (2.0 ** -8 * np.abs(r) + (2.0 ** -8 + 2 * dx[..., None] + 2.0 ** -16) * ra +
             2.0 ** -11 * S_)
    assert np.isfinite(g).all()
    err = np.abs(g - r)
    assert (err <= bound).all(), (float((err / np.maximum(bound, 1e-30)).max()),
                                  np.unravel_index(np.argmax(err - bound), err.shape))
    if lse is not None:
        gl = to_f64(lse)
        empty = np.isneginf(rl)
        np.testing.assert_array_equal(np.isneginf(gl), empty)
        e = np.abs(np.where(empty, 0, gl) - np.where(empty, 0, rl))
        assert (e <= dx.T + 2.0 ** -20 * (1 + np.abs(np.where(empty, 0, rl)))).all(), e.max()


def build(T, lens, Hkv, d, page, seed, spare=2, width=None):
    """A cache with the sequences' pages in shuffled order, unwritten slots NaN."""
    import torch
    per = [-(-n // page) for n in lens]
    n_pages = sum(per) + spare
    order = S.rng(seed, 50).permutation(n_pages).astype(np.int32)
    width = width or max(1, max(per))
    table = np.full((len(lens), width), -7, np.int32)   # never read: would be flagged
    cache = cache_of(T, n_pages, page, Hkv, d)
    ks, vs, at = [], [], 0
    for b, n in enumerate(lens):
        table[b, :per[b]] = order[at:at + per[b]]
        at += per[b]
        k, v = outlier_rows((1, n, Hkv, d), seed + b), S.normal((1, n, Hkv, d), seed + b, 3)
        if n:
            j = np.arange(n)
            slots = (table[b, j // page] * page + j % page).astype(np.int32)[None]
            T.kv4_store(to_dev(k), to_dev(v), to_dev(slots), cache, page)
        ks.append(O.kv4_values(k)[0])
        vs.append(O.kv4_values(v)[0])
    return (cache, to_dev(table), torch.tensor(lens, dtype=torch.int32, device="cuda"), ks, vs)


def run_case(T, lens, Nq, Hq, Hkv, d, page, mask, window, seed=70, scale=0.0, **kw):
    cache, table, sl, ks, vs = build(T, lens, Hkv, d, page, seed)
    q = S.normal((len(lens), Nq, Hq, d), seed, 9)
    o, lse = T.mha_fwd_kv4(to_dev(q), cache, table, sl, Hkv, page, mask=mask, window=window,
                           scale=scale, return_lse=True, **kw)
    assert T.device_error() == 0
    for b in range(len(lens)):
        check_rows(T, o[b], lse[b], q[b], ks[b], vs[b], mask, window, scale or None)
    return o, lse


EDGE_LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 64, 100, 255, 257]


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("mask,window", [(0, 0), (1, 0), (2, 1), (2, 16), (2, 37)])
def test_single_token_edges(T, d, mask, window):
    run_case(T, EDGE_LENS, 1, 3, 3, d, 16, mask, window)


@pytest.mark.parametrize("Nq,Hq,Hkv", [(1, 4, 1), (1, 14, 2), (1, 8, 8), (2, 6, 2), (3, 5, 5),
                                       (4, 8, 2), (5, 21, 3), (9, 1, 1), (17, 4, 2), (40, 2, 2),
                                       (8, 32, 4)])
@pytest.mark.parametrize("mask,window", [(0, 0), (1, 0), (2, 20)])
def test_several_tokens_and_shared_heads(T, Nq, Hq, Hkv, mask, window):
    run_case(T, [0, 1, 5, 16, 40, 130], Nq, Hq, Hkv, 64, 32, mask, window)


@pytest.mark.parametrize("d", [32, 96, 128])
@pytest.mark.parametrize("Nq,Hq,Hkv", [(2, 2, 2), (1, 3, 1), (4, 2, 2), (1, 7, 1), (3, 4, 1),
                                       (1, 16, 1), (5, 5, 1)])
def test_column_forms(T, d, Nq, Hq, Hkv):
    """Each number of columns (new token x query head of a key head) that takes a
    form of its own: 1, 2, 3-4, 5-8, 9-16, more; every d."""
    run_case(T, [3, 75, 260], Nq, Hq, Hkv, d, 16, T.MASK_CAUSAL, 0)


@pytest.mark.parametrize("Nq,Hq,Hkv,d", [(1, 8, 8, 128), (4, 8, 2, 128), (1, 2, 1, 64),
                                         (16, 2, 1, 96), (2, 16, 1, 32)])
@pytest.mark.parametrize("page", [16, 48, 128])
def test_long_and_ragged(T, Nq, Hq, Hkv, d, page):
    run_case(T, [5000, 3, 1777, 2048, 0, 4095], Nq, Hq, Hkv, d, page, T.MASK_CAUSAL, 0)


def test_one_very_long_sequence(T):
    run_case(T, [70001], 1, 2, 2, 128, 64, T.MASK_CAUSAL, 0)
    run_case(T, [33333], 3, 2, 1, 64, 16, T.MASK_CAUSAL_WINDOW, 9000)


def test_many_short_sequences(T):
    lens = [int(x) for x in S.rng(5).integers(0, 70, 300)]
    run_case(T, lens, 1, 4, 2, 64, 16, T.MASK_CAUSAL, 0)


def test_scale_argument_and_large_scores(T):
    run_case(T, [100, 300], 1, 2, 2, 64, 16, T.MASK_CAUSAL, 0, scale=2.5)
    run_case(T, [100, 300], 1, 2, 2, 64, 16, T.MASK_CAUSAL, 0, scale=1e-4)


@pytest.mark.parametrize("Hq", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("kind", ["v_huge_hidden_by_softmax", "v_groups", "v_zero", "v_top",
                                  "q_large", "q_small", "mixed_tokens"])
def test_extreme_ranges(T, kind, Hq):
    """Scales far apart within a head: what a token that gets no weight holds, or
    another group, must not cost the others their digits."""
    import torch
    n, d, page = 150, 128, 16
    k = S.normal((n, 1, d), 180, 0, dtype="f32")
    v = S.normal((n, 1, d), 180, 1, dtype="f32")
    q = S.normal((1, Hq, d), 180, 2, dtype="f32")
    if kind == "v_huge_hidden_by_softmax":
        k[5] = -40.0 * q[0, 0] / np.abs(q[0, 0]).max()   # gets p ~ 0 from query 0
        q[0, 1:] = q[0, :1] * np.float32(1.25)
        v[5] *= np.float32(1e30)
        k[5] *= np.float32(8.0)                          # p underflows to 0 exactly
    elif kind == "v_groups":
        v *= np.repeat(np.float32([1e-20, 1.0, 1e20, 1e-3]), 32)
    elif kind == "v_zero":
        v[:, :, 32:64] = 0.0
        v[:100, :, 64:96] = 0.0
    elif kind == "v_top":
        v *= np.float32(8e36)                            # just below the largest bf16 scale
    elif kind == "q_large":
        q *= np.float32(1e20)
        k *= np.float32(1e-20)
    elif kind == "q_small":
        q *= np.float32(1e-30)
        k *= np.float32(1e30)
    else:
        v *= np.float32(10.0) ** S.rng(3).integers(-12, 12, (n, 1, 1)).astype(np.float32)
        k *= np.float32(0.2)
    kb, vb, qb = (S.f32_to_bf16_bits(x) for x in (k, v, q))
    cache = cache_of(T, 10, page, 1, d)
    T.kv4_store(to_dev(kb[None]), to_dev(vb[None]), to_dev(np.arange(n, dtype=np.int32)[None]),
                cache, page)
    table = torch.arange(10, dtype=torch.int32, device="cuda")[None]
    o, lse = T.mha_fwd_kv4(to_dev(qb[None]), cache, table,
                           torch.tensor([n], dtype=torch.int32, device="cuda"), 1, page,
                           return_lse=True)
    kv, vv = O.kv4_values(kb), O.kv4_values(vb)
    if kind != "v_huge_hidden_by_softmax":
        check_rows(T, o[0], lse[0], qb, kv, vv, T.MASK_CAUSAL, 0)
        return
    keep = np.r_[0:5, 6:n]                               # token 5 has weight 0
    check_rows(T, o[0], lse[0], qb, kv[keep], vv[keep], T.MASK_NONE, 0)


def test_strided_query_and_output(T):
    import torch
    lens, Nq, H, d, page = [50, 33], 2, 4, 64, 16
    cache, table, sl, ks, vs = build(T, lens, H, d, page, 90)
    qkv = S.normal((2, Nq, 3, H, d), 91, 0)
    out = torch.full((2, H + 1, Nq, d + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    ov = out[:, :H, :, :d].permute(0, 2, 1, 3)
    T.mha_fwd_kv4(to_dev(qkv)[:, :, 0], cache, table, sl, H, page, out=ov)
    for b in range(2):
        check_rows(T, ov[b], None, qkv[b, :, 0], ks[b], vs[b], T.MASK_CAUSAL, 0)
    assert torch.all(out[:, H] == 5.0) and torch.all(out[..., d:] == 5.0)


def test_hidden_rows_that_hold_nan_do_not_matter(T):
    """Keys after a token's position, before its window, and rows of the last
    page that were never written hold NaN scales."""
    import torch
    H, d, page, n = 2, 128, 16, 90
    k, v = S.normal((1, n, H, d), 95, 0), S.normal((1, n, H, d), 95, 1)
    kn, vn = k.copy(), v.copy()
    kn[0, :30], vn[0, :30] = 0x7FC0, 0x7FC0
    kn[0, 70:], vn[0, 70:] = 0x7F80, 0x7FC0
    q = S.normal((1, 40, H, d), 95, 2)
    table = torch.arange(6, dtype=torch.int32, device="cuda")[None]
    slots = to_dev(np.arange(n, dtype=np.int32)[None])
    sl = torch.tensor([n], dtype=torch.int32, device="cuda")
    outs = []
    for kk, vv in ((k, v), (kn, vn)):
        cache = cache_of(T, 6, page, H, d)
        T.kv4_store(to_dev(kk), to_dev(vv), slots, cache, page)
        outs.append(T.mha_fwd_kv4(to_dev(q), cache, table, sl, H, page,
                                  mask=T.MASK_CAUSAL_WINDOW, window=20, return_lse=True))
    # tokens at positions 50 .. 69 with a window of 20 see keys 31 .. 69 only
    assert torch.equal(outs[0][0][:, :20], outs[1][0][:, :20])
    assert torch.equal(outs[0][1][..., :20], outs[1][1][..., :20])
    assert torch.isnan(outs[1][0][:, 20:]).all()         # and the others do see them


def test_bad_pages_and_lengths_are_flagged(T):
    import torch
    H, d, page = 2, 64, 16
    cache, table, sl, ks, vs = build(T, [64, 64, 64], H, d, page, 97, width=5)
    q = S.normal((3, 1, H, d), 97, 9)
    t2 = table.clone()
    t2[1, 1], t2[1, 2] = 1 << 20, -1                     # keys 16 .. 47 of sequence 1 hidden
    o, lse = T.mha_fwd_kv4(to_dev(q), cache, t2, sl, H, page, return_lse=True)
    assert T.device_error() == 8
    check_rows(T, o[0], lse[0], q[0], ks[0], vs[0], T.MASK_CAUSAL, 0)
    keep = np.r_[0:16, 48:64]
    check_rows(T, o[1], lse[1], q[1], ks[1][keep], vs[1][keep], T.MASK_NONE, 0)
    bad = torch.tensor([64, -5, 64], dtype=torch.int32, device="cuda")
    o, lse = T.mha_fwd_kv4(to_dev(q), cache, table, bad, H, page, return_lse=True)
    assert T.device_error() == 8
    assert not o[1].any() and torch.isinf(lse[1]).all()
    check_rows(T, o[2], lse[2], q[2], ks[2], vs[2], T.MASK_CAUSAL, 0)
    long = torch.tensor([64, 64, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    T.mha_fwd_kv4(to_dev(q), cache, table[:, :4].contiguous(), long, H, page)
    assert T.device_error() == 8
    assert T.device_error() == 0


def test_workspace_is_reused_and_calls_are_repeatable(T):
    """One workspace through calls of different shapes, results bit for bit the
    same as with a fresh one."""
    import torch
    ws = None
    shapes = [([70000], 1, 2, 2, 128), ([100, 0, 5000], 4, 8, 2, 64), ([9] * 64, 1, 4, 4, 32),
              ([3000, 2900], 1, 40, 40, 128)]
    need = max(T.mha_fwd_kv4_workspace_bytes(len(l), n, hq, hk, d) for l, n, hq, hk, d in shapes)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for rep in range(2):
        for i, (lens, Nq, Hq, Hkv, d) in enumerate(shapes):
            cache, table, sl, _, _ = build(T, lens, Hkv, d, 16, 110 + i)
            q = to_dev(S.normal((len(lens), Nq, Hq, d), 110 + i, 9))
            a = T.mha_fwd_kv4(q, cache, table, sl, Hkv, 16, return_lse=True)
            b = T.mha_fwd_kv4(q, cache, table, sl, Hkv, 16, return_lse=True, workspace=ws)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert T.device_error() == 0


def test_captured_call_replays_with_new_lengths_and_pages(T):
    """Two graphs share a workspace and replay one after the other; lengths,
    pages and cache contents change between replays."""
    import torch
    H, d, page, B = 4, 128, 16, 3
    lens = [700, 64, 1500]
    cache, table, sl, ks, vs = build(T, lens, H, d, page, 120)
    q = S.normal((B, 1, H, d), 120, 9)
    qd = to_dev(q)
    ws = torch.zeros(T.mha_fwd_kv4_workspace_bytes(B, 1, H, H, d), dtype=torch.uint8,
                     device="cuda")
    outs = [torch.zeros_like(qd) for _ in range(2)]
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        T.mha_fwd_kv4(qd, cache, table, sl, H, page, out=outs[0], workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            T.mha_fwd_kv4(qd, cache, table, sl, H, page, out=outs[i], workspace=ws,
                          mask=T.MASK_CAUSAL if i == 0 else T.MASK_CAUSAL_WINDOW, window=100)
        graphs.append(g)
    for step in range(3):
        now = [max(1, n - 300 * step) for n in lens]
        sl.copy_(torch.tensor(now, dtype=torch.int32))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for b in range(B):
            check_rows(T, outs[0][b], None, q[b], ks[b][:now[b]], vs[b][:now[b]], T.MASK_CAUSAL, 0)
            check_rows(T, outs[1][b], None, q[b], ks[b][:now[b]], vs[b][:now[b]],
                       T.MASK_CAUSAL_WINDOW, 100)
    assert T.device_error() == 0


def test_streams(T):
    """Calls on a stream other than the current one, results made in the call."""
    import torch
    lens, H, d, page = [300, 20], 4, 64, 16
    cache, table, sl, ks, vs = build(T, lens, H, d, page, 130)
    q = S.normal((2, 1, H, d), 130, 9)
    qd = to_dev(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [T.mha_fwd_kv4(qd, cache, table, sl, H, page, stream=s) for _ in range(4)]
    slots = (table[:1, :1] * page + torch.arange(16, device="cuda")).to(torch.int32)
    s.wait_stream(torch.cuda.current_stream())
    got = T.kv4_load(cache, slots, H, d, page, dtype=torch.float32, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for o in outs:
        for b in range(2):
            check_rows(T, o[b], None, q[b], ks[b], vs[b], T.MASK_CAUSAL, 0)
    np.testing.assert_array_equal(to_f64(got[0])[0], ks[0][:16])


def test_two_calls_at_once(T):
    """Two streams, a workspace each, calls of different shapes in flight together."""
    import torch
    page = 16
    shapes = [([20000, 300], 1, 8, 8, 128), ([3000] * 9, 2, 8, 2, 64)]
    cases = []
    for i, (lens, Nq, Hq, Hkv, d) in enumerate(shapes):
        cache, table, sl, ks, vs = build(T, lens, Hkv, d, page, 190 + 20 * i)
        q = S.normal((len(lens), Nq, Hq, d), 190 + i, 9)
        ws = torch.zeros(T.mha_fwd_kv4_workspace_bytes(len(lens), Nq, Hq, Hkv, d),
                         dtype=torch.uint8, device="cuda")
        qd = to_dev(q)
        ref = T.mha_fwd_kv4(qd, cache, table, sl, Hkv, page, workspace=ws)
        cases.append((qd, cache, table, sl, Hkv, ws, torch.cuda.Stream(), ref, q, ks, vs))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(30):
        for o, (qd, cache, table, sl, Hkv, ws, st, *_r) in zip(outs, cases):
            o.append(T.mha_fwd_kv4(qd, cache, table, sl, Hkv, page, workspace=ws, stream=st))
    torch.cuda.synchronize()
    for o, c in zip(outs, cases):
        assert all(torch.equal(x, c[7]) for x in o)
        for b in range(len(c[9])):
            check_rows(T, c[7][b], None, c[8][b], c[9][b], c[10][b], T.MASK_CAUSAL, 0)
    assert T.device_error() == 0


def test_captured_decode_step(T):
    """One graph of premix, store and attention; positions, slots and lengths move
    on between replays, and each replay equals the calls made one by one."""
    import torch
    B, H, P, d, page, n0, steps = 3, 4, 2, 64, 16, 30, 5
    HP = H * P
    i32 = dict(dtype=torch.int32, device="cuda")
    width = 4
    table = torch.arange(B * width, **i32).flip(0).view(B, width).contiguous()
    x = [to_dev(S.normal((steps, B, 1, H, d), 200, t)) for t in range(3)]
    ws = [to_dev(S.premix_weight(H, P, 201, t)) for t in range(3)]
    k0, v0 = (to_dev(S.normal((B, n0, HP, d), 202, t)) for t in range(2))
    j = torch.arange(width * page, device="cuda")
    every = (table[:, j // page] * page + j % page).to(torch.int32)
    caches = [cache_of(T, B * width, page, HP, d) for _ in range(2)]
    for c in caches:
        T.kv4_store(k0, v0, every[:, :n0].contiguous(), c, page)
    scratch = [torch.zeros(T.mha_fwd_kv4_workspace_bytes(B, 1, HP, HP, d), dtype=torch.uint8,
                           device="cuda") for _ in range(2)]
    xin = [t[0].clone() for t in x]
    pos, slots, lens = torch.zeros((B, 1), **i32), torch.zeros((B, 1), **i32), torch.zeros(B, **i32)
    y = [torch.empty((B, 1, HP, d), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    o = torch.empty_like(y[0])

    def step(xs, ys, out, cache, work):
        T.premix_fwd_qkv_at(xs, ws, P, pos, out=ys)
        T.kv4_store(ys[1], ys[2], slots, cache, page)
        T.mha_fwd_kv4(ys[0], cache, table, lens, HP, page, out=out, workspace=work)

    def move(i):
        pos.fill_(n0 + i)
        slots.copy_(every[:, n0 + i:n0 + i + 1])
        lens.fill_(n0 + i + 1)
        for a, b in zip(xin, x):
            a.copy_(b[i])

    move(0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(xin, y, o, caches[0], scratch[0])
    y2, o2 = [torch.empty_like(t) for t in y], torch.empty_like(o)
    for i in range(steps):
        move(i)
        g.replay()
        step(xin, y2, o2, caches[1], scratch[1])
        assert all(torch.equal(a, b) for a, b in zip(y, y2)) and torch.equal(o, o2)
        assert torch.isfinite(o.float()).all()
    assert torch.equal(caches[0], caches[1])
    assert T.device_error() == 0


# ------------------------------------------------------------------ premix at positions
@pytest.mark.parametrize("B,N,H,P,d,dtype", [
    (1, 1, 20, 4, 128, "bf16"), (3, 5, 20, 4, 128, "bf16"), (7, 1, 4, 2, 64, "bf16"),
    (2, 3, 32, 4, 64, "bf16"), (1, 9, 8, 1, 32, "bf16"), (2, 4, 4, 2, 32, "f32"),
    (1, 3, 20, 4, 128, "f32"), (64, 1, 5, 3, 128, "bf16"), (13, 5, 5, 3, 128, "bf16"),
    (2, 32, 1, 1, 64, "bf16"), (5, 13, 32, 4, 64, "bf16")])
def test_premix_at_positions(T, B, N, H, P, d, dtype):
    xs = [S.normal((B, N, H, d), 140, t, dtype=dtype) for t in range(3)]
    ws = [S.premix_weight(H, P, 141, t) for t in range(3)]
    pos = S.rng(142).integers(0, 200000, (B, N)).astype(np.int32)
    pos[0, 0] = 0
    ys = T.premix_fwd_qkv_at([to_dev(x) for x in xs], [to_dev(w) for w in ws], P, to_dev(pos))
    for t in range(3):
        r = O.premix_at(xs[t], ws[t], P, pos) if t < 2 else O.premix_fwd(xs[t], ws[t], P)
        if dtype == "bf16":
            assert_bf16_close(to_f64(ys[t]), r, f"premix at {t}")
        else:
            np.testing.assert_allclose(to_f64(ys[t]), r, atol=1e-5, rtol=0)


@pytest.mark.parametrize("n,H,P,d", [(51, 20, 4, 128), (52, 20, 4, 128), (32, 32, 4, 64),
                                     (33, 32, 4, 64), (256, 8, 2, 64), (257, 8, 2, 64)])
def test_premix_at_where_the_kernels_change(T, n, H, P, d):
    """The largest call of the kernel for few tokens, and the next."""
    xs = [S.normal((n, 1, H, d), 145, t) for t in range(3)]
    ws = [S.premix_weight(H, P, 146, t) for t in range(3)]
    pos = S.rng(147).integers(0, 130000, (n, 1)).astype(np.int32)
    ys = T.premix_fwd_qkv_at([to_dev(x) for x in xs], [to_dev(w) for w in ws], P, to_dev(pos))
    for t in range(3):
        r = O.premix_at(xs[t], ws[t], P, pos) if t < 2 else O.premix_fwd(xs[t], ws[t], P)
        assert_bf16_close(to_f64(ys[t]), r, f"premix at {t}")


def test_premix_at_consecutive_positions_is_the_premix(T):
    import torch
    B, N, H, P, d = 2, 37, 20, 4, 128
    xs = [to_dev(S.normal((B, N, H, d), 150, t)) for t in range(3)]
    ws = [to_dev(S.premix_weight(H, P, 151, t)) for t in range(3)]
    pos = torch.arange(N, dtype=torch.int32, device="cuda").expand(B, N).contiguous()
    a = T.premix_fwd_qkv(xs, ws, P, rope=True)
    b = T.premix_fwd_qkv_at(xs, ws, P, pos)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


# ------------------------------------------------------------------ together, as a decode loop
@pytest.mark.parametrize("H,P,d,window", [(20, 4, 128, 0), (4, 2, 64, 40)])
def test_decode_loop_of_one_layer(T, H, P, d, window):
    """Prompt: premix, store.  Then token by token: premix at the position, store,
    attention; each step against the oracle's premix of that token and its
    attention over what the cache holds."""
    import torch
    B, n0, steps, page, HP = 2, 61, 6, 16, H * P
    n = n0 + steps
    xs = [S.normal((B, n, H, d), 160, t) for t in range(3)]
    ws = [S.premix_weight(H, P, 161, t) for t in range(3)]
    xd, wd = [to_dev(x) for x in xs], [to_dev(w) for w in ws]
    width = -(-n // page)
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").flip(0).view(B, width)
    table = table.contiguous()
    cache = cache_of(T, B * width, page, HP, d)
    ws4 = torch.zeros(T.mha_fwd_kv4_workspace_bytes(B, 1, HP, HP, d), dtype=torch.uint8,
                      device="cuda")
    mask = T.MASK_CAUSAL_WINDOW if window else T.MASK_CAUSAL

    def slots(a, b):
        j = torch.arange(a, b, device="cuda")
        return (table[:, j // page] * page + j % page).to(torch.int32).contiguous()

    _, kp, vp = T.premix_fwd_qkv([x[:, :n0].contiguous() for x in xd], wd, P, rope=True)
    T.kv4_store(kp, vp, slots(0, n0), cache, page)
    held = [[to_f64(kp)], [to_f64(vp)]]
    for i in range(n0, n):
        pos = torch.full((B, 1), i, dtype=torch.int32, device="cuda")
        q, k, v = T.premix_fwd_qkv_at([x[:, i:i + 1].contiguous() for x in xd], wd, P, pos)
        T.kv4_store(k, v, slots(i, i + 1), cache, page)
        sl = torch.full((B,), i + 1, dtype=torch.int32, device="cuda")
        o, lse = T.mha_fwd_kv4(q, cache, table, sl, HP, page, mask=mask, window=window,
                               return_lse=True, workspace=ws4)
        for t, y in enumerate((q, k)):
            r = O.premix_at(xs[t][:, i:i + 1], ws[t], P, np.full((B, 1), i))
            assert_bf16_close(to_f64(y), r, f"premix {t} at {i}")
        held[0].append(to_f64(k))
        held[1].append(to_f64(v))
        qb = q.cpu().view(torch.int16).numpy().view(np.uint16)
        for b in range(B):
            kv, vv = (O.kv4_values(np.concatenate(h, 1)[b].astype(np.float32)) for h in held)
            check_rows(T, o[b], lse[b], qb[b], kv, vv, mask, window)
    gk, gv = T.kv4_load(cache, slots(0, n), HP, d, page, dtype=torch.float32)
    for got, h in ((gk, held[0]), (gv, held[1])):
        np.testing.assert_array_equal(to_f64(got),
                                      O.kv4_values(np.concatenate(h, 1).astype(np.float32)))
    assert T.device_error() == 0


def test_joint_variant_decodes_its_pseudo_tokens(T):
    """The interleaved layout: a token is P pseudo-tokens of H heads; the P
    queries of the last token see pseudo-tokens up to their own."""
    import torch
    B, N, H, P, d, page = 1, 30, 4, 4, 64, 16
    xs = [S.normal((B, N, H, d), 170, t) for t in range(3)]
    ws = [S.premix_weight(H, P, 171, t) for t in range(3)]
    yq, yk, yv = T.premix_fwd_qkv_interleaved([to_dev(x) for x in xs], [to_dev(w) for w in ws], P,
                                              rope=True)
    q, k, v = (y.view(B, N * P, H, d) for y in (yq, yk, yv))
    cache = cache_of(T, 8, page, H, d)
    T.kv4_store(k, v, torch.arange(N * P, dtype=torch.int32, device="cuda")[None], cache, page)
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    sl = torch.tensor([N * P], dtype=torch.int32, device="cuda")
    o = T.mha_fwd_kv4(q[:, -P:], cache, table, sl, H, page)
    qb = q[:, -P:].contiguous().cpu().view(torch.int16).numpy().view(np.uint16)
    check_rows(T, o[0], None, qb[0], O.kv4_values(to_f64(k)[0].astype(np.float32)),
               O.kv4_values(to_f64(v)[0].astype(np.float32)), T.MASK_CAUSAL, 0)


# ------------------------------------------------------------------ the binding's checks
def test_binding_refusals(T):
    import torch
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")
    i32 = torch.int32
    cache = cache_of(T, 2, 16, 2, 64)
    k, slots = z(1, 3, 2, 64), z(1, 3, dt=i32)
    ok = dict(q=z(1, 1, 2, 64), cache=cache, block_table=z(1, 2, dt=i32), seq_lens=z(1, dt=i32),
              Hkv=2, page=16)
    for bad in (dict(k=k, v=z(1, 3, 2, 32)), dict(k=k, v=k.float()), dict(k=k.half(), v=k.half()),
                dict(k=k[0], v=k[0])):
        with pytest.raises((ValueError, TypeError)):
            T.kv4_store(bad["k"], bad["v"], slots, cache, 16)
    with pytest.raises(ValueError):
        T.kv4_store(k, k.clone(), slots.long(), cache, 16)
    with pytest.raises(ValueError):
        T.kv4_store(k, k.clone(), z(3, 1, dt=i32), cache, 16)
    with pytest.raises(ValueError):
        T.kv4_store(k, k.clone(), slots, cache, 32)              # page does not match the cache
    with pytest.raises(ValueError):
        T.kv4_store(k, k.clone(), slots, cache.cpu(), 16)
    with pytest.raises(ValueError):
        T.kv4_store(k.transpose(2, 3), k.transpose(2, 3), slots, cache, 16)
    with pytest.raises(ValueError):
        T.kv4_load(cache, slots[0], 2, 64, 16)
    with pytest.raises(ValueError):
        T.kv4_load(cache, slots, 2, 64, 16, out=(k, k.clone()[:, :2]))
    for change in (dict(q=z(1, 1, 2, 64, dt=torch.float32)), dict(q=z(1, 2, 64)),
                   dict(block_table=z(2, 2, dt=i32)), dict(seq_lens=z(2, dt=i32)),
                   dict(seq_lens=z(1, dt=torch.int64)), dict(page=24), dict(Hkv=3),
                   dict(out=z(1, 1, 2, 32)), dict(lse=z(1, 2, 2, dt=torch.float32)),
                   dict(workspace=z(16, dt=torch.float32)),
                   dict(workspace=z(16, dt=torch.uint8)), dict(q=z(1, 1, 3, 64)),
                   dict(mask=T.MASK_CAUSAL_WINDOW)):
        with pytest.raises((ValueError, T.IHAError)):
            T.mha_fwd_kv4(**{**ok, **change})
    x, w = [z(1, 2, 4, 32)] * 3, [z(4, 2, 4, dt=torch.float32)] * 3
    with pytest.raises(ValueError):
        T.premix_fwd_qkv_at(x, w, 2, z(2, 1, dt=i32))
    with pytest.raises(ValueError):
        T.premix_fwd_qkv_at(x, w, 2, z(1, 2, dt=torch.int64))
    assert T.device_error() == 0
