"""GPU parity of the 8-bit cache (kv8_append, kv8_load, mha_fwd_kv8, kv8_evict) with
the oracle, through the Python binding.

Tolerances.  What the cache holds, which keys are kept and their weights: exact.
Attention, with u = 2^-23: a score is a sum of d exact products in d / 16 matrix
instructions, each of which adds 16 products and truncates at most 17 times by u of the
sum of their magnitudes, and three scalings of u / 2:
  dx = scale (17 d / 16 + 2) u max over keys of sum_f |q_f k_f|,
moves p by 2 dx (its own and the sum's) and lse by dx; exp2 and the sums of p add less
than 2^-16 (blocks of 16 keys a warp: up to 30 here).  Each term p v of O is rounded
once to fp16, 2^-11 of itself or 2^-30 of the largest p s times a code up to 448, and
the result to bf16:
  |o - r|   <= 2^-8 |r| + (2^-11 + 2 dx + 2^-16) sum p |v| + n 2^-30 448 max(p) max(s)
  |lse - r| <= dx + 2^-20 (1 + |r|)
  |w - r|   <= (2 dx + 2^-19 (1 + |lse|)) times what the call adds + 2^-23 |r| + 2^-120,
the last for up to 64 probabilities below 2^-126, the smallest normal number of fp32 (one
of 1.6e-71, a row whose scores are 160 apart, is 0)."""
import math

import numpy as np
import pytest

import oracle as O
import synthetic as S
from helpers import to_dev, to_f64

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


def ints(a):
    import torch
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def cache_of(T, n_pages, page, H, d, fill=0xFF):
    """0xFF: every code and scale of a page that was never written is a NaN."""
    import torch
    return torch.full((n_pages, T.kv8_page_bytes(page, H, d)), fill, dtype=torch.uint8,
                      device="cuda")


def rows(shape, seed, dtype="bf16", stream=0):
    """Rows with channels of unequal size, whose size drifts from row to row."""
    x = S.normal(shape, seed, stream, dtype="f32")
    ch = S.normal(shape[-2:], seed, stream + 20, dtype="f32")
    row = S.normal(shape[:-1] + (1,), seed, stream + 21, dtype="f32")
    x = (x * np.exp(ch) * np.exp(0.7 * row)).astype(np.float32)
    return S.f32_to_bf16_bits(x) if dtype == "bf16" else x


def tables(lens, page, seed, spare=2, width=None):
    """Pages in shuffled order; entries that no key needs are never read."""
    per = [-(-n // page) for n in lens]
    n_pages = sum(per) + spare
    order = S.rng(seed, 50).permutation(n_pages).astype(np.int32)
    table = np.full((len(lens), width or max(1, max(per))), -7, np.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    return table, n_pages, order[at:]


def slots_of(table, b, n, page):
    j = np.arange(n)
    return (table[b, j // page] * page + j % page).astype(np.int32)[None]


def assert_held(T, cache, table, b, page, ref_k, ref_v, what=""):
    """Everything that sequence b holds equals the oracle's rows, in fp32 and in bf16."""
    import torch
    n, H, d = ref_k.values.shape
    if n == 0:
        return
    for dt in (torch.float32, torch.bfloat16):
        got = T.kv8_load(cache, to_dev(slots_of(table, b, n, page)), H, d, page, dtype=dt)
        for g, r in zip(got, (ref_k.values, ref_v.values)):
            r = r if dt == torch.float32 else O.round_bf16(r.astype(np.float32)).reshape(r.shape)
            np.testing.assert_array_equal(to_f64(g)[0], r, err_msg=what)


# ------------------------------------------------------------------ append and load
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("page", [16, 48])
def test_appends_of_any_length(T, dtype, d, page):
    """Sequences that grow by 1, 15, 16, 17, 40, ... rows a call, out of step, each
    block's scale growing as its rows come."""
    H, steps = 3, [1, 15, 16, 17, 3, 40, 1, 1, 2, 33]
    starts = [0, 5, 16, 31]
    lens = [s + sum(steps) for s in starts]
    table, n_pages, _ = tables(lens, page, 3)
    cache = cache_of(T, n_pages, page, H, d)
    B = len(starts)
    refs = [(O.Kv8Rows(H, d), O.Kv8Rows(H, d)) for _ in range(B)]
    at = [0] * B
    for i, N in enumerate([max(starts)] + steps):
        k, v = rows((B, N, H, d), 100 + i, dtype), rows((B, N, H, d), 200 + i, dtype, 3)
        counts = starts if i == 0 else [N] * B
        at = [a + c for a, c in zip(at, counts)]
        T.kv8_append(to_dev(k), to_dev(v), to_dev(table), ints(at), cache, page,
                     counts=ints(counts) if i == 0 else None)
        for b in range(B):
            for r, x in zip(refs[b], (k, v)):
                if counts[b]:
                    r.append(x[b, N - counts[b]:])
    assert T.device_error() == 0
    for b in range(B):
        assert_held(T, cache, table, b, page, *refs[b], f"sequence {b}")


@pytest.mark.parametrize("N,H,d,dtype", [(3301, 10, 128, "bf16"), (777, 80, 128, "f32"),
                                         (1500, 7, 96, "bf16"), (1025, 1, 32, "f32")])
def test_a_prompt(T, N, H, d, dtype):
    page = 64
    table, n_pages, _ = tables([N], page, 4)
    cache = cache_of(T, n_pages, page, H, d)
    k, v = rows((1, N, H, d), 5, dtype), S.normal((1, N, H, d), 6, 0, dtype=dtype)
    T.kv8_append(to_dev(k), to_dev(v), to_dev(table), ints([N]), cache, page)
    assert_held(T, cache, table, 0, page, O.Kv8Rows(H, d).append(k[0]), O.Kv8Rows(H, d).append(v[0]))


def test_padding_counts_and_bytes_that_stay(T):
    """Rows before the first key are padding; a count of 0 adds nothing; pages and heads
    that get no row keep every byte; the rest of a fresh block is zeros."""
    import torch
    H, d, page, N = 2, 64, 32, 7
    table = np.array([[3, 1], [0, 5], [2, 4]], np.int32)
    cache = cache_of(T, 7, page, H, d, 0x5A)
    before = cache.clone()
    k, v = rows((3, N, H, d), 8), rows((3, N, H, d), 9)
    T.kv8_append(to_dev(k), to_dev(v), to_dev(table), ints([0, 20, 9]), cache, page,
                 counts=ints([7, 0, 0]))
    assert T.device_error() == 0 and torch.equal(cache, before)
    T.kv8_append(to_dev(k), to_dev(v), to_dev(table), ints([4, 33, 9]), cache, page,
                 counts=ints([7, 1, 0]))
    assert T.device_error() == 0
    changed = (cache != before).any(1).tolist()
    assert changed == [False, False, False, True, False, True, False]
    assert_held(T, cache, table, 0, page, O.Kv8Rows(H, d).append(k[0, 3:]),
                O.Kv8Rows(H, d).append(v[0, 3:]))
    # key 32 of sequence 1 is the first of page 5; rows 1 .. 15 of its block are zeros
    got = T.kv8_load(cache, ints([list(range(5 * page, 5 * page + 16))]), H, d, page,
                     dtype=torch.float32)
    for g, x in zip(got, (k, v)):
        np.testing.assert_array_equal(to_f64(g)[0, 0],
                                      O.Kv8Rows(H, d).append(x[1, -1:]).values[0])
        assert not g[0, 1:].any()
    blocks = cache[5, :2 * H * 32 * d].view(H, 2, -1)  # the other block of each head in page 5
    assert bool((blocks[:, 1] == 0x5A).all()) and bool((blocks[:, 0] != 0x5A).any())
    tails = cache[5, 2 * H * 32 * d:].view(-1, 16)[:2 * H].view(H, 2, 16)
    assert bool((tails[:, 1] == 0x5A).all()) and bool((tails[:, 0] != 0x5A).any())
    assert bool((cache[5, 2 * H * (32 * d + 16):] == 0x5A).all())


def test_bad_lengths_counts_and_pages_are_flagged(T):
    import torch
    H, d, page = 1, 32, 16
    cache = cache_of(T, 2, page, H, d, 0)
    before = cache.clone()
    k = to_dev(rows((1, 20, H, d), 10))
    T.kv8_append(k, k, ints([[2, -1]]), ints([20]), cache, page)
    assert T.device_error() == 8 and torch.equal(cache, before)
    T.kv8_append(k, k, ints([[0, 1]]), ints([33]), cache, page, counts=ints([0]))
    assert T.device_error() == 8 and torch.equal(cache, before)
    T.kv8_append(k, k, ints([[0, 1]]), ints([-3]), cache, page)
    assert T.device_error() == 8 and torch.equal(cache, before)
    T.kv8_append(k, k, ints([[0, 1]]), ints([3]), cache, page, counts=ints([-1]))
    assert T.device_error() == 8 and torch.equal(cache, before)
    T.kv8_append(k, k, ints([[0, 7]]), ints([16]), cache, page, counts=ints([21]))
    assert T.device_error() == 8
    got = T.kv8_load(cache, ints([[-1, 32, -2, 5]]), H, d, page)[0]
    assert T.device_error() == 8 and not got[0, :3].any() and got[0, 3].any()
    assert T.device_error() == 0


def test_rows_that_are_not_finite_and_extreme_ones(T):
    import torch
    H, d, page = 1, 128, 16
    x = np.ones((1, 9, H, d), np.float32)
    x[0, 0, 0, 3] = np.inf
    x[0, 2, 0, 127] = np.nan
    x[0, 3] *= np.float32(2.0 ** -130)
    x[0, 4] *= np.float32(3.0e38)
    x[0, 5] *= np.float32(2.0 ** -99)
    x[0, 6, 0, :] = 0.0
    x[0, 6, 0, 0] = -0.0
    for xx in (x, S.f32_to_bf16_bits(x)):
        for order in (slice(None), [8, 7, 6, 5, 4, 3, 2, 1, 0], [3, 5, 6, 3, 5, 6, 3, 5, 6]):
            xs = np.ascontiguousarray(xx[:, order])
            cache = cache_of(T, 1, page, H, d)
            r = O.Kv8Rows(H, d)
            for a, b in ((0, 4), (4, 5), (5, 9)):
                c = np.ascontiguousarray(xs[:, a:b])
                T.kv8_append(to_dev(c), to_dev(c), ints([[0]]), ints([b]), cache, page)
                r.append(c[0])
            assert_held(T, cache, np.array([[0]]), 0, page, r, r)
    # a row written over one of NaN
    cache = cache_of(T, 1, page, H, d)
    T.kv8_append(to_dev(x[:, :3]), to_dev(x[:, :3]), ints([[0]]), ints([3]), cache, page)
    T.kv8_append(to_dev(x[:, 1:2]), to_dev(x[:, 1:2]), ints([[0]]), ints([3]), cache, page)
    got = T.kv8_load(cache, ints([[0, 1, 2]]), H, d, page, dtype=torch.float32)[0]
    assert torch.isnan(got[0, 0]).all() and bool((got[0, 1:] == 1.0).all())


def test_strided_views_and_five_dimensions(T):
    import torch
    B, N, H, d, page = 2, 9, 4, 64, 16
    qkv = rows((B, N, 3, H, d), 21)
    t = to_dev(qkv)
    table = np.array([[1], [0]], np.int32)
    cache = cache_of(T, 2, page, H, d)
    T.kv8_append(t[:, :, 1], t[:, :, 2], to_dev(table), ints([N, N]), cache, page)
    out = torch.full((B, N, 2, H + 1, d + 8), 9.0, dtype=torch.float32, device="cuda")
    slots = to_dev(np.concatenate([slots_of(table, b, N, page) for b in range(B)]))
    T.kv8_load(cache, slots, H, d, page, out=(out[:, :, 0, :H, :d], out[:, :, 1, :H, :d]))
    for b in range(B):
        for i in range(2):
            np.testing.assert_array_equal(to_f64(out[b, :, i, :H, :d]),
                                          O.Kv8Rows(H, d).append(qkv[b, :, 1 + i]).values)
    assert torch.all(out[..., H, :] == 9.0) and torch.all(out[..., d:] == 9.0)
    one = to_dev(rows((1, 1, H, d), 22))
    T.kv8_append(one.expand(2, 4, H, d), one.expand(2, 4, H, d), to_dev(table), ints([4, 4]),
                 cache, page)
    s5 = ints([[[0, 1], [16, 17]], [[3, 2], [-1, 19]]])
    gk, _ = T.kv8_load(cache, s5, H, d, page, dtype=torch.float32)
    assert gk.shape == (2, 2, 2, H, d) and not gk[1, 1, 0].any()
    assert torch.equal(gk[0], gk[:1, :1, :1].expand(1, 2, 2, H, d)[0])
    assert T.device_error() == 0


def test_cache_longer_than_4_gib(T):
    """Offsets past 32 bits: append, read, attend and evict in the last pages of 5 GiB."""
    import torch
    H, d, page = 80, 128, 128
    pb = T.kv8_page_bytes(page, H, d)
    n_pages = (5 << 30) // pb
    cache = torch.empty((n_pages, pb), dtype=torch.uint8, device="cuda")
    cache[-4:] = 0xFF
    cache[:2] = 0xFF
    n = 130
    table = np.array([[n_pages - 2, n_pages - 1]], np.int32)
    k, v = rows((1, n, H, d), 31), rows((1, n, H, d), 32)
    T.kv8_append(to_dev(k), to_dev(v), to_dev(table), ints([n]), cache, page)
    rk, rv = O.Kv8Rows(H, d).append(k[0]), O.Kv8Rows(H, d).append(v[0])
    assert_held(T, cache, table, 0, page, rk, rv)
    q = S.normal((1, 1, H, d), 33, 0)
    w = torch.zeros((1, H, 2 * page), device="cuda")
    o, w = T.mha_fwd_kv8(to_dev(q), cache, to_dev(table), ints([n]), H, page, weights=w)
    check_rows(o[0], None, q[0], rk.values, rv.values, T.MASK_CAUSAL, 0)
    dest = np.array([[n_pages - 3]], np.int32)
    lens, kept, _ = T.kv8_evict(cache, to_dev(table), ints([n]), w, to_dev(dest), H, d, page, 100, 9)
    ids = O.kv8_kept(to_f64(w)[0, :, :n], 100, 9)
    np.testing.assert_array_equal(kept[0].cpu().numpy(), ids)
    assert_held(T, cache, dest, 0, page, rk.evicted(ids), rv.evicted(ids))
    assert bool((cache[:2] == 0xFF).all()) and T.device_error() == 0


# ------------------------------------------------------------------ attention
def score_error(q, k, scale):
    """dx of each row and query head [Nq, Hq]."""
    Nq, Hq, d = q.shape
    G = Hq // k.shape[1]
    qa = np.abs(q.astype(np.float64))
    ka = np.abs(np.nan_to_num(k))
    most = np.stack([(qa[:, h] @ ka[:, h // G].T).max(1, initial=0.0) for h in range(Hq)], 1)
    return scale * (17 * d / 16 + 2) * 2.0 ** -23 * most


def check_rows(o, lse, q, k, v, mask, window, scale=None, w=None, w0=None):
    """One sequence: o [Nq, Hq, d], lse [Hq, Nq], w [Hkv, n], against the oracle."""
    Nq, Hq, d = q.shape
    n, Hkv, _ = k.shape
    G = Hq // Hkv
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    qf = S.bf16_bits_to_f32(q)
    r, rl, ra = O.kv4_attention(q, k, v, mask, window, scale)
    dx = score_error(qf, k, sc)
    s = np.abs(v).max((0, 2), initial=0.0) / 224          # a block's scale, at most [Hkv]
    flat = n * 2.0 ** -30 * 448 * np.repeat(s, G)[None, :, None]
    bound = 2.0 ** -8 * np.abs(r) + (2.0 ** -11 + 2 * dx[..., None] + 2.0 ** -16) * ra + flat
    g = to_f64(o)
    assert np.isfinite(g).all()
    err = np.abs(g - r)
    assert (err <= bound).all(), (float((err / np.maximum(bound, 1e-30)).max()),
                                  np.unravel_index(np.argmax(err - bound), err.shape))
    empty = np.isneginf(rl)
    rl0 = np.where(empty, 0, rl)
    if lse is not None:
        gl = to_f64(lse)
        np.testing.assert_array_equal(np.isneginf(gl), empty)
        e = np.abs(np.where(empty, 0, gl) - rl0)
        assert (e <= dx.T + 2.0 ** -20 * (1 + np.abs(rl0))).all(), e.max()
    if w is not None:
        add = O.kv8_weights(q, k, mask, window, scale)
        rel = (2 * dx + 2.0 ** -19 * (1 + np.abs(rl0.T))).max(0).reshape(Hkv, G).max(1)[:, None]
        rw = w0 + add
        e = np.abs(w - rw)
        over = e - (rel * add + 2.0 ** -23 * rw + 2.0 ** -120)
        bad = np.argwhere(over > 0)[:3].tolist()
        assert not bad, [(i, e[tuple(i)], add[tuple(i)], rw[tuple(i)]) for i in bad]


def build(T, lens, Hkv, d, page, seed, spare=2, width=None):
    table, n_pages, free = tables(lens, page, seed, spare, width)
    cache = cache_of(T, n_pages, page, Hkv, d)
    ks, vs = [], []
    for b, n in enumerate(lens):
        k, v = rows((1, n, Hkv, d), seed + b), rows((1, n, Hkv, d), seed + b, stream=3)
        if n:
            T.kv8_append(to_dev(k), to_dev(v), to_dev(table[b:b + 1]), ints([n]), cache, page)
        ks.append(O.Kv8Rows(Hkv, d).append(k[0]))
        vs.append(O.Kv8Rows(Hkv, d).append(v[0]))
    return cache, to_dev(table), ints(lens), ks, vs, free


def run_case(T, lens, Nq, Hq, Hkv, d, page, mask, window, seed=70, scale=0.0, weigh=True):
    import torch
    cache, table, sl, ks, vs, _ = build(T, lens, Hkv, d, page, seed)
    q = S.normal((len(lens), Nq, Hq, d), seed, 9)
    cap = table.shape[1] * page
    weigh = weigh and Nq * Hq // Hkv <= 64
    w0 = S.rng(seed, 60).random((len(lens), Hkv, cap), np.float32) if weigh else None
    kw = dict(weights=to_dev(w0)) if weigh else {}
    res = T.mha_fwd_kv8(to_dev(q), cache, table, sl, Hkv, page, mask=mask, window=window,
                        scale=scale, return_lse=True, **kw)
    assert T.device_error() == 0
    o, lse = res[:2]
    for b, n in enumerate(lens):
        w = to_f64(res[2])[b] if weigh else None
        check_rows(o[b], lse[b], q[b], ks[b].values, vs[b].values, mask, window, scale or None,
                   None if w is None else w[:, :n], None if w is None else w0[b, :, :n])
        if weigh:
            np.testing.assert_array_equal(w[:, n:], w0[b, :, n:])
    if weigh:  # without weights, the same bits
        plain = T.mha_fwd_kv8(to_dev(q), cache, table, sl, Hkv, page, mask=mask, window=window,
                              scale=scale)
        assert torch.equal(plain, o)
    return o, lse


EDGE_LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 64, 100, 255, 257]


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("mask,window", [(0, 0), (1, 0), (2, 1), (2, 16), (2, 37)])
def test_single_token_edges(T, d, mask, window):
    run_case(T, EDGE_LENS, 1, 3, 3, d, 16, mask, window)


@pytest.mark.parametrize("Nq,Hq,Hkv", [(1, 4, 1), (1, 14, 2), (1, 8, 8), (2, 6, 2), (3, 5, 5),
                                       (4, 8, 2), (5, 21, 3), (9, 1, 1), (17, 4, 2), (40, 2, 2),
                                       (8, 32, 4), (70, 1, 1)])
@pytest.mark.parametrize("mask,window", [(0, 0), (1, 0), (2, 20)])
def test_several_tokens_and_shared_heads(T, Nq, Hq, Hkv, mask, window):
    run_case(T, [0, 1, 5, 16, 40, 130], Nq, Hq, Hkv, 64, 32, mask, window)


@pytest.mark.parametrize("d", [32, 96, 128])
@pytest.mark.parametrize("Nq,Hq,Hkv", [(2, 2, 2), (1, 3, 1), (4, 2, 2), (1, 7, 1), (3, 4, 1),
                                       (1, 16, 1), (5, 5, 1)])
def test_column_forms(T, d, Nq, Hq, Hkv):
    run_case(T, [3, 75, 260], Nq, Hq, Hkv, d, 16, T.MASK_CAUSAL, 0)


@pytest.mark.parametrize("Nq,Hq,Hkv,d", [(1, 8, 8, 128), (4, 8, 2, 128), (1, 2, 1, 64),
                                         (16, 2, 1, 96), (2, 16, 1, 32)])
@pytest.mark.parametrize("page", [16, 48, 128])
def test_long_and_ragged(T, Nq, Hq, Hkv, d, page):
    run_case(T, [5000, 3, 1777, 2048, 0, 4095], Nq, Hq, Hkv, d, page, T.MASK_CAUSAL, 0)


def test_one_long_sequence(T):
    run_case(T, [20001], 1, 2, 2, 128, 64, T.MASK_CAUSAL, 0)
    run_case(T, [13333], 3, 2, 1, 64, 16, T.MASK_CAUSAL_WINDOW, 9000)


def test_many_short_sequences(T):
    lens = [int(x) for x in S.rng(5).integers(0, 70, 300)]
    run_case(T, lens, 1, 4, 2, 64, 16, T.MASK_CAUSAL, 0)


def test_scale_argument_and_large_scores(T):
    run_case(T, [100, 300], 1, 2, 2, 64, 16, T.MASK_CAUSAL, 0, scale=2.5)
    run_case(T, [100, 300], 1, 2, 2, 64, 16, T.MASK_CAUSAL, 0, scale=1e-4)


def test_a_key_alone_gives_its_value(T):
    """One visible key: o is exactly the value that the cache holds."""
    for d in (32, 64, 96, 128):
        H, n, page = 4, 50, 16
        cache, table, sl, ks, vs, _ = build(T, [n], H, d, page, 40)
        q = S.normal((1, 3, H, d), 41, 0)
        o = T.mha_fwd_kv8(to_dev(q), cache, table, sl, H, page, mask=T.MASK_CAUSAL_WINDOW, window=1)
        np.testing.assert_array_equal(to_f64(o)[0], vs[0].values[-3:])


@pytest.mark.parametrize("kind", ["falling", "rising", "far", "tiny", "huge"])
@pytest.mark.parametrize("Hq", [1, 4, 12])
def test_scales_of_v_and_scores_that_move_apart(T, kind, Hq):
    """V's block scales run over 2^60 while the scores favour now the one end, now the
    other; blocks far below and above the range of fp16."""
    import torch
    n, d, page = 700, 64, 16
    q = S.normal((1, 1, Hq, d), 81, 0)
    k, v = S.normal((1, n, 1, d), 81, 1, dtype="f32"), S.normal((1, n, 1, d), 81, 2, dtype="f32")
    ramp = np.linspace(-30, 30, n)[None, :, None, None]
    if kind == "falling":
        v = v * 2.0 ** -ramp
    elif kind == "rising":
        v = v * 2.0 ** ramp
    elif kind == "far":
        v = v * np.where(np.arange(n) % 100 < 50, 2.0 ** -40, 2.0 ** 40)[None, :, None, None]
    else:
        v = v * 2.0 ** (-90 if kind == "tiny" else 100)
    k = k + 0.5 * ramp / 30 * S.normal((d,), 81, 3, dtype="f32")
    k, v = (S.f32_to_bf16_bits(x.astype(np.float32)) for x in (k, v))
    table, n_pages, _ = tables([n], page, 82)
    cache = cache_of(T, n_pages, page, 1, d)
    T.kv8_append(to_dev(k), to_dev(v), to_dev(table), ints([n]), cache, page)
    rk, rv = O.Kv8Rows(1, d).append(k[0]), O.Kv8Rows(1, d).append(v[0])
    o = T.mha_fwd_kv8(to_dev(q), cache, to_dev(table), ints([n]), 1, page)
    r, _, ra = O.kv4_attention(q[0], rk.values, rv.values)
    dx = score_error(S.bf16_bits_to_f32(q[0]), rk.values, d ** -0.5)
    # terms below 2^-19 of the largest p s so far are off by 2^-30 of it, times 448
    p = O.kv8_weights(q[0], rk.values) if Hq == 1 else np.ones((1, n))
    ps = (np.minimum(p, 1.0) * np.ldexp(1.0, np.repeat(rv.e[:, 0], 16)[:n])).max()
    bound = (2.0 ** -8 * np.abs(r) + (2.0 ** -11 + 2 * dx[..., None] + 2.0 ** -16) * ra +
             n * 2.0 ** -30 * 448 * ps)
    g = to_f64(o)[0]
    assert np.isfinite(g).all() and (np.abs(g - r) <= bound).all(), (np.abs(g - r) / bound).max()


def test_strided_query_and_output(T):
    import torch
    B, Nq, H, d, page = 2, 3, 4, 64, 16
    cache, table, sl, ks, vs, _ = build(T, [40, 7], H, d, page, 90)
    x = S.normal((B, Nq, 3, H, d), 91, 0)
    out = torch.full((B, H, Nq, d + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    o = out[..., :d].transpose(1, 2)
    T.mha_fwd_kv8(to_dev(x)[:, :, 1], cache, table, sl, H, page, out=o)
    for b in range(B):
        check_rows(o[b], None, np.ascontiguousarray(x[b, :, 1]), ks[b].values, vs[b].values, 1, 0)
    assert bool((out[..., d:] == 9.0).all())


def test_rows_of_nan_count_only_where_they_are_seen(T):
    """A drafted token whose K or V is not finite does not touch the tokens before it; a
    window that has passed it does not see it; where it is seen, everything is NaN (of V:
    O, of K: O, lse and weights)."""
    import torch
    n, d, page, Nq = 45, 64, 16, 6
    for which in (0, 1):
        x = [rows((1, n, 1, d), 95), rows((1, n, 1, d), 96)]
        f = [S.bf16_bits_to_f32(a) for a in x]
        f[which][0, 41, 0, 5] = np.nan
        f[which][0, 20, 0, 5] = -np.inf
        x = [S.f32_to_bf16_bits(a) for a in f]
        cache = cache_of(T, 3, page, 1, d)
        table = ints([[2, 0, 1]])
        T.kv8_append(to_dev(x[0]), to_dev(x[1]), table, ints([n]), cache, page)
        ref = [O.Kv8Rows(1, d).append(a[0]) for a in x]
        q = S.normal((1, Nq, 1, d), 97, 0)
        w = torch.zeros((1, 1, 3 * page), device="cuda")
        o, lse, w = T.mha_fwd_kv8(to_dev(q), cache, table, ints([n]), 1, page,
                                  mask=T.MASK_CAUSAL_WINDOW, window=10, return_lse=True, weights=w)
        # rows 39 .. 44; keys 30 .. 44 at most: 41 is seen from row 41 on, 20 never
        assert not torch.isnan(o[0, :2]).any() and torch.isnan(o[0, 2:]).all()
        assert torch.isnan(lse[0, 0]).tolist() == [False, False] + [which == 0] * 4
        clean = [np.nan_to_num(a.values[:41]) for a in ref]
        check_rows(o[0, :2], lse[0, :, :2], q[0, :2], *clean, T.MASK_CAUSAL_WINDOW, 10)
        assert not torch.isnan(w[0, 0, :30]).any()
        assert torch.isnan(w[0, 0, 32:45]).all() == (which == 0)
        o = T.mha_fwd_kv8(to_dev(q[:, :1]), cache, table, ints([40]), 1, page)
        assert torch.isnan(o).all()                     # all keys: 20 is among them
        o = T.mha_fwd_kv8(to_dev(q[:, :1]), cache, table, ints([20]), 1, page)
        check_rows(o[0], None, q[0, :1], *(a.values[:20] for a in ref), 1, 0)
    assert T.device_error() == 0


def test_bad_pages_and_lengths_are_flagged(T):
    import torch
    H, d, page = 2, 64, 16
    cache, table, sl, ks, vs, _ = build(T, [64, 40], H, d, page, 120)
    q = S.normal((2, 1, H, d), 121, 0)
    bad = table.clone()
    bad[0, 1], bad[0, 3] = 10 ** 6, -1
    w = torch.zeros((2, H, 64), device="cuda")
    o, w = T.mha_fwd_kv8(to_dev(q), cache, bad, sl, H, page, weights=w)
    assert T.device_error() == 8
    keep = np.r_[0:16, 32:48]
    check_rows(o[0], None, q[0], ks[0].values[keep], vs[0].values[keep], 0, 0)
    assert not w[0, :, 16:32].any() and not w[0, :, 48:].any()
    assert abs(float(w[0].sum()) - H) < 1e-4
    check_rows(o[1], None, q[1], ks[1].values, vs[1].values, 1, 0)
    o2 = T.mha_fwd_kv8(to_dev(q), cache, table, ints([1000, -5]), H, page)
    assert T.device_error() == 8
    check_rows(o2[0], None, q[0], ks[0].values, vs[0].values, 1, 0)
    assert not o2[1].any()
    allbad, lse, w = T.mha_fwd_kv8(to_dev(q), cache, torch.full_like(table, -1), sl, H, page,
                                   return_lse=True, weights=torch.zeros_like(w))
    assert T.device_error() == 8 and not allbad.any() and bool((lse == -math.inf).all())
    assert not w.any()


def test_weights_in_place_and_workspaces(T):
    """In place equals apart; one workspace, zeroed once, for calls of many shapes."""
    import torch
    ws = torch.zeros(T.mha_fwd_kv8_workspace_bytes(3, 4, 8, 2, 64, 512), dtype=torch.uint8,
                     device="cuda")
    ws[4096:] = 0xFF
    for i, (lens, Nq, Hq, Hkv) in enumerate([([300, 2, 77], 4, 8, 2), ([511], 1, 2, 2),
                                             ([64, 0, 500], 2, 4, 2)] * 2):
        cache, table, sl, ks, vs, _ = build(T, lens, Hkv, 64, 16, 130 + i, width=32)
        q = to_dev(S.normal((len(lens), Nq, Hq, 64), 131, 0))
        w = torch.rand((len(lens), Hkv, 512), device="cuda")
        o, w1 = T.mha_fwd_kv8(q, cache, table, sl, Hkv, 16, weights=w, workspace=ws)
        o2, w2 = T.mha_fwd_kv8(q, cache, table, sl, Hkv, 16, weights=w, weights_out=w)
        assert w2 is w and torch.equal(w1, w) and torch.equal(o, o2)
    assert T.device_error() == 0


def test_weights_of_a_table_far_wider_than_its_sequences(T):
    """Weights apart and in place; each CTA of the sum takes several stretches of keys."""
    import torch
    lens, H, d, page = [37, 20000], 40, 32, 64
    cache, table, sl, ks, vs, _ = build(T, lens, H, d, page, 137, width=700)
    q = S.normal((2, 1, H, d), 138, 0)
    w = torch.rand((2, H, 700 * page), device="cuda")
    w0 = to_f64(w)
    o, w1 = T.mha_fwd_kv8(to_dev(q), cache, table, sl, H, page, weights=w)
    o, w2 = T.mha_fwd_kv8(to_dev(q), cache, table, sl, H, page, weights=w, weights_out=w)
    assert w2 is w and torch.equal(w1, w)
    g = to_f64(w1)
    for b, n in enumerate(lens):
        check_rows(o[b], None, q[b], ks[b].values, vs[b].values, 1, 0, None, g[b, :, :n],
                   w0[b, :, :n])
        np.testing.assert_array_equal(g[b, :, n:], w0[b, :, n:])


def test_a_cache_off_128_bytes_and_a_workspace_of_both_caches(T):
    """A cache that starts on 16 bytes only gives the same bits; one workspace serves the
    attentions over both caches, one after the other."""
    import torch
    lens, H, d, page = [100, 33], 2, 96, 48
    cache, table, sl, ks, vs, free = build(T, lens, H, d, page, 145, spare=6)
    moved = torch.empty(cache.numel() + 16, dtype=torch.uint8, device="cuda")[16:].view(cache.shape)
    moved.copy_(cache)
    q = to_dev(S.normal((2, 2, 4, d), 146, 0))
    w = torch.rand((2, H, table.shape[1] * page), device="cuda")
    a = T.mha_fwd_kv8(q, cache, table, sl, H, page, weights=w, return_lse=True)
    b = T.mha_fwd_kv8(q, moved, table, sl, H, page, weights=w, return_lse=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    dest = ints([free[:3].tolist(), free[3:6].tolist()])
    for c in (cache, moved):
        T.kv8_evict(c, table, sl, w, dest, H, d, page, 40, 5)
        T.kv8_append(q[:, :, :H].contiguous(), q[:, :, 2:], dest, ints([42, 35]), c, page)
    assert torch.equal(*(T.kv8_load(c, ints([[i * page + j for j in range(42)] for i in
                                             (dest[0, 0].item(), dest[1, 0].item())]), H, d,
                                    page)[0] for c in (cache, moved)))
    k4 = torch.zeros((8, T.kv4_page_bytes(page, H, d)), dtype=torch.uint8, device="cuda")
    slots = torch.arange(100, dtype=torch.int32, device="cuda")[None]
    kv = [to_dev(rows((1, 100, H, d), 147 + i)) for i in range(2)]
    T.kv4_store(*kv, slots, k4, page)
    t4, l4 = ints([[0, 1, 2]]), ints([100])
    ref = T.mha_fwd_kv4(q[:1], k4, t4, l4, H, page)
    ws = torch.zeros(max(T.mha_fwd_kv8_workspace_bytes(2, 2, 4, H, d, w.shape[2]),
                         T.mha_fwd_kv4_workspace_bytes(1, 2, 4, H, d)), dtype=torch.uint8,
                     device="cuda")
    cache, table, sl, *_ = build(T, lens, H, d, page, 145)
    for _ in range(3):
        c = T.mha_fwd_kv8(q, cache, table, sl, H, page, weights=w, return_lse=True, workspace=ws)
        assert all(torch.equal(x, y) for x, y in zip(a, c))
        assert torch.equal(T.mha_fwd_kv4(q[:1], k4, t4, l4, H, page, workspace=ws), ref)
    assert T.device_error() == 0


def test_two_calls_at_once(T):
    """Two streams, a workspace each, in flight together; then each on its own."""
    import torch
    sets = []
    for i, (lens, Nq, Hq, Hkv) in enumerate([([3000, 40], 1, 8, 8), ([900, 1200, 5], 4, 8, 2)]):
        cache, table, sl, _, _, _ = build(T, lens, Hkv, 128, 64, 140 + i)
        q = to_dev(S.normal((len(lens), Nq, Hq, 128), 141, i))
        keys = table.shape[1] * 64
        ws = torch.zeros(T.mha_fwd_kv8_workspace_bytes(len(lens), Nq, Hq, Hkv, 128, keys),
                         dtype=torch.uint8, device="cuda")
        w = torch.zeros((len(lens), Hkv, keys), device="cuda")
        sets.append(((q, cache, table, sl, Hkv, 64), dict(workspace=ws, weights=w)))
    alone = [T.mha_fwd_kv8(*a, **kw) for a, kw in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(20):
        for i, (a, kw) in enumerate(sets):
            got[i].append(T.mha_fwd_kv8(*a, stream=streams[i], **kw))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(r, alone[i]))
    assert T.device_error() == 0


# ------------------------------------------------------------------ eviction
@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (16, 5), (33, 0), (33, 33), (100, 7),
                                         (1000, 100)])
def test_evictions(T, d, keep, recent):
    """Kept positions, lengths, weights and rows, of sequences shorter than, equal to and
    longer than what is kept; ties, NaN, infinities and both zeros among the weights."""
    import torch
    H, page = 3, 32
    lens = [0, 1, 33, 100, 101, 700, 2100]
    width = -(-keep // page) + 1
    cache, table, sl, ks, vs, free = build(T, lens, H, d, page, 150, spare=len(lens) * width)
    dest = free[:len(lens) * width].reshape(len(lens), width)
    cap = table.shape[1] * page
    w = S.normal((len(lens), H, cap), 151, 0, dtype="f32")
    w[:, 1] = np.round(w[:, 1])                          # many ties
    w[:, 2, ::5] = np.nan
    w[:, 2, 1::7] = -np.inf
    w[:, 2, 2::11] = -0.0
    w[:, 2, 3::13] = 0.0
    w[:, 2, 4::97] = np.inf
    before = cache.clone()
    nl, kept, wo = T.kv8_evict(cache, table, sl, to_dev(w), to_dev(dest), H, d, page, keep, recent)
    assert T.device_error() == 0
    assert nl.tolist() == [min(n, keep) for n in lens]
    for b, n in enumerate(lens):
        ids = O.kv8_kept(w[b, :, :n], keep, recent)
        m = ids.shape[1]
        got = kept[b].cpu().numpy()
        np.testing.assert_array_equal(got[:, :m], ids, err_msg=str(b))
        assert (got[:, m:] == -1).all()
        gw = wo[b].cpu().numpy()
        np.testing.assert_array_equal(gw[:, :m], np.take_along_axis(w[b], ids, 1))
        assert not gw[:, m:].any()
        assert_held(T, cache, dest, b, page, ks[b].evicted(ids), vs[b].evicted(ids), str(b))
        for i in range(-(-n // page)):                   # sources keep every byte
            pg = int(table[b, i])
            assert torch.equal(cache[pg], before[pg])


@pytest.mark.parametrize("H,n,keep,recent", [
    (2, 20000, 5000, 100), (2, 50000, 700, 0), (2, 50000, 45000, 20000), (2, 16389, 16388, 3),
    (40, 9000, 4000, 4000), (160, 45000, 3000, 10), (160, 5000, 4999, 0)])
@pytest.mark.parametrize("kind", ["close", "equal", "zeros", "spread", "misaligned"])
def test_which_keys_stay_of_many(T, H, n, keep, recent, kind):
    """The selection alone, by one and by several CTAs a head and past what they hold in
    shared memory: weights that agree in their first 11 or 22 bits, all equal, mostly
    zeros, of all sizes and signs."""
    import torch
    d, page = 32, 128
    width, dw = -(-n // page), -(-keep // page)
    cache = torch.zeros((width + dw, T.kv8_page_bytes(page, H, d)), dtype=torch.uint8, device="cuda")
    table = torch.arange(width, dtype=torch.int32, device="cuda")[None].contiguous()
    dest = (torch.arange(dw, dtype=torch.int32, device="cuda") + width)[None].contiguous()
    g = S.rng(155)
    cap = width * page
    if kind == "close":
        w = np.stack([1 + g.integers(0, 1 << 12, cap) * 2.0 ** -23,
                      1 + g.random(cap) / 5] * (H // 2)).astype(np.float32)
    elif kind == "equal":
        w = np.full((H, cap), 0.25, np.float32)
    elif kind == "zeros":
        w = (g.random((H, cap)) * (g.random((H, cap)) < 0.01)).astype(np.float32)
    else:
        w = (g.standard_normal((H, cap)) * 10.0 ** g.integers(-30, 30, (H, cap))).astype(np.float32)
    wd = torch.empty(H * cap + 4, device="cuda")
    wd = wd[1:-3] if kind == "misaligned" else wd[:-4]
    wd = wd.view(1, H, cap).copy_(to_dev(w)[None])
    nl, kept, wo = T.kv8_evict(cache, table, ints([n]), wd, dest, H, d, page, keep, recent)
    for h in sorted({0, 1, H // 2, H - 1}):
        x = w[h, :n - recent].astype(np.float64)
        ids = np.sort(np.argsort(-x, kind="stable")[:keep - recent])
        ids = np.concatenate([ids, np.arange(n - recent, n)])
        np.testing.assert_array_equal(kept[0, h].cpu().numpy(), ids)
        np.testing.assert_array_equal(wo[0, h, :keep].cpu().numpy(), w[h, ids])
        assert not wo[0, h, keep:].any()
    assert nl.tolist() == [keep] and T.device_error() == 0


def test_rows_behind_an_evicted_sequence_and_its_growth(T):
    """The last block's other rows are zeros; the shortened sequence grows on."""
    import torch
    H, d, page, n, keep = 2, 64, 16, 60, 21
    cache, table, sl, ks, vs, free = build(T, [n], H, d, page, 160, spare=4)
    dest = free[:2][None]
    w = to_dev(S.rng(161).random((1, H, 64), np.float32))
    nl, kept, wo = T.kv8_evict(cache, table, sl, w, to_dev(dest), H, d, page, keep, 4)
    got = T.kv8_load(cache, to_dev(slots_of(dest, 0, 32, page)), H, d, page, dtype=torch.float32)
    assert not got[0][0, keep:].any() and not got[1][0, keep:].any()
    ids = kept[0].cpu().numpy()
    rk, rv = ks[0].evicted(ids), vs[0].evicted(ids)
    k, v = rows((1, 7, H, d), 162), rows((1, 7, H, d), 163)
    T.kv8_append(to_dev(k), to_dev(v), to_dev(dest), nl + 7, cache, page)
    assert_held(T, cache, dest, 0, page, rk.append(k[0]), rv.append(v[0]))
    assert T.device_error() == 0


def test_evictions_of_rows_of_nan_and_shared_pages(T):
    """A kept row of NaN stays one and leaves its neighbours alone; two sequences that
    share their pages are evicted each to its own; bad pages are flagged."""
    import torch
    H, d, page = 1, 32, 16
    x = rows((1, 40, H, d), 170)
    f = S.bf16_bits_to_f32(x)
    f[0, 3, 0, 1], f[0, 30, 0, 2] = np.nan, np.inf
    x = S.f32_to_bf16_bits(f)
    cache = cache_of(T, 8, page, H, d)
    table = ints([[4, 2, 0], [4, 2, 0]])
    T.kv8_append(to_dev(x), to_dev(x), table[:1].contiguous(), ints([40]), cache, page)
    r = O.Kv8Rows(H, d).append(x[0])
    w = S.rng(171).random((2, H, 48)).astype(np.float32)
    w[:, :, 3] = w[:, :, 30] = 5.0
    dest = np.array([[7], [1]], np.int32)
    nl, kept, _ = T.kv8_evict(cache, table, ints([40, 33]), to_dev(w), to_dev(dest), H, d, page, 9, 2)
    for b, n in enumerate((40, 33)):
        ids = O.kv8_kept(w[b, :, :n], 9, 2)
        np.testing.assert_array_equal(kept[b].cpu().numpy(), ids)
        assert 3 in ids and 30 in ids
        assert_held(T, cache, dest, b, page, r.evicted(ids), r.evicted(ids))
    assert T.device_error() == 0
    before = cache.clone()
    T.kv8_evict(cache, table, ints([40, 33]), to_dev(w), ints([[9], [-1]]), H, d, page, 9, 2)
    assert T.device_error() == 8 and torch.equal(cache, before)
    T.kv8_evict(cache, ints([[4, -2, 0], [99, 99, 99]]), ints([40, 90]), to_dev(w), to_dev(dest), H,
                d, page, 9, 2)
    assert T.device_error() == 8


# ------------------------------------------------------------------ a run of them together
def decode_step(T, s, q, k, v, rope, pos, page, Hkv):
    """One token of each sequence: rotate, append, attend, gather weights."""
    T.rope_fwd(q, k, pos, rope, out=(q, k))
    T.kv8_append(k, v, s["table"], s["lens"], s["cache"], page)
    o, w = T.mha_fwd_kv8(q, s["cache"], s["table"], s["lens"], Hkv, page, out=s["o"],
                         weights=s["w"], weights_out=s["w"], workspace=s["ws"])
    return o


@pytest.mark.parametrize("captured", [False, True])
def test_a_run_of_decode_steps_with_evictions(T, captured):
    """Prompts, then steps of rotation, append and attention with weights, an eviction
    each time a sequence reaches its limit, against the oracle step by step; the steps
    eager or as one captured graph whose positions and lengths move on."""
    import torch
    B, Hq, Hkv, d, page, keep, recent, limit = 3, 4, 2, 64, 16, 40, 12, 48
    width = limit // page
    prompt = [30, 47, 5]
    rope = T.Rope(48, interleaved=True, scaling="linear", factor=2.0)
    w_, _ = O.rope_frequencies(48, 10000.0, "linear", 2.0)
    tab = [np.arange(B * width, dtype=np.int32).reshape(B, width) + i * B * width for i in range(2)]
    cache = cache_of(T, 2 * B * width, page, Hkv, d)
    s = dict(cache=cache, table=to_dev(tab[0]), lens=ints(prompt),
             w=torch.zeros((B, Hkv, limit), device="cuda"),
             o=torch.zeros((B, 1, Hq, d), dtype=torch.bfloat16, device="cuda"),
             ws=torch.zeros(T.mha_fwd_kv8_workspace_bytes(B, 1, Hq, Hkv, d, limit),
                            dtype=torch.uint8, device="cuda"))
    N = max(prompt)
    pos = np.maximum(np.arange(N)[None] - N + np.array(prompt)[:, None], 0).astype(np.int32)
    k, v = rows((B, N, Hkv, d), 180), rows((B, N, Hkv, d), 181)
    kd = to_dev(k)
    T.rope_fwd(kd, None, to_dev(pos), rope, out=(kd, None))
    T.kv8_append(kd, to_dev(v), s["table"], s["lens"], cache, page)
    kr = kd.cpu().view(torch.int16).numpy().view(np.uint16)
    refs = [[O.Kv8Rows(Hkv, d).append(kr[b, N - n:]), O.Kv8Rows(Hkv, d).append(v[b, N - n:])]
            for b, n in enumerate(prompt)]
    lens, at, cur = list(prompt), list(prompt), 0
    q1, k1, v1 = (torch.zeros((B, 1, h, d), dtype=torch.bfloat16, device="cuda")
                  for h in (Hq, Hkv, Hkv))
    p1 = ints([[n] for n in at])
    graph = None
    for step in range(25):
        x = [rows((B, 1, h, d), 200 + step, stream=i) for i, h in enumerate((Hq, Hkv, Hkv))]
        w0 = to_f64(s["w"])
        for t, a in zip((q1, k1, v1), x):
            t.copy_(to_dev(a))
        lens = [n + 1 for n in lens]
        s["lens"].copy_(ints(lens))
        p1.copy_(ints([[n] for n in at]))
        if not captured:
            decode_step(T, s, q1, k1, v1, rope, p1, page, Hkv)
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    decode_step(T, s, q1, k1, v1, rope, p1, page, Hkv)
            graph.replay()
        at = [a + 1 for a in at]
        qr, kr = (t.cpu().view(torch.int16).numpy().view(np.uint16) for t in (q1, k1))
        for t, a in zip((qr, kr), x):                    # the rotation itself
            want = O.rotate(a, np.array(at)[:, None] - 1, w_, 1.0, True)
            f = S.bf16_bits_to_f32(t)
            assert (np.abs(f - want) <= 2.0 ** -8 * np.abs(want) +
                    2.0 ** -20 * np.abs(S.bf16_bits_to_f32(a)).max()).all()
        for b in range(B):
            refs[b][0].append(kr[b])
            refs[b][1].append(x[2][b])
            check_rows(s["o"][b], None, qr[b], refs[b][0].values, refs[b][1].values, 1, 0, None,
                       to_f64(s["w"])[b, :, :lens[b]], w0[b, :, :lens[b]])
        if max(lens) == limit:
            cur = 1 - cur
            wd = to_f64(s["w"])
            nl, kept, wo = T.kv8_evict(cache, s["table"], s["lens"], s["w"], to_dev(tab[cur]), Hkv,
                                       d, page, keep, recent)
            s["w"].copy_(wo)
            s["table"].copy_(to_dev(tab[cur]))
            for b in range(B):
                ids = O.kv8_kept(wd[b, :, :lens[b]], keep, recent)
                np.testing.assert_array_equal(kept[b, :, :ids.shape[1]].cpu().numpy(), ids)
                refs[b] = [r.evicted(ids) for r in refs[b]]
            lens = [min(n, keep) for n in lens]
            assert nl.tolist() == lens
    for b in range(B):
        assert_held(T, cache, tab[cur], b, page, *refs[b])
    assert T.device_error() == 0


def test_a_captured_eviction_replays_with_other_lengths_and_weights(T):
    """Append, attention with weights, eviction and reading back in one graph."""
    import torch
    H, d, page, keep, n0 = 2, 64, 16, 30, 100
    table, n_pages, free = tables([n0], page, 195, spare=3)
    dest = free[:2][None]
    cache = cache_of(T, n_pages, page, H, d)
    rk, rv = O.Kv8Rows(H, d), O.Kv8Rows(H, d)
    k, v = rows((1, n0, H, d), 196), rows((1, n0, H, d), 197)
    lens = ints([70])
    kd, vd = to_dev(k[:, :70]), to_dev(v[:, :70])
    T.kv8_append(kd, vd, to_dev(table), lens, cache, page)
    rk.append(k[0, :70]), rv.append(v[0, :70])
    td, dd = to_dev(table), to_dev(dest)
    q = to_dev(S.normal((1, 1, H, d), 198, 0))
    k1, v1 = to_dev(k[:, :1]), to_dev(v[:, :1])
    w = torch.zeros((1, H, table.shape[1] * page), device="cuda")
    ws = torch.zeros(T.mha_fwd_kv8_workspace_bytes(1, 1, H, H, d, w.shape[2]), dtype=torch.uint8,
                     device="cuda")
    nl, kept = torch.zeros_like(lens), torch.zeros((1, H, keep), dtype=torch.int32, device="cuda")
    wo, o = torch.zeros((1, H, 32), device="cuda"), torch.zeros_like(q)
    back = torch.zeros((1, keep, H, d), device="cuda"), torch.zeros((1, keep, H, d), device="cuda")
    slots = to_dev(slots_of(dest, 0, keep, page))

    def step():
        T.kv8_append(k1, v1, td, lens, cache, page)
        T.mha_fwd_kv8(q, cache, td, lens, H, page, out=o, weights=w, weights_out=w, workspace=ws)
        T.kv8_evict(cache, td, lens, w, dd, H, d, page, keep, 5, nl, kept, wo)
        T.kv8_load(cache, slots, H, d, page, out=back)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(70, n0):
        k1.copy_(to_dev(k[:, n:n + 1]))
        v1.copy_(to_dev(v[:, n:n + 1]))
        lens.fill_(n + 1)
        graph.replay()
        rk.append(k[0, n:n + 1]), rv.append(v[0, n:n + 1])
        torch.cuda.synchronize()
        ids = O.kv8_kept(to_f64(w)[0, :, :n + 1], keep, 5)
        np.testing.assert_array_equal(kept[0].cpu().numpy(), ids)
        np.testing.assert_array_equal(to_f64(wo)[0, :, :keep],
                                      np.take_along_axis(to_f64(w)[0], ids, 1))
        np.testing.assert_array_equal(to_f64(back[0])[0], rk.evicted(ids).values)
        np.testing.assert_array_equal(to_f64(back[1])[0], rv.evicted(ids).values)
        assert nl.tolist() == [keep]
    assert T.device_error() == 0


def test_many_sequences_and_misaligned_weights(T):
    """More sequences than a CTA has threads, weights off 16 bytes."""
    import torch
    lens = [int(x) for x in S.rng(6).integers(0, 50, 300)]
    H, d, page = 2, 32, 16
    cache, table, sl, ks, vs, _ = build(T, lens, H, d, page, 210)
    q = S.normal((300, 1, 4, d), 211, 0)
    cap = table.shape[1] * page
    w = torch.rand(300 * H * cap + 3, device="cuda")
    wi = w[1:-2].view(300, H, cap)
    wo = torch.zeros(300 * H * cap + 3, device="cuda")[3:].view(300, H, cap)
    o, wo = T.mha_fwd_kv8(to_dev(q), cache, table, sl, H, page, weights=wi, weights_out=wo)
    g, g0 = to_f64(wo), to_f64(wi)
    for b, n in enumerate(lens):
        check_rows(o[b], None, q[b], ks[b].values, vs[b].values, 1, 0, None, g[b, :, :n],
                   g0[b, :, :n])
        np.testing.assert_array_equal(g[b, :, n:], g0[b, :, n:])
    # one call adds one row to each of them
    k, v = rows((300, 1, H, d), 212), rows((300, 1, H, d), 213)
    t2, n_pages, _ = tables([n + 1 for n in lens], page, 214)
    c2 = cache_of(T, n_pages, page, H, d)
    for b, n in enumerate(lens):
        if n:
            x = [to_dev(rows((1, n, H, d), 210 + b, stream=s)) for s in (0, 3)]
            T.kv8_append(*x, to_dev(t2[b:b + 1]), ints([n]), c2, page)
    T.kv8_append(to_dev(k), to_dev(v), to_dev(t2), sl + 1, c2, page)
    for b in range(0, 300, 7):
        assert_held(T, c2, t2, b, page, ks[b].append(k[b]), vs[b].append(v[b]), str(b))
    assert T.device_error() == 0


def test_streams(T):
    """Calls on a stream other than the current one, results made in the call."""
    import torch
    H, d, page, n = 4, 64, 16, 90
    s = torch.cuda.Stream()
    table, n_pages, free = tables([n], page, 190, spare=8)
    cache = cache_of(T, n_pages, page, H, d)
    k, v = rows((1, n, H, d), 191), rows((1, n, H, d), 192)
    q = to_dev(S.normal((1, 1, H, d), 193, 0))
    kd, vd, td, ld = to_dev(k), to_dev(v), to_dev(table), ints([n])
    dest = to_dev(free[:2][None])
    w = torch.rand((1, H, table.shape[1] * page), device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    T.kv8_append(kd, vd, td, ld, cache, page, stream=s)
    o, w1 = T.mha_fwd_kv8(q, cache, td, ld, H, page, weights=w, stream=s)
    nl, kept, w2 = T.kv8_evict(cache, td, ld, w1, dest, H, d, page, 20, 4, stream=s)
    got = T.kv8_load(cache, to_dev(slots_of(table, 0, n, page)), H, d, page, stream=s)
    s.synchronize()
    rk, rv = O.Kv8Rows(H, d).append(k[0]), O.Kv8Rows(H, d).append(v[0])
    check_rows(o[0], None, q[0].cpu().view(torch.int16).numpy().view(np.uint16), rk.values,
               rv.values, 1, 0)
    np.testing.assert_array_equal(to_f64(got[0])[0], rk.values)
    np.testing.assert_array_equal(kept[0].cpu().numpy(), O.kv8_kept(to_f64(w1)[0, :, :n], 20, 4))
    assert nl.tolist() == [20]


def test_binding_refusals(T):
    import torch
    H, d, page = 2, 64, 16
    cache = cache_of(T, 4, page, H, d, 0)
    k = torch.zeros((1, 3, H, d), dtype=torch.bfloat16, device="cuda")
    table, lens = ints([[0, 1]]), ints([3])
    w = torch.zeros((1, H, 32), device="cuda")
    for a in ((k[0], k, table, lens, cache, page), (k, k[:, :2], table, lens, cache, page),
              (k, k.float(), table, lens, cache, page), (k, k, table[0], lens, cache, page),
              (k, k, table.long(), lens, cache, page), (k, k, table, ints([1, 2]), cache, page),
              (k, k, table, lens, cache[:, :-16], page), (k, k, table, lens, cache, 32),
              (k, k, table, lens.cpu(), cache, page), (k.cpu(), k, table, lens, cache, page),
              (k.transpose(2, 3), k.transpose(2, 3), table, lens, cache, page)):
        with pytest.raises((ValueError, T.IHAError)):
            T.kv8_append(*a)
    with pytest.raises(ValueError):
        T.kv8_append(k, k, table, lens, cache, page, counts=ints([[1]]))
    q = torch.zeros((1, 1, 4, d), dtype=torch.bfloat16, device="cuda")
    for kw in (dict(weights=w[:, :1]), dict(weights=w.double()), dict(weights_out=w),
               dict(weights=w, weights_out=w[..., :16]), dict(workspace=w),
               dict(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")),
               dict(out=q[..., :32]), dict(lse=w), dict(mask=7), dict(mask=2, window=0)):
        with pytest.raises((ValueError, T.IHAError)):
            T.mha_fwd_kv8(q, cache, table, lens, H, page, **kw)
    with pytest.raises((ValueError, T.IHAError)):
        T.mha_fwd_kv8(q.float(), cache, table, lens, H, page)
    dest = ints([[2]])
    for a in ((table, lens, w[:, :1], dest, H, d, page, 5, 1), (table, lens, w, dest, H, d, page, 0, 0),
              (table, lens, w, dest, H, d, page, 5, 6), (table, lens, w, dest, H, d, page, 17, 1),
              (table, ints([[3]]), w, dest, H, d, page, 5, 1), (table, lens, w, dest[0], H, d, page, 5, 1),
              (table, lens, w, dest, H, 32, page, 5, 1)):
        with pytest.raises((ValueError, T.IHAError)):
            T.kv8_evict(cache, *a)
    with pytest.raises(ValueError):
        T.kv8_load(cache, ints([0]), H, d, page)
    with pytest.raises(ValueError):
        T.kv8_load(cache, table, H, d, page, out=(k,))
    assert T.device_error() == 0
