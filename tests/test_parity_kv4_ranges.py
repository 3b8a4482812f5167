"""GPU parity of mha_fwd_kv4 where V's scales and the scores move apart along a
sequence: a token that weighed much when it was read and is overtaken later must
not cost the later ones their digits.

Tolerances, per element, p normalised, r the exact result, ra = sum_j p_j |v_j|,
sp = sum_j p_j s_j of the feature's group (v_j = s_j c_j, |c_j| <= 7):
  the output                 2^-8 |r|           (bf16)
  scores                     2 dx ra            (as in test_parity_kv4.py), exp2 and
                                                fp32 products 2^-16 ra
  up to 4 columns            2^-11 ra           (fp16 P)
                           + 2^-11 sp           (256 tokens of codes n <= 15: 16 MMAs of
                                                17 truncations of 2^-23 of 15 sp of them;
                                                16 * 17 * 15 * 2^-23 < 2^-11)
                           + 7 n 2^-30 sp       (P below fp16's normal range: half of
                                                2^-24, where the largest P is at least 2^5)
  more columns               2^-8 ra            (bf16 P)
                           + (n / 16 + 2) 17 2^-23 ra   (truncations, codes exact)
Nothing is granted to a key whose weight is nothing.
"""
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


SEQS = 3001  # so many that a warp takes whole sequences, and cuts fall on every block


def attend(T, kb, vb, qb, page=16):
    """SEQS sequences that share the pages of the rows kb, vb [n, 1, d] (bf16 bits),
    each with the queries qb [1, Hq, d].  Returns the distinct results."""
    import torch
    n, _, d = kb.shape
    pages = -(-n // page)
    cache = torch.full((pages, T.kv4_page_bytes(page, 1, d)), 0xFF, dtype=torch.uint8,
                       device="cuda")
    T.kv4_store(to_dev(kb[None]), to_dev(vb[None]), to_dev(np.arange(n, dtype=np.int32)[None]),
                cache, page)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(SEQS, 1)
    o, lse = T.mha_fwd_kv4(to_dev(qb[None]).expand(SEQS, -1, -1, -1), cache, table,
                           torch.full((SEQS,), n, dtype=torch.int32, device="cuda"), 1, page,
                           return_lse=True)
    assert T.device_error() == 0
    both = torch.cat((o[:, 0].float(), lse), -1)                # [SEQS, Hq, d + 1]
    both = to_f64(torch.unique(both, dim=0))
    return both[..., :d], both[..., d]


def check(T, kb, vb, qb):
    n, _, d = kb.shape
    Hq = qb.shape[1]
    kv, vv = O.kv4_values(kb)[:, 0], O.kv4_values(vb)[:, 0]                     # [n, d]
    g, gl = attend(T, kb, vb, qb)
    q = S.bf16_bits_to_f32(qb).astype(np.float64)[0]                            # [Hq, d]
    sc = 1.0 / math.sqrt(d)
    x = sc * q @ kv.T                                                           # [Hq, n]
    m = x.max(1, keepdims=True)
    p = np.exp(x - m)
    l = p.sum(1, keepdims=True)
    p /= l
    r, ra = p @ vv, p @ np.abs(vv)
    rl = (m + np.log(l))[:, 0]
    sv = np.abs(vv).reshape(n, d // 32, 32).max(-1) / 7 * (1 + 2.0 ** -7)       # >= the scale
    sp = np.repeat(p @ sv, 32, 1)
    qa = np.abs(q).reshape(Hq, d // 32, 32).sum(-1)
    ks = np.abs(kv).reshape(n, d // 32, 32).max(-1).max(0) / 7
    dx = (sc * (143 * 2.0 ** -21 + 7 * 2.0 ** -20) * (qa * ks).sum(-1))[:, None]
    bound = 2.0 ** -8 * np.abs(r) + (2 * dx + 2.0 ** -16) * ra
    if Hq <= 4:
        bound += 2.0 ** -11 * ra + (2.0 ** -11 + 7 * n * 2.0 ** -30) * sp
    else:
        bound += (2.0 ** -8 + (n / 16 + 2) * 17 * 2.0 ** -23) * ra
    err = np.abs(g - r)
    assert np.isfinite(g).all()
    assert (err <= bound).all(), float((err / np.maximum(bound, 1e-300)).max())
    assert (np.abs(gl - rl) <= dx[:, 0] + 2.0 ** -20 * (1 + np.abs(rl))).all()


def rows(n, d, Hq, seed):
    """K nearly orthogonal to the queries, V of order 1, queries of one direction."""
    k = 0.05 * S.normal((n, 1, d), seed, 0, dtype="f32")
    v = S.normal((n, 1, d), seed, 1, dtype="f32")
    q = np.repeat(S.normal((1, 1, d), seed, 2, dtype="f32"), Hq, 1)
    q *= (1 + 0.125 * np.arange(Hq) / Hq).astype(np.float32)[None, :, None]
    return k, v, q


def lift(k, q, at, nats):
    """Keys `at` score about `nats` with query 0."""
    d = q.shape[-1]
    k[at] += np.float32(nats * math.sqrt(d) / (q[0, 0] ** 2).sum()) * q[0, 0]


def bits(*xs):
    return [S.f32_to_bf16_bits(x.astype(np.float32)) for x in xs]


COLUMNS = [1, 2, 4, 8, 16]


@pytest.mark.parametrize("Hq", COLUMNS)
@pytest.mark.parametrize("ratio", [2.0 ** 12, 2.0 ** 16, 2.0 ** 20, 2.0 ** 24, 1e10, 1e20])
@pytest.mark.parametrize("d", [32, 96, 128])
def test_a_heavy_value_overtaken_by_higher_scores(T, d, ratio, Hq):
    """Token 0 has weight when it is read, and a V scale `ratio` times the others';
    tokens from 64 on score so much higher that nothing of it is left."""
    n = 150
    k, v, q = rows(n, d, Hq, 300)
    v[0] *= np.float32(ratio)
    lift(k, q, slice(64, n), 60.0 + math.log(ratio))
    check(T, *bits(k, v, q))


@pytest.mark.parametrize("Hq", COLUMNS)
@pytest.mark.parametrize("step", [1e-6, 1e-3, 1e3])
def test_scores_that_climb_while_scales_change(T, step, Hq):
    """Every 32 tokens the scores rise by 25 and V changes by a factor: the reference
    moves again and again, and what is left of earlier tokens fades or stays."""
    n, d = 224, 128
    k, v, q = rows(n, d, Hq, 301)
    for i in range(n // 32):
        at = slice(32 * i, 32 * i + 32)
        lift(k, q, at, 25.0 * i)
        v[at] *= np.float32(step ** (i - 3))
    check(T, *bits(k, v, q))


@pytest.mark.parametrize("Hq", COLUMNS)
def test_an_overtaken_value_that_still_weighs(T, Hq):
    """The heavy token's weight and its scale cancel: both ends of the sequence count."""
    n, d = 150, 128
    k, v, q = rows(n, d, Hq, 302)
    v[0] *= np.float32(2.0 ** 60)
    lift(k, q, slice(64, n), 60 * math.log(2.0) - math.log(n - 64.0))
    check(T, *bits(k, v, q))


@pytest.mark.parametrize("Hq", COLUMNS)
@pytest.mark.parametrize("top", [1e-25, 1e30])
def test_groups_that_take_turns(T, top, Hq):
    """Each group of 32 features has its heavy token at another place."""
    n, d = 260, 128
    k, v, q = rows(n, d, Hq, 303)
    v *= np.float32(top)
    for j in range(4):
        v[40 * j, 0, 32 * j:32 * j + 32] *= np.float32(1e6)
        lift(k, q, slice(40 * j + 24, n), 12.0)
    lift(k, q, slice(200, n), 30.0)
    check(T, *bits(k, v, q))


@pytest.mark.parametrize("Hq", COLUMNS)
def test_values_of_zero_then_small_ones(T, Hq):
    """All of V is zero (or nearly) where the scores are low, ordinary behind."""
    n, d = 150, 96
    k, v, q = rows(n, d, Hq, 304)
    v[:70] = 0.0
    v[:70, :, :32] = 2.0 ** -99
    lift(k, q, slice(70, n), 40.0)
    check(T, *bits(k, v, q))
