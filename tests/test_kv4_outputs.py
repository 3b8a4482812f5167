"""Outputs of kv4_load and mha_fwd_kv4 that overlap are refused, and slices of
one tensor that do not are taken.

The host's decision is compared with brute force over every pair of rows.  A
layout that is taken goes on to the launch, so that comparison runs only where
there is no GPU to launch on (status 4); the addresses are made up."""
import ctypes as C
import itertools
import random

import pytest

import synthetic as S
import transformer_attention_iha_gb300 as T
from helpers import to_dev

A = 0x100000000


def gpu():
    import torch
    return torch.cuda.is_available()


@pytest.fixture(scope="module")
def L():
    T.build()
    return T.lib()


def starts(n, s):
    return [sum(i * x for i, x in zip(idx, s)) for idx in itertools.product(*map(range, n))]


def load(L, n, sk, sv, delta, d):
    """kv4_load of [n0, n1, n2] tokens and n3 heads, v starting `delta` elements after k."""
    return L.kv4_load(C.c_void_p(A), C.c_void_p(2 * A), C.c_void_p(4 * A),
                      C.c_void_p(4 * A + 2 * delta), n[0], n[1], n[2], 64, 64, n[3], d,
                      T.Strides(*sk), T.Strides(*sv), T.BF16, None)


def attend(L, n, so, d):
    st = T.Strides(n[1] * n[2] * d, 0, n[2] * d, d)
    return L.mha_fwd_kv4(C.c_void_p(A), C.c_void_p(2 * A), C.c_void_p(3 * A), C.c_void_p(4 * A),
                         C.c_void_p(5 * A), None, C.c_void_p(6 * A), 1 << 40, n[0], n[1], n[2],
                         n[2], d, 64, 64, 1, st, T.Strides(so[0], 0, so[1], so[2]), 0.0, 1, 0,
                         T.BF16, None)


def test_overlapping_outputs_are_refused(L):
    d = 32
    n, dense = (2, 1, 3, 4), (3 * 4 * d, 0, 4 * d, d)
    for delta in (0, 8, d, 5 * d, 11 * d + 8, 23 * d):
        assert load(L, n, dense, dense, delta, d) == 1, delta
        assert load(L, n, dense, dense, -delta, d) == 1, -delta
    assert "outputs overlap" in L.iha_last_error().decode()
    pairs = (6 * 4 * d, 0, 2 * 4 * d, d)                    # rows of another in between
    assert load(L, n, pairs, pairs, 4 * d - 8, d) == 1
    assert load(L, n, pairs, pairs, 3 * d, d) == 1
    for s in ((96 * d, 0, 2 * d, d), (96 * d, 0, 4 * d, 24), (2 * 4 * d, 0, 4 * d, d)):
        assert load(L, n, s, dense, 10 ** 6 * 8, d) == 1, s
        assert load(L, n, dense, s, 10 ** 6 * 8, d) == 1, s
        assert "rows of an output" in L.iha_last_error().decode()
    for so in ((96 * d, 2 * d, d), (96 * d, 4 * d, 24), (8 * d, 4 * d, d), (96 * d, d, d)):
        assert attend(L, (2, 3, 4), so, d) == 1, so
        assert "rows of the output" in L.iha_last_error().decode()


@pytest.mark.skipif(gpu(), reason="layouts that are taken would be launched")
def test_decision_against_brute_force(L):
    rng = random.Random(5)
    seen = [0, 0, 0]
    for _ in range(4000):
        d = rng.choice([32, 64])
        n = tuple(rng.choice([1, 1, 2, 3, 5]) for _ in range(4))
        some = [8, 24, d, d + 8, 2 * d, 3 * d, 4 * d, 5 * d, 6 * d, 7 * d + 16, 12 * d, 30 * d]
        sk = tuple(rng.choice(some) for _ in n)
        sv = sk if rng.random() < 0.6 else tuple(rng.choice(some) for _ in n)
        delta = 8 * rng.randrange(-200, 200)
        k, v = starts(n, sk), starts(n, sv)
        inner = [min((abs(a - b) for a, b in itertools.combinations(r, 2)), default=d) < d
                 for r in (k, v)]
        cross = min(abs(a - b - delta) for a in k for b in v) < d
        st = load(L, n, sk, sv, delta, d)
        assert st == (1 if any(inner) or cross else 4), (n, sk, sv, delta, d, st)
        seen[0 if any(inner) else 1 if cross else 2] += 1
        o = starts(n[1:], sk[1:])
        bad = min((abs(a - b) for a, b in itertools.combinations(o, 2)), default=d) < d
        assert attend(L, n[1:], sk[1:], d) == (1 if bad else 4), (n, sk, d)
    assert min(seen) > 100


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["token", "head", "feature", "not_nested"])
def test_slices_of_one_tensor(form):
    import torch
    B, N, H, d, page = 2, 5, 3, 64, 16
    cache = torch.zeros((1, T.kv4_page_bytes(page, H, d)), dtype=torch.uint8, device="cuda")
    kd, vd = (to_dev(S.normal((B, N, H, d), 500, t)) for t in range(2))
    slots = torch.arange(B * N, dtype=torch.int32, device="cuda").view(B, N)
    T.kv4_store(kd, vd, slots, cache, page)
    rk, rv = T.kv4_load(cache, slots, H, d, page)
    z = lambda *s: torch.full(s, 9.0, dtype=torch.bfloat16, device="cuda")
    if form == "token":
        t = z(B, N, 2, H, d)
        k, v = t[:, :, 0], t[:, :, 1]
    elif form == "head":
        t = z(B, N, H, 2, d)
        k, v = t[..., 0, :], t[..., 1, :]
    elif form == "feature":
        t = z(B, N, H, 2 * d + 8)
        k, v = t[..., :d], t[..., d:2 * d]
    else:  # two batch rows 3 d apart, heads 2 d apart: 0, 2, 4 and 3, 5, 7
        t = z(B * N * 16 * d)
        k, v = (t.as_strided((B, N, H, d), (3 * d, 16 * d, 2 * d, 1), at * d) for at in (0, 8))
    T.kv4_load(cache, slots, H, d, page, out=(k, v))
    assert torch.equal(k, rk) and torch.equal(v, rv)
    with pytest.raises(T.IHAError):
        T.kv4_load(cache, slots, H, d, page, out=(k, k))
    assert T.device_error() == 0
