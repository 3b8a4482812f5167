"""What the keys' weights do not depend on: the oracle gives a row's later keys nothing (CPU),
and a V row that is not finite leaves every weight as it is (GPU; tolerances as in
test_parity_kv8.py)."""
import math

import numpy as np
import pytest

import oracle as O
import synthetic as S


@pytest.mark.parametrize("mask,window", [(O.MASK_CAUSAL, 0), (O.MASK_CAUSAL_WINDOW, 4),
                                         (O.MASK_NONE, 0)])
def test_oracle_gives_hidden_keys_nothing(mask, window):
    n, Nq, Hq, Hkv, d = 9, 3, 4, 2, 32
    q = S.normal((Nq, Hq, d), 5, 0)
    k = S.normal((n, Hkv, d), 5, 1, dtype="f32").astype(np.float64)
    f = S.bf16_bits_to_f32(q).astype(np.float64)
    want = np.zeros((Hkv, n))
    for t in range(Nq):
        at = n - Nq + t                                  # the token's own position
        row = O.kv8_weights(q[t:t + 1], k[:at + 1], mask, window)
        first = max(0, at - window + 1) if window else 0
        last = n - 1 if mask == O.MASK_NONE else at
        if mask != O.MASK_NONE:                          # on its own the token is the last key
            assert (row[:, :first] == 0).all() and (row[:, first:] > 0).all()
        for h in range(Hq):
            x = np.array([f[t, h] @ k[j, h // 2] / math.sqrt(d) for j in range(first, last + 1)])
            p = np.exp(x) / np.exp(x).sum()
            want[h // 2, first:last + 1] += p
    got = O.kv8_weights(q, k, mask, window)
    np.testing.assert_allclose(got, want, rtol=1e-12, atol=0)
    if mask != O.MASK_NONE:                              # the last key is seen by the last row only
        one = O.kv8_weights(q[-1:], k, mask, window)
        np.testing.assert_allclose(got[:, -1], one[:, -1], rtol=1e-12)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq", [1, 4])
def test_weights_do_not_see_v(Hq):
    import torch
    import transformer_attention_iha_gb300 as T
    from helpers import to_dev, to_f64
    from test_parity_kv8 import check_rows
    n, d, page, Nq = 45, 64, 16, 6
    k, v = S.normal((1, n, 1, d), 195, 0), S.normal((1, n, 1, d), 195, 1)
    bad = S.bf16_bits_to_f32(v).copy()
    bad[0, 41, 0, 5], bad[0, 33, 0, 5] = np.nan, np.inf
    q = S.normal((1, Nq, Hq, d), 197, 0)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    sl = torch.tensor([n], dtype=torch.int32, device="cuda")
    got = []
    for x in (v, S.f32_to_bf16_bits(bad)):
        cache = torch.full((3, T.kv8_page_bytes(page, 1, d)), 0xFF, dtype=torch.uint8,
                           device="cuda")
        T.kv8_append(to_dev(k), to_dev(x), table, sl, cache, page)
        w = torch.zeros((1, 1, 3 * page), device="cuda")
        got.append(T.mha_fwd_kv8(to_dev(q), cache, table, sl, 1, page, mask=T.MASK_CAUSAL_WINDOW,
                                 window=10, return_lse=True, weights=w))
    (o, lse, w), (o2, lse2, w2) = got
    assert torch.isnan(o2[0, 2:]).all() and not torch.isnan(w2).any()
    assert torch.equal(w, w2) and torch.equal(lse, lse2)
    ref = [O.Kv8Rows(1, d).append(a[0]) for a in (k, v)]
    check_rows(o[0], lse[0], q[0], ref[0].values, ref[1].values, T.MASK_CAUSAL_WINDOW, 10, None,
               to_f64(w2)[0, :, :n], np.zeros((1, n)))
    assert T.device_error() == 0
