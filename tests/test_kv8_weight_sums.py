"""GPU test that the keys' weights of mha_fwd_kv8 are the softmax's, however large the
scores: those that a call adds sum up to its rows.

Tolerance.  A weight is 2^(x - r) / l of a score x that is rounded already, so what x lost
does not count; l is the sum of the same 2^(x - r).  With u = 2^-24: both exponents are off
by u |x - r|, and so their weighted mean by u (8 + log2 n) ln 2 < 14 u each; exp2f and ex2
are within 2^-22, 4 u; a lane adds up to 40 probabilities of these cases, 40 u; joins, the
reciprocal and the two products 20 u: together less than 96 u.  A key's sum over `cols`
rows adds cols u:
  |sum w - rows| <= (96 + cols) 2^-24 rows."""
import numpy as np
import pytest

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


@pytest.mark.parametrize("lens,Nq,Hq,Hkv", [([300, 17], 1, 2, 2), ([5000], 1, 1, 1),
                                            ([300, 64, 4000], 4, 8, 2), ([500, 33], 8, 16, 2)])
@pytest.mark.parametrize("size", [1.0, 300.0, 2500.0, 40000.0])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("with_lse", [False, True])
def test_weights_sum_to_the_rows(T, lens, Nq, Hq, Hkv, size, sign, with_lse):
    """Scores about `size` or -size, a few units apart, so that many keys have a part."""
    import torch
    d, page, B = 64, 16, len(lens)
    width = -(-max(lens) // page)
    cache = torch.zeros((B * width, T.kv8_page_bytes(page, Hkv, d)), dtype=torch.uint8,
                        device="cuda")
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k = S.normal((B, max(lens), Hkv, d), 610, 0, dtype="f32")
    k[..., 0] = 256.0                                      # exact in 8 bits beside the others
    k[..., 1:] *= 4.0
    q = S.normal((B, Nq, Hq, d), 610, 1, dtype="f32")
    q[..., 0] = sign * size * 8.0 / 256.0 * (1.0 + 0.01 * np.arange(Hq))
    q[..., 1:] *= 0.1
    T.kv8_append(to_dev(S.f32_to_bf16_bits(k)), to_dev(S.normal(k.shape, 610, 2)), table, sl,
                 cache, page, counts=sl)
    w = torch.zeros((B, Hkv, width * page), device="cuda")
    res = T.mha_fwd_kv8(to_dev(S.f32_to_bf16_bits(q)), cache, table, sl, Hkv, page, weights=w,
                        return_lse=with_lse)
    g, rows = to_f64(res[-1]), Nq * Hq // Hkv
    for b, n in enumerate(lens):
        assert not g[b, :, n:].any()
        # (more than one key has a part: the sum is not one probability of 1)
        assert (g[b, :, :n].max(1) < 0.99 * rows).all()
        err = np.abs(g[b].sum(1) - rows)
        assert (err <= (96 + rows) * 2.0 ** -24 * rows).all(), (err / rows).max()
    assert T.device_error() == 0
