"""GPU parity of a chunk that continues a prompt, by the calls that README shows:
premix at positions, store, the prefix and the chunk read back, attention without
a mask over the prefix and causal over the chunk, joined by their LSEs.  In bf16
against the oracle and mha_fwd_kv4 over the same cache; in float32, which
mha_fwd_kv4 does not take, against the oracle."""
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
    return T


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,n0,C,H,P,d,page", [(1, 1, 1, 4, 2, 64, 16), (2, 45, 19, 4, 2, 64, 16),
                                               (1, 300, 130, 3, 1, 128, 32),
                                               (1, 131, 257, 2, 2, 64, 64)])
def test_chunk_after_a_prefix(T, B, n0, C, H, P, d, page, dtype):
    import torch
    n, HP = n0 + C, H * P
    xs = [to_dev(S.normal((B, n, H, d), 520, t, dtype=dtype)) for t in range(3)]
    ws = [to_dev(S.premix_weight(H, P, 521, t)) for t in range(3)]
    width = -(-n // page)
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").flip(0).view(B, width)
    table = table.contiguous()
    j = torch.arange(n, device="cuda")
    slots = (table[:, j // page] * page + j % page).to(torch.int32)
    before, new = slots[:, :n0].contiguous(), slots[:, n0:].contiguous()
    cache = torch.zeros((B * width, T.kv4_page_bytes(page, HP, d)), dtype=torch.uint8,
                        device="cuda")
    _, k, v = T.premix_fwd_qkv([x[:, :n0].contiguous() for x in xs], ws, P, rope=True)
    T.kv4_store(k, v, before, cache, page)

    pos = torch.arange(n0, n, dtype=torch.int32, device="cuda").expand(B, C).contiguous()
    q, k, v = T.premix_fwd_qkv_at([x[:, n0:].contiguous() for x in xs], ws, P, pos)
    T.kv4_store(k, v, new, cache, page)
    o1, l1 = T.mha_fwd(q, *T.kv4_load(cache, before, HP, d, page, dtype=q.dtype), return_lse=True)
    o2, l2 = T.mha_fwd(q, *T.kv4_load(cache, new, HP, d, page, dtype=q.dtype),
                       mask=T.MASK_CAUSAL, return_lse=True)
    w = torch.sigmoid(l1 - l2).view(B, HP, C).transpose(1, 2).unsqueeze(-1)  # of the prefix
    o = torch.lerp(o2.float(), o1.float(), w).to(q.dtype)
    lse = torch.logaddexp(l1, l2).view(B, HP, C)

    held = [to_f64(t) for t in T.kv4_load(cache, slots, HP, d, page, dtype=torch.float32)]
    qf = to_f64(q).astype(np.float32)
    for b in range(B):
        r, rl, _ = O.kv4_attention(qf[b], held[0][b], held[1][b], O.MASK_CAUSAL)
        if dtype == "bf16":
            assert_bf16_close(to_f64(o)[b], r, "chunk")
            # 2e-3 as for mha_fwd; and K, read back in bf16, is off by 2^-8 of itself
            # (half a step), so a score, and with it the lse, by at most
            # scale 2^-8 sum_f |q_f| |k_jf|, j the worst key
            dk = 2.0 ** -8 / d ** 0.5 * np.einsum("thf,jhf->htj", np.abs(qf[b]),
                                                  np.abs(held[0][b])).max(-1)
            assert (np.abs(to_f64(lse)[b] - rl) <= 2e-3 + dk).all()
        else:
            np.testing.assert_allclose(to_f64(o)[b], r, atol=1e-5, rtol=0)
            np.testing.assert_allclose(to_f64(lse)[b], rl, atol=1e-5, rtol=1e-6)
    if dtype == "bf16":
        sl = torch.full((B,), n, dtype=torch.int32, device="cuda")
        o4 = T.mha_fwd_kv4(q, cache, table, sl, HP, page)
        assert_bf16_close(to_f64(o), to_f64(o4), "chunk and mha_fwd_kv4")
    assert T.device_error() == 0
