"""GPU parity of calls at the edges of what the header allows: positions up to
2^24 either way, batches without a key, chunks of many columns, more new tokens
than a sequence has keys, pages that sequences share."""
import numpy as np
import pytest

import oracle as O
import synthetic as S
from helpers import assert_bf16_close, to_dev, to_f64
from test_parity_kv4 import build, check_rows, run_case

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


# the kernel for few tokens, the tensor-core kernel, the CUDA-core kernel (bf16, float32)
@pytest.mark.parametrize("n,H,P,d,dtype", [(9, 20, 4, 128, "bf16"), (70, 20, 4, 128, "bf16"),
                                           (300, 8, 2, 64, "bf16"), (20, 4, 2, 32, "bf16"),
                                           (20, 4, 2, 64, "f32")])
def test_premix_at_far_and_negative_positions(T, n, H, P, d, dtype):
    xs = [S.normal((1, n, H, d), 540, t, dtype=dtype) for t in range(3)]
    ws = [S.premix_weight(H, P, 541, t) for t in range(3)]
    top = 2 ** 24 - 1
    pos = S.rng(542).integers(-top, top + 1, (1, n)).astype(np.int32)
    pos[0, :4] = [top, -top, -1, 2 ** 23 + 1]
    ys = T.premix_fwd_qkv_at([to_dev(x) for x in xs], [to_dev(w) for w in ws], P, to_dev(pos))
    for t in range(3):
        r = O.premix_at(xs[t], ws[t], P, pos) if t < 2 else O.premix_fwd(xs[t], ws[t], P)
        if dtype == "bf16":
            assert_bf16_close(to_f64(ys[t]), r, f"premix at {t}")
        else:
            np.testing.assert_allclose(to_f64(ys[t]), r, atol=1e-5, rtol=0)


@pytest.mark.parametrize("B,Nq,Hq,Hkv", [(1, 1, 1, 1), (1, 1, 80, 80), (200, 1, 4, 2), (3, 9, 2, 1)])
@pytest.mark.parametrize("mask,window", [(0, 0), (1, 0), (2, 3)])
def test_batches_without_a_key(T, B, Nq, Hq, Hkv, mask, window):
    o, lse = run_case(T, [0] * B, Nq, Hq, Hkv, 64, 16, mask, window)
    assert not o.any() and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("lens,Nq,Hq,Hkv,d,window", [([150, 40], 130, 3, 1, 64, 0),
                                                     ([300], 257, 2, 2, 32, 31),
                                                     ([20, 77], 100, 4, 2, 96, 0)])
def test_chunks_of_many_columns(T, lens, Nq, Hq, Hkv, d, window):
    """Longer than the sequence too: the first rows see nothing."""
    run_case(T, lens, Nq, Hq, Hkv, d, 16, T.MASK_CAUSAL_WINDOW if window else T.MASK_CAUSAL, window)


@pytest.mark.parametrize("Nq,Hq,Hkv", [(1, 2, 2), (1, 8, 2), (2, 10, 2)])
def test_sequences_that_share_pages(T, Nq, Hq, Hkv):
    """A common prefix: the page table names the same pages for every sequence."""
    import torch
    d, page = 128, 16
    cache, table, _, ks, vs = build(T, [500], Hkv, d, page, 550)
    lens = [500, 16, 333, 0, 499]
    q = S.normal((len(lens), Nq, Hq, d), 551, 0)
    o, lse = T.mha_fwd_kv4(to_dev(q), cache, table.repeat(len(lens), 1),
                           torch.tensor(lens, dtype=torch.int32, device="cuda"), Hkv, page,
                           return_lse=True)
    assert T.device_error() == 0
    for b, n in enumerate(lens):
        check_rows(T, o[b], lse[b], q[b], ks[0][:n], vs[0][:n], T.MASK_CAUSAL, 0)
