"""Of mha_fwd_kv4's workspace only the first 4096 bytes have to be zero at first:
with NaN bits in all the rest, results are the same and the counters in those bytes
are left at zero."""
import pytest

import synthetic as S
from helpers import to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import transformer_attention_iha_gb300 as T
    T.lib()
    return T


def problem(T, lens, Nq, Hq, Hkv, d):
    import torch
    B, page = len(lens), 32
    width = -(-max(lens) // page)
    cache = torch.zeros((B * width, T.kv4_page_bytes(page, Hkv, d)), dtype=torch.uint8,
                        device="cuda")
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    n = B * width * page
    k, v = (to_dev(S.normal((1, n, Hkv, d), 530, t)) for t in range(2))
    T.kv4_store(k, v, torch.arange(n, dtype=torch.int32, device="cuda")[None], cache, page)
    q = to_dev(S.normal((B, Nq, Hq, d), 530, 2))
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return lambda **kw: T.mha_fwd_kv4(q, cache, table, sl, Hkv, page, return_lse=True, **kw)


@pytest.mark.parametrize("lens,Nq,Hq,Hkv,d", [([20000], 1, 2, 2, 128), ([9000, 0, 33], 2, 8, 2, 64),
                                              ([5000, 700], 1, 7, 1, 96), ([3000], 5, 6, 2, 32)])
def test_only_the_first_bytes_need_zeros(T, lens, Nq, Hq, Hkv, d):
    import torch
    call = problem(T, lens, Nq, Hq, Hkv, d)
    size = T.mha_fwd_kv4_workspace_bytes(len(lens), Nq, Hq, Hkv, d)
    clean = call(workspace=torch.zeros(size, dtype=torch.uint8, device="cuda"))
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:4096] = 0
    for _ in range(3):
        got = call(workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(clean, got))
        assert not ws[:1920].any()
    assert T.device_error() == 0
