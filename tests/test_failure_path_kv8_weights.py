"""GPU test of mha_fwd_kv8's failure path with the keys' weights, made without any GPU
fault (one stage of copies never counts as complete, every wait of that launch ends
after 20 ms): weights that are gathered over many calls stay as they were when a call
gave up, in place and apart, and the call after it adds its own once."""
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


# one unit a warp; units that span CTAs; one and several columns; weights off 16 bytes
@pytest.mark.parametrize("lens,Nq,Hq,Hkv", [([40] * 3, 1, 2, 2), ([9000], 1, 1, 1),
                                            ([3000, 0, 700], 2, 8, 2), ([5000], 4, 4, 1)])
@pytest.mark.parametrize("off", [0, 1])
def test_a_call_that_gave_up_leaves_the_weights(T, lens, Nq, Hq, Hkv, off):
    import torch
    d, page, B = 64, 16, len(lens)
    width = -(-max(lens) // page)
    cache = torch.zeros((B * width, T.kv8_page_bytes(page, Hkv, d)), dtype=torch.uint8,
                        device="cuda")
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k, v = (to_dev(S.normal((B, max(lens), Hkv, d), 410, t)) for t in range(2))
    T.kv8_append(k, v, table, sl, cache, page)
    q = to_dev(S.normal((B, Nq, Hq, d), 410, 2))
    keys = width * page
    ws = torch.zeros(T.mha_fwd_kv8_workspace_bytes(B, Nq, Hq, Hkv, d, keys), dtype=torch.uint8,
                     device="cuda")
    n = B * Hkv * keys
    w = torch.rand(n + 4, device="cuda")[off:off + n].view(B, Hkv, keys)
    w0 = w.clone()

    def call(out):
        return T.mha_fwd_kv8(q, cache, table, sl, Hkv, page, weights=w, weights_out=out,
                             workspace=ws)

    good = call(torch.empty_like(w0))[1]
    assert T.device_error(clear=True) == 0 and not torch.equal(good, w0)
    apart = torch.full_like(w0, 7.0)
    for out, before in ((w, w0), (apart, apart.clone())):
        assert T.lib().iha_test_fail_next_wait(20000) == 0    # 20 ms limit, one launch
        call(out)
        assert T.device_error(clear=True) == 2                 # a bounded wait gave up
        assert torch.equal(w, w0) and torch.equal(out, before)
        ws[:4096].zero_()
    assert torch.equal(call(apart)[1], good)
    assert torch.equal(call(w)[1], good)
    assert T.device_error() == 0
