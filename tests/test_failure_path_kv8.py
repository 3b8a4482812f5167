"""GPU test of mha_fwd_kv8's failure path, made without any GPU fault: a test
hook lets one stage of copies never count as complete and shortens every wait
of that launch to 20 ms.  The launch must give up, report device error 2 and
leave the context usable; with its workspace zeroed again, the next call must
match the one before."""
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


# one unit a warp; a unit that spans CTAs; one and several columns
@pytest.mark.parametrize("lens,Nq,Hq,Hkv", [([40] * 3, 1, 2, 2), ([9000], 1, 1, 1),
                                            ([3000, 0, 700], 2, 8, 2), ([5000], 4, 4, 1)])
def test_withheld_stage_times_out_and_the_next_call_is_clean(T, lens, Nq, Hq, Hkv):
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
    w = torch.zeros((B, Hkv, keys), device="cuda")

    def call():
        return T.mha_fwd_kv8(q, cache, table, sl, Hkv, page, return_lse=True, weights=w,
                             workspace=ws)

    good = call()
    assert T.device_error(clear=True) == 0
    assert T.lib().iha_test_fail_next_wait(20000) == 0       # 20 ms limit, one launch
    call()
    assert T.device_error(clear=True) == 2                    # a bounded wait gave up
    ws.zero_()
    for _ in range(2):                                        # the hook was one-shot
        again = call()
        assert all(torch.equal(a, b) for a, b in zip(good, again))
    assert T.device_error() == 0
