"""How many keys kv8_evict can be told to keep: what is refused (on the CPU, before any
launch), and more than a table has."""
import ctypes as C

import pytest

import oracle as O
import synthetic as S
import transformer_attention_iha_gb300 as T


@pytest.fixture(scope="module")
def L():
    T.build()
    return T.lib()


def _p(i):
    return C.c_void_p((1 << 44) + (i << 38))      # apart, never dereferenced


@pytest.mark.parametrize("keep", [(1 << 30) + 1, (1 << 31) - 8192, (1 << 31) - 1])
@pytest.mark.parametrize("recent", [0, 7])
def test_more_keys_than_a_table_can_hold_are_refused(L, keep, recent):
    """A list of so many positions could not be counted through in 32 bits."""
    st = L.kv8_evict(_p(0), _p(1), _p(2), _p(3), _p(4), _p(5), _p(6), _p(7), 1, 8, 16, 4, 4, 1, 64,
                     keep, recent, None)
    assert st == 2 and "2^30" in L.iha_last_error().decode()


@pytest.mark.gpu
@pytest.mark.parametrize("keep,recent", [(65, 3), (4000, 0), (4000, 4000)])
def test_more_keys_than_the_table_has(L, keep, recent):
    """Every sequence is kept whole; the list goes on with -1, the weights with 0."""
    import torch
    from helpers import to_dev, to_f64
    H, d, page, width, lens = 2, 64, 16, 4, [64, 17, 0]
    B = len(lens)
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    cache = torch.full((2 * B * width, T.kv8_page_bytes(page, H, d)), 0xFF, dtype=torch.uint8,
                       device="cuda")
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k, v = S.normal((B, 64, H, d), 600, 0), S.normal((B, 64, H, d), 600, 1)
    T.kv8_append(to_dev(k), to_dev(v), table, sl, cache, page, counts=sl)
    w = torch.rand((B, H, width * page), device="cuda")
    nl, kept, wo = T.kv8_evict(cache, table, sl, w, table + B * width, H, d, page, keep, recent)
    assert nl.tolist() == lens and kept.shape == (B, H, keep)
    for b, n in enumerate(lens):
        for h in range(H):
            assert kept[b, h].tolist() == list(range(n)) + [-1] * (keep - n)
        assert torch.equal(wo[b, :, :n], w[b, :, :n]) and not wo[b, :, n:].any()
        if n == 0:
            continue
        slots = ((table[b].long() + B * width)[:, None] * page +
                 torch.arange(page, device="cuda")).reshape(-1)[:n].to(torch.int32)[None]
        got = T.kv8_load(cache, slots, H, d, page, dtype=torch.float32)
        for g, x in zip(got, (k, v)):
            assert (to_f64(g)[0] == O.Kv8Rows(H, d).append(x[b, 64 - n:]).values).all()
    assert T.device_error() == 0
