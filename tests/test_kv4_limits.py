"""The largest calls of mha_fwd_kv4: what its 32-bit counts cannot hold is refused.
A call that is taken goes on to the launch, so these run only where there is no
GPU to launch on (status 4); the addresses are made up."""
import ctypes as C

import pytest

import transformer_attention_iha_gb300 as T

A = 1 << 42


def gpu():
    import torch
    return torch.cuda.is_available()


@pytest.fixture(scope="module")
def L():
    T.build()
    return T.lib()


def attend(L, B, page, table_width=1, d=32):
    """One head, one new token of each of B sequences, q broadcast over them."""
    return L.mha_fwd_kv4(*(C.c_void_p(i * A) for i in range(1, 6)), None, C.c_void_p(6 * A),
                         1 << 40, B, 1, 1, 1, d, 1, page, table_width, T.Strides(0, 0, 0, 0),
                         T.Strides(d, 0, 0, 0), 0.0, 1, 0, T.BF16, None)


@pytest.mark.skipif(gpu(), reason="a call that is taken would be launched")
def test_positions_of_a_cta_fit_32_bits(L):
    """Without a device the grid is 3 CTAs of 4 warps.  95 sequences of 2^26 blocks
    are 531 million positions a warp: four shares and a unit of 2^26 pass 2^31."""
    assert attend(L, 32, 1 << 30) == 4
    assert attend(L, 95, 1 << 30) == 2
    assert "one launch" in L.iha_last_error().decode()


def test_more_sequences_than_the_scan_can_count(L):
    """Its index moves in steps of 128 and would pass 2^31 - 1 (refused everywhere)."""
    for B in ((1 << 30) + 1, (1 << 31) - 1):
        assert attend(L, B, 16) == 2
        assert "sequences" in L.iha_last_error().decode()
