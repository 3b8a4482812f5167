"""GPU parity of rotary positions (iha_rope_fwd, iha_rope_bwd) with the oracle.

Tolerance.  An angle modulo a turn is held to 2^-32 turns; the rest of up to an eighth of a
turn behind the nearest quarter is read as fp32, 2^-28 turns off: together less than
2 pi * 2^-25 < 2^-22 radians; sine and cosine are good to 2^-23
more, the gain's product and the two products and their sum to 4 roundings of 2^-24:
  |y - r| <= gain * (|a| + |b|) * (2^-22 + 2^-23 + 4 * 2^-24) < 2^-21 gain (|a| + |b|),
and bf16 results 2^-8 |r| more.  The oracle's own angle, a product in float64, is off by
2^-53 |position * w|."""
import numpy as np
import pytest

import oracle as O
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


def f32(x):
    return S.bf16_bits_to_f32(x) if x.dtype == np.uint16 else x


def check(got, x, pos, w, gain, inter, back):
    n = len(w)
    r = O.rotate(x, pos, w, gain, inter, back)
    a = np.abs(f32(x).astype(np.float64))
    pair = np.zeros_like(a)
    lo, hi = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if inter else (slice(0, n), slice(n, 2 * n))
    pair[..., lo] = pair[..., hi] = a[..., lo] + a[..., hi]
    far = 2.0 ** -52 * np.abs(pos.astype(np.float64)).max() * w.max()
    bound = gain * pair * (2.0 ** -21 + far)
    if x.dtype == np.uint16:
        bound = bound + 2.0 ** -8 * np.abs(r)
    g = to_f64(got)
    assert (np.abs(g - r) <= bound).all(), np.abs(g - r).max()
    np.testing.assert_array_equal(g[..., 2 * n:], f32(x)[..., 2 * n:])  # copied, bit for bit


CASES = [  # B, N, Hq, Hk, d, rot: vectors and single pairs, one head to many, no k
    (1, 1, 1, 0, 8, 2), (2, 3, 4, 1, 16, 16), (1, 33, 3, 3, 64, 64), (3, 5, 32, 8, 128, 128),
    (2, 7, 5, 2, 96, 48), (1, 9, 2, 7, 80, 80), (1, 4, 80, 80, 128, 64), (2, 3, 3, 1, 256, 256),
    (1, 5, 2, 1, 64, 6), (1, 2, 2, 2, 256, 254), (4, 1, 20, 20, 128, 32), (1, 700, 9, 1, 32, 32),
    (1, 900, 21, 3, 80, 50)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_shapes_layouts_and_directions(T, dtype, inter, case):
    B, N, Hq, Hk, d, rot = case
    q, k = S.normal((B, N, Hq, d), 1, 0, dtype=dtype), S.normal((B, N, max(1, Hk), d), 1, 1, dtype=dtype)
    pos = S.rng(2).integers(0, 9000, (B, N)).astype(np.int32)
    rope = T.Rope(rot, interleaved=inter)
    w, _ = O.rope_frequencies(rot)
    for back, call in ((False, T.rope_fwd), (True, T.rope_bwd)):
        yq, yk = call(to_dev(q), to_dev(k) if Hk else None, to_dev(pos), rope)
        check(yq, q, pos, w, 1.0, inter, back)
        assert (yk is None) == (Hk == 0)
        if Hk:
            check(yk, k, pos, w, 1.0, inter, back)


@pytest.mark.parametrize("scaling,factor,trained", [("linear", 4.0, 0), ("base", 8.0, 0),
                                                    ("parts", 8.0, 4096), ("parts", 1.0, 64)])
def test_scaled_for_long_contexts_at_far_and_negative_positions(T, scaling, factor, trained):
    import torch
    q = S.normal((2, 6, 3, 64), 3, 0, dtype="f32")
    pos = np.array([[0, 1, 1 << 20, (1 << 24) + 1, 123456789, 2 ** 31 - 1],
                    [-1, -2, -70000, -(1 << 24) - 1, -123456789, -2 ** 31]], np.int32)
    rope = T.Rope(64, scaling=scaling, factor=factor, trained=trained)
    w, gain = O.rope_frequencies(64, 10000.0, scaling, factor, trained)
    for back, call in ((False, T.rope_fwd), (True, T.rope_bwd)):
        y, _ = call(to_dev(q), None, to_dev(pos), rope)
        check(y[:, :4], q[:, :4], pos[:, :4], w, gain, False, back)
        # farther out the table's own 53 bits count: w * position to 2^-51 or so
        check(y[:, 4:], q[:, 4:], pos[:, 4:], w, gain, False, back)
    y2, _ = T.rope_fwd(to_dev(q), None, to_dev(pos), T.Rope(64, gain=2.0))
    y1, _ = T.rope_fwd(to_dev(q), None, to_dev(pos), T.Rope(64))
    assert torch.equal(y2, 2 * y1)


def test_gradient_against_differences(T):
    """<dy, rope(x + h e)> - <dy, rope(x)> over h, for the formula that the backward pass
    states: the map is linear, so differences are exact but for rounding."""
    import torch
    x = S.normal((1, 3, 2, 32), 4, 0, dtype="f32")
    dy = S.normal((1, 3, 2, 32), 4, 1, dtype="f32")
    pos = to_dev(np.array([[5, 77, 4000]], np.int32))
    rope = T.Rope(24, interleaved=True, scaling="parts", factor=4.0, trained=128)
    dx, _ = T.rope_bwd(to_dev(dy), None, pos, rope)
    y0 = to_f64(T.rope_fwd(to_dev(x), None, pos, rope)[0])
    g = to_f64(dx)
    for n, h, f in ((0, 0, 0), (1, 1, 7), (2, 0, 23), (2, 1, 31), (1, 0, 12)):
        e = x.copy()
        e[0, n, h, f] += 1.0
        y1 = to_f64(T.rope_fwd(to_dev(e), None, pos, rope)[0])
        num = ((y1 - y0) * dy.astype(np.float64)).sum()
        # four values of at most |x| + 1 < 8, each off by 2^-20 of itself
        assert abs(num - g[0, n, h, f]) <= 2.0 ** -16 * np.abs(dy[0, n, h]).max()
    # there and back with the gain of each: gain^2 x on the rotated features
    y, _ = T.rope_fwd(to_dev(x), None, pos, rope)
    z = to_f64(T.rope_bwd(y, None, pos, rope)[0])
    assert np.abs(z[..., :24] - rope.gain ** 2 * x[..., :24]).max() <= 2.0 ** -17
    np.testing.assert_array_equal(z[..., 24:], x[..., 24:])


@pytest.mark.parametrize("rot", [48, 50])
def test_views_in_place_and_default_positions(T, rot):
    """q and k as slices of one projection's output, turned in place; a broadcast input;
    results written into slices; everything around them untouched."""
    import torch
    B, N, Hq, Hk, d = 2, 5, 4, 2, 64
    x = S.normal((B, N, Hq + 2 * Hk, d), 5, 0)
    t = to_dev(x)
    rope = T.Rope(rot)
    w, _ = O.rope_frequencies(rot)
    pos = np.broadcast_to(np.arange(N), (B, N))
    q, k = t[:, :, :Hq], t[:, :, Hq:Hq + Hk]
    yq, yk = T.rope_fwd(q, k, None, rope, out=(q, k))
    assert yq.data_ptr() == t.data_ptr()
    check(t[:, :, :Hq], x[:, :, :Hq], pos, w, 1.0, False, False)
    check(t[:, :, Hq:Hq + Hk], x[:, :, Hq:Hq + Hk], pos, w, 1.0, False, False)
    np.testing.assert_array_equal(to_f64(t[:, :, Hq + Hk:]), f32(x)[:, :, Hq + Hk:])
    one = S.normal((1, 1, 1, d), 5, 1)
    out = torch.full((B, N, 3, d + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    T.rope_bwd(to_dev(one).expand(B, N, 3, d), None, None, rope, out=(out[..., :d], None))
    check(out[..., :d], np.broadcast_to(one, (B, N, 3, d)), pos, w, 1.0, False, True)
    assert bool((out[..., d:] == 9.0).all())
    # rows of k between rows of q in one buffer, apart but interleaved
    both = to_dev(S.normal((B, N, 2, 3, d), 5, 2))
    ref = T.rope_fwd(both[:, :, 0].contiguous(), both[:, :, 1].contiguous(), None, rope)
    T.rope_fwd(both[:, :, 0], both[:, :, 1], None, rope, out=(both[:, :, 0], both[:, :, 1]))
    assert torch.equal(both[:, :, 0], ref[0]) and torch.equal(both[:, :, 1], ref[1])


def test_many_rows_past_32_bit_offsets(T):
    """5 GB of rows: the last ones, and a few drawn among the others."""
    import torch
    N, H, d = 1 << 18, 80, 128
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    q = torch.empty((1, N, H, d), dtype=torch.bfloat16, device="cuda")
    pick = np.array([0, 1, 4097, N // 2, N - 2, N - 1])
    x = S.normal((1, len(pick), H, d), 6, 0)
    q[:, torch.from_numpy(pick).cuda()] = to_dev(x)
    rope = T.Rope(d)
    w, _ = O.rope_frequencies(d)
    T.rope_fwd(q, None, None, rope, out=(q, None))
    check(q[:, torch.from_numpy(pick).cuda()], x, pick[None], w, 1.0, False, False)


def test_stream_graph_and_non_finite(T):
    import torch
    x = S.normal((2, 3, 4, 64), 7, 0, dtype="f32")
    x[0, 0, 0, 3], x[1, 2, 3, 40] = np.inf, np.nan
    rope = T.Rope(64)
    xd, pos = to_dev(x), to_dev(np.full((2, 3), 11, np.int32))
    ref, _ = T.rope_fwd(xd, None, pos, rope)
    g = to_f64(ref)
    bad = ~np.isfinite(g)
    want = np.zeros_like(bad)
    want[0, 0, 0, [3, 35]] = want[1, 2, 3, [8, 40]] = True
    np.testing.assert_array_equal(bad, want)            # its own pair only
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, _ = T.rope_fwd(xd, None, pos, rope, stream=s)
    s.synchronize()
    assert torch.equal(y.nan_to_num(7.0), ref.nan_to_num(7.0))
    out = torch.empty_like(xd)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        T.rope_fwd(xd, None, pos, rope, out=(out, None))
    pos.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.nan_to_num(7.0)[1, 0], xd[1, 0])


def test_binding_refusals(T):
    import torch
    q = torch.zeros((1, 2, 3, 64), device="cuda")
    k = torch.zeros((1, 2, 1, 64), device="cuda")
    pos = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    rope = T.Rope(64)
    for a in ((q[0], k, pos, rope), (q, k[0], pos, rope), (q, k[:, :1], pos, rope),
              (q, k[..., :32], pos, rope), (q, k.bfloat16(), pos, rope), (q, k, pos[:, :1], rope),
              (q, k, pos.long(), rope), (q.cpu(), k, pos, rope), (q, k, pos.cpu(), rope),
              (q[..., ::2], None, pos, T.Rope(32)), (q.transpose(2, 3), None, pos, rope)):
        with pytest.raises(ValueError):
            T.rope_fwd(*a)
    for out in ((q,), (q, None), (torch.zeros_like(q), q), (torch.zeros_like(q[:, :1]), k)):
        with pytest.raises((ValueError, T.IHAError)):
            T.rope_fwd(q, k, pos, rope, out=out)
    with pytest.raises(TypeError):
        T.rope_fwd(q, k, pos, 64)
    with pytest.raises(TypeError):
        T.rope_fwd(q.half(), None, pos, rope)
    with pytest.raises(T.IHAError):
        T.rope_fwd(q, k, pos, T.Rope(128))
