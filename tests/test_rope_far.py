"""The rotation's table in all of its 64 bits, against arithmetic of 90 digits, and angles
at positions so far out that a table of 53 bits shows.

An entry is turns per position times 2^64, rounded: off by half a unit, and at 2^31
positions by 2^-34 turns.  The kernel drops what lies below 2^-32 turns and reads the rest of
an eighth of a turn as fp32, 2^-28 turns off; sine and cosine are good to 2^-23, products
and sums to 4 roundings of 2^-24:
  |y - r| <= gain (|a| + |b|) (2 pi (2^-28 + 2^-32 + 2^-34) + 2^-23 + 2^-22)
          <  gain (|a| + |b|) 2^-21."""
import math
from decimal import Decimal, getcontext, localcontext

import numpy as np
import pytest

import synthetic as S
import transformer_attention_iha_gb300 as T

getcontext().prec = 90


def pi():
    """Machin's formula."""
    def arctan_of_inverse(n):
        x = total = Decimal(1) / n
        k, sign = 1, -1
        while abs(x) > Decimal(10) ** -88:
            x /= n * n
            k += 2
            total += sign * x / k
            sign = -sign
        return total
    return 4 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))


def turns(rot, base=10000.0, scaling=None, factor=1.0, trained=0, fast=32.0, slow=1.0):
    """Turns per position of each pair, from the formulas."""
    f, two_pi = Decimal(factor), 2 * pi()
    out = []
    for i in range(rot // 2):
        x = Decimal(base).ln()
        if scaling == "base":
            x += f.ln() * rot / (rot - 2)
        t = (x * (-2 * i) / rot).exp() / two_pi
        if scaling == "linear":
            t /= f
        if scaling == "parts":
            g = (trained * t - Decimal(slow)) / (Decimal(fast) - Decimal(slow))
            g = min(Decimal(1), max(Decimal(0), g))
            t *= g + (1 - g) / f
        out.append(t)
    return out


CASES = [dict(rot=2), dict(rot=64), dict(rot=128, base=500000.0), dict(rot=256, base=1e6),
         dict(rot=250, base=1.0000001), dict(rot=6, base=1.7e308), dict(rot=256, base=1.7e308),
         dict(rot=128, scaling="linear", factor=7.3), dict(rot=8, scaling="linear", factor=9e29),
         dict(rot=4, scaling="base", factor=8.0), dict(rot=96, scaling="base", factor=2.7),
         dict(rot=256, base=1e5, scaling="base", factor=1e20), dict(rot=2, scaling="parts",
                                                                    factor=3.0, trained=64),
         dict(rot=128, scaling="parts", factor=8.0, trained=4096),
         dict(rot=128, base=150000.0, scaling="parts", factor=40.0, trained=4095, fast=31.7,
              slow=0.3),
         dict(rot=64, scaling="parts", factor=1.0, trained=2048),
         dict(rot=64, scaling="parts", factor=5.0, trained=2 ** 31 - 1, fast=1e9, slow=0.0)]


@pytest.mark.parametrize("case", CASES)
def test_every_bit_of_the_table(case):
    T.build()
    r = T.Rope(**case)
    for i, t in enumerate(turns(**case)):
        off = Decimal(int(r._c.turn[i])) - t * 2 ** 64
        assert abs(off) <= Decimal("0.500001"), (i, float(off))


@pytest.mark.gpu
@pytest.mark.parametrize("case", [dict(rot=64), dict(rot=64, interleaved=True),
                                  dict(rot=64, scaling="parts", factor=8.0, trained=4096),
                                  dict(rot=48, scaling="base", factor=6.5)])
def test_angles_at_the_farthest_positions(case):
    import torch
    from helpers import to_dev, to_f64
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 3571, 2000000011, -1999999973, 1 << 30, 123456789, 1]
    x = S.normal((1, len(pos), 3, 64), 700, 0, dtype="f32")
    rope = T.Rope(**case)
    y = to_f64(T.rope_fwd(to_dev(x), None, torch.tensor([pos], dtype=torch.int32, device="cuda"),
                          rope)[0])[0]
    rot, inter = case["rot"], case.get("interleaved", False)
    ts = turns(**{k: v for k, v in case.items() if k != "interleaved"})
    x = x[0].astype(np.float64)
    for n, p in enumerate(pos):
        for i, t in enumerate(ts):
            with localcontext():
                a = p * t
                a = 2 * math.pi * float(a - a.to_integral_value())
            c, s = rope.gain * math.cos(a), rope.gain * math.sin(a)
            ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
            u, v = x[n, :, ia], x[n, :, ib]
            bound = rope.gain * (np.abs(u) + np.abs(v)) * 2.0 ** -21
            assert (np.abs(y[n, :, ia] - (u * c - v * s)) <= bound).all(), (p, i)
            assert (np.abs(y[n, :, ib] - (v * c + u * s)) <= bound).all(), (p, i)
