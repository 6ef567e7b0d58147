"""kvq_rope_table at far positions and for frequencies of every size, against angles of 400 bits.

A value is off by at most 2^-22 of the amplitude: 2.0e-7 by the angle's three roundings, the series and the last sum and
product (test_rope_gpu.py counts them), and the phase, a multiple of 2^-64 turns, by half of one a position: below 2^-34
turns, 3.7e-10, at positions below 2^31.  2^-22 is 2.38e-7.
"""
import math
from fractions import Fraction

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def K():
    from compress_kv_write_gb300 import build
    build.build()
    import compress_kv_write_gb300 as K
    K.lib()
    return K


def _pi(bits):
    """pi 2^bits, rounded down, by Machin's formula."""
    one = 1 << (bits + 32)

    def arctan_of_one_over(n):
        t = total = one // n
        k, sign = 1, -1
        while t:
            t //= n * n
            k += 2
            total += sign * (t // k)
            sign = -sign
        return total
    return (16 * arctan_of_one_over(5) - 4 * arctan_of_one_over(239)) >> 32


PI = _pi(400)


def angle(freq, position):
    """position * freq, less whole turns, as a double."""
    f = Fraction(freq) * position
    turns = Fraction(f.numerator << 400, f.denominator * 2 * PI)
    return 2 * math.pi * float(turns - turns.numerator // turns.denominator)


# from one radian a position down, as models have them; faster and slower than any; turned the other way; none
PLAIN = [10000.0 ** (-2 * i / 64) for i in range(32)]
ODD = [0.994, 3.0, math.pi, 1e4, 1e6, 123456789.123, 2.0 ** 40 + 2.0 ** -12, 1e13 + 0.3125, 2.0 ** 52, 1.9e16, 1e-9, 1e-12, 1e-17, 5e-20,
       1e-300, 5e-324, 0.0, -0.0, -1.0, -0.03, -1e-4, -1e-10, -7e-17, -1e6, -12345.678, 2 * math.pi, -2 * math.pi, 4.0 * math.pi,
       math.pi / 2, -math.pi / 4, 6.2831853, 1e-8]


@pytest.mark.parametrize("freq", [PLAIN, ODD], ids=["plain", "odd"])
@pytest.mark.parametrize("first", [0, 65521, 1000003, 2 ** 27 - 9, 2 ** 31 - 1 - 37])
@pytest.mark.parametrize("amplitude", [1.0, -1.3466])
def test_every_position_and_frequency(K, freq, first, amplitude):
    rows, h = 37, len(freq)
    table = torch.full((rows, 2 * h), 7.0, device=DEV)
    K.kvq_rope_table(torch.tensor(freq, dtype=torch.float64, device=DEV), table, first=first, amplitude=amplitude)
    got = table.cpu().double()
    amplitude = torch.tensor(amplitude, dtype=torch.float32).item()
    x = torch.tensor([[angle(f, first + r) for f in freq] for r in range(rows)], dtype=torch.float64)
    off = (got - amplitude * torch.cat((x.cos(), x.sin()), 1)).abs()
    assert off.max() <= 2.0 ** -22 * abs(amplitude), (off.max().item() * 2 ** 22, [freq[i % h] for i in off.amax(0).topk(3).indices.tolist()])


def test_no_fraction_of_a_turn_is_left(K):
    freq = [2.0 ** 52 * 2 * math.pi, 1e17, -1e300, math.inf, -math.inf, math.nan, 2.0 ** 52 * 6.28, 1.0]
    table = torch.zeros((3, 16), device=DEV)
    K.kvq_rope_table(torch.tensor(freq, dtype=torch.float64, device=DEV), table, first=5)
    nan = table.cpu().isnan()
    assert nan[:, [0, 1, 2, 3, 4, 5, 8, 9, 10, 11, 12, 13]].all() and not nan[:, [6, 7, 14, 15]].any()
