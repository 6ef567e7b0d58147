"""rope_frequencies(how="blend") where the border of the slow pairs lies past the last pair: the ramp goes on to that border."""
import math

import pytest
import torch

from compress_kv_write_gb300 import rope_frequencies

# (rot, original, factor, first, last): the pairs between which the two are mixed are those that turn 32 times and once within
# `original` positions, at rot ln(original / (2 pi n)) / (2 ln base), rounded down and up, the second at most rot - 1:
# with a base of 10,000 for (rot, original)
#    64,  65536: 20.105, 32.146     64,  50000: 19.165, 31.206     64, 131072: 22.513, 34.554     128, 65536: 40.210, 64.292
#    64, 262144: 24.921, 36.962     16,  32768:  4.424,  7.434     64,   4096: 10.472, 22.513
# and with a base of 16, 8, 1024: 2.348, 7.348 (8, so 7)
SETTINGS = [(64, 65536, 16, 20, 33, 1e4), (64, 50000, 16, 19, 32, 1e4), (64, 131072, 8, 22, 35, 1e4), (128, 65536, 16, 40, 65, 1e4),
            (64, 262144, 4, 24, 37, 1e4), (16, 32768, 4, 4, 8, 1e4), (64, 4096, 32, 10, 23, 1e4), (8, 1024, 4, 2, 7, 16.0)]


@pytest.mark.parametrize("rot,original,factor,first,last,base", SETTINGS)
def test_ramp(rot, original, factor, first, last, base):
    got = rope_frequencies(rot, base, factor=factor, original=original)
    for i in range(rot // 2):
        plain = base ** (-2 * i / rot)
        share = min(max((i - first) / (last - first), 0.0), 1.0)   # of the divided one
        assert math.isclose(got[i], plain * (1 - share) + plain / factor * share, rel_tol=1e-12), i
        if original * plain / (2 * math.pi) > 1:                   # turns more than `slow` times
            assert got[i] > plain / factor * (1 + 1e-9), i


def test_last_pair_by_hand():
    # rot 64, 65,536 positions, factor 16: pair 31 is 11 / 13 of the way, (1 - 11 / 13) + 11 / 13 / 16 = 43 / 208 of its frequency
    got = rope_frequencies(64, factor=16, original=65536)[31]
    assert math.isclose(got, 10000.0 ** (-62 / 64) * 43 / 208, rel_tol=1e-12)
    # 131,072 positions, factor 8: 9 / 13 of the way, 4 / 13 + 9 / 104 = 41 / 104
    got = rope_frequencies(64, factor=8, original=131072)[31]
    assert math.isclose(got, 10000.0 ** (-62 / 64) * 41 / 104, rel_tol=1e-12)
    # every pair turns 32 times and more: nothing changes
    assert torch.equal(rope_frequencies(8, factor=4, original=2 ** 26)[:4], rope_frequencies(8))


@pytest.mark.parametrize("original,slow,fast", [(4, 1, 32), (6, 1, 32), (100, 16, 32), (1, 1, 2)])
def test_no_pair_turns_so_often(original, slow, fast):
    """The fastest pair turns original / (2 pi) times: where that is not more than `slow`, every pair is divided."""
    got = rope_frequencies(64, factor=4, original=original, slow=slow, fast=fast)
    assert original / (2 * math.pi) <= slow
    assert torch.allclose(got, rope_frequencies(64) / 4, rtol=1e-12, atol=0)
