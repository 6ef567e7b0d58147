"""Rotary positions without a GPU: scaled frequencies against their formulas, and the calls that the host refuses."""
import math

import pytest
import torch

A = 0x10000          # a 16-byte aligned fake device address (never dereferenced)


@pytest.fixture(scope="module")
def L():
    from compress_kv_write_gb300 import build
    build.build()
    from compress_kv_write_gb300 import kvq
    return kvq.lib()


def test_frequencies():
    from compress_kv_write_gb300 import rope_frequencies
    plain = [10000.0 ** (-2 * i / 64) for i in range(32)]
    assert torch.allclose(rope_frequencies(64), torch.tensor(plain, dtype=torch.float64), rtol=1e-15)
    assert torch.allclose(rope_frequencies(64, factor=8, how="linear"), torch.tensor(plain, dtype=torch.float64) / 8, rtol=1e-15)
    f = rope_frequencies(64, factor=8, how="base")
    assert f[0] == 1 and math.isclose(f[-1], plain[-1] / 8, rel_tol=1e-12)
    f = rope_frequencies(64, factor=32, original=4096)
    turns = [4096 * p / (2 * math.pi) for p in plain]
    for i in range(32):
        if turns[i] > 32 * 1.4:            # more than one index above the border
            assert math.isclose(f[i], plain[i], rel_tol=1e-12)
        elif turns[i] < 1 / 1.4:
            assert math.isclose(f[i], plain[i] / 32, rel_tol=1e-12)
        else:
            assert plain[i] / 32 * (1 - 1e-12) <= f[i] <= plain[i] * (1 + 1e-12)
    assert (f[1:] < f[:-1]).all() and f.dtype == torch.float64
    assert torch.equal(rope_frequencies(2), torch.ones(1, dtype=torch.float64))


@pytest.mark.parametrize("bad", [dict(rot=3), dict(rot=0), dict(rot=64, base=0.0), dict(rot=64, factor=0.5),
                                 dict(rot=64, how="x"), dict(rot=2, factor=2, how="base"),
                                 dict(rot=64, factor=2, fast=1, slow=1)])
def test_frequencies_refused(bad):
    from compress_kv_write_gb300 import rope_frequencies
    with pytest.raises(ValueError):
        rope_frequencies(**bad)


def _table(L, freq=A, rot=64, first=0, rows=8, amplitude=1.0, table=A):
    return L.kvq_rope_table(freq, rot, first, rows, amplitude, table, None)


@pytest.mark.parametrize("bad,status", [
    (dict(freq=None), 1), (dict(freq=A + 4), 1), (dict(rot=0), 1), (dict(rot=63), 1), (dict(rot=1026), 2), (dict(first=-1), 1),
    (dict(rows=-1), 1), (dict(first=2 ** 31 - 8), 2), (dict(rows=2 ** 31), 2), (dict(amplitude=float("nan")), 1),
    (dict(amplitude=float("inf")), 1), (dict(table=None), 1), (dict(table=A + 8), 1), (dict(rows=0, table=None), 0)])
def test_table_on_the_host(L, bad, status):
    assert _table(L, **bad) == status, bad


def _rope(L, x=A, dtype=1, n=4, heads=8, dim=512, xt=4096, xh=512, start=448, rot=64, flags=0, cs=A, rows=8, pos=A,
          out=A, ot=4096, oh=512, err=None):
    return L.kvq_rope(x, dtype, n, heads, dim, xt, xh, start, rot, flags, cs, rows, pos, out, ot, oh, err, None)


BIG = 1 << 30


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), 1), (dict(n=-1), 1), (dict(heads=0), 1), (dict(dim=1), 1), (dict(rot=0), 1), (dict(rot=7), 1),
    (dict(start=-2), 1), (dict(start=450), 1), (dict(start=0, rot=514), 1), (dict(flags=4), 1), (dict(cs=None), 1),
    (dict(cs=A + 4), 1), (dict(rows=-1), 1), (dict(pos=None), 1), (dict(pos=A + 2), 1), (dict(x=None), 1), (dict(x=A + 1), 1),
    (dict(out=None), 1), (dict(dtype=0, out=A + 2), 1), (dict(xt=-1), 1), (dict(xh=-1), 1), (dict(err=A + 1), 1),
    (dict(dim=1 << 17, rot=64, start=0), 2), (dict(dim=4096, rot=2048, start=0), 2), (dict(heads=1 << 17), 2),
    (dict(out=BIG, ot=512), 1), (dict(out=BIG, oh=256), 1), (dict(out=BIG, ot=600, oh=700), 1),   # rows of out overlap
    (dict(out=A + 16), 1), (dict(ot=8192), 1), (dict(out=A + 1024 * 8), 1),                        # partly x's rows
    (dict(xt=0, xh=0, out=A), 1),
    (dict(n=0, x=None, out=None, pos=None), 0)])
def test_rope_on_the_host(L, bad, status):
    assert _rope(L, **bad) == status, bad


def test_sizes_past_64_bits_are_refused(L):
    assert _table(L, first=2 ** 63 - 1, rows=1) == 2
    assert _table(L, first=2 ** 62, rows=2 ** 62) == 2
    assert _rope(L, n=2 ** 31, xt=2 ** 40, out=BIG, ot=2 ** 40) == 1
    assert _rope(L, n=2, heads=2 ** 16, xt=512, xh=2 ** 60, out=BIG) == 1
