"""kvq_evict_select and kvq_evict_move without a GPU: the calls that the host refuses."""
import pytest

A = 0x10000          # a 16-byte aligned fake device address (never dereferenced)
B = 1 << 40


@pytest.fixture(scope="module")
def L():
    from compress_kv_write_gb300 import build
    build.build()
    from compress_kv_write_gb300 import kvq
    return kvq.lib()


def _select(L, mass=A, mrows=4, width=100, mstride=100, rows=None, kv_len=A, n_seq=4, keep=10, first=2, last=3, kept=A,
            kstride=10, count=A, err=None):
    return L.kvq_evict_select(mass, mrows, width, mstride, rows, kv_len, n_seq, keep, first, last, kept, kstride, count, err, None)


@pytest.mark.parametrize("bad,status", [
    (dict(mass=None), 1), (dict(mass=A + 2), 1), (dict(mrows=-1), 1), (dict(mrows=3), 1), (dict(width=-1), 1),
    (dict(mstride=99), 1), (dict(rows=A + 1), 1), (dict(kv_len=None), 1), (dict(kv_len=A + 2), 1), (dict(n_seq=-1), 1),
    (dict(keep=0), 1), (dict(first=-1), 1), (dict(last=-1), 1), (dict(first=8), 1), (dict(first=11, last=0), 1),
    (dict(kept=None), 1), (dict(kept=A + 2), 1), (dict(kstride=9), 1), (dict(count=None), 1), (dict(count=A + 2), 1),
    (dict(err=A + 1), 1), (dict(width=2 ** 30 + 1, mstride=2 ** 31), 2), (dict(keep=2 ** 30 + 1, kstride=2 ** 31), 2),
    (dict(n_seq=2 ** 20 + 1, mrows=2 ** 21), 2), (dict(n_seq=0, mass=None, kv_len=None, kept=None, count=None), 0)])
def test_select_on_the_host(L, bad, status):
    assert _select(L, **bad) == status, bad


def _move(L, layout=1, pb=6, pool=A, pages=8, table=A, trows=4, width=3, stride=3, req=None, new=A, nwidth=1, nstride=1,
          kept=A, n_seq=4, keep=10, kstride=10, mass=None, mrows=0, mwidth=0, mstride=0, rows=None, out=None, ostride=0,
          err=None):
    return L.kvq_evict_move(layout, pb, pool, pages, table, trows, width, stride, req, new, nwidth, nstride, kept, n_seq,
                            keep, kstride, mass, mrows, mwidth, mstride, rows, out, ostride, err, None)


M = dict(mass=A, mrows=4, mwidth=192, mstride=192, out=B, ostride=10)


@pytest.mark.parametrize("bad,status", [
    (dict(layout=0), 1), (dict(layout=3), 1), (dict(pb=5), 2), (dict(pb=0), 1), (dict(pool=None), 1), (dict(pool=A + 8), 1),
    (dict(pages=0), 1), (dict(table=None), 1), (dict(table=A + 2), 1), (dict(trows=3), 1), (dict(trows=-1), 1),
    (dict(width=-1), 1), (dict(stride=2), 1), (dict(req=A + 1), 1), (dict(new=None), 1), (dict(new=A + 1), 1),
    (dict(nwidth=0), 1), (dict(keep=65, kstride=65), 1), (dict(nwidth=2, nstride=1), 1), (dict(kept=None), 1),
    (dict(kept=A + 2), 1), (dict(n_seq=-1), 1), (dict(keep=0), 1), (dict(kstride=9), 1), (dict(err=A + 2), 1),
    (dict(mass=A), 1), (dict(out=A), 1), (dict(rows=A), 1), (M | dict(mass=A + 2), 1), (M | dict(out=B + 2), 1),
    (M | dict(mrows=3), 1), (M | dict(mstride=191), 1), (M | dict(ostride=9), 1), (M | dict(rows=A + 2), 1),
    (M | dict(out=A + 64), 1), (dict(width=2 ** 24 + 1, stride=2 ** 25), 2),
    (dict(n_seq=2 ** 20 + 1, trows=2 ** 21), 2), (dict(n_seq=0, table=None, trows=0, new=None, kept=None), 0)])
def test_move_on_the_host(L, bad, status):
    assert _move(L, **bad) == status, bad
