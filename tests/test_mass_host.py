"""kvq_attend_mass without a GPU: the calls that the host refuses, and the workspace."""
import pytest

A = 0x10000          # a 16-byte aligned fake device address (never dereferenced)
B = 1 << 40
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    from compress_kv_write_gb300 import build
    build.build()
    from compress_kv_write_gb300 import kvq
    return kvq.lib()


def test_workspace(L):
    for bad in ((0, 200, 10), (4, 0, 10), (4, 200, 0), (-1, 200, 10)):
        assert L.kvq_mass_workspace(*bad) == 0
    assert all(L.kvq_mass_workspace(4, r, 1000) == 0 for r in (1, 64, 128))
    assert L.kvq_mass_workspace(4, 129, 1000) == 4 * 2 * 1000 * 4
    assert L.kvq_mass_workspace(3, 2048, 1001) == 3 * 16 * 1004 * 4


def _mass(L, layout=1, pb=6, q=A, q_tok=8192, q_head=512, n_seq=4, q_len=1, heads=16, lse=A, pool=A, pages=8, table=A, trows=4,
          width=2, stride=2, req=None, kv_len=A, mask=None, scale=0.04, mass=A, mrows=4, mwidth=128, mstride=128, rows=None, prev=None,
          pstride=0, decay=1.0, ws=None, ws_bytes=0, err=None):
    return L.kvq_attend_mass(layout, pb, q, q_tok, q_head, n_seq, q_len, heads, lse, pool, pages, table, trows, width, stride,
                             req, kv_len, mask, scale, mass, mrows, mwidth, mstride, rows, prev, pstride, decay, ws, ws_bytes, err, None)


@pytest.mark.parametrize("bad,status", [
    (dict(layout=0), 1), (dict(layout=3), 1), (dict(pb=0), 1), (dict(pb=17), 1), (dict(pb=5), 2), (dict(q=None), 1),
    (dict(q=A + 8), 1), (dict(q_tok=-8), 1), (dict(q_tok=516), 1), (dict(q_head=4), 1), (dict(n_seq=-1), 1), (dict(q_len=0), 1),
    (dict(heads=0), 1), (dict(heads=1025), 2), (dict(n_seq=65536, trows=65536, mrows=65536), 2),
    (dict(n_seq=1 << 12, q_len=1 << 13), 2), (dict(mask=A + 4), 1), (dict(mask=A, q_len=1025), 2), (dict(lse=None), 1), (dict(lse=A + 2), 1), (dict(pool=None), 1), (dict(pool=A + 4), 1),
    (dict(pages=0), 1), (dict(table=None), 1), (dict(table=A + 2), 1), (dict(trows=-1), 1), (dict(trows=3), 1), (dict(width=-1), 1),
    (dict(stride=1), 1), (dict(req=A + 1), 1), (dict(kv_len=None), 1), (dict(kv_len=A + 2), 1), (dict(scale=NAN), 1),
    (dict(scale=INF), 1), (dict(mass=None), 1), (dict(mass=A + 2), 1), (dict(mrows=3), 1), (dict(mrows=-1), 1), (dict(mwidth=-1), 1),
    (dict(mstride=127), 1), (dict(rows=A + 2), 1), (dict(prev=B + 2, pstride=128), 1), (dict(prev=B, pstride=127), 1),
    (dict(prev=A + 64, pstride=128), 1), (dict(prev=A, pstride=256), 1), (dict(prev=B, pstride=128, decay=NAN), 1),
    (dict(prev=B, pstride=128, decay=INF), 1), (dict(heads=129), 1), (dict(heads=129, ws=A + 8, ws_bytes=1 << 20), 1),
    (dict(heads=129, ws=A, ws_bytes=4 * 2 * 128 * 4 - 1), 1), (dict(err=A + 2), 1),
    (dict(n_seq=0, q=None, lse=None, kv_len=None, mass=None, table=None), 0)])
def test_mass_on_the_host(L, bad, status):
    assert _mass(L, **bad) == status, bad
