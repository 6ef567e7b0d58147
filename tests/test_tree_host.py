"""kvq_tree_mask and kvq_attend_tree without a GPU: the calls that the host refuses."""
import pytest

A = 0x10000          # a 16-byte aligned fake device address (never dereferenced)


@pytest.fixture(scope="module")
def L():
    from compress_kv_write_gb300 import build
    build.build()
    from compress_kv_write_gb300 import kvq
    return kvq.lib()


def _mask(L, parent=A, n=4, q_len=9, stride=9, kv_len=A, mask=A, pos=A, err=None):
    return L.kvq_tree_mask(parent, n, q_len, stride, kv_len, mask, pos, err, None)


@pytest.mark.parametrize("bad,status", [
    (dict(parent=None), 1), (dict(parent=A + 2), 1), (dict(n=-1), 1), (dict(q_len=0), 1), (dict(q_len=1025, stride=1025), 2),
    (dict(stride=8), 1), (dict(kv_len=A + 2), 1), (dict(mask=None), 1), (dict(mask=A + 4), 1), (dict(pos=A + 2), 1),
    (dict(err=A + 1), 1), (dict(n=(1 << 24) + 1), 2), (dict(n=0, parent=None, mask=None), 0)])
def test_mask_on_the_host(L, bad, status):
    assert _mask(L, **bad) == status, bad


def _tree(L, layout=1, page_bits=6, q=A, q_tok=8192, q_head=512, n_seq=4, q_len=3, heads=16, pool=A, pages=8,
          table=A, rows=4, width=2, stride=2, req=None, kv_len=A, mask=A, scale=0.04, out=A, out_dtype=1, out_tok=8192,
          out_head=512, lse=None, ws=A, ws_bytes=None, err=None):
    if ws_bytes is None:
        ws_bytes = L.kvq_attend_workspace(max(q_len * heads, 1))
    return L.kvq_attend_tree(layout, page_bits, q, q_tok, q_head, n_seq, q_len, heads, pool, pages, table, rows, width,
                             stride, req, kv_len, mask, scale, out, out_dtype, out_tok, out_head, lse, ws, ws_bytes, err, None)


@pytest.mark.parametrize("bad,status", [
    (dict(mask=None), 1), (dict(mask=A + 4), 1), (dict(q_len=1025), 2), (dict(layout=3), 1), (dict(page_bits=5), 2),
    (dict(q=None), 1), (dict(q_tok=516), 1), (dict(pool=None), 1), (dict(table=None), 1), (dict(rows=3), 1),
    (dict(kv_len=None), 1), (dict(scale=float("nan")), 1), (dict(out_tok=512), 1), (dict(ws=None), 1), (dict(ws_bytes=100), 1),
    (dict(heads=1025), 2), (dict(err=A + 2), 1), (dict(n_seq=0, q=None, out=None, mask=None, kv_len=None, ws=None), 0)])
def test_tree_on_the_host(L, bad, status):
    assert _tree(L, **bad) == status, bad
