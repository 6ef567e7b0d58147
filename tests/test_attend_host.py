"""kvq_attend, kvq_attend_slots and kvq_norm_quant without a GPU: the calls
that are refused on the host, and the sizes (no call here reaches a launch)."""
import pytest

A = 0x10000          # a 16-byte aligned fake device address (never dereferenced)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    from compress_kv_write_gb300 import build
    build.build()
    from compress_kv_write_gb300 import kvq
    return kvq.lib()


def test_workspace_size(L):
    assert L.kvq_attend_workspace(0) == 0 and L.kvq_attend_workspace(-3) == 0
    sizes = [L.kvq_attend_workspace(r) for r in (1, 16, 17, 64, 65, 4096)]
    assert all(s > 0 and s % 16 == 0 for s in sizes)
    assert sizes == sorted(sizes) and sizes[3] == sizes[5]     # bounded, whatever the number of rows
    assert sizes[-1] < 64 << 20


def _attend(L, layout=1, page_bits=6, q=A, q_tok=8192, q_head=512, n_seq=4, q_len=1, heads=16, pool=A, pages=8,
            table=A, rows=4, width=2, stride=2, req=None, kv_len=A, scale=0.04, out=A, out_dtype=1, out_tok=8192,
            out_head=512, lse=None, ws=A, ws_bytes=None, err=None):
    if ws_bytes is None:
        ws_bytes = L.kvq_attend_workspace(max(q_len * heads, 1))
    return L.kvq_attend(layout, page_bits, q, q_tok, q_head, n_seq, q_len, heads, pool, pages, table, rows, width,
                        stride, req, kv_len, scale, out, out_dtype, out_tok, out_head, lse, ws, ws_bytes, err, None)


@pytest.mark.parametrize("bad", [
    dict(layout=0), dict(layout=3), dict(page_bits=0), dict(page_bits=17), dict(n_seq=-1), dict(q_len=0),
    dict(heads=0), dict(q=None), dict(q=A + 8), dict(q_tok=-8), dict(q_tok=516), dict(q_head=4), dict(pool=None),
    dict(pool=A + 4), dict(pages=0), dict(table=None), dict(table=A + 2), dict(rows=-1), dict(width=-1),
    dict(stride=1), dict(rows=3), dict(req=A + 1), dict(kv_len=None), dict(kv_len=A + 2), dict(scale=NAN),
    dict(scale=INF), dict(scale=-INF), dict(out=None), dict(out=A + 8), dict(out_dtype=2), dict(out_tok=504),
    dict(out_tok=8196), dict(out_head=256), dict(out_head=516), dict(lse=A + 2), dict(ws=None), dict(ws=A + 8),
    dict(err=A + 2), dict(out_tok=512), dict(out_tok=7680), dict(out_tok=512, out_head=1536),
])
def test_attend_rejects_on_host(L, bad):
    assert _attend(L, **bad) == 1, bad


def test_attend_rejects_small_workspace(L):
    need = L.kvq_attend_workspace(16)
    assert _attend(L, ws_bytes=need - 1) == 1
    assert _attend(L, ws_bytes=0) == 1


def test_attend_unsupported_and_empty(L):
    assert _attend(L, page_bits=5) == 2
    assert _attend(L, heads=1025) == 2
    assert _attend(L, n_seq=1 << 24, q_len=2) == 2
    assert _attend(L, n_seq=0, q=None, out=None, kv_len=None, table=None, rows=0, ws=None) == 0
    assert _attend(L, n_seq=0, scale=NAN) == 1            # a bad value is refused in an empty call too


def _slots(L, layout=2, page_bits=6, q=A, q_tok=8192, q_head=512, n=4, heads=16, pool=A, slots_n=128, slots=A, dt=0,
           n_sel=32, stride=32, scale=0.04, out=A, out_dtype=1, out_tok=8192, out_head=512, lse=None, ws=A,
           ws_bytes=None, err=None):
    if ws_bytes is None:
        ws_bytes = L.kvq_attend_workspace(heads)
    return L.kvq_attend_slots(layout, page_bits, q, q_tok, q_head, n, heads, pool, slots_n, slots, dt, n_sel, stride,
                              scale, out, out_dtype, out_tok, out_head, lse, ws, ws_bytes, err, None)


@pytest.mark.parametrize("bad", [
    dict(layout=7), dict(page_bits=-1), dict(q=None), dict(q_head=511), dict(n=-1), dict(heads=0), dict(pool=A + 1),
    dict(slots_n=0), dict(slots_n=100), dict(slots=None), dict(slots=A + 2), dict(slots=A + 4, dt=1), dict(dt=2),
    dict(n_sel=-1), dict(n_sel=0x7FFFFFFF), dict(n_sel=(1 << 30) + 1, stride=1 << 31), dict(stride=-1), dict(scale=NAN), dict(out=A + 2), dict(out_dtype=-1),
    dict(out_head=510), dict(ws=None), dict(ws_bytes=8), dict(lse=A + 1), dict(err=A + 3),
])
def test_attend_slots_rejects_on_host(L, bad):
    assert _slots(L, **bad) == 1, bad


def test_attend_slots_unsupported_and_empty(L):
    assert _slots(L, page_bits=7) == 2
    assert _slots(L, n=0, q=None, out=None, slots=None, ws=None) == 0


def _norm(L, x=A, dt=1, n=4, dim=512, xs=512, res=A, rs=512, ro=A, ros=512, w=A, eps=1e-6, codes=A, cs=512, scales=A,
          ss=16):
    return L.kvq_norm_quant(x, dt, n, dim, xs, res, rs, ro, ros, w, eps, codes, cs, scales, ss, None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x=A + 8), dict(dt=2), dict(n=-1), dict(dim=0), dict(dim=48), dict(dim=-32), dict(xs=511),
    dict(xs=516), dict(res=None), dict(ro=None), dict(res=A + 8), dict(rs=256), dict(ros=500), dict(w=None),
    dict(w=A + 4), dict(eps=-1.0), dict(eps=NAN), dict(codes=None), dict(codes=A + 4), dict(cs=508), dict(cs=516),
    dict(scales=None), dict(ss=15),
])
def test_norm_quant_rejects_on_host(L, bad):
    assert _norm(L, **bad) == 1, bad


def test_norm_quant_unsupported_and_empty(L):
    assert _norm(L, dim=16416, xs=16416) == 2
    assert _norm(L, n=0, x=None, res=None, ro=None, w=None, codes=None, scales=None) == 0
