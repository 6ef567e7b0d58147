"""Attention calls whose waits give up: the call ends, reports KVQ_DEVERR_WAIT, and the next one is right.

With a limit of 0 every wait inside the kernel ends at once, as if its time had
run out: the warps run through their loops over whatever their buffers hold, all
at addresses that do not depend on data, wait for the products they issued and
return.  What the call should have written is NaN then, so that a caller without
an error word sees it too.
"""
import contextlib

import pytest
import torch

from test_attend_gpu import DEV, FP4, V41, K, Paged, check, make_pool, queries, run_slots, want_slots  # noqa: F401

pytestmark = pytest.mark.gpu
DEVERR_WAIT = 16


@contextlib.contextmanager
def no_waiting(K):
    before = K.attend_wait_limit(0)
    try:
        yield
    finally:
        K.attend_wait_limit(before)


CASES = [(16, 1, [70]), (5, 1, [1, 0, 64]), (32, 1, [5000, 3]), (64, 1, [700, 64, 9000]), (40, 2, [130, 0, 2000])]


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads,q_len,lens", CASES)
def test_reported_and_the_next_call_is_right(K, layout, heads, q_len, lens):
    c = Paged(layout, 6, lens, heads, q_len, seed=heads)
    ws = torch.empty(K.attend_workspace(q_len * heads), dtype=torch.uint8, device=DEV)
    want = c.want()
    for _ in range(3):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        with no_waiting(K):
            c.run(K, err=err, ws=ws)
        assert err.item() == DEVERR_WAIT
        err.zero_()
        out, lse = c.run(K, err=err, ws=ws)
        assert err.item() == 0
        check(out, lse, want, "after a call that gave up")


@pytest.mark.parametrize("layout", [V41, FP4])
def test_by_slots(K, layout):
    pool = make_pool(layout, 6, 512, 3)
    q, s = queries(7, 24, 5), torch.arange(7 * 300, dtype=torch.int32).view(7, 300) % 512
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    with no_waiting(K):
        run_slots(K, layout, 6, pool, 512, q, s, err=err)
    assert err.item() == DEVERR_WAIT
    err.zero_()
    out, lse = run_slots(K, layout, 6, pool, 512, q, s, err=err)
    assert err.item() == 0
    check(out, lse, want_slots(layout, 6, pool, 512, q, s), "after a call that gave up")


def test_other_bits_stay_beside_it(K):
    """A bad length is reported with the wait, and behind the batch nothing is written."""
    c = Paged(V41, 6, [70, 90], 16, seed=3)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    big = torch.full((4, 16, 512), 3.0, dtype=torch.bfloat16, device=DEV)
    with no_waiting(K):
        c.run(K, out=big[:2], kv_len=torch.tensor([70, -1], dtype=torch.int32, device=DEV), err=err)
    assert err.item() == DEVERR_WAIT + 64
    assert (big[2:] == 3).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads,q_len,lens", CASES)
def test_rows_are_nan(K, layout, dtype, heads, q_len, lens):
    """Whole tiles, tiles that are joined, empty sequences: all of q's rows, and nothing behind them."""
    c = Paged(layout, 6, lens, heads, q_len, seed=heads)
    n = len(lens) * q_len
    big = torch.full((n + 1, heads + 1, 520), 3.0, dtype=dtype, device=DEV)
    with no_waiting(K):
        out, lse = c.run(K, out=big[:n, :heads, :512])
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    big[:n, :heads, :512] = 3
    assert (big == 3).all()


@pytest.mark.parametrize("layout", [V41, FP4])
def test_rows_by_slots_are_nan(K, layout):
    pool = make_pool(layout, 6, 512, 3)
    s = torch.arange(300 * 300, dtype=torch.int32).view(300, 300) % 512
    s[7] = -1
    with no_waiting(K):
        out, lse = run_slots(K, layout, 6, pool, 512, queries(300, 24, 5), s, out=torch.zeros((300, 24, 512), device=DEV))
    assert torch.isnan(out).all() and torch.isnan(lse).all()
