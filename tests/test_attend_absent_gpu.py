"""What the pool's first row holds does not reach the rows that do not see it.

The kernels read that row in the place of a token that is not there (behind a
length, padding of a list, a bad page or slot), so it may hold anything: codes
and scales that are NaN, or scales that fp16 cannot hold.  Results are compared
with the same call's over a pool whose first row is an ordinary one, bit by bit.
"""
import numpy as np
import pytest
import torch

import oracle as O
from test_attend_gpu import DEV, FP4, V41, K, Paged, check, make_pool, queries, run_slots, want_slots  # noqa: F401

pytestmark = pytest.mark.gpu

# (layout, code byte, scale byte): NaN codes and scales; V41 scales of 2^15 (above fp16's largest after the factor 2) to
# 2^127 over ordinary codes; FP4's NaN scale as kvq_store writes it
ROWS = [(V41, 0xFF, 0xFF), (V41, 0x38, 0xFF), (V41, 0x38, 142), (V41, 0x7E, 200), (V41, 0x38, 254), (V41, 0x7F, 127),
        (FP4, 0xFF, 0xFF), (FP4, 0x22, 0x7F), (FP4, 0x77, 0x7E)]


def first_row(layout, page_bits, pool, code, scale):
    cb, used = (512, 16) if layout == V41 else (256, 16)
    pool[:cb] = code
    pool[(cb << page_bits):(cb << page_bits) + used] = scale


def without_page_0(c):
    """Moves what page 0 holds, so that no sequence has it."""
    used = {int(p) for i, n in enumerate(c.lens) for p in c.table[i][:-(-n // (1 << c.pb))]}
    free = next(p for p in range(c.pages) if p not in used)
    pool = c.pool.reshape(c.pages, -1)
    pool[free] = pool[0]
    c.table[c.table == 0] = free
    return c


@pytest.mark.parametrize("layout,code,scale", ROWS)
@pytest.mark.parametrize("heads,q_len,lens,pb", [
    (16, 1, [70, 0, 1, 129], 6),
    (33, 1, [63, 64, 100], 4),
    (64, 1, [300, 3], 2),
    (16, 3, [2, 70, 129], 6),
    (8, 1, [20000, 40, 90], 6),         # split over CTAs and joined
])
def test_paged(K, layout, code, scale, heads, q_len, lens, pb):
    c = without_page_0(Paged(layout, pb, lens, heads, q_len, seed=heads + q_len))
    clean, lse = c.run(K)
    first_row(layout, pb, c.pool, code, scale)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got, lse2 = c.run(K, err=err)
    assert err.item() == 0
    assert torch.equal(got, clean) and torch.equal(lse2, lse)
    check(got, lse2, c.want(), "beside the first row")


@pytest.mark.parametrize("layout,code,scale", ROWS)
def test_bad_pages_and_table_rows(K, layout, code, scale):
    c = without_page_0(Paged(layout, 6, [200, 90, 100], 16, seed=3))
    table = torch.from_numpy(c.table.copy())
    table[0, 1], table[1, 0] = c.pages, -1
    req = torch.tensor([0, 1, 7], dtype=torch.int32, device=DEV)
    clean, lse = c.run(K, table=table.to(DEV), req=req)
    first_row(layout, 6, c.pool, code, scale)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got, lse2 = c.run(K, table=table.to(DEV), req=req, err=err)
    assert err.item() == 4 + 32
    assert torch.equal(got, clean) and torch.equal(lse2, lse) and torch.isfinite(got).all()
    assert (got[2] == 0).all() and torch.isneginf(lse2[2]).all()


@pytest.mark.parametrize("layout,code,scale", ROWS)
@pytest.mark.parametrize("heads,n_sel", [(16, 100), (32, 129), (64, 40), (64, 2000)])
def test_slots(K, layout, code, scale, heads, n_sel):
    """Padding, a list of padding alone, a bad slot, and a width that is no multiple of 64."""
    slots_n = 512
    pool = make_pool(layout, 6, slots_n, 5)
    rng = np.random.default_rng(n_sel)
    s = torch.from_numpy(rng.integers(1, slots_n, (4, n_sel))).to(torch.int32)
    s[torch.from_numpy(rng.random(s.shape) < 0.2)] = -1
    s[1] = -1
    s[2, 5] = slots_n
    q = queries(4, heads, 7)
    clean, lse = run_slots(K, layout, 6, pool, slots_n, q, s)
    first_row(layout, 6, pool, code, scale)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got, lse2 = run_slots(K, layout, 6, pool, slots_n, q, s, err=err)
    assert err.item() == 1
    assert torch.equal(got, clean) and torch.equal(lse2, lse)
    check(got, lse2, want_slots(layout, 6, pool, slots_n, q, s), "beside slot 0")


@pytest.mark.parametrize("layout", [V41, FP4])
def test_a_row_that_is_not_a_number_as_the_store_writes_it(K, layout):
    """kvq_store of a NaN row to slot 0 of the pool, which is no sequence's: every other row attends as before."""
    c = without_page_0(Paged(layout, 6, [130, 65, 1], 16, seed=9))
    clean, lse = c.run(K)
    pool = torch.from_numpy(c.pool).to(DEV)
    x = torch.full((1, 512), float("nan"), dtype=torch.bfloat16, device=DEV)
    K.kvq_store(layout, 6, 0, x, torch.zeros(1, dtype=torch.int64, device=DEV), pool, c.pages * 64)
    torch.cuda.synchronize()
    c.pool = pool.cpu().numpy()
    assert O.bytes_per_token(layout) * 64 * c.pages == c.pool.size
    got, lse2 = c.run(K)
    assert torch.equal(got, clean) and torch.equal(lse2, lse)
