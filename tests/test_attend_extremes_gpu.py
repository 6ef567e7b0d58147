"""The largest and smallest calls that the attention takes: 2^30 cached tokens (by a table and by a list that repeat a few
pages), a million sequences, 1,024 heads, a table without columns."""
import math

import numpy as np
import pytest
import torch

from test_attend_gpu import DEV, FP4, V41, K, decode, make_pool, row_power  # noqa: F401

pytestmark = pytest.mark.gpu
PAGES = 8


def mean_of(K, layout, heads, n, many, slots):
    """The call with a scale of 0 over n tokens a sequence, the pool's slots in turn: (out, lse, mean, its tolerance).  Equal
    weights are exact; a CTA adds sums of 256 blocks (2^-14 of them at most, see test_attend_tail_gpu) to nearest, less
    than 2^9 times."""
    pool = make_pool(layout, 6, PAGES * 64, 5)
    rows = decode(layout, 6, pool, np.arange(PAGES * 64))
    q = torch.ones((1, 1, 512), dtype=torch.bfloat16, device=DEV).expand(many, heads, 512)
    out, lse = torch.full((many, heads, 512), float("nan"), device=DEV), torch.full((many, heads), float("nan"), device=DEV)
    ws = torch.empty(K.attend_workspace(heads), dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pool_d = torch.from_numpy(pool).to(DEV)
    if slots:
        s = torch.arange(n, dtype=torch.int32, device=DEV) % (PAGES * 64)
        K.kvq_attend_slots(layout, 6, q, pool_d, PAGES * 64, s.expand(many, n), out, ws, scale=0.0, lse=lse, err=err)
    else:
        table = (torch.arange(-(-n // 64), dtype=torch.int32, device=DEV) % PAGES)[None]
        K.kvq_attend(layout, 6, q, pool_d, PAGES, table, torch.full((many,), n, dtype=torch.int32, device=DEV), out, ws,
                     scale=0.0, req=torch.zeros(many, dtype=torch.int32, device=DEV), lse=lse, err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    seen = rows[:min(n, rows.shape[0])]
    assert n % rows.shape[0] == 0 or n <= rows.shape[0]
    tol = (2.0 ** -14 + 2.0 ** -15) * np.abs(seen).mean(0) + (2.0 ** -25 * row_power(layout, seen).mean() if layout == V41 else 0)
    return out, lse, torch.from_numpy(seen.mean(0)).to(DEV), torch.from_numpy(np.broadcast_to(tol, (512,)).copy()).to(DEV)


@pytest.mark.parametrize("layout,heads,n,many,slots", [
    (V41, 16, 1 << 30, 1, False), (FP4, 64, 1 << 30, 1, False), (V41, 24, 1 << 30, 1, True),
    (FP4, 1, 64, 1 << 20, False), (V41, 3, 7, 1 << 18, True), (FP4, 1024, 512, 3, False), (V41, 1, 1, 1, False),
])
def test_means(K, layout, heads, n, many, slots):
    out, lse, want, tol = mean_of(K, layout, heads, n, many, slots)
    for i in range(0, many, 1 << 16):
        assert ((out[i:i + (1 << 16)].double() - want).abs() <= tol).all()
    assert (lse.double() - math.log(n)).abs().max() <= 2.0 ** -18


@pytest.mark.parametrize("rows,n", [(2, 2), (5, 2), (0, 0)])
def test_a_table_without_columns(K, rows, n):
    """No sequence can hold a token, so all are empty; one that claims to is reported."""
    pool = torch.zeros(64 * 528, dtype=torch.uint8, device=DEV)
    out, lse = torch.full((n, 16, 512), 3.0, device=DEV), torch.full((n, 16), 3.0, device=DEV)
    ws, err = torch.empty(K.attend_workspace(16), dtype=torch.uint8, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    for lens, bit in (([0] * n, 0), ([1] * n, 64 if n else 0)):
        K.kvq_attend(V41, 6, torch.ones((n, 16, 512), dtype=torch.bfloat16, device=DEV), pool, 1,
                     torch.zeros((rows, 0), dtype=torch.int32, device=DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                     out, ws, scale=1.0, lse=lse, err=err)
        torch.cuda.synchronize()
        assert (out == 0).all() and torch.isneginf(lse).all() and err.item() == bit
