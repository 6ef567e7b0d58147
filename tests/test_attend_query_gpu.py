"""Query rows that are not finite: their scores are infinite or NaN over every
token, so the softmax, and with it the row, is NaN wherever they see one, and a
zero row with lse = -inf, as any other, where they see none."""
import pytest
import torch

import numpy as np
import oracle as O
from test_attend_gpu import DEV, FP4, V41, K, Paged, check  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("heads,q_len,lens", [(16, 1, [1, 0, 130]), (33, 1, [64, 700]), (8, 3, [2, 70]), (64, 1, [9000, 1])])
def test_rows_are_nan_alone(K, layout, value, heads, q_len, lens):
    """Dim 7 of every cached row is negative, so one infinite value there makes all scores of a row -inf or +inf."""
    c = Paged(layout, 6, lens, heads, q_len, seed=heads)
    x = torch.randn((c.pages * 64, 512), generator=torch.Generator().manual_seed(3))
    x[:, 7] = -x[:, 7].abs() - 0.5
    x = x.to(torch.bfloat16)
    assert O.store(layout, 6, 0, x.view(torch.int16).numpy().view(np.uint16), np.arange(c.pages * 64), c.pool) == O.OK
    want = c.want()
    bad = [(t, h) for t in range(len(lens) * q_len) for h in range(t % 3, heads, 5)]
    q = c.q.clone()
    for t, h in bad:
        q[t, h, 7] = value
    out, lse = c.run(K, q=q.to(DEV))
    for t, h in bad:
        i, j = divmod(t, q_len)
        if lens[i] - (q_len - 1 - j) > 0:
            assert torch.isnan(out[t, h]).all() and torch.isnan(lse[t, h]), (t, h)
        else:
            assert (out[t, h] == 0).all() and lse[t, h] == float("-inf"), (t, h)
        out[t, h], lse[t, h] = 0, 0
        for a in want[t]:
            a[h] = 0
    check(out, lse, want, "the other rows")
