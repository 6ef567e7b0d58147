"""V41 rows at both ends of bf16's range: the scores' scaling and the softmax sums.

A V41 row is decoded relative to its largest scale, a power of two between
2^-47 and 2^113, which goes back into the scores and the weights.  Tolerances
are test_attend_gpu's: they count the roundings of the computation, and hold
whatever the rows' powers are.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from test_attend_gpu import DEV, V41, K, Paged, check, decode, queries, row_power, run_slots, want_slots  # noqa: F401

pytestmark = pytest.mark.gpu


def store(c, x):
    x = x.to(torch.bfloat16)
    assert torch.isfinite(x).all()
    assert O.store(V41, c.pb, 0, x.view(torch.int16).numpy().view(np.uint16), np.arange(c.pages << c.pb), c.pool) == O.OK


def rows(c, seed):
    return torch.randn((c.pages << c.pb, 512), generator=torch.Generator().manual_seed(seed))


def fp32_out(c):
    return torch.full(c.q.shape, float("nan"), device=DEV)


# ------------------------------------------------------- the scores' scaling

@pytest.mark.parametrize("heads,q_len", [(16, 1), (24, 1), (40, 2)])
@pytest.mark.parametrize("row,query", [(90, -90), (104, -104), (112, -112), (118, -118), (-40, 40), (-50, 50), (-38, 110)])
def test_large_rows_and_small_queries(K, heads, q_len, row, query):
    """Rows near 2^row with query rows near 2^query: the scores are moderate, products of partial factors are not."""
    c = Paged(V41, 6, [200, 67, 1], heads, q_len=q_len, seed=37)
    store(c, rows(c, 41) * 2.0 ** row)
    c.q = (queries(3 * q_len, heads, 43).float() * 2.0 ** query).to(torch.bfloat16)
    if row + query:
        c.scale *= 2.0 ** -(row + query)
    out, lse = c.run(K, out=fp32_out(c))
    check(out, lse, c.want(), (row, query))


@pytest.mark.parametrize("row,scale", [(100, -100), (118, -118), (-40, 40), (-40, 80)])
def test_large_and_small_scales(K, row, scale):
    """The same with the factor in `scale`, and queries that make up for the rest."""
    c = Paged(V41, 6, [200, 67, 1], 16, seed=47)
    store(c, rows(c, 53) * 2.0 ** row)
    c.scale *= 2.0 ** scale
    c.q = (queries(3, 16, 59).float() * 2.0 ** -(row + scale)).to(torch.bfloat16)
    out, lse = c.run(K, out=fp32_out(c))
    check(out, lse, c.want(), (row, scale))


@pytest.mark.parametrize("power", [20, 40, 80])
@pytest.mark.parametrize("heads", [16, 64])
def test_huge_scores(K, heads, power):
    """Scores near 2^(25 + power): a row whose only token's score leaves no room for any offset is that token's row, and
    of several tokens the one with the largest score is all that counts."""
    c = Paged(V41, 6, [1, 130], heads, seed=61)
    x = rows(c, 67) * 2.0 ** 20
    first, best = c.slots(0, 1)[0], c.slots(1, 130)[77]
    x[best] = x[best].abs() * 4
    store(c, x)
    c.q = (queries(2, heads, 71).float() * 2.0 ** power).to(torch.bfloat16)
    c.q[1] = c.q[1].abs()
    out, lse = c.run(K, out=fp32_out(c))
    kept = decode(V41, 6, c.pool, [first, best])
    s = np.einsum("thd,td->th", c.q.double().numpy(), kept) * c.scale
    for t in range(2):
        # one weight, rounded to fp16; the row as it is decoded
        tol = (2.0 ** -11 + 2.0 ** -18) * np.abs(kept[t]) + 2.0 ** -25 * row_power(V41, kept[t:t + 1])
        assert (np.abs(out[t].double().cpu().numpy() - kept[t]) <= tol).all()
        assert (np.abs(lse[t].double().cpu().numpy() - s[t]) <= 2.0 ** -12 * np.abs(s[t])).all()


# ------------------------------------------------------- sums over rows of very different powers

@pytest.mark.parametrize("heads,q_len", [(16, 1), (32, 1), (40, 2)])
@pytest.mark.parametrize("low,high", [(0, 116), (-40, 100), (-38, 118), (-60, 110)])
@pytest.mark.parametrize("order", ["first", "last", "alone"])
def test_equal_weights_of_unequal_rows(K, heads, q_len, low, high, order):
    """Zero queries weigh every visible token alike, so lse is log n and the
    large rows' share of the output is 1 / n each, wherever they stand: in a
    tile's first block, in its last, or one among many."""
    lens = [500, 130, 64]
    c = Paged(V41, 6, lens, heads, q_len=q_len, seed=73)
    x = rows(c, 79)
    s = torch.full((c.pages * 64, 1), 2.0 ** low)
    for i, n in enumerate(lens):
        at = c.slots(i, n - q_len + 1 if order == "last" else n)
        s[{"first": at[:40], "last": at[-30:], "alone": at[n // 2:n // 2 + 1]}[order]] = 2.0 ** high
    store(c, x * s)
    c.q[:] = 0
    out, lse = c.run(K, out=fp32_out(c))
    check(out, lse, c.want(), (low, high, order))


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("big_at", [[3], [20000], [9000, 20990]])
def test_joined_parts_of_unequal_rows(K, heads, big_at):
    """The same where a tile is split over CTAs: the parts' maxima differ by more than fp32 holds."""
    c = Paged(V41, 6, [21001], heads, seed=83)
    x = rows(c, 89) * 2.0 ** -36
    big = c.slots(0, 21001)[big_at]
    x[big] = rows(c, 91)[big] * 2.0 ** 114
    store(c, x)
    c.q[:, ::2] = 0
    c.q[:, 1::2] = (c.q[:, 1::2].float() * 2.0 ** -112).to(torch.bfloat16)
    out, lse = c.run(K, out=fp32_out(c))
    check(out, lse, c.want(), big_at)
    assert abs(lse[0, 0].item() - math.log(21001)) < 1e-5


def test_by_slots(K):
    c = Paged(V41, 6, [512], 24, seed=97)
    x = rows(c, 101)
    x[::7] *= 2.0 ** 114
    x[3::11] *= 2.0 ** -50
    store(c, x)
    q = torch.zeros((3, 24, 512), dtype=torch.bfloat16)
    q[1, ::2] = (queries(1, 12, 103)[0].float() * 2.0 ** -115).to(torch.bfloat16)
    g = torch.Generator().manual_seed(107)
    s = torch.randint(0, 512, (3, 700), generator=g, dtype=torch.int32)
    out, lse = run_slots(K, V41, 6, c.pool, c.pages * 64, q, s, out=torch.empty(q.shape, device=DEV))
    check(out, lse, want_slots(V41, 6, c.pool, c.pages * 64, q, s), "slots")
