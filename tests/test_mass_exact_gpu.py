"""kvq_attend_mass where the scores' products sum exactly, so that a weight is off by its exponent's own roundings alone.

A row has two dims that a query sees, of power-of-two and 6 * power-of-two values, and a query two that are not zero: a score
s is two products whose sum has no more than 24 bits, and lse is one of the scores.  exp(s - lse) is off by
* 2^-23 |s - lse| in the exponent: log2(e) scale and log2(e) lse rounded to fp32 (2^-24 of s and of lse; their difference is
  what is left once both are made up for), and the sum of the two products rounded (2^-24 of it);
* 2^-20 relative: two hardware exponentials of 2^-22 and their product, and the sum over the heads.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from test_attend_gpu import DEV, FP4, V41, K, decode  # noqa: F401
from test_mass_gpu import Mass, check

pytestmark = pytest.mark.gpu
SMALL = [0.0, 1.5, -3.0, 6.0, -12.0, -0.75, 0.375]   # dim 40 of the tokens: 6 * 2^j


def pool_of(layout, large, small):
    """numpy pool, one slot a token: dim 5 holds large[t] (a power of two), dim 6, which no query sees, 1.5 of it (6 * 2^j, so
    that a V41_FP4 block's scale is exact), dim 40, in a block of its own, small[t]."""
    n = -(-len(large) // 64) * 64
    x = torch.zeros((n, 512))
    x[:len(large), 5] = torch.tensor(large)
    x[:len(large), 6] = 1.5 * x[:len(large), 5].abs()
    x[:len(large), 40] = torch.tensor(small)
    pool = np.zeros(n * O.bytes_per_token(layout), np.uint8)
    assert O.store(layout, 6, 0, x.to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16), np.arange(n), pool) == O.OK
    rows = decode(layout, 6, pool, np.arange(len(large)))
    assert (rows == x[:len(large)].double().numpy()).all()      # nothing was rounded
    return pool, rows


def run(K, layout, pool, n, q, lse, scale):
    mass = torch.full((1, n + 1), -7.0, device=DEV)
    K.kvq_attend_mass(layout, 6, q.to(DEV), lse.to(DEV), torch.from_numpy(pool).to(DEV), -(-n // 64),
                      torch.arange(-(-n // 64), dtype=torch.int32, device=DEV)[None], torch.tensor([n], dtype=torch.int32, device=DEV),
                      mass, scale=scale)
    assert mass[0, n] == -7
    return mass[0, :n].cpu().double().numpy()


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads", [1, 16, 20, 64, 128])
@pytest.mark.parametrize("scale", [1.0, 0.7, 512 ** -0.5, -0.3])
@pytest.mark.parametrize("power", [0, 3, 5, 9, 12])
def test_exponent(K, layout, heads, scale, power):
    scale = float(np.float32(scale))
    small = [SMALL[t % len(SMALL)] for t in range(150)]
    large = [32.0] * 150
    pool, rows = pool_of(layout, large, small)
    q = torch.zeros((1, heads, 512))
    q[0, :, 5] = torch.tensor([2.0 ** max(power - h % 4, 0) for h in range(heads)])
    q[0, :, 40] = 1.0
    s = q[0].double().numpy() @ rows.T * scale
    lse = torch.from_numpy(s[:, 0]).float()[None]
    # dim 40 is 0 in token 0: its score is a power of two times the scale, its weight 1
    assert (lse[0].double().numpy() == s[:, 0]).all()
    got = run(K, layout, pool, 150, q.to(torch.bfloat16), lse, scale)
    d = s - s[:, :1]
    want = np.exp(d)
    tol = (want * np.expm1(2.0 ** -23 * np.abs(d) + 2.0 ** -20)).sum(0) + heads * 2.0 ** -24 * want.sum(0)
    assert (np.abs(got - want.sum(0)) <= tol).all(), (np.abs(got - want.sum(0)) / tol).max()


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("lse", [-3.0, 0.0, 11.5129, 20.0, 60.0])
def test_flat(K, layout, lse):
    """Scores of zero, whatever lse is."""
    pool, rows = pool_of(layout, [4.0] * 70, [0.0] * 70)
    q = torch.zeros((1, 16, 512))
    q[0, :, 100] = 3.0
    lse = torch.full((1, 16), lse)
    got = run(K, layout, pool, 70, q.to(torch.bfloat16), lse, 0.125)
    l = lse[0].double().numpy()
    want = np.exp(-l).sum()
    tol = want * (math.expm1(2.0 ** -23 * abs(l[0]) + 2.0 ** -20) + 16 * 2.0 ** -24)
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads", [1, 64, 128])
@pytest.mark.parametrize("scale", [1.0, 0.7, -0.3, 0.9, 1.1])
@pytest.mark.parametrize("power", [24, 29, 34, 60])
def test_scores_that_fp32_cannot_tell_apart(K, layout, heads, scale, power):
    """|lse| of 2^24 to 2^60, where a unit in its last place is 2 and more: no weight is NaN, a token far below lse has none, and up
    to 2^28 the token whose score lse is has 1, within 2^-20 and what the second-order terms, 2^-46 of lse, come to."""
    scale = float(np.float32(scale))
    top = 32.0 if layout == FP4 else 2.0 ** 20
    pool, rows = pool_of(layout, [top, -top, top / 2, top / 4] * 20, [0.0] * 80)
    q = torch.zeros((1, heads, 512))
    q[0, :, 5] = 2.0 ** power / top
    s = q[0].double().numpy() @ rows.T * scale
    for at in range(4):
        lse = torch.from_numpy(s[:, at]).float()[None]
        assert (lse[0].double().numpy() == s[:, at]).all()
        got = run(K, layout, pool, 80, q.to(torch.bfloat16), lse, scale)
        assert not np.isnan(got).any() and (got >= 0).all()
        assert (got[s[0] < s[0, at]] == 0).all()
        if power <= 28:
            assert (np.abs(got[s[0] == s[0, at]] - heads) <= heads * (2.0 ** -20 + heads * 2.0 ** -24 + abs(s[0, at]) * 2.0 ** -46)).all()


@pytest.mark.parametrize("heads,q_len", [(16, 1), (32, 1), (64, 1), (128, 1), (64, 3)])
@pytest.mark.parametrize("e", [-30, -8, 10, 13, 20, 60, 100])
def test_rows_of_other_powers(K, heads, q_len, e):
    """V41 rows far from one beside rows near it, every other token's, queries that bring the large ones' scores back."""
    c = Mass(V41, 6, [200, 333], heads, q_len=q_len, seed=29)
    pool = c.pool.reshape(c.pages, -1)
    scales = pool[:, 64 * 512:].reshape(c.pages, 64, 16).astype(np.int32)
    scales[:, ::2] = np.clip(scales[:, ::2] + e, 0, 254)
    pool[:, 64 * 512:] = scales.astype(np.uint8).reshape(c.pages, -1)
    if e > 0:
        c.q = (c.q.double() * 2.0 ** -e).to(torch.bfloat16)
    lse = c.lses()
    check(c.run(K, lse), c.lens, c.want(lse), e)


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads", [16, 32, 64, 128])
@pytest.mark.parametrize("scale", [0.125, 0.0, -0.0, 1e-38, 1e30])
def test_rows_without_scores(K, layout, heads, scale):
    """Queries of zeros, scales of zero and near it, lse infinite, of the largest size or absent, rows beside plain ones."""
    scale = float(np.float32(scale))
    pool, rows = pool_of(layout, [4.0, -8.0, 16.0] * 30, [0.0, 1.5, -3.0] * 30)
    q = torch.zeros((1, heads, 512))
    q[0, ::2, 5] = 0.5 if scale < 1 else 2.0 ** -110
    lse = torch.full((1, heads), 1.25)
    lse[0, 1], lse[0, 2], lse[0, 3], lse[0, 4] = math.inf, -math.inf, 3e38, 80.0
    s = q[0].double().numpy() @ rows.T * scale
    l = lse[0].double().numpy()[:, None]
    with np.errstate(over="ignore"):
        p = np.where(np.isneginf(l), 0.0, np.exp(s - l))
    got = run(K, layout, pool, 90, q.to(torch.bfloat16), lse, scale)
    tol = np.where(p > 0, p * np.expm1(2.0 ** -23 * np.where(np.isinf(l), 0, np.minimum(np.abs(s - l), 1e3)) + 2.0 ** -20) + 2.0 ** -126, 0)
    assert (np.abs(got - p.sum(0)) <= tol.sum(0) + heads * 2.0 ** -24 * p.sum(0)).all()
    lse[0, 5] = math.nan
    assert np.isnan(run(K, layout, pool, 90, q.to(torch.bfloat16), lse, scale)).all()


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads", [20, 64])
def test_few_tries(K, layout, heads):
    """Waits that give up, for the tiles of 32 and 64 rows: the call ends, weights are right or, where the error word says so, NaN."""
    c = Mass(layout, 6, [3000, 30, 0, 900], heads, seed=43)
    lse = c.lses()
    want = c.want(lse)
    for limit in (0, 1, 3, 10, 50, 200):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        before = K.attend_wait_limit(limit)
        try:
            got = c.run(K, lse, err=err)
        finally:
            K.attend_wait_limit(before)
        assert err.item() in (0, 16)
        if err.item() == 0:
            check(got, c.lens, want, limit)
        for i, (total, tol) in enumerate(want):
            row = got[i, :c.lens[i]].cpu().double().numpy()
            assert (np.isnan(row) | (np.abs(row - total) <= tol)).all() and (got[i, c.lens[i]:] == -7).all()
    check(c.run(K, lse), c.lens, want, "after")


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads,q_len", [(16, 1), (32, 1), (64, 1), (128, 1), (64, 6)])
def test_tiles_of_one_block(K, layout, heads, q_len):
    """Many tiles of one block and a few of more, so that a CTA's tiles, with constants of their own, follow each other closely: every
    sequence as in a call of its own, bit for bit."""
    lens = [1 + (37 * i) % 128 if i % 5 else 129 + 53 * i % 400 for i in range(400 if q_len == 1 else 150)]
    c = Mass(layout, 6, lens, heads, q_len=q_len, seed=61)
    # rows of a sequence have scores, and sums, of a size of their own
    size = torch.tensor([2.0 ** (i % 7 - 3) for i in range(len(lens))]).repeat_interleave(q_len)[:, None, None]
    c.q = (c.q.float() * size).to(torch.bfloat16)
    lse = c.lses()   # (with scores to 100 above some other number, weights pass fp32)
    got = c.run(K, lse)
    check(got, c.lens, c.want(lse), "all")
    whole_q, whole_table = c.q, c.table
    for i in (0, 1, 5, 77, 149):
        c.q, c.table, c.lens = whole_q[i * q_len:(i + 1) * q_len], whole_table[i:i + 1], lens[i:i + 1]
        one = c.run(K, lse[i * q_len:(i + 1) * q_len])
        assert torch.equal(one[0, :lens[i]], got[i, :lens[i]])
