"""A sink token and a long flat tail: weights that are tiny one by one and not in all.

The sink's key has score d ln 2 and the n others have score 0, so each of them
weighs 2^-d of the sink, and the tail has n 2^-d of its mass.  The sink's row
is zero in the dims that the output is read in, so what comes out there is the
tail's share alone.  A weight (for V41 times t, its row's power of two) is
rounded to fp16: relative 2^-11, or, where that is more, by an amount that is so
small that it comes to no more than 2^-13 of the largest over all n tokens (and
to no more than 2^-25 for each), so

  |out - exact| <= (2^-11 + 2^-18) sum p |k| / l + min(2^-13, n 2^-25) max(p t) max(|k| / t) / l

(2^-18: the exponentials and fp32 sums in up to 2^14 blocks, which round to
nearest one by one) plus a V41 value's own decoding.  Weights of 2^-25 each that
were left out would be ten times that.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from test_attend_gpu import DEV, FP4, V41, K, decode, row_power  # noqa: F401

pytestmark = pytest.mark.gpu
PAGES = 9           # page 0: the sink and padding; 1 to 8: the tail's rows, repeated


def problem(layout, d, seed, spread=0):
    """(pool, decoded rows [PAGES * 64, 512], query [512]): scale * q k is d ln 2 for slot 0 and 0 for slots 64 on."""
    g = torch.Generator().manual_seed(seed)
    x = 1 + 0.25 * torch.randn((PAGES * 64, 512), generator=g)
    x *= torch.exp2(torch.randint(-spread, 1, (PAGES * 64, 1), generator=g).float())
    x[:, :32] = 0
    x[0] = 0
    x[0, :32] = 1.5        # exact in both layouts, and as large as the tail's values
    x = x.to(torch.bfloat16)
    pool = np.zeros(PAGES * 64 * O.bytes_per_token(layout), np.uint8)
    assert O.store(layout, 6, 0, x.view(torch.int16).numpy().view(np.uint16), np.arange(PAGES * 64), pool) == O.OK
    q = torch.zeros(512)
    q[:32] = 2
    return pool, decode(layout, 6, pool, np.arange(PAGES * 64)), q, d * math.log(2) / (32 * 3)


def expect(layout, rows, count, d):
    """count[s]: how often slot s is seen (slot 0 once).  (out, lse, tolerance)."""
    p = count * np.where(np.arange(rows.shape[0]) == 0, 1.0, 2.0 ** -d)
    l, t = p.sum(), row_power(layout, rows)
    out = p @ rows / l
    one = np.where(np.arange(rows.shape[0]) == 0, 1.0, 2.0 ** -d)
    seen = count > 0
    tol = (2.0 ** -11 + 2.0 ** -18) * (p @ np.abs(rows)) / l + \
        min(2.0 ** -13, count.sum() * 2.0 ** -25) * (one * t)[seen].max() * (np.abs(rows) / t[:, None])[seen].max(0) / l
    if layout == V41:
        tol = tol + 2.0 ** -25 * (p @ t) / l
    return out, d * math.log(2) + math.log(l), tol


def compare(out, lse, want, tag):
    o, l, tol = want
    got = out.double().cpu().numpy()
    tail = np.abs(o[32:])
    assert not tail.any() or (tol[32:] < 0.25 * tail).all(), "the tail shows"
    off = np.abs(got - o)
    assert (off <= tol + 2.0 ** -22 * np.abs(o)).all(), (tag, (off / np.maximum(tol, 1e-300)).max())
    off = np.abs(lse.double().cpu().numpy() - l).max()
    assert off <= 2.0 ** -17 + 2.0 ** -20 * abs(l), (tag, off)


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads,q_len", [(16, 1), (32, 1), (40, 2)])
@pytest.mark.parametrize("n,d", [(3000, 20.0), (1 << 17, 25.5), (1 << 20, 28.5)])
def test_paged(K, layout, heads, q_len, n, d):
    pool, rows, q, scale = problem(layout, d, 3)
    table = 1 + torch.arange(1 + n // 64, dtype=torch.int32)[None] % 8
    table[0, 0] = 0
    # the first page: the sink, and tail rows in its other slots
    head = torch.from_numpy(pool.copy())
    cb, sb = (512, 16) if layout == V41 else (256, 32)
    head[cb:64 * cb] = head[64 * (cb + sb) + cb:64 * (cb + sb) + 64 * cb]
    head[64 * cb + sb:64 * (cb + sb)] = head[64 * (cb + sb) + 64 * cb + sb:128 * (cb + sb)]
    length = 64 * table.shape[1]
    rows = decode(layout, 6, head.numpy(), np.arange(PAGES * 64))
    many = 160                           # as many sequences as SMs, so that one CTA sums most of a sequence
    out = torch.full((many * q_len, heads, 512), float("nan"), device=DEV)
    lse = torch.full((many * q_len, heads), float("nan"), device=DEV)
    ws = torch.empty(K.attend_workspace(q_len * heads), dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    K.kvq_attend(layout, 6, q.to(torch.bfloat16).to(DEV).expand(many * q_len, heads, 512), head.to(DEV), PAGES,
                 table.to(DEV), torch.full((many,), length, dtype=torch.int32, device=DEV), out, ws, scale=scale, q_len=q_len,
                 req=torch.zeros(many, dtype=torch.int32, device=DEV), lse=lse, err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    for j in range(q_len):
        seen = length - (q_len - 1 - j)
        at = np.arange(seen)
        count = np.bincount(table[0].numpy()[at >> 6] * 64 + (at & 63), minlength=PAGES * 64).astype(np.float64)
        want = expect(layout, rows, count, d)
        for i in (0, 1, 77, many - 1):
            compare(out[i * q_len + j], lse[i * q_len + j], want, (n, d, i, j))


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("where", ["first", "last", "none but the sink"])
def test_slots(K, layout, where):
    """The sink at either end of a list (with a sink last, the maximum moves after the tail is summed), and rows whose
    powers of two differ."""
    n, d, heads, many = 1 << 17, 25.5, 24, 160
    pool, rows, q, scale = problem(layout, d, 7, spread=3)
    s = 64 + torch.arange(n, dtype=torch.int32) % (8 * 64)
    if where == "none but the sink":
        s[:] = -1
    s[0 if where != "last" else n - 1] = 0
    out, lse = torch.empty((many, heads, 512), device=DEV), torch.empty((many, heads), device=DEV)
    ws = torch.empty(K.attend_workspace(heads), dtype=torch.uint8, device=DEV)
    K.kvq_attend_slots(layout, 6, q.to(torch.bfloat16).to(DEV).expand(many, heads, 512), torch.from_numpy(pool).to(DEV),
                       PAGES * 64, s.to(DEV).expand(many, n), out, ws, scale=scale, lse=lse)
    torch.cuda.synchronize()
    count = np.bincount(s[s >= 0].numpy(), minlength=PAGES * 64).astype(np.float64)
    for i in (0, 1, 77, many - 1):
        compare(out[i], lse[i], expect(layout, rows, count, d), (where, i))


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads", [16, 32, 64])
@pytest.mark.parametrize("n,many", [(313 * 64 - 5, 300), (1 << 20, 160)])
def test_sums_of_many_equal_weights(K, layout, heads, n, many):
    """Equal weights are exact, so what the mean is off by is the sums': a CTA that sums most of a sequence, or several,
    in up to 2^14 blocks.  The tensor cores add 16 tokens at a time and drop what is below 2^-23 of the sum, which is
    half of the final one on average; over at most 256 blocks that is 256 * 4 * 2^-23 / 2 = 2^-14.  The rest is rounded
    to nearest (2^-18, with the final division), and a V41 value is off by its decoding."""
    pool, rows, q, _ = problem(layout, 0.0, 11)
    table = 1 + torch.arange(-(-n // 64), dtype=torch.int32)[None] % 8
    out, lse = torch.full((many, heads, 512), float("nan"), device=DEV), torch.full((many, heads), float("nan"), device=DEV)
    ws = torch.empty(K.attend_workspace(heads), dtype=torch.uint8, device=DEV)
    K.kvq_attend(layout, 6, q.to(torch.bfloat16).to(DEV).expand(many, heads, 512), torch.from_numpy(pool).to(DEV), PAGES,
                 table.to(DEV), torch.full((many,), n, dtype=torch.int32, device=DEV), out, ws, scale=0.0,
                 req=torch.zeros(many, dtype=torch.int32, device=DEV), lse=lse)
    torch.cuda.synchronize()
    at = np.arange(n)
    count = np.bincount(table[0].numpy()[at >> 6] * 64 + (at & 63), minlength=PAGES * 64).astype(np.float64)
    want = count @ rows / n
    tol = (2.0 ** -14 + 2.0 ** -18) * (count @ np.abs(rows)) / n
    if layout == V41:
        tol = tol + 2.0 ** -25 * (count @ row_power(layout, rows)) / n
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
    assert np.abs(lse.double().cpu().numpy() - math.log(n)).max() <= 2.0 ** -18


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads", [16, 64])
def test_maxima_that_move_late(K, layout, heads):
    """Scores that rise along a part of many blocks, so that sums already put aside are brought to later maxima: the
    tokens of each quarter of the sequence weigh 2^12 of the quarter before."""
    n, many = 64 * 1500, 152
    pool, rows, q, _ = problem(layout, 0.0, 13)
    x = np.zeros((PAGES * 64, 512), np.float32)
    g = np.random.default_rng(17)
    x[:, 32:] = 1 + 0.25 * g.standard_normal((PAGES * 64, 480))
    for page in range(1, 5):
        x[page * 64:(page + 1) * 64, :32] = 0.375 * (page - 1)
    x = torch.from_numpy(x).to(torch.bfloat16)
    pool = np.zeros(PAGES * 64 * O.bytes_per_token(layout), np.uint8)
    assert O.store(layout, 6, 0, x.view(torch.int16).numpy().view(np.uint16), np.arange(PAGES * 64), pool) == O.OK
    rows = decode(layout, 6, pool, np.arange(PAGES * 64))
    assert all((rows[p * 64:(p + 1) * 64, :32] == 0.375 * (p - 1)).all() for p in range(1, 5))
    scale = 12 * math.log(2) / (32 * 2 * 0.375)
    table = (1 + torch.arange(n // 64, dtype=torch.int32) * 4 // (n // 64))[None]
    out, lse = torch.full((many, heads, 512), float("nan"), device=DEV), torch.full((many, heads), float("nan"), device=DEV)
    ws = torch.empty(K.attend_workspace(heads), dtype=torch.uint8, device=DEV)
    K.kvq_attend(layout, 6, q.to(torch.bfloat16).to(DEV).expand(many, heads, 512), torch.from_numpy(pool).to(DEV), PAGES,
                 table.to(DEV), torch.full((many,), n, dtype=torch.int32, device=DEV), out, ws, scale=scale,
                 req=torch.zeros(many, dtype=torch.int32, device=DEV), lse=lse)
    torch.cuda.synchronize()
    p = np.exp2(12.0 * (np.arange(PAGES * 64) // 64 - 4))
    p[:64] = p[5 * 64:] = 0
    count = np.where(p > 0, n / 256, 0.0)
    l = (p * count).sum()
    want = (p * count) @ rows / l
    t = row_power(layout, rows)
    # weights 2^-11, sums as above, the smallest weights 2^-13 of the largest in all
    tol = (2.0 ** -11 + 2.0 ** -14 + 2.0 ** -18) * want + 2.0 ** -13 * (p * t).max() * (rows / t[:, None])[p > 0].max(0) / l
    if layout == V41:
        tol = tol + 2.0 ** -25 * ((p * count) @ t) / l
    assert (np.abs(out.double().cpu().numpy() - want) <= tol + 1e-30).all()
    exact = math.log(l) + 3 * 12 * math.log(2)
    assert np.abs(lse.double().cpu().numpy() - exact).max() <= 2.0 ** -17 + 2.0 ** -20 * exact
