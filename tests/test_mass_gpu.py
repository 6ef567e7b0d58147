"""kvq_attend_mass against the definition in 64 bits.

Rows are decoded by the oracle; a weight is exp(s - lse) with the lse that the
call is given.  The tolerance counts the roundings, u = 2^-k for a half step:

* the score is off by 512 * 2^-23 * scale * sum |q k| + 2^-22 |s| (fp32 sum of
  exact products, truncating accumulators, and its scaling), for V41 by another
  scale * sum |q| * 2^-25 t, t the power of two that the row is decoded relative
  to (fp16's subnormals);
* the exponent's constants and its sum: 2^-23 (|s| + |lse|) + 2^-23 |s - lse|;
* the exponential 2^-21 relative, zero below 2^-126;
* a token's sum over R rows: R * 2^-24 of it, whatever the order, and twice
  2^-23 for what was there before (decay * prev, which counts by its magnitude).
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from test_attend_gpu import DEV, FP4, V41, K, Paged, decode, row_power  # noqa: F401

pytestmark = pytest.mark.gpu


def weights(layout, q, lse, rows, scale):
    """(weights, tolerance) of one query token: q float64 [h, 512], lse float64 [h], rows [n, 512]; both [h, n]."""
    s = q @ rows.T * scale
    with np.errstate(invalid="ignore"):
        p = np.where(np.isneginf(lse)[:, None], 0.0, np.exp(s - lse[:, None]))
        t = row_power(layout, rows)
        d = 512 * 2.0 ** -23 * abs(scale) * (np.abs(q) @ np.abs(rows).T) + 2.0 ** -22 * np.abs(s)
        if layout == V41:
            d = d + abs(scale) * np.abs(q).sum(1)[:, None] * 2.0 ** -25 * t
        d = d + 2.0 ** -23 * (np.abs(s) + np.abs(lse)[:, None]) + 2.0 ** -23 * np.abs(s - lse[:, None]) + 2.0 ** -21
        tol = np.where(np.isneginf(lse)[:, None], 0.0, p * np.expm1(d) + 2.0 ** -125)
    return p, tol


class Mass(Paged):
    def lses(self):
        """float32 [tokens, heads]: the log-sums, rounded."""
        got, q = [], self.q.double().numpy()
        for i, n in enumerate(self.lens):
            rows = decode(self.layout, self.pb, self.pool, self.slots(i, n))
            for j in range(self.q_len):
                vis = max(0, n - (self.q_len - 1 - j))
                if vis == 0:
                    got.append(np.full(self.heads, -math.inf))
                    continue
                s = q[i * self.q_len + j] @ rows[:vis].T * self.scale
                m = s.max(1)
                got.append(m + np.log(np.exp(s - m[:, None]).sum(1)))
        return torch.from_numpy(np.stack(got).astype(np.float32))

    def want(self, lse, prev=None, decay=1.0, missing=()):
        """[(mass, tolerance)] of each sequence; `missing`: (sequence, token) pairs that are not there."""
        got, q, l = [], self.q.double().numpy(), lse.double().numpy()
        for i, n in enumerate(self.lens):
            rows = decode(self.layout, self.pb, self.pool, self.slots(i, n)) if n else np.zeros((0, 512))
            total, tol = np.zeros(n), np.zeros(n)
            for j in range(self.q_len):
                vis, at = max(0, n - (self.q_len - 1 - j)), i * self.q_len + j
                p, d = weights(self.layout, q[at], l[at], rows[:vis], self.scale)
                total[:vis] += p.sum(0)
                tol[:vis] += d.sum(0)
            for s, t in missing:
                if s == i:
                    total[t] = tol[t] = 0
            tol += self.q_len * self.heads * 2.0 ** -24 * total
            if prev is not None:
                before = decay * prev[i, :n].double().numpy()
                tol += 2.0 ** -22 * (np.abs(before) + total)
                total = total + before
            got.append((total, tol + 1e-36))
        return got

    def run(self, K, lse, mass=None, prev=None, decay=1.0, rows=None, req=None, table=None, kv_len=None, q=None, err=None, ws=None,
            mask=None):
        width = self.width << self.pb
        if mass is None:
            mass = torch.full((len(self.lens), width), -7.0, device=DEV)
        table = torch.from_numpy(self.table).to(DEV) if table is None else table
        kv_len = torch.tensor(self.lens, dtype=torch.int32, device=DEV) if kv_len is None else kv_len
        size = K.mass_workspace(kv_len.numel(), self.q_len * self.heads, min(table.shape[1] << self.pb, mass.shape[-1]))
        if ws is None:   # stale contents mean nothing
            ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
        K.kvq_attend_mass(self.layout, self.pb, self.q.to(DEV) if q is None else q, lse.to(DEV), torch.from_numpy(self.pool).to(DEV),
                          self.pages, table, kv_len, mass, ws, scale=self.scale, q_len=self.q_len, req=req, rows=rows, prev=prev,
                          decay=decay, mask=mask, err=err)
        torch.cuda.synchronize()
        return mass


def check(mass, lens, want, tag, behind=-7.0):
    got = mass.cpu().double().numpy()
    for i, (total, tol) in enumerate(want):
        n = lens[i]
        assert np.isfinite(got[i, :n]).all(), (tag, i)
        bad = np.abs(got[i, :n] - total) > tol
        assert not bad.any(), (tag, i, int(bad.sum()), np.flatnonzero(bad)[:4], (np.abs(got[i, :n] - total) / tol).max())
        assert behind is None or (got[i, n:] == behind).all(), (tag, i)


CASES = [
    (16, 1, [100], 6),
    (1, 1, [1], 6),
    (5, 1, [0, 1, 31, 32, 33, 63, 64, 65], 6),
    (16, 1, [127, 128, 129, 255, 256, 257, 0, 2], 6),
    (17, 1, [300, 5], 4),
    (33, 1, [1000, 3, 130], 2),
    (64, 1, [640, 129, 1, 0, 77], 8),
    (65, 1, [300, 128, 1], 6),
    (128, 1, [511, 2, 200], 4),
    (8, 4, [1, 3, 4, 5, 128, 131, 260], 6),       # sequences shorter than their query
    (7, 3, [130, 0, 2], 2),
    (64, 5, [257, 64, 400], 6),                   # three tiles of 128 rows a sequence
    (3, 70, [200, 69, 33, 300], 8),
    (128, 3, [290, 0, 1, 129], 6),
]


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads,q_len,lens,pb", CASES)
def test_lengths(K, layout, heads, q_len, lens, pb):
    c = Mass(layout, pb, lens, heads, q_len, seed=heads + q_len)
    lse = c.lses()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = c.run(K, lse, err=err)
    assert err.item() == 0
    check(got, lens, c.want(lse), "overwritten")
    # every query row's weights are one in all: what the tolerances let through would show here
    for i, n in enumerate(lens):
        rows = sum(max(0, n - (q_len - 1 - j)) > 0 for j in range(q_len)) * heads
        assert abs(got[i, :n].double().sum().item() - rows) <= 1e-4 * rows
    prev = torch.rand(got.shape, generator=torch.Generator().manual_seed(1))
    added = c.run(K, lse, prev=prev.to(DEV), decay=0.75)
    check(added, lens, c.want(lse, prev, 0.75), "added")
    same = prev.to(DEV)
    c.run(K, lse, mass=same, prev=same, decay=0.75)
    for i, n in enumerate(lens):
        assert torch.equal(same[i, :n], added[i, :n]) and torch.equal(same[i, n:].cpu(), prev[i, n:])


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads,q_len", [(16, 1), (32, 1), (64, 1), (128, 1), (40, 8)])
def test_many_blocks_a_cta(K, layout, heads, q_len):
    """More blocks than CTAs, in long tiles and in short ones: every ring goes round several times; twice the same bits."""
    c = Mass(layout, 6, [128 * 152 * 5 + 5, 0, 700] if q_len == 1 else [128 * 152 + 77, 700], heads, q_len=q_len, seed=51)
    lse = c.lses()
    got = c.run(K, lse)
    check(got, c.lens, c.want(lse), (heads, "long"))
    assert torch.equal(c.run(K, lse), got)
    lens = [128 * ((7 * i) % 6) + (i % 3) for i in range(300 if q_len == 1 else 40)]
    c = Mass(layout, 6, lens, heads, q_len=q_len, seed=53)
    lse = c.lses()
    check(c.run(K, lse), lens, c.want(lse), (heads, "short"))


@pytest.mark.parametrize("layout", [V41, FP4])
def test_many_sequences(K, layout):
    """More sequences than threads of a CTA, most of them short or empty, small pages."""
    rng = np.random.default_rng(5)
    lens = [int(n) for n in rng.integers(0, 40, 1300)]
    lens[700] = 900
    c = Mass(layout, 2, lens, 4, seed=7)
    lse = c.lses()
    check(c.run(K, lse), lens, c.want(lse), "many")


@pytest.mark.parametrize("layout", [V41, FP4])
def test_after_attention_over_steps(K, layout):
    """With the lse that kvq_attend leaves, added up over steps of growing sequences, rows by index; then the caches are cut
    and attention over what is left equals attention over the kept tokens' slots."""
    heads, keep = 24, 70
    c = Mass(layout, 6, [200, 90, 140], heads, seed=11)
    rows = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    width = c.width * 64
    mass = torch.zeros((5, width), device=DEV)
    table = torch.from_numpy(c.table).to(DEV).clamp(0, c.pages - 1)
    pool = torch.from_numpy(c.pool).to(DEV)
    total = [np.zeros(n) for n in c.lens]
    tol = [np.zeros(n) for n in c.lens]
    full = list(c.lens)
    g = torch.Generator().manual_seed(3)
    ws = torch.empty(K.attend_workspace(heads), dtype=torch.uint8, device=DEV)
    for step in range(3):
        lens = [n - 2 + step for n in full]
        c.lens = lens
        c.q = (2 * torch.randn((3, heads, 512), generator=g)).to(torch.bfloat16)
        q, kv = c.q.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
        out, lse = torch.empty_like(q), torch.empty((3, heads), device=DEV)
        K.kvq_attend(layout, 6, q, pool, c.pages, table, kv, out, ws, scale=c.scale, lse=lse)
        K.kvq_attend_mass(layout, 6, q, lse, pool, c.pages, table, kv, mass, scale=c.scale, rows=rows, prev=mass, decay=0.5)
        for i, (w, d) in enumerate(c.want(lse.cpu())):
            n = lens[i]
            total[i][:n] = 0.5 * total[i][:n] + w
            tol[i][:n] = 0.5 * tol[i][:n] + d + 2.0 ** -22 * total[i][:n]
    for i, r in enumerate([4, 0, 2]):
        assert (np.abs(mass[r, :full[i]].cpu().double().numpy() - total[i]) <= tol[i]).all()
        assert (mass[r, full[i]:] == 0).all()
    assert (mass[1] == 0).all() and (mass[3] == 0).all()
    # cut to the tokens of most weight
    kv = torch.tensor(full, dtype=torch.int32, device=DEV)
    kept, count = torch.empty((3, keep), dtype=torch.int32, device=DEV), torch.empty(3, dtype=torch.int32, device=DEV)
    K.kvq_evict_select(mass, kv, kept, count, first=2, last=10, rows=rows)
    big = torch.cat((pool, torch.zeros(6 * 64 * O.bytes_per_token(layout), dtype=torch.uint8, device=DEV)))
    new = (torch.arange(6, dtype=torch.int32, device=DEV) + c.pages).view(3, 2)
    left = torch.zeros((3, keep), device=DEV)
    K.kvq_evict_move(layout, 6, big, c.pages + 6, table, new, kept, mass=mass, rows=rows, mass_out=left)
    out, lse = torch.empty_like(q), torch.empty((3, heads), device=DEV)
    K.kvq_attend(layout, 6, q, big, c.pages + 6, new, count, out, ws, scale=c.scale, lse=lse)
    slots = table.long().gather(1, (kept >> 6).clamp_min(0).long()) * 64 + (kept & 63)
    slots = torch.where(kept >= 0, slots, -1)
    out2, lse2 = torch.empty_like(q), torch.empty((3, heads), device=DEV)
    K.kvq_attend_slots(layout, 6, q, pool, c.pages * 64, slots, out2, ws, scale=c.scale, lse=lse2)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert torch.equal(left[0], mass[4][kept[0].long()])


@pytest.mark.parametrize("layout", [V41, FP4])
def test_what_is_not_seen_may_hold_anything(K, layout):
    """NaN rows behind the lengths and in unused pages change nothing; one in a sequence makes its own weight NaN alone, and
    a NaN or infinite query row, or lse, the weights of the tokens that it sees."""
    c = Mass(layout, 6, [70, 129, 200], 16, q_len=3, seed=19)
    lse = c.lses()
    clean = c.run(K, lse)
    check(clean, c.lens, c.want(lse), "clean")
    bpt = O.bytes_per_token(layout)
    pool = c.pool.reshape(c.pages, -1)
    used = {int(p) for i, n in enumerate(c.lens) for p in c.table[i][:-(-n // 64)]}
    cb = 512 if layout == V41 else 256
    sb = bpt - cb

    def poison(i, t):
        p, r = c.table[i][t >> 6], t & 63
        pool[p, r * cb:(r + 1) * cb] = 0xFF
        pool[p, 64 * cb + r * sb:64 * cb + r * sb + 16] = 0xFF
    for p in range(c.pages):
        if p not in used:
            pool[p] = 0xFF
    for i, n in enumerate(c.lens):
        for t in range(n, -(-n // 64) * 64):
            poison(i, t)
    assert torch.equal(c.run(K, lse), clean)
    poison(1, 30)
    poison(2, 199)       # the last query token alone sees it
    got = c.run(K, lse)
    assert got[1, 30].isnan() and got[2, 199].isnan()
    got[1, 30], got[2, 199] = clean[1, 30], clean[2, 199]
    assert torch.equal(got, clean)
    for odd in (float("nan"), float("inf")):
        c2 = Mass(layout, 6, [70, 129, 200], 16, q_len=3, seed=19)
        c2.q[3, 5, 100] = odd              # sequence 1, its first query token: sees 127 of 129
        got = c2.run(K, lse)
        assert got[1, :127].isnan().all() and torch.equal(got[1, 127:], clean[1, 127:])
        assert torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])
    bad = lse.clone()
    bad[7, 2] = float("nan")               # sequence 2, its second query token: sees 199 of 200
    c2 = Mass(layout, 6, [70, 129, 200], 16, q_len=3, seed=19)
    got = c2.run(K, bad)
    assert got[2, :199].isnan().all() and torch.equal(got[2, 199:], clean[2, 199:]) and torch.equal(got[:2], clean[:2])
    # rows without a sum have no weight, even over a token that is not a number
    none = torch.full_like(lse, -math.inf)
    got = c.run(K, none)
    assert all((got[i, :n] == 0).all() for i, n in enumerate(c.lens))


def test_no_weight_without_a_sum(K):
    c = Mass(V41, 6, [70, 300], 20, seed=23)
    lse = c.lses()
    lse[0, 3], lse[1, :] = -math.inf, -math.inf
    got = c.run(K, lse)
    check(got, c.lens, c.want(lse), "some")
    assert (got[1, :300] == 0).all()


@pytest.mark.parametrize("e", [-30, 20, 60, 100])
def test_rows_of_other_powers(K, e):
    """V41 rows far from one, queries that bring the scores back."""
    c = Mass(V41, 6, [200], 16, seed=29)
    pool = c.pool.reshape(c.pages, -1)
    pool[:, 64 * 512:] = np.clip(pool[:, 64 * 512:].astype(np.int32) + e, 0, 254).astype(np.uint8)
    c.q = (c.q.double() * 2.0 ** -e).to(torch.bfloat16)
    lse = c.lses()
    check(c.run(K, lse), c.lens, c.want(lse), e)


def test_bad_lengths_pages_and_rows(K):
    c = Mass(V41, 6, [200, 90, 100, 70, 60, 50], 16, seed=31)
    lse = c.lses()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = torch.from_numpy(c.table.copy())
    table[0, 1], table[1, 0] = c.pages, -1
    lens = torch.tensor([200, 90, -1, 64 * c.width + 1, 60, 50], dtype=torch.int32, device=DEV)
    got = c.run(K, lse, table=table.to(DEV), kv_len=lens, req=torch.tensor([0, 1, 2, 3, 6, 5], dtype=torch.int32, device=DEV),
                rows=torch.tensor([0, 1, 2, 3, 4, -1], dtype=torch.int32, device=DEV), err=err)
    assert err.item() == 4 | 32 | 64
    assert (got[2:] == -7).all()
    c.lens = [200, 90]
    check(got, c.lens, c.want(lse, missing=[(0, t) for t in range(64, 128)] + [(1, t) for t in range(64)]), "pages")
    # a weights' row that is shorter than the table is a limit too
    err.zero_()
    c = Mass(V41, 6, [200, 90], 16, seed=31)
    short = torch.full((2, 150), -7.0, device=DEV)
    c.run(K, c.lses(), mass=short, err=err)
    assert err.item() == 64 and (short[0] == -7).all() and (short[1, :90] != -7).all()


def test_strides_and_rows_behind(K):
    c = Mass(FP4, 6, [200, 90], 6, q_len=2, seed=37)
    lse = c.lses()
    want = c.run(K, lse)
    wide = torch.zeros((4, 6, 640), dtype=torch.bfloat16, device=DEV)
    wide[..., :512] = c.q.to(DEV)
    big = torch.full((5, 400), -7.0, device=DEV)
    strided = torch.full((4, c.width + 3), -1, dtype=torch.int32)
    strided[3, :c.width], strided[1, :c.width] = torch.from_numpy(c.table[0]), torch.from_numpy(c.table[1])
    got = c.run(K, lse, q=wide[..., :512], mass=big[:, :300], table=strided.to(DEV)[:, :c.width],
                req=torch.tensor([3, 1], dtype=torch.int32, device=DEV), rows=torch.tensor([4, 1], dtype=torch.int32, device=DEV))
    assert torch.equal(got[4, :200], want[0, :200]) and torch.equal(got[1, :90], want[1, :90])
    assert (big[:, 300:] == -7).all() and (big[[0, 2, 3]] == -7).all() and (big[1, 90:] == -7).all()
    head_major = c.q.to(DEV).permute(1, 0, 2).contiguous().permute(1, 0, 2)
    assert torch.equal(c.run(K, lse, q=head_major), want)


@pytest.mark.parametrize("heads,q_len", [(16, 1), (64, 3)])
def test_captured(K, heads, q_len):
    c = Mass(V41, 6, [200, 90, 300], heads, q_len=q_len, seed=41)
    q, lse = torch.zeros_like(c.q, device=DEV), torch.zeros((3 * q_len, heads), device=DEV)
    pool, table = torch.from_numpy(c.pool).to(DEV), torch.from_numpy(c.table).to(DEV).clamp(0, c.pages - 1)
    kv = torch.zeros(3, dtype=torch.int32, device=DEV)
    mass = torch.full((3, c.width * 64), -7.0, device=DEV)
    ws = torch.empty(K.mass_workspace(3, heads * q_len, c.width * 64), dtype=torch.uint8, device=DEV)

    def step():
        K.kvq_attend_mass(V41, 6, q, lse, pool, c.pages, table, kv, mass, ws, scale=c.scale, q_len=q_len)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([200, 90, 300], [0, 64, 129]):
        c.lens = lens
        l = c.lses()
        q.copy_(c.q)
        lse.copy_(l)
        kv.copy_(torch.tensor(lens))
        mass.fill_(-7.0)
        graph.replay()
        torch.cuda.synchronize()
        check(mass, lens, c.want(l), lens)


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads,q_len,lens", [(4, 7, [7, 100, 0, 130, 3]), (2, 63, [63, 64, 127, 200]), (3, 70, [70, 133, 400]),
                                              (64, 5, [69, 300])])
def test_trees(K, layout, heads, q_len, lens):
    """With a tree's masks, any mask among them, and the lse that kvq_attend_tree leaves."""
    from test_tree_gpu import Tree
    rng = np.random.default_rng(heads)
    for sees in (None, [[np.flatnonzero(rng.random(q_len) < (0.3 if j % 4 else 0.0)).tolist() for j in range(q_len)] for _ in lens]):
        c = Tree(layout, 6, lens, heads, q_len, seed=5, sees=sees)
        out, lse = c.run(K)
        mass = torch.full((len(lens), c.width * 64), -7.0, device=DEV)
        ws = torch.full((K.mass_workspace(len(lens), q_len * heads, c.width * 64),), 0xFF, dtype=torch.uint8, device=DEV)
        K.kvq_attend_mass(layout, 6, c.q.to(DEV), lse, torch.from_numpy(c.pool).to(DEV), c.pages, torch.from_numpy(c.table).to(DEV),
                          torch.tensor(lens, dtype=torch.int32, device=DEV), mass, ws, scale=c.scale, mask=c.mask.to(DEV))
        q, l = c.q.double().numpy(), lse.cpu().double().numpy()
        want = []
        for i, n in enumerate(lens):
            rows = decode(layout, 6, c.pool, c.slots(i, n)) if n else np.zeros((0, 512))
            total, tol = np.zeros(n), np.zeros(n)
            for j in range(q_len):
                t = np.array(c.seen(i, j) if n else [], np.int64)
                p, d = weights(layout, q[i * q_len + j], l[i * q_len + j], rows[t], c.scale)
                total[t] += p.sum(0)
                tol[t] += d.sum(0)
            want.append((total, tol + q_len * heads * 2.0 ** -24 * total + 1e-36))
        check(mass, lens, want, sees is None)


def test_a_wait_that_gives_up(K):
    """With a limit of 0 every wait gives up: the weights are NaN and the error word says so; the next call is sound."""
    for heads, q_len in ((16, 1), (64, 3)):
        c = Mass(FP4, 6, [700, 30], heads, q_len=q_len, seed=43)
        lse = c.lses()
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        before = K.attend_wait_limit(0)
        try:
            got = c.run(K, lse, err=err)
        finally:
            K.attend_wait_limit(before)
        assert err.item() == 16
        for i, n in enumerate(c.lens):
            assert got[i, :n].isnan().all() and (got[i, n:] == -7).all()
        err.zero_()
        check(c.run(K, lse, err=err), c.lens, c.want(lse), "after")
        assert err.item() == 0


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads,q_len", [(16, 1), (128, 1), (64, 3)])
def test_a_few_tries(K, layout, heads, q_len):
    """With a few tries some waits give up and some do not: the call ends, and a weight is right or, where the error word
    says so, NaN."""
    c = Mass(layout, 6, [3000, 30, 0, 900], heads, q_len=q_len, seed=43)
    lse = c.lses()
    want = c.want(lse)
    for limit in (1, 2, 5, 20, 100):
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


def test_binding_refuses(K):
    c = Mass(V41, 6, [20, 9], 4, seed=47)
    lse = c.lses()
    m = torch.zeros((2, 64), device=DEV)
    for bad in (dict(mass=m[:1]), dict(mass=m.double()), dict(mass=m[0]), dict(prev=m[:, :32]), dict(prev=m.double()),
                dict(rows=torch.zeros(1, dtype=torch.int32, device=DEV)), dict(err=m), dict(q=c.q.to(DEV).float()),
                dict(kv_len=torch.zeros(3, dtype=torch.int32, device=DEV)), dict(ws=m), dict(mask=m),
                dict(mask=torch.zeros((1, 1, 1), dtype=torch.int64, device=DEV)),
                dict(mask=torch.zeros((2, 2, 1), dtype=torch.int64, device=DEV))):
        with pytest.raises((TypeError, ValueError)):
            c.run(K, lse, **({"mass": torch.zeros((2, 64), device=DEV)} | bad))
    with pytest.raises((TypeError, ValueError)):
        c.run(K, lse[:, :2])
    with pytest.raises(K.KVQError):      # prev across mass's rows
        big = torch.zeros((3, 64), device=DEV)
        c.run(K, lse, mass=big[:2], prev=big[1:])
    with pytest.raises(K.KVQError):      # no workspace where there has to be one
        c = Mass(V41, 6, [20, 9], 64, q_len=3, seed=47)
        c.run(K, c.lses(), ws=torch.zeros(0, dtype=torch.uint8, device=DEV))
