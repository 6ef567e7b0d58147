"""kvq_attend_tree against the definition in 64 bits, with kvq_attend's tolerances (test_attend_gpu says where they come
from), and kvq_tree_mask against a walk from child to parent."""
import numpy as np
import pytest
import torch

import oracle as O
from test_attend_gpu import DEV, FP4, V41, K, Paged, check, decode, reference  # noqa: F401

pytestmark = pytest.mark.gpu


def lines(parent):
    """Of each token, itself and its ancestors."""
    got = []
    for j in range(len(parent)):
        line, at = [], j
        while at >= 0:
            line.append(at)
            at = int(parent[at])
        got.append(sorted(line))
    return got


def words_of(sees, q_len):
    """int64 [q_len, ceil(q_len / 64)] of lists of seen tokens."""
    w = np.zeros((q_len, (q_len + 63) // 64), np.uint64)
    for j, line in enumerate(sees):
        for k in line:
            w[j, k // 64] |= np.uint64(1) << np.uint64(k % 64)
    return w.view(np.int64)


def some_parents(n, q_len, seed, deep=False):
    rng = np.random.default_rng(seed)
    p = np.empty((n, q_len), np.int32)
    for j in range(q_len):
        p[:, j] = j - 1 if deep else rng.integers(-1, j, n)
    return p


class Tree(Paged):
    """`sees[i][j]`: the drafted tokens that query token j of sequence i sees."""

    def __init__(self, layout, pb, lens, heads, q_len, seed=0, sees=None, width_more=0):
        super().__init__(layout, pb, lens, heads, q_len, seed, width_more)
        if sees is None:
            sees = [lines(p) for p in some_parents(len(lens), q_len, seed)]
        self.sees = sees
        self.mask = torch.from_numpy(np.stack([words_of(s, q_len) for s in sees]))

    def seen(self, i, j):
        base = self.lens[i] - self.q_len
        return [t for t in range(max(0, base))] + [base + k for k in self.sees[i][j] if base + k >= 0]

    def want(self):
        got, q = [], self.q.double().numpy()
        for i, n in enumerate(self.lens):
            rows = decode(self.layout, self.pb, self.pool, self.slots(i, n))
            for j in range(self.q_len):
                t = np.array(self.seen(i, j) if n else [], np.int64)
                got.append(reference(self.layout, q[i * self.q_len + j], rows[t], self.scale))
        return got

    def run(self, K, out=None, q=None, table=None, req=None, mask=None, err=None, ws=None, kv_len=None):
        q = self.q.to(DEV) if q is None else q
        out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV) if out is None else out
        lse = torch.full(q.shape[:2], float("nan"), device=DEV)
        if ws is None:
            ws = torch.full((K.attend_workspace(self.q_len * self.heads),), 0xFF, dtype=torch.uint8, device=DEV)
        table = torch.from_numpy(self.table).to(DEV) if table is None else table
        kv_len = torch.tensor(self.lens, dtype=torch.int32, device=DEV) if kv_len is None else kv_len
        K.kvq_attend_tree(self.layout, self.pb, q, torch.from_numpy(self.pool).to(DEV), self.pages, table, kv_len,
                          (self.mask if mask is None else mask).to(DEV), out, ws, scale=self.scale, req=req, lse=lse, err=err)
        torch.cuda.synchronize()
        return out, lse


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads,q_len,lens,pb", [
    (1, 1, [1], 6),
    (16, 1, [0, 1, 64, 65], 6),
    (16, 7, [700], 6),
    (5, 2, [2, 3, 63, 64, 65, 66], 6),
    (8, 24, [24, 0, 25, 100, 130, 64], 4),
    (3, 63, [63, 64, 126, 127, 128, 200], 2),
    (4, 64, [64, 128, 129, 127, 65], 6),
    (2, 65, [65, 128, 129, 193, 90], 8),
    (1, 130, [130, 200, 0, 257], 6),
    (64, 5, [69, 300], 6),
    (33, 3, [5, 700, 3], 6),
    (128, 2, [2, 130], 6),
    (7, 9, [3, 8, 9, 1, 0], 6),                    # fewer cached tokens than drafted ones
])
def test_trees(K, layout, heads, q_len, lens, pb):
    c = Tree(layout, pb, lens, heads, q_len, seed=heads + q_len)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = c.run(K, err=err)
    assert err.item() == 0
    check(out, lse, c.want(), "tree")


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("q_len,lens", [(20, [20, 21, 100, 147]), (70, [70, 133, 400])])
def test_any_mask(K, layout, q_len, lens):
    """Masks that are no tree's: random ones, also of later tokens, and rows that see nothing at all."""
    rng = np.random.default_rng(q_len)
    sees = [[np.flatnonzero(rng.random(q_len) < (0.3 if j % 4 else 0.0)).tolist() for j in range(q_len)] for _ in lens]
    c = Tree(layout, 6, lens, 4, q_len, seed=3, sees=sees)
    out, lse = c.run(K)
    want = c.want()
    check(out, lse, want, "any")
    rows = out.view(len(lens), q_len, 4, 512)
    assert (rows[0, ::4] == 0).all() and torch.isneginf(lse.view(len(lens), q_len, 4)[0, ::4]).all()


@pytest.mark.parametrize("layout", [V41, FP4])
def test_split_over_ctas(K, layout):
    """Long sequences of several tiles, split over many CTAs and joined; fp32 output, twice the same bits."""
    c = Tree(layout, 6, [20003, 30, 0, 5000], 10, 30, seed=5)
    out = torch.full(c.q.shape, float("nan"), device=DEV)
    out, lse = c.run(K, out=out)
    check(out, lse, c.want(), "split")
    again, lse2 = c.run(K, out=torch.empty_like(out))
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_a_chain_is_causal(K):
    """A tree without branches is kvq_attend's causal mask: the same values up to both calls' tolerance."""
    c = Tree(FP4, 6, [300, 77, 9, 0], 6, 9, seed=7, sees=[lines(p) for p in some_parents(4, 9, 0, deep=True)])
    out, lse = c.run(K, out=torch.empty(c.q.shape, device=DEV))
    check(out, lse, Paged.want(c), "chain")
    got, lse2 = Paged.run(c, K, out=torch.empty(c.q.shape, device=DEV))
    check(got, lse2, Paged.want(c), "causal")


@pytest.mark.parametrize("layout", [V41, FP4])
def test_unseen_tokens_may_hold_anything(K, layout):
    """NaN rows in drafted tokens reach the query rows that see them and no others; what lies behind the last token, and in
    the mask's bits behind the last drafted token, does not matter."""
    q_len, lens = 12, [100, 12, 64]
    c = Tree(layout, 6, lens, 16, q_len, seed=11)
    clean, lse = c.run(K)
    check(clean, lse, c.want(), "clean")
    bpt = O.bytes_per_token(layout)
    pool = c.pool.reshape(c.pages, -1)
    cb = 512 if layout == V41 else 256
    sb = bpt - cb

    def poison(i, t):
        p, r = c.table[i][t >> 6], t & 63
        pool[p, r * cb:(r + 1) * cb] = 0xFF
        pool[p, 64 * cb + r * sb:64 * cb + r * sb + 16] = 0xFF
    for i, n in enumerate(lens):
        for t in range(n, -(-n // 64) * 64):
            poison(i, t)
    more = c.mask | ~((1 << q_len) - 1)
    got, lse2 = c.run(K, mask=more)
    assert torch.equal(got, clean) and torch.equal(lse, lse2)
    for i, n in enumerate(lens):
        poison(i, n - q_len + 4)
    got, lse2 = c.run(K)
    for i in range(len(lens)):
        for j in range(q_len):
            at = i * q_len + j
            if 4 in c.sees[i][j]:
                assert got[at].isnan().all() and lse2[at].isnan().all()
            else:
                assert torch.equal(got[at], clean[at]) and torch.equal(lse2[at], lse[at]), (i, j)


def test_bad_lengths_pages_and_rows(K):
    c = Tree(V41, 6, [200, 90, 100], 8, 5, seed=13)
    table = torch.from_numpy(c.table.copy())
    table[0, 1] = c.pages
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = torch.tensor([200, 90, 64 * c.width + 1], dtype=torch.int32, device=DEV)
    got, lse = c.run(K, table=table.to(DEV), kv_len=lens, req=torch.tensor([0, 3, 2], dtype=torch.int32, device=DEV), err=err)
    assert err.item() == 4 | 32 | 64
    assert (got[5:] == 0).all() and torch.isneginf(lse[5:]).all()
    rows = decode(V41, 6, c.pool, c.slots(0, 200))
    want = []
    for j in range(5):
        t = np.array([t for t in c.seen(0, j) if not 64 <= t < 128])
        want.append(reference(V41, c.q.double().numpy()[j], rows[t], c.scale))
    check(got[:5], lse[:5], want, "without a page")


def test_shared_tables_strides_and_rows_behind(K):
    c = Tree(FP4, 6, [200, 90], 6, 4, seed=17)
    want, lse = c.run(K)
    check(want, lse, c.want(), "plain")
    wide = torch.zeros((8, 6, 640), dtype=torch.bfloat16, device=DEV)
    wide[..., :512] = c.q.to(DEV)
    big = torch.full((10, 6, 512), 3.0, dtype=torch.bfloat16, device=DEV)
    strided = torch.full((5, c.width + 3), -1, dtype=torch.int32)
    strided[3, :c.width], strided[1, :c.width] = torch.from_numpy(c.table[0]), torch.from_numpy(c.table[1])
    got, lse2 = c.run(K, q=wide[..., :512], out=big[:8], table=strided.to(DEV)[:, :c.width],
                      req=torch.tensor([3, 1], dtype=torch.int32, device=DEV))
    assert torch.equal(got, want) and torch.equal(lse, lse2) and (big[8:] == 3).all()


@pytest.mark.parametrize("q_len", [1, 2, 31, 63, 64, 65, 128, 129, 300, 1024])
@pytest.mark.parametrize("deep", [False, True])
def test_tree_mask(K, q_len, deep):
    n = 5
    parent = some_parents(n, q_len, q_len, deep)
    wide = torch.full((n, q_len + 3), 99, dtype=torch.int32, device=DEV)
    wide[:, :q_len] = torch.from_numpy(parent).to(DEV)
    words = (q_len + 63) // 64
    mask = torch.full((n + 1, q_len, words), -7, dtype=torch.int64, device=DEV)
    pos = torch.full((n + 1, q_len), -7, dtype=torch.int32, device=DEV)
    lens = [q_len, q_len + 1000, 0, q_len // 2, q_len + 5]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    K.kvq_tree_mask(wide[:, :q_len], mask[:n], kv_len=torch.tensor(lens, dtype=torch.int32, device=DEV), pos=pos[:n], err=err)
    assert err.item() == 0 and (mask[n] == -7).all() and (pos[n] == -7).all()
    for i in range(n):
        sees = lines(parent[i])
        assert np.array_equal(mask[i].cpu().numpy(), words_of(sees, q_len))
        assert pos[i].tolist() == [max(0, lens[i] - q_len + len(s) - 1) for s in sees]
    K.kvq_tree_mask(wide[:, :q_len], mask[:n])
    K.kvq_tree_mask(wide[:, :q_len], mask[:n], pos=pos[:n])
    assert pos[0].tolist() == [len(s) - 1 for s in lines(parent[0])]


def test_tree_mask_bad_parents(K):
    """A parent that is no earlier token counts as -1."""
    parent = torch.tensor([[-1, 0, 2, 7, -2, 4], [-1, 0, 1, 2, 3, 4]], dtype=torch.int32, device=DEV)
    mask = torch.empty((2, 6, 1), dtype=torch.int64, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    K.kvq_tree_mask(parent, mask, err=err)
    assert err.item() == 32
    assert mask[0, :, 0].tolist() == [1, 3, 4, 8, 16, 48] and mask[1, :, 0].tolist() == [1, 3, 7, 15, 31, 63]


def test_tree_captured(K):
    """Mask and attention in a graph, replayed over other trees and lengths."""
    c = Tree(V41, 6, [200, 90, 30], 8, 20, seed=23)
    q, pool, table = c.q.to(DEV), torch.from_numpy(c.pool).to(DEV), torch.from_numpy(c.table).to(DEV)
    table.clamp_(0, c.pages - 1)
    parent = torch.zeros((3, 20), dtype=torch.int32, device=DEV) - 1
    lens = torch.zeros(3, dtype=torch.int32, device=DEV)
    mask, pos = torch.zeros((3, 20, 1), dtype=torch.int64, device=DEV), torch.zeros((3, 20), dtype=torch.int32, device=DEV)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=DEV)
    ws = torch.empty(K.attend_workspace(160), dtype=torch.uint8, device=DEV)

    def step():
        K.kvq_tree_mask(parent, mask, kv_len=lens, pos=pos)
        K.kvq_attend_tree(V41, 6, q, pool, c.pages, table, lens, mask, out, ws, scale=c.scale, lse=lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed, ls in ((1, [200, 90, 30]), (2, [20, 0, 25])):
        p = some_parents(3, 20, seed)
        parent.copy_(torch.from_numpy(p))
        lens.copy_(torch.tensor(ls))
        graph.replay()
        torch.cuda.synchronize()
        c.lens, c.sees = ls, [lines(x) for x in p]
        check(out, lse, c.want(), seed)


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads,q_len,lens", [(16, 1, [70]), (4, 8, [5000, 0, 9]), (64, 3, [700, 64, 9000])])
def test_a_wait_that_gives_up(K, layout, heads, q_len, lens):
    """With a limit of 0 every wait gives up: all rows are NaN, nothing behind them is written, and the next call is right."""
    c = Tree(layout, 6, lens, heads, q_len, seed=31)
    n = len(lens) * q_len
    big = torch.full((n + 1, heads, 512), 3.0, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    before = K.attend_wait_limit(0)
    try:
        out, lse = c.run(K, out=big[:n], err=err)
    finally:
        K.attend_wait_limit(before)
    assert err.item() == 16 and out.isnan().all() and lse.isnan().all() and (big[n] == 3).all()
    err.zero_()
    out, lse = c.run(K, err=err)
    assert err.item() == 0
    check(out, lse, c.want(), "after")


def test_binding_refuses(K):
    c = Tree(V41, 6, [20, 9], 4, 3, seed=29)
    m = c.mask
    for bad in (m[:1], m[:, :2], m[..., 0], m.int(), torch.cat((m, m), 2)):
        with pytest.raises((TypeError, ValueError)):
            c.run(K, mask=bad)
    parent = torch.zeros((2, 3), dtype=torch.int32, device=DEV)
    mask = torch.zeros((2, 3, 1), dtype=torch.int64, device=DEV)
    for bad in (dict(parent=parent.long()), dict(mask=mask[:1]), dict(mask=mask.int()), dict(pos=parent[:1]), dict(pos=mask),
                dict(kv_len=parent[0]), dict(parent=parent.T), dict(err=mask), dict(mask=mask.cpu())):
        with pytest.raises((TypeError, ValueError)):
            K.kvq_tree_mask(**(dict(parent=parent, mask=mask) | bad))
