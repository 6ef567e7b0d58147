"""A speculative decode step as a server makes it: positions and masks from the tree, queries rotated, the drafted tokens'
rows rotated and stored, attention, the outputs turned back, the weights added up; and in between a cache cut to its tokens
of most weight.  Checked against 64 bits, then captured into a graph and replayed over other inputs with the eager calls'
bits.  Then what lies far out in memory, and empty calls."""
import numpy as np
import pytest
import torch

import oracle as O
from test_attend_gpu import DEV, FP4, V41, K, decode, reference  # noqa: F401
from test_attend_gpu import check as check_rows
from test_mass_gpu import Mass, weights
from test_mass_gpu import check as check_mass
from test_rope_gpu import bits, turned
from test_tree_gpu import Tree, lines, some_parents

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", [V41, FP4])
def test_step(K, layout):
    n, q_len, heads, width, pages, keep = 3, 9, 16, 6, 40, 90
    scale = 512 ** -0.5
    g = torch.Generator().manual_seed(5)
    table = torch.randperm(pages, generator=g)[:n * width].view(n, width).to(torch.int32)
    new = torch.tensor([p for p in range(pages) if p not in set(table.view(-1).tolist())][:2 * n], dtype=torch.int32).view(n, 2)
    td, nd = table.to(DEV), new.to(DEV)
    cs = torch.empty((4096, 64), device=DEV)
    K.kvq_rope_table(K.rope_frequencies(64, factor=8, original=1024).to(DEV), cs, amplitude=1.1)
    parent, lens = torch.zeros((n, q_len), dtype=torch.int32, device=DEV) - 1, torch.zeros(n, dtype=torch.int32, device=DEV)
    q, k = (torch.zeros((n * q_len, h, 512), dtype=torch.bfloat16, device=DEV) for h in (heads, 1))
    first = torch.randn((pages * 64, 512), generator=g).to(torch.bfloat16).to(DEV)

    def buffers():
        b = dict(pool=torch.zeros(pages * 64 * O.bytes_per_token(layout), dtype=torch.uint8, device=DEV),
                 mask=torch.zeros((n, q_len, 1), dtype=torch.int64, device=DEV), pos=torch.zeros((n, q_len), dtype=torch.int32, device=DEV),
                 q=torch.zeros_like(q), out=torch.zeros_like(q), turned=torch.zeros_like(q), lse=torch.zeros(q.shape[:2], device=DEV),
                 mass=torch.zeros((n, width * 64), device=DEV), kept=torch.zeros((n, keep), dtype=torch.int32, device=DEV),
                 count=torch.zeros(n, dtype=torch.int32, device=DEV), left=torch.zeros((n, keep), device=DEV),
                 out2=torch.zeros((n, heads, 512), dtype=torch.bfloat16, device=DEV), err=torch.zeros(1, dtype=torch.int32, device=DEV),
                 ws=torch.zeros(K.attend_workspace(q_len * heads), dtype=torch.uint8, device=DEV),
                 ws2=torch.zeros(K.mass_workspace(n, q_len * heads, width * 64), dtype=torch.uint8, device=DEV))
        K.kvq_store(layout, 6, 0, first, torch.arange(pages * 64, device=DEV), b["pool"], pages * 64)
        return b

    def step(b):
        K.kvq_tree_mask(parent, b["mask"], kv_len=lens, pos=b["pos"], err=b["err"])
        K.kvq_rope(q, b["pos"].view(-1), cs, b["q"], start=448, err=b["err"])
        at = (lens[:, None] - q_len + torch.arange(q_len, device=DEV)).long()
        loc = (td.long().gather(1, at >> 6) * 64 + (at & 63)).view(-1)
        K.kvq_store(layout, 6, K.FLAG_ROPE, k[:, 0], loc, b["pool"], pages * 64, cos_sin=cs, pos=b["pos"].view(-1), err=b["err"])
        K.kvq_attend_tree(layout, 6, b["q"], b["pool"], pages, td, lens, b["mask"], b["out"], b["ws"], scale=scale, lse=b["lse"],
                          err=b["err"])
        K.kvq_rope(b["out"], b["pos"].view(-1), cs, b["turned"], start=448, inverse=True, err=b["err"])
        K.kvq_attend_mass(layout, 6, b["q"], b["lse"], b["pool"], pages, td, lens, b["mass"], b["ws2"], scale=scale, mask=b["mask"],
                          prev=b["mass"], decay=0.5, err=b["err"])
        K.kvq_evict_select(b["mass"], lens, b["kept"], b["count"], first=2, last=q_len, err=b["err"])
        K.kvq_evict_move(layout, 6, b["pool"], pages, td, nd, b["kept"], mass=b["mass"], mass_out=b["left"], err=b["err"])
        K.kvq_attend(layout, 6, b["q"][::q_len], b["pool"], pages, nd, b["count"], b["out2"], b["ws"], scale=scale, err=b["err"])

    def fill(seed, ls):
        h = torch.Generator().manual_seed(seed)
        q.copy_((2 * torch.randn(q.shape, generator=h)).to(torch.bfloat16))
        k.copy_(torch.randn(k.shape, generator=h).to(torch.bfloat16))
        parent.copy_(torch.from_numpy(some_parents(n, q_len, seed)))
        lens.copy_(torch.tensor(ls))

    eager, captured = buffers(), buffers()
    fill(1, [300, 80, 9])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(buffers())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(captured)
    total = np.zeros((n, width * 64))
    tol = np.zeros((n, width * 64))
    for seed, ls in ((2, [300, 80, 9]), (3, [309, 89, 18]), (4, [318, 98, 27])):
        fill(seed, ls)
        step(eager)
        graph.replay()
        torch.cuda.synchronize()
        for name in eager:
            if name not in ("ws", "ws2"):
                assert torch.equal(eager[name], captured[name]), (seed, name)
        b = eager
        assert b["err"].item() == 0
        sees = [lines(p) for p in parent.tolist()]
        pos = b["pos"].cpu()
        assert pos.tolist() == [[ls[i] - q_len + len(s) - 1 for s in sees[i]] for i in range(n)]
        assert torch.equal(bits(b["q"]), bits(turned(q.cpu(), pos.view(-1), cs.cpu(), 448, False, False)))
        assert torch.equal(bits(b["turned"]), bits(turned(b["out"].cpu(), pos.view(-1), cs.cpu(), 448, False, True)))
        pool, qd, ld = b["pool"].cpu().numpy(), b["q"].cpu().double().numpy(), b["lse"].cpu().double().numpy()
        want, mass = [], []
        total *= 0.5
        tol = 0.5 * tol + 2.0 ** -22 * total
        for i, m in enumerate(ls):
            t = np.arange(m)
            rows = decode(layout, 6, pool, table[i].numpy().astype(np.int64)[t >> 6] * 64 + (t & 63))
            for j in range(q_len):
                s = np.array(list(range(m - q_len)) + [m - q_len + d for d in sees[i][j]])
                want.append(reference(layout, qd[i * q_len + j], rows[s], scale))
                p, d = weights(layout, qd[i * q_len + j], ld[i * q_len + j], rows[s], scale)
                total[i][s] += p.sum(0)
                tol[i][s] += d.sum(0) + 2.0 ** -20 * p.sum(0)
            mass.append((total[i][:m].copy(), tol[i][:m] + 2.0 ** -20 * total[i][:m] + 1e-36))
        check_rows(b["out"], b["lse"], want, seed)
        check_mass(b["mass"], ls, mass, seed, behind=None)
        assert b["count"].tolist() == [min(m, keep) for m in ls]
        kept = b["kept"].cpu()
        after = []
        for i, m in enumerate(ls):
            t = kept[i][kept[i] >= 0].numpy().astype(np.int64)
            assert (np.diff(t) > 0).all() and t[0] == 0 and t[-1] == m - 1
            rows = decode(layout, 6, pool, table[i].numpy().astype(np.int64)[t >> 6] * 64 + (t & 63))
            after.append(reference(layout, qd[i * q_len], rows, scale))
        check_rows(b["out2"], None, after, (seed, "cut"))


@pytest.mark.parametrize("layout", [V41, FP4])
def test_pools_beyond_32_bits(K, layout):
    """Pages behind the first 4 GB, weights behind 2^32 bytes: the same bits as over a small pool."""
    c = Tree(layout, 6, [200, 90, 77], 8, 5, seed=3)
    want, lse = c.run(K)
    m = Mass(layout, 6, [200, 90, 77], 8, q_len=5, seed=3)
    mass = m.run(K, lse.cpu(), mask=c.mask.to(DEV))
    bpp = 64 * O.bytes_per_token(layout)
    pages = (1 << 32) // bpp + 40
    assert pages * bpp > 1 << 32
    big = torch.zeros(pages * bpp, dtype=torch.uint8, device=DEV)
    shift = pages - c.pages
    big[shift * bpp:] = torch.from_numpy(c.pool).to(DEV).view(-1)
    table = torch.from_numpy(np.where(c.table < c.pages, c.table + shift, c.table)).to(DEV)
    kv = torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    q, out, l2 = c.q.to(DEV), torch.empty_like(want), torch.empty_like(lse)
    ws = torch.empty(K.attend_workspace(40), dtype=torch.uint8, device=DEV)
    K.kvq_attend_tree(layout, 6, q, big, pages, table, kv, c.mask.to(DEV), out, ws, scale=c.scale, lse=l2)
    assert torch.equal(out, want) and torch.equal(l2, lse)
    wide = torch.empty(2 * ((1 << 30) + 64) + 1024, device=DEV).as_strided((3, 256), ((1 << 30) + 64, 1))
    K.kvq_attend_mass(layout, 6, q, lse, big, pages, table, kv, wide, scale=c.scale, mask=c.mask.to(DEV))
    for i, n in enumerate(c.lens):
        assert torch.equal(wide[i, :n], mass[i, :n])
    kept, count = torch.empty((3, 50), dtype=torch.int32, device=DEV), torch.empty(3, dtype=torch.int32, device=DEV)
    K.kvq_evict_select(wide, kv, kept, count, first=1)
    small, c2 = torch.empty_like(kept), torch.empty_like(count)
    K.kvq_evict_select(mass, kv, small, c2, first=1)
    assert torch.equal(kept, small) and torch.equal(count, c2)
    left = torch.empty((3, 50), device=DEV)
    new = torch.tensor([[shift - 1], [shift - 2], [0]], dtype=torch.int32, device=DEV)
    K.kvq_evict_move(layout, 6, big, pages, table, new, kept, mass=wide, mass_out=left)
    got = torch.empty((150, 512), dtype=torch.bfloat16, device=DEV)
    src = torch.empty_like(got)
    K.kvq_dequant_slots(layout, 6, big, pages * 64, (new.long() * 64 + torch.arange(50, device=DEV)).view(-1).contiguous(), got)
    slots = table.long().gather(1, kept.long() >> 6) * 64 + (kept & 63)
    K.kvq_dequant_slots(layout, 6, big, pages * 64, slots.view(-1).contiguous(), src)
    assert torch.equal(got, src) and torch.equal(left, mass.gather(1, kept.long()))


def test_empty_calls(K):
    """No sequences, no tokens, tables without columns: nothing is written, nothing is refused."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    pool = torch.zeros(2 * 64 * 528, dtype=torch.uint8, device=DEV)
    q0, q2 = torch.zeros((0, 4, 512), dtype=torch.bfloat16, device=DEV), torch.zeros((2, 4, 512), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(K.attend_workspace(8), dtype=torch.uint8, device=DEV)
    K.kvq_rope(q0, i32(0), torch.zeros((3, 64), device=DEV), torch.empty_like(q0), start=0)
    K.kvq_rope_table(torch.ones(4, dtype=torch.float64, device=DEV), torch.zeros((0, 8), device=DEV))
    K.kvq_tree_mask(i32(0, 3), torch.zeros((0, 3, 1), dtype=torch.int64, device=DEV))
    K.kvq_attend_tree(V41, 6, q0, pool, 2, i32(0, 1), i32(0), torch.zeros((0, 3, 1), dtype=torch.int64, device=DEV), torch.empty_like(q0),
                      ws, scale=1.0)
    K.kvq_attend_mass(V41, 6, q0, torch.zeros((0, 4), device=DEV), pool, 2, i32(0, 1), i32(0), torch.zeros((0, 64), device=DEV), scale=1.0)
    K.kvq_evict_select(torch.zeros((0, 64), device=DEV), i32(0), i32(0, 5), i32(0))
    K.kvq_evict_move(V41, 6, pool, 2, i32(0, 1), i32(0, 1), i32(0, 5))
    # sequences over a table of no pages are empty ones
    out, lse = torch.full((2, 4, 512), 3.0, device=DEV), torch.zeros((2, 4), device=DEV)
    K.kvq_attend_tree(V41, 6, q2, pool, 2, i32(2, 0), i32(2), torch.ones((2, 1, 1), dtype=torch.int64, device=DEV), out, ws, scale=1.0, lse=lse)
    assert (out == 0).all() and torch.isneginf(lse).all()
    mass = torch.full((2, 64), 5.0, device=DEV)
    K.kvq_attend_mass(V41, 6, q2, lse, pool, 2, i32(2, 0), i32(2), mass, scale=1.0)
    assert (mass == 5).all()
    kept, count = i32(2, 5), i32(2) + 9
    K.kvq_evict_select(torch.zeros((2, 0), device=DEV), i32(2), kept, count)
    assert (kept == -1).all() and (count == 0).all()
    K.kvq_evict_move(V41, 6, pool, 2, i32(2, 0), i32(2, 1), kept)
    assert (pool == 0).all()


def test_other_streams(K):
    """Tensors made on one stream, calls given another: they run there."""
    c = Tree(FP4, 6, [500, 90], 16, 3, seed=9)
    want, lse = c.run(K)
    side = torch.cuda.Stream()
    q, pool = c.q.to(DEV), torch.from_numpy(c.pool).to(DEV)
    table, kv = torch.from_numpy(c.table).to(DEV), torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    parent = torch.tensor([[max(-1, s[-2] if len(s) > 1 else -1) for s in x] for x in c.sees], dtype=torch.int32, device=DEV)
    mask, out, l2 = torch.zeros((2, 3, 1), dtype=torch.int64, device=DEV), torch.empty_like(want), torch.empty_like(lse)
    ws = torch.empty(K.attend_workspace(48), dtype=torch.uint8, device=DEV)
    mass = torch.zeros((2, c.width * 64), device=DEV)
    kept, count = torch.zeros((2, 40), dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    K.kvq_tree_mask(parent, mask, stream=side)
    K.kvq_attend_tree(FP4, 6, q, pool, c.pages, table, kv, mask, out, ws, scale=c.scale, lse=l2, stream=side)
    K.kvq_attend_mass(FP4, 6, q, l2, pool, c.pages, table, kv, mass, scale=c.scale, mask=mask, stream=side)
    K.kvq_evict_select(mass, kv, kept, count, stream=side)
    side.synchronize()
    assert torch.equal(mask.cpu(), c.mask) and torch.equal(out, want) and torch.equal(l2, lse)
    assert count.tolist() == [40, 40] and abs(mass.double().sum().item() - 2 * 48) < 1e-2


@pytest.mark.parametrize("layout", [V41, FP4])
def test_two_streams_at_once(K, layout):
    """Calls with buffers and workspaces of their own, under way on two streams together: the results of one at a time."""
    probs = [Tree(layout, 6, lens, heads, q_len, seed=heads) for lens, heads, q_len in (([3000, 90, 7], 16, 5), ([700, 0, 1500], 64, 3))]
    runs = []
    for c in probs:
        n, rows, width = len(c.lens), c.q_len * c.heads, c.width * 64
        runs.append(dict(c=c, q=c.q.to(DEV), pool=torch.from_numpy(c.pool).to(DEV), table=torch.from_numpy(c.table).to(DEV),
                         kv=torch.tensor(c.lens, dtype=torch.int32, device=DEV), mask=c.mask.to(DEV), out=torch.empty_like(c.q, device=DEV),
                         lse=torch.empty(c.q.shape[:2], device=DEV), mass=torch.zeros((n, width), device=DEV),
                         kept=torch.zeros((n, 200), dtype=torch.int32, device=DEV), count=torch.zeros(n, dtype=torch.int32, device=DEV),
                         ws=torch.empty(K.attend_workspace(rows), dtype=torch.uint8, device=DEV),
                         ws2=torch.empty(K.mass_workspace(n, rows, width), dtype=torch.uint8, device=DEV), stream=torch.cuda.Stream()))

    def go(r, stream):
        c = r["c"]
        K.kvq_attend_tree(layout, 6, r["q"], r["pool"], c.pages, r["table"], r["kv"], r["mask"], r["out"], r["ws"], scale=c.scale,
                          lse=r["lse"], stream=stream)
        K.kvq_attend_mass(layout, 6, r["q"], r["lse"], r["pool"], c.pages, r["table"], r["kv"], r["mass"], r["ws2"], scale=c.scale,
                          mask=r["mask"], stream=stream)
        K.kvq_evict_select(r["mass"], r["kv"], r["kept"], r["count"], last=9, stream=stream)

    alone = []
    for r in runs:
        go(r, None)
        torch.cuda.synchronize()
        alone.append([r[k].clone() for k in ("out", "lse", "mass", "kept", "count")])
        for k in ("out", "lse", "mass", "kept", "count"):
            r[k].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for r in runs:
            go(r, r["stream"])
    torch.cuda.synchronize()
    for r, want in zip(runs, alone):
        for k, w in zip(("out", "lse", "mass", "kept", "count"), want):
            assert torch.equal(r[k], w), k
