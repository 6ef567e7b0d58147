"""kvq_evict_select and kvq_evict_move: whole numbers and bytes, compared for equality with plain Python."""
import numpy as np
import pytest
import torch

import oracle as O
from test_attend_gpu import DEV, FP4, V41, K  # noqa: F401

pytestmark = pytest.mark.gpu


def chosen(row, n, keep, first, last):
    """The tokens that stay, from the definition."""
    if n <= keep:
        return list(range(n))
    free = list(range(first, n - last))
    value = [np.inf if np.isnan(row[t]) else float(row[t]) for t in free]
    nan = [bool(np.isnan(row[t])) for t in free]
    order = sorted(range(len(free)), key=lambda i: (not nan[i], -value[i], free[i]))
    return sorted(list(range(first)) + [free[i] for i in order[:keep - first - last]] + list(range(n - last, n)))


def select(K, mass, lens, keep, first, last, rows=None, err=None):
    kept = torch.full((len(lens), keep), -7, dtype=torch.int32, device=DEV)
    count = torch.full((len(lens),), -7, dtype=torch.int32, device=DEV)
    K.kvq_evict_select(mass.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), kept, count, first=first, last=last,
                       rows=rows, err=err)
    torch.cuda.synchronize()
    return kept.cpu().numpy(), count.cpu().tolist()


def weights(kind, n, width, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "spread":
        return torch.exp(3 * torch.randn((n, width), generator=g))
    if kind == "zeros":
        return torch.where(torch.rand((n, width), generator=g) < 0.9, 0.0, torch.rand((n, width), generator=g))
    if kind == "few":      # a handful of values, both zeros, both signs
        return torch.tensor([0.0, -0.0, 1.0, -1.0, 1e-40, -1e-40, 3.0])[torch.randint(0, 7, (n, width), generator=g)]
    if kind == "odd":
        m = torch.randn((n, width), generator=g)
        m[:, ::7], m[:, 3::11], m[:, 5::13] = float("nan"), float("inf"), -float("inf")
        return m
    if kind == "near":     # differ in the last bits alone
        return (torch.randint(0, 3000, (n, width), generator=g) + 0x3F800000).to(torch.int32).view(torch.float32)
    return torch.full((n, width), 0.25)


@pytest.mark.parametrize("kind", ["spread", "zeros", "few", "odd", "near", "same"])
@pytest.mark.parametrize("lens,keep,first,last", [
    ([1], 1, 0, 0), ([2], 1, 0, 0), ([2], 1, 1, 0), ([2], 1, 0, 1), ([0, 1, 5, 6, 7], 6, 2, 2), ([33, 64, 65, 31], 32, 0, 0),
    ([1000, 999, 10, 0, 501], 500, 4, 100), ([4097, 4096, 2049], 2048, 4, 128), ([5000], 4999, 0, 0), ([5000], 1, 0, 0),
    ([20001, 8193, 300], 701, 0, 33), ([40000, 39999], 20000, 20000, 0), ([32768], 16000, 7, 15000)])
def test_select(K, kind, lens, keep, first, last):
    width = max(lens) + 3
    mass = weights(kind, len(lens), width, keep)
    kept, count = select(K, mass, lens, keep, first, last)
    for i, n in enumerate(lens):
        want = chosen(mass[i].numpy(), n, keep, first, last)
        assert count[i] == len(want)
        assert kept[i].tolist() == want + [-1] * (keep - len(want)), (kind, i)


@pytest.mark.parametrize("n,keep", [(131072, 65536), (400003, 1000), (400003, 399000)])
def test_select_long(K, n, keep):
    """Sequences longer than a cluster's CTAs hold in shared memory; numpy's stable sort."""
    mass = weights("zeros", 2, n + 64, 5)
    kept, count = select(K, mass, [n, n - 1], keep, 16, 512)
    for i, length in enumerate((n, n - 1)):
        free = np.argsort(-mass[i, 16:length - 512].numpy(), kind="stable")[:keep - 528] + 16
        want = np.concatenate((np.arange(16), np.sort(free), np.arange(length - 512, length)))
        assert count[i] == keep and np.array_equal(kept[i], want)


def test_select_rows_and_bad_ones(K):
    mass = weights("spread", 5, 200, 6)
    rows = torch.tensor([4, 0, 4, -1, 5, 2, 1], dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = [150, 60, 200, 50, 50, 201, -3]
    kept, count = select(K, mass, lens, 40, 1, 2, rows=rows, err=err)
    assert err.item() == 32 | 64
    for i, r in enumerate([4, 0, 4]):      # the same row twice is only read
        assert kept[i].tolist() == chosen(mass[r].numpy(), lens[i], 40, 1, 2)
    assert count[3:] == [0] * 4 and (kept[3:] == -1).all()
    # strided rows of weights and of the output
    big = torch.zeros((3, 300), device=DEV)
    big[:, :200] = mass[:3].to(DEV)
    out = torch.full((3, 64), -7, dtype=torch.int32, device=DEV)
    n = torch.tensor([200, 0, 41], dtype=torch.int32, device=DEV)
    c = torch.empty(3, dtype=torch.int32, device=DEV)
    K.kvq_evict_select(big[:, :200], n, out[:, :40], c, first=1, last=2)
    assert (out[:, 40:] == -7).all() and c.tolist() == [40, 0, 40]
    assert out[0, :40].tolist() == chosen(mass[0].numpy(), 200, 40, 1, 2) and out[2, :40].tolist() == chosen(mass[2].numpy(), 41, 40, 1, 2)


def moved(pool, layout, pb, pages, table, new, kept):
    """The pool after the move, byte by byte."""
    P, bpt = 1 << pb, O.bytes_per_token(layout)
    cb = 512 if layout == V41 else 256
    sb = bpt - cb
    src = pool.reshape(pages, P * bpt)
    got = src.copy()
    for i in range(kept.shape[0]):
        for k, t in enumerate(kept[i]):
            if t < 0:
                continue
            a, b, r, d = table[i][t >> pb], new[i][k >> pb], t & (P - 1), k & (P - 1)
            got[b, d * cb:(d + 1) * cb] = src[a, r * cb:(r + 1) * cb]
            got[b, P * cb + d * sb:P * cb + (d + 1) * sb] = src[a, P * cb + r * sb:P * cb + (r + 1) * sb]
    return got.reshape(-1)


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("pb", [2, 4, 6, 8])
def test_move(K, layout, pb):
    rng = np.random.default_rng(pb)
    P, n_seq, keep, width = 1 << pb, 3, 77, -(-300 // (1 << pb))
    need = -(-keep // P)
    pages = n_seq * (width + need) + 2
    pool = rng.integers(0, 256, pages * P * O.bytes_per_token(layout), dtype=np.uint8)
    perm = rng.permutation(pages)
    table = perm[:n_seq * width].reshape(n_seq, width).astype(np.int32)
    new = perm[n_seq * width:n_seq * (width + need)].reshape(n_seq, need).astype(np.int32)
    kept = np.full((n_seq, keep), -1, np.int32)
    for i, c in enumerate((77, 1, 40)):
        kept[i, :c] = np.sort(rng.permutation(300)[:c])
    mass = torch.rand((n_seq, width * P))
    out = torch.full((n_seq, keep + 3), 9.0, device=DEV)
    d = torch.from_numpy(pool).to(DEV)
    K.kvq_evict_move(layout, pb, d, pages, torch.from_numpy(table).to(DEV), torch.from_numpy(new).to(DEV),
                     torch.from_numpy(kept).to(DEV), mass=mass.to(DEV), mass_out=out)
    assert np.array_equal(d.cpu().numpy(), moved(pool, layout, pb, pages, table, new, kept))
    for i in range(n_seq):
        live = torch.from_numpy(kept[i] >= 0)
        want = torch.where(live, mass[i][torch.from_numpy(kept[i]).long().clamp_min(0)], 9.0)
        assert torch.equal(out[i, :keep].cpu(), want) and (out[i, keep:] == 9).all()
    d = torch.from_numpy(pool).to(DEV)      # without weights, table rows by way of req
    req = torch.tensor([2, 2, 0], dtype=torch.int32, device=DEV)
    K.kvq_evict_move(layout, pb, d, pages, torch.from_numpy(table).to(DEV), torch.from_numpy(new).to(DEV),
                     torch.from_numpy(kept).to(DEV), req=req)
    assert np.array_equal(d.cpu().numpy(), moved(pool, layout, pb, pages, table[[2, 2, 0]], new, kept))


def test_move_bad_entries(K):
    """Bad pages, entries and rows move nothing, and say so."""
    rng = np.random.default_rng(3)
    pages, keep = 12, 70
    pool = rng.integers(0, 256, pages * 64 * 528, dtype=np.uint8)
    table = np.array([[0, 1, 2], [3, 99, 4], [5, 6, 7]], np.int32)
    new = np.array([[8, 9], [10, -1], [11, 11]], np.int32)
    kept = np.tile(np.arange(keep, dtype=np.int32), (3, 1))
    kept[0, 5], kept[0, 6] = 192, -9
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(req=None):
        d = torch.from_numpy(pool).to(DEV)
        err.zero_()
        K.kvq_evict_move(V41, 6, d, pages, torch.from_numpy(table).to(DEV), torch.from_numpy(new[:, :2].copy()).to(DEV),
                         torch.from_numpy(kept).to(DEV), req=req, err=err)
        return d.cpu().numpy()
    want = kept.copy()
    want[0, 5:7] = -1
    want[1, 64:] = -1
    t2 = table.copy()
    t2[1, 1] = 0
    got = run(torch.tensor([0, 1, 3], dtype=torch.int32, device=DEV))
    want[2] = -1
    assert err.item() == 1 | 4 | 32
    assert np.array_equal(got, moved(pool, V41, 6, pages, t2, np.maximum(new, 0), want))


def test_rows_that_stay_where_they_are(K):
    """The new table may begin with old pages of which every row stays."""
    rng = np.random.default_rng(4)
    pool = rng.integers(0, 256, 6 * 64 * 288, dtype=np.uint8)
    table, new = np.array([[2, 0, 4]], np.int32), np.array([[2, 5]], np.int32)
    kept = np.concatenate((np.arange(64), np.arange(70, 128), [190, 191])).astype(np.int32)[None]
    d = torch.from_numpy(pool).to(DEV)
    K.kvq_evict_move(FP4, 6, d, 6, torch.from_numpy(table).to(DEV), torch.from_numpy(new).to(DEV), torch.from_numpy(kept).to(DEV))
    assert np.array_equal(d.cpu().numpy(), moved(pool, FP4, 6, 6, table, new, kept))


def test_select_and_move_captured(K):
    """Both calls in a graph, replayed over other weights and lengths."""
    n, width, keep = 3, 512, 100
    mass, lens = torch.zeros((n, width), device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
    kept, count = torch.zeros((n, keep), dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
    rng = np.random.default_rng(7)
    pool = rng.integers(0, 256, 32 * 64 * 528, dtype=np.uint8)
    table = torch.arange(24, dtype=torch.int32).view(3, 8)
    new = torch.arange(24, 30, dtype=torch.int32).view(3, 2)
    d, td, nd = torch.from_numpy(pool).to(DEV), table.to(DEV), new.to(DEV)
    out = torch.zeros((n, keep), device=DEV)

    def step():
        K.kvq_evict_select(mass, lens, kept, count, first=2, last=5)
        K.kvq_evict_move(V41, 6, d, 32, td, nd, kept, mass=mass, mass_out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed, ls in ((1, [512, 100, 7]), (2, [0, 101, 511])):
        m = weights("spread", n, width, seed)
        mass.copy_(m)
        lens.copy_(torch.tensor(ls))
        d.copy_(torch.from_numpy(pool))
        graph.replay()
        torch.cuda.synchronize()
        want = np.full((n, keep), -1, np.int32)
        for i in range(n):
            c = chosen(m[i].numpy(), ls[i], keep, 2, 5)
            want[i, :len(c)] = c
        assert np.array_equal(kept.cpu().numpy(), want)
        assert np.array_equal(d.cpu().numpy(), moved(pool, V41, 6, 32, table.numpy(), new.numpy(), want))


@pytest.mark.parametrize("width", [20000, 100000, 200000])
def test_select_captured_in_clusters(K, width):
    """Sequences that a cluster's CTAs share, in a graph, replayed over other weights and lengths."""
    keep = width // 3
    mass, lens = torch.zeros((2, width), device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    kept, count = torch.zeros((2, keep), dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        K.kvq_evict_select(mass, lens, kept, count, first=3, last=50)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.kvq_evict_select(mass, lens, kept, count, first=3, last=50)
    for seed, ls in ((1, [width, width // 2]), (2, [keep, width - 1])):
        m = weights("zeros", 2, width, seed)
        mass.copy_(m)
        lens.copy_(torch.tensor(ls))
        graph.replay()
        torch.cuda.synchronize()
        for i, n in enumerate(ls):
            if n <= keep:
                want = np.arange(n)
            else:
                free = np.argsort(-m[i, 3:n - 50].numpy(), kind="stable")[:keep - 53] + 3
                want = np.concatenate((np.arange(3), np.sort(free), np.arange(n - 50, n)))
            assert count[i] == want.size and np.array_equal(kept[i, :want.size].cpu().numpy(), want)


def test_binding_refuses(K):
    mass, lens = torch.zeros((2, 64), device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    kept, count = torch.zeros((2, 8), dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    for bad in (dict(mass=mass.double()), dict(mass=mass[0]), dict(mass=mass[:1]), dict(kept=kept[:1]), dict(kept=kept.long()),
                dict(count=count[:1]), dict(kv_len=lens.long()), dict(kv_len=lens.cpu()), dict(rows=lens[:1]), dict(first=9),
                dict(mass=mass.T), dict(err=lens.float())):
        a = dict(mass=mass, kv_len=lens, kept=kept, count=count) | bad
        with pytest.raises((TypeError, ValueError, K.KVQError)):
            K.kvq_evict_select(**a)
    pool = torch.zeros(4 * 64 * 528, dtype=torch.uint8, device=DEV)
    table, new = torch.zeros((2, 1), dtype=torch.int32, device=DEV), torch.ones((2, 1), dtype=torch.int32, device=DEV)
    for bad in (dict(pool=pool[1:]), dict(pool_pages=5), dict(page_table=table[:1]), dict(new_table=new[:1]), dict(kept=kept[:1]),
                dict(mass=mass), dict(mass_out=mass), dict(rows=lens), dict(mass=mass, mass_out=mass), dict(layout=5),
                dict(page_bits=3), dict(mass=mass, mass_out=torch.zeros((2, 7), device=DEV)), dict(req=lens[:1])):
        a = dict(layout=V41, page_bits=6, pool=pool, pool_pages=4, page_table=table, new_table=new, kept=kept) | bad
        with pytest.raises((TypeError, ValueError, K.KVQError)):
            K.kvq_evict_move(**a)
