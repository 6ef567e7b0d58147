"""kvq_rope and kvq_rope_table against their definitions.

The rotation is (u c - v s, v c + u s) in fp32 with every product and sum
rounded, then rounded to the rows' type: torch's elementwise operations on the
CPU do the same, so the bits are compared.

A table's value is off by at most 2^-22 of the amplitude: the angle x within
pi / 4 by 3 roundings of 2^-24 (its conversion, the factor and the product), of
which the derivative leaves |x cos x| or |x sin x| <= 0.56 of it, 1.0e-7; the
phase's 32 bits 1.5e-9; the series' end 4e-9; its last sum 2^-25; the
amplitude's product 2^-24: 2.0e-7 in all, below 2^-22 = 2.4e-7.  The angle
itself is p f in 64 bits, off by 2^-52 of it on either side.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def K():
    from compress_kv_write_gb300 import build
    build.build()
    import compress_kv_write_gb300 as K
    K.lib()
    return K


def turned(x, pos, table, start, half, inverse):
    """The definition on the CPU, bit for bit."""
    rot = table.shape[1]
    r = rot // 2
    z = x.float().clone()
    c, s = table[pos.long(), None, :r], table[pos.long(), None, r:]
    if inverse:
        s = -s
    part = z[..., start:start + rot]
    u, v = (part[..., :r].clone(), part[..., r:].clone()) if half else (part[..., 0::2].clone(), part[..., 1::2].clone())
    a, b = u * c - v * s, v * c + u * s
    if half:
        part[..., :r], part[..., r:] = a, b
    else:
        part[..., 0::2], part[..., 1::2] = a, b
    return z.to(x.dtype)


def bits(t):
    return t.cpu().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def table_of(rot, rows=97):
    a = torch.arange(rows, dtype=torch.float64)[:, None] * 10000.0 ** (-2 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    return torch.cat((a.cos(), a.sin()), 1).float()


def problem(n, heads, dim, rot, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, heads, dim), generator=g).to(dtype)
    pos = torch.randint(0, 97, (n,), generator=g).to(torch.int32)
    return x, pos, table_of(rot)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("n,heads,dim,start,rot", [
    (1, 1, 64, 0, 64), (1, 16, 512, 448, 64), (3, 5, 512, 448, 64), (700, 3, 128, 0, 64), (2, 128, 512, 448, 64),
    (5, 7, 192, 32, 96), (4, 3, 66, 2, 62), (3, 2, 7, 1, 6), (2, 9, 2, 0, 2), (1, 130, 40, 0, 16), (2, 2, 4096, 1000, 1024),
    (2, 3, 24, 8, 16), (1, 1, 8200, 4, 20), (9, 1, 512, 0, 512), (6, 5, 128, 88, 40), (3, 4, 44, 4, 24), (2, 3, 20, 2, 12),
    (5, 300, 36, 0, 36), (2, 2, 6000, 0, 8)])
def test_rope(K, dtype, half, inverse, n, heads, dim, start, rot):
    x, pos, table = problem(n, heads, dim, rot, dtype, n * 31 + dim)
    want = turned(x, pos, table, start, half, inverse)
    xd = x.to(DEV)
    out = torch.full((n + 1, heads, dim), 7.0, dtype=dtype, device=DEV)
    K.kvq_rope(xd, pos.to(DEV), table.to(DEV), out[:n], start=start, half=half, inverse=inverse)
    torch.cuda.synchronize()
    assert torch.equal(bits(out[:n]), bits(want)) and (out[n] == 7).all() and torch.equal(bits(xd), bits(x))
    K.kvq_rope(xd, pos.to(DEV), table.to(DEV), xd, start=start, half=half, inverse=inverse)
    torch.cuda.synchronize()
    assert torch.equal(bits(xd), bits(want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("half", [False, True])
def test_rope_strides(K, dtype, half):
    n, heads, dim, rot = 6, 4, 96, 32
    x, pos, table = problem(n, heads, dim, rot, dtype, 3)
    want = turned(x, pos, table, 64, half, False)
    p, t = pos.to(DEV), table.to(DEV)
    # heads outermost, and rows beside others
    by_head = torch.zeros((heads, n, dim), dtype=dtype, device=DEV).transpose(0, 1)
    wide = torch.full((n, heads, 2 * dim), 5.0, dtype=dtype, device=DEV)
    wide[..., :dim] = x.to(DEV)
    K.kvq_rope(wide[..., :dim], p, t, by_head, start=64, half=half)
    assert torch.equal(bits(by_head), bits(want))
    # out beside x within the same rows
    K.kvq_rope(wide[..., :dim], p, t, wide[..., dim:], start=64, half=half)
    assert torch.equal(bits(wide[..., dim:]), bits(want)) and torch.equal(bits(wide[..., :dim]), bits(x))
    # in place in a part of wider rows, the rest as it was
    wide[..., dim:] = 5.0
    K.kvq_rope(wide[..., :dim], p, t, wide[..., :dim], start=64, half=half)
    assert torch.equal(bits(wide[..., :dim]), bits(want)) and (wide[..., dim:] == 5).all()
    # a row repeated by stride 0, an odd offset
    flat = torch.zeros(dim + 1, dtype=dtype, device=DEV)
    flat[1:] = x[0, 0].to(DEV)
    out = torch.zeros((n, heads, dim), dtype=dtype, device=DEV)
    K.kvq_rope(flat[1:].expand(n, heads, dim), p, t, out, start=64, half=half)
    assert torch.equal(bits(out), bits(turned(x[:1, :1].expand(n, heads, dim), pos, table, 64, half, False)))


@pytest.mark.parametrize("dim", [96, 97])
def test_rope_bad_positions_and_nan(K, dim):
    n, heads, rot = 5, 3, 64
    x, pos, table = problem(n, heads, dim, rot, torch.bfloat16, 4)
    x[0, 0, 0], x[1, 1, 40], x[2, 2, 33] = float("nan"), float("inf"), -float("inf")
    want = turned(x, pos, table, 32, False, False)
    bad = pos.clone()
    bad[3], bad[4] = -1, 97
    out = torch.full((n, heads, dim), 7.0, dtype=torch.bfloat16, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    K.kvq_rope(x.to(DEV), bad.to(DEV), table.to(DEV), out, start=32, err=err)
    assert err.item() == 2 and (out[3:] == 7).all()
    a, b = out[:3].float().cpu(), want[:3].float()
    assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a[~a.isnan()], b[~b.isnan()])
    K.kvq_rope(x.to(DEV), bad.to(DEV), table.to(DEV), out, start=32)     # without an error word
    empty = torch.zeros((0, 64), device=DEV)
    err.zero_()
    K.kvq_rope(x.to(DEV), pos.to(DEV), empty, out, start=32, err=err)    # a table of no rows: every position is bad
    assert err.item() == 2


def test_rope_back_and_forth_and_gradient(K):
    """Turning back undoes the turn up to roundings (4 a value of each call), and is the gradient: <R x, y> = <x, R^T y>,
    also against differences, of which a linear map has the exact ones."""
    n, heads, dim, rot = 33, 4, 128, 96
    x, pos, table = problem(n, heads, dim, rot, torch.float32, 5)
    y = torch.randn((n, heads, dim), generator=torch.Generator().manual_seed(6))
    a = [t.to(DEV) for t in (x, y, pos, table)]
    for half in (False, True):
        rx = K.kvq_rope(a[0], a[2], a[3], torch.empty_like(a[0]), start=0, half=half)
        ry = K.kvq_rope(a[1], a[2], a[3], torch.empty_like(a[1]), start=0, half=half, inverse=True)
        back = K.kvq_rope(rx, a[2], a[3], torch.empty_like(rx), start=0, half=half, inverse=True)
        scale = a[0].abs().amax()
        assert (back - a[0]).abs().amax() <= 12 * 2.0 ** -24 * 2 * scale
        lhs, rhs = (rx.double() * a[1].double()).sum(), (a[0].double() * ry.double()).sum()
        assert abs(lhs - rhs) <= 6 * 2.0 ** -24 * (a[0].double().norm() * a[1].double().norm()) * 2
        step = torch.zeros_like(a[0])
        step[:, :, 5] = 1.0
        diff = (K.kvq_rope(a[0] + step, a[2], a[3], torch.empty_like(rx), start=0, half=half) - rx).double()
        # d <R x, y> / d x[5] = (R^T y)[5]; the difference's roundings are 2^-22 of the largest value
        got = (diff * a[1].double()).sum(-1)
        assert (got - ry[..., 5].double()).abs().amax() <= 2.0 ** -20 * (1 + scale) * a[1].abs().amax() * 4


@pytest.mark.parametrize("rot,rows,first", [(64, 1, 0), (64, 8192, 0), (64, 1000, 1048576 - 1000), (2, 100, 3), (6, 777, 5),
                                            (1024, 33, 100000), (128, 70000, 12345), (64, 10, 2 ** 31 - 11), (40, 5000, 0)])
@pytest.mark.parametrize("factor,amplitude", [(1.0, 1.0), (32.0, 1.3465735902799727)])
def test_table(K, rot, rows, first, factor, amplitude):
    freq = K.rope_frequencies(rot, factor=factor)
    table = torch.full((rows + 1, rot), 7.0, device=DEV)
    K.kvq_rope_table(freq.to(DEV), table[:rows], first=first, amplitude=amplitude)
    p = torch.arange(first, first + rows, dtype=torch.float64)[:, None]
    angle = p * freq
    want = torch.cat((angle.cos(), angle.sin()), 1) * amplitude
    tol = amplitude * (2.0 ** -22 + 2.0 ** -50 * torch.cat((angle, angle), 1))
    assert ((table[:rows].cpu().double() - want).abs() <= tol).all() and (table[rows] == 7).all()


def test_table_odd_frequencies(K):
    """Negative, zero and large frequencies; those of which no fraction of a turn is left give NaN, and no other column."""
    freq = torch.tensor([-0.5, 0.0, 1e6, 6.283185307179586, float("nan"), float("inf"), 1e300, 3.0], dtype=torch.float64)
    table = torch.empty((50, 16), device=DEV)
    K.kvq_rope_table(freq.to(DEV), table)
    got = table.cpu().double()
    angle = torch.arange(50, dtype=torch.float64)[:, None] * freq
    want = torch.cat((angle.cos(), angle.sin()), 1)
    odd = torch.tensor([4, 5, 6, 12, 13, 14])
    assert got[:, odd].isnan().all()
    rest = [c for c in range(16) if c not in odd.tolist()]
    tol = 2.0 ** -22 + 2.0 ** -50 * torch.cat((angle, angle), 1).abs()
    assert ((got - want).abs() <= tol)[:, rest].all()


def test_table_serves_the_store(K):
    """Rows stored with the table rotate as rows that kvq_rope turned and the store only quantised."""
    g = torch.Generator().manual_seed(8)
    x = torch.randn((70, 512), generator=g).to(torch.bfloat16).to(DEV)
    pos = torch.randint(0, 5000, (70,), generator=g).to(torch.int32).to(DEV)
    table = torch.empty((5000, 64), device=DEV)
    K.kvq_rope_table(K.rope_frequencies(64, factor=16).to(DEV), table)
    a, b = (torch.zeros(128 * 528, dtype=torch.uint8, device=DEV) for _ in range(2))
    loc = torch.arange(70, device=DEV)
    K.kvq_store(K.V41, 6, K.FLAG_ROPE, x, loc, a, 128, cos_sin=table, pos=pos)
    turned_ = K.kvq_rope(x[:, None], pos, table, torch.empty_like(x[:, None]), start=448)
    K.kvq_store(K.V41, 6, 0, turned_[:, 0], loc, b, 128)
    assert torch.equal(a, b) and a.any()


def test_rope_captured_and_streams(K):
    x, pos, table = problem(40, 6, 512, 64, torch.bfloat16, 9)
    p, t = pos.to(DEV), table.to(DEV)
    xd, out = torch.zeros_like(x, device=DEV), torch.zeros_like(x, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        K.kvq_rope(xd, p, t, out, start=448)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.kvq_rope(xd, p, t, out, start=448)
    xd.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(out), bits(turned(x, pos, table, 448, False, False)))
    out.zero_()
    K.kvq_rope(xd, p, t, out, start=448, stream=side)
    side.synchronize()
    assert torch.equal(bits(out), bits(turned(x, pos, table, 448, False, False)))


def test_rope_binding_refuses(K):
    x = torch.zeros((2, 3, 64), dtype=torch.bfloat16, device=DEV)
    p, t = torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros((4, 64), device=DEV)
    for bad in (dict(x=x[0]), dict(x=x.half()), dict(out=x.float()), dict(out=x[:1]), dict(pos=p[:1]), dict(pos=p.long()),
                dict(cos_sin=t.double()), dict(cos_sin=t[0]), dict(x=x.cpu()), dict(cos_sin=t.cpu()), dict(err=p.long()),
                dict(x=x.transpose(1, 2)), dict(start=2), dict(start=-2), dict(out=x[:, :, :])):
        a = dict(x=x, pos=p, cos_sin=t, out=torch.zeros_like(x), start=0, err=None) | bad
        if "out" in bad and bad["out"].data_ptr() == x.data_ptr() and bad["out"].shape == x.shape and bad["out"].dtype == x.dtype:
            K.kvq_rope(**a)      # x itself is no mistake
            continue
        with pytest.raises((TypeError, ValueError, K.KVQError)):
            K.kvq_rope(**a)
    with pytest.raises(K.KVQError):
        big = torch.zeros((4, 3, 64), dtype=torch.bfloat16, device=DEV)
        K.kvq_rope(big[:2], p, t, big[1:3], start=0)
