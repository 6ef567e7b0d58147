"""kvq_norm_quant against the definition in 64 bits.

y = z * rsqrt(mean z^2 + eps) * w is computed in fp32: the sum of squares over
dim values (at most dim/256 + 13 sequential roundings of positive terms), the
division, the addition of eps, a reciprocal square root good to 2^-22 and two
products, so y is off by at most (dim/512 + 16) * 2^-24 + 2^-22 relative; call
it dy.  A code may then differ from the 64-bit one only where y lies within dy
of the middle between two codes, and a scale only where the block's largest
magnitude lies within dy of a power of two.  What the code and scale stand for
is therefore within half an e4m3 step of y (1 +- dy), or saturated at 448.
"""
import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def K():
    from compress_kv_write_gb300 import build
    build.build()
    import compress_kv_write_gb300 as K
    K.lib()
    return K


def check(codes, scales, z, w, eps, dim):
    """codes, scales numpy uint8; z float64 [n, dim], the exact sum."""
    n = z.shape[0]
    dy = (dim / 512 + 16) * 2.0 ** -24 + 2.0 ** -22
    y = z / np.sqrt((z * z).mean(1, keepdims=True) + eps) * w
    yb, cb = y.reshape(n, -1, 32), codes.reshape(n, -1, 32)
    amax = np.abs(yb).max(2)
    lo, hi = (np.clip(np.frexp(amax * (1 + s * dy))[1] - 1 + 127 - 8, 0, None) for s in (-1, 1))
    lo, hi = np.where(amax > 0, lo, 0), np.where(amax > 0, hi, 0)
    sc = scales.astype(np.int64)
    assert ((sc == lo) | (sc == hi)).all()
    assert (lo != hi).mean() < 0.01
    v = O.e4m3_decode(codes).astype(np.float64).reshape(yb.shape)
    u = yb * np.exp2(127.0 - sc)[..., None]
    u = np.clip(u, -448, 448)
    step = np.exp2(np.maximum(np.frexp(u)[1] - 1, -6) - 3.0)
    assert (np.abs(v - u) <= step / 2 + np.abs(u) * dy).all()
    # and to nearest: codes of the 64-bit value wherever it is not within dy of a border
    r = np.round(u / step) * step
    sure = np.abs(np.abs(u / step - np.floor(u / step)) - 0.5) * step > 2 * dy * np.abs(u)
    assert (v == r)[sure].all() and (~sure).mean() < 0.01
    assert (cb[yb == 0] & 0x7F == 0).all()


def bits(t):
    return t.cpu().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("n,dim", [(1, 32), (3, 64), (9, 256), (5, 288), (17, 512), (2, 544), (1, 1056), (33, 2048),
                                   (3, 2080), (7, 4096), (2, 4128), (5, 8192), (1, 8224), (3, 16384), (700, 96), (2, 992), (2050, 4000), (5, 768),
                                   (11, 1280), (4, 1504), (6, 1792)])
def test_norm_quant(K, dtype, residual, n, dim):
    g = torch.Generator().manual_seed(n * 131 + dim)
    x = torch.randn((n, dim), generator=g).to(dtype)
    r = (torch.randn((n, dim), generator=g) * 3).to(dtype)
    w = 1 + 0.1 * torch.randn(dim, generator=g)
    codes = torch.full((n + 1, dim), 0xAA, dtype=torch.uint8, device=DEV)
    scales = torch.full((n + 1, dim // 32), 0xAA, dtype=torch.uint8, device=DEV)
    total = torch.full((n + 1, dim), 9.0, dtype=dtype, device=DEV)
    K.kvq_norm_quant(x.to(DEV), w.to(DEV), codes[:n], scales[:n], eps=1e-5, residual=r.to(DEV) if residual else None,
                     residual_out=total[:n] if residual else None)
    torch.cuda.synchronize()
    # the sum is one fp32 addition: z as the kernel has it
    z = x.float() + r.float() if residual else x.float()
    if residual:
        assert torch.equal(bits(total[:n]), bits(z.to(dtype)))
    assert (codes[n] == 0xAA).all() and (scales[n] == 0xAA).all() and (total[n] == 9).all()
    check(codes[:n].cpu().numpy(), scales[:n].cpu().numpy(), z.double().numpy(), w.double().numpy(), 1e-5, dim)


def test_in_place_and_strided(K):
    n, dim = 37, 1056
    g = torch.Generator().manual_seed(1)
    x = torch.randn((n, dim + 64), generator=g).to(torch.bfloat16).to(DEV)
    r = torch.randn((n, dim), generator=g).to(torch.bfloat16).to(DEV)
    w = (1 + 0.1 * torch.randn(dim, generator=g)).to(DEV)
    codes = torch.zeros((n, dim + 8), dtype=torch.uint8, device=DEV)
    scales = torch.zeros((n, dim // 32 + 3), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(r)
    xs = x[:, 64:]
    K.kvq_norm_quant(xs, w, codes[:, :dim], scales[:, :dim // 32], residual=r, residual_out=out)
    assert (codes[:, dim:] == 0).all() and (scales[:, dim // 32:] == 0).all()
    for target in ("residual", "x"):
        r2, x2 = r.clone(), xs.contiguous()
        c2, s2 = torch.empty((n, dim), dtype=torch.uint8, device=DEV), torch.empty((n, dim // 32), dtype=torch.uint8, device=DEV)
        to = r2 if target == "residual" else x2
        K.kvq_norm_quant(x2, w, c2, s2, residual=r2, residual_out=to)
        torch.cuda.synchronize()
        assert torch.equal(to, out) and torch.equal(c2, codes[:, :dim]) and torch.equal(s2, scales[:, :dim // 32])


def test_zero_rows_extremes_and_the_cache_codec(K):
    """Zero rows give zero codes and scales; large and tiny rows keep their
    codes (the norm cancels the factor); a row of unit scale is quantised as
    kvq_store quantises it."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn((8, 512), generator=g)
    w = torch.ones(512)
    x[0] = 0
    x[2] = x[1] * 2.0 ** 50
    x[3] = x[1] * 2.0 ** -8
    codes = torch.empty((8, 512), dtype=torch.uint8, device=DEV)
    scales = torch.empty((8, 16), dtype=torch.uint8, device=DEV)
    K.kvq_norm_quant(x.to(DEV), w.to(DEV), codes, scales, eps=0.0)
    torch.cuda.synchronize()
    c, s = codes.cpu(), scales.cpu()
    assert torch.equal(c[1], c[2]) and torch.equal(c[1], c[3]) and torch.equal(s[1], s[2]) and torch.equal(s[1], s[3])
    K.kvq_norm_quant(x.to(DEV), w.to(DEV), codes, scales, eps=1e-6)
    torch.cuda.synchronize()
    c, s = codes.cpu(), scales.cpu()
    assert ((c[0] & 0x7F) == 0).all() and (s[0] == 0).all()
    check(c.numpy()[1:], s.numpy()[1:], x.double().numpy()[1:], np.ones(512), 1e-6, 512)
    # rows of +-1 are their own norm up to eps = 0, so both calls quantise the same values
    y = torch.where(torch.rand((64, 512), generator=g) < 0.5, -1.0, 1.0)
    codes, scales = torch.empty((64, 512), dtype=torch.uint8, device=DEV), torch.empty((64, 16), dtype=torch.uint8, device=DEV)
    K.kvq_norm_quant(y.to(DEV), w.to(DEV), codes, scales, eps=0.0)
    pool = torch.zeros(64 * 528, dtype=torch.uint8, device=DEV)
    K.kvq_store(K.V41, 6, 0, y.to(DEV), torch.arange(64, device=DEV), pool, 64)
    torch.cuda.synchronize()
    assert torch.equal(pool[:64 * 512].view(64, 512), codes) and torch.equal(pool[64 * 512:].view(64, 16), scales)


def test_captured_and_refused(K):
    x = torch.randn((5, 128), device=DEV).to(torch.bfloat16)
    w = torch.ones(128, device=DEV)
    codes, scales = torch.zeros((5, 128), dtype=torch.uint8, device=DEV), torch.zeros((5, 4), dtype=torch.uint8, device=DEV)
    K.kvq_norm_quant(x, w, codes, scales)
    want = codes.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.kvq_norm_quant(x, w, codes, scales)
    codes.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(codes, want)
    K.kvq_norm_quant(x[:0], w, codes[:0], scales[:0])
    for bad in (dict(x=x.half()), dict(weight=w.double()), dict(codes=codes.int())):
        with pytest.raises(TypeError):
            K.kvq_norm_quant(**{**dict(x=x, weight=w, codes=codes, scales=scales), **bad})
    for bad in (dict(codes=codes[:, :64]), dict(scales=scales[:4]), dict(residual=x), dict(x=x[:, :64])):
        with pytest.raises(ValueError):
            K.kvq_norm_quant(**{**dict(x=x, weight=w, codes=codes, scales=scales), **bad})
