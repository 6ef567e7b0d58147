"""kvq_norm_quant with residual_out in or beside its inputs' memory gives the bits of separate buffers."""
import pytest
import torch

from test_norm_quant_gpu import DEV, K, bits  # noqa: F401

pytestmark = pytest.mark.gpu


def run(K, x, w, r, out):
    n, dim = x.shape
    codes = torch.zeros((n, dim), dtype=torch.uint8, device=DEV)
    scales = torch.zeros((n, dim // 32), dtype=torch.uint8, device=DEV)
    K.kvq_norm_quant(x, w, codes, scales, residual=r, residual_out=out)
    torch.cuda.synchronize()
    return codes, scales, out.clone()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,dim", [(1, 96), (700, 512), (4100, 1056), (300, 4096), (65, 16384)])
def test_placements(K, dtype, n, dim):
    g = torch.Generator().manual_seed(n + dim)
    x, r = (torch.randn((n, dim), generator=g).to(dtype).to(DEV) for _ in range(2))
    w = (1 + 0.1 * torch.randn(dim, generator=g)).to(DEV)
    want = run(K, x, w, r, torch.empty_like(x))

    def same(x, r, out, tag):
        got = run(K, x, w, r, out)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), tag
        assert torch.equal(bits(got[2]), bits(want[2])), tag
    x2, r2 = x.clone(), r.clone()
    same(x, r2, r2, "the residual")
    same(x2, r, x2, "x")
    wide = torch.zeros((n, 3 * dim + 64), dtype=dtype, device=DEV)      # columns of one buffer, and in place there
    a, b, c = wide[:, :dim], wide[:, dim:2 * dim], wide[:, 2 * dim + 64:]
    a.copy_(x), b.copy_(r)
    same(a, b, c, "columns of one buffer")
    same(a, b, b, "in place in columns")
    if n > 1:
        # strides that differ, rows that do not touch: x every second row, the sums in between, two apart
        buf = torch.zeros((4 * n, dim), dtype=dtype, device=DEV)
        a, c = buf[0::4], buf[1::2][:n]
        a.copy_(x)
        same(a, r, c, "rows of different strides")
    both = x.clone()
    got = run(K, both, w, both, both)                                   # x is the residual too
    assert torch.equal(bits(got[2]), bits((x.float() + x.float()).to(dtype)))


def test_overlaps_are_refused(K):
    buf = torch.zeros((40, 512), dtype=torch.bfloat16, device=DEV)
    x, w = torch.zeros((8, 512), dtype=torch.bfloat16, device=DEV), torch.ones(512, device=DEV)
    for r, out in ((buf[:8], buf[1:9]), (buf[0:16:2], buf[0:24:3]), (buf[:8], buf[0:16:2])):
        with pytest.raises(K.KVQError):
            run(K, x, w, r, out)
    run(K, x, w, buf[:8], buf[8:16])
    run(K, x, w, buf[0:16:2], buf[1:17:2])
