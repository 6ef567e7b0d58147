"""KVQ_ROPE_INVERSE is the transpose: with a table of amplitude A it turns back what a table of amplitude 1 / A turned, and after
the same table it leaves A * A.

A pair of length r is turned with three roundings a value, 2^-24 of at most A r each, and by cosines and sines that are off by
2^-22 A; there and back that is below 2^-19 times the two amplitudes times r.
"""
import pytest
import torch

from test_rope_gpu import DEV, K  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("amplitude", [1.0, 1.1, 1.3465735902799727, 0.5])
def test_there_and_back(K, half, amplitude):
    n, heads, dim, rot = 40, 3, 96, 64
    g = torch.Generator().manual_seed(2)
    x = torch.randn((n, heads, dim), generator=g)
    pos = torch.randint(0, 5000, (n,), generator=g).to(torch.int32).to(DEV)
    tables = []
    for a in (amplitude, 1 / amplitude):
        tables.append(torch.empty((5000, rot), device=DEV))
        K.kvq_rope_table(K.rope_frequencies(rot, factor=8, original=1024).to(DEV), tables[-1], amplitude=a)
    part = x[..., 16:16 + rot].double()
    u, v = (part[..., :rot // 2], part[..., rot // 2:]) if half else (part[..., 0::2], part[..., 1::2])
    r = (u * u + v * v).sqrt()
    r = torch.cat((r, r), -1) if half else r.repeat_interleave(2, -1)
    for back, left in ((tables[0], amplitude * amplitude), (tables[1], 1.0)):
        there, got = torch.empty((n, heads, dim), device=DEV), torch.empty((n, heads, dim), device=DEV)
        K.kvq_rope(x.to(DEV), pos, tables[0], there, start=16, half=half)
        K.kvq_rope(there, pos, back, got, start=16, half=half, inverse=True)
        off = (got[..., 16:16 + rot].cpu().double() - left * part).abs()
        assert (off <= 2.0 ** -19 * left * r).all()
        assert torch.equal(got[..., :16].cpu(), x[..., :16]) and torch.equal(got[..., 16 + rot:].cpu(), x[..., 16 + rot:])
