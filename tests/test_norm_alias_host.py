"""kvq_norm_quant's residual_out beside its inputs, without a GPU: rows that overlap an input's without being them are
refused on the host (no call here reaches a launch)."""
import pytest

from test_attend_host import L, _norm  # noqa: F401

X, RES, RO, CODES, SCALES = 0x100000, 0x200000, 0x300000, 0x400000, 0x500000


def call(L, **kw):
    return _norm(L, **{**dict(x=X, res=RES, ro=RO, codes=CODES, scales=SCALES, w=0x600000), **kw})


# bf16 rows of 512 elements (1024 bytes), 4 of them, 512 elements apart unless said
@pytest.mark.parametrize("bad", [
    dict(ro=RES, ros=1024), dict(ro=X, ros=520), dict(ro=RES, rs=1024), dict(ro=X, xs=2048),   # another stride
    dict(ro=RES + 1024), dict(ro=RES - 1024), dict(ro=X + 3 * 1024), dict(ro=X - 3 * 1024),    # shifted by rows
    dict(ro=RES + 16), dict(ro=X - 512), dict(ro=X + 3 * 1024 + 1008), dict(ro=RES - 4096 + 16),  # by parts of one
    dict(ro=RES + 1008, ros=1024, rs=1024), dict(ro=RES + 1040, ros=1024, rs=1024),            # within wider rows
    dict(ro=RES + 2 * 1024, ros=1536, rs=1024), dict(n=1, ro=X + 16), dict(n=1, ro=RES - 1008),
    dict(ro=X, ros=1024, res=X), dict(n=1000, ro=RES + 999 * 1024),
])
def test_overlaps_are_refused(L, bad):
    assert call(L, **bad) == 1, bad
