"""kvq_attend and kvq_attend_slots against the definition in 64 bits.

Rows are decoded by the oracle (exact in bf16) and attended in numpy float64.
The tolerance counts the roundings of the computation, u = 2^-k for a half
step:

* a score s = scale * sum q k is a 512-term fp32 sum of exact products: off by
  at most 512 * 2^-23 * scale * sum |q k| (2^-23, not 2^-24, for accumulators
  that truncate), plus 2^-22 |s| for its scaling.  Call the largest such bound
  of a row ds;
* a weight p = exp(s - m) is off by 2 ds relative (numerator and the sum),
  2^-21 for the exponential and the exponent's rounding at |s - m| <= 64, and
  the rounding of p * t to fp16, where t is the power of two that the token's
  row is decoded relative to (V41_FP4: 1; V41: the one that brings the row's
  largest scale to 2^7): 2^-11, or below 2^-14 of the largest p * t of the row
  2^-25 of that one;
* a value of a V41 row is decoded as fp16 relative to t, whose subnormals are
  multiples of 2^-24: off by at most 2^-25 t (where no block's scale is 2^-32 of
  the row's largest or less, as here);
* out is a weighted mean of the rows: off by that relative error times
  sum p |k|, 512-step-like accumulation 2^-22 * (blocks + 16) of the same sum,
  and its own rounding, 2^-8 |out| for bf16;
* lse = log(sum): ds + 2^-20 + 2^-22 |lse|.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
V41, FP4 = 1, 2


@pytest.fixture(scope="module")
def K():
    from compress_kv_write_gb300 import build
    build.build()
    import compress_kv_write_gb300 as K
    K.lib()
    return K


def bf16_to_f64(u16):
    return (u16.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def decode(layout, page_bits, pool, slots):
    """float64 [n, 512] rows of a numpy pool."""
    slots = np.asarray(slots, np.int64)
    bpt, P = O.bytes_per_token(layout), 1 << page_bits
    cb = 512 if layout == V41 else 256
    sb = bpt - cb
    # the oracle reads pages of 64: copy the rows into pages of its own
    n = max(64, -(-slots.size // 64) * 64)
    mine = np.zeros(n * bpt, np.uint8)
    for i, s in enumerate(slots):
        src, dst = (s >> page_bits) * P * bpt, (i >> 6) * 64 * bpt
        r, d = s & (P - 1), i & 63
        mine[dst + d * cb:dst + (d + 1) * cb] = pool[src + r * cb:src + (r + 1) * cb]
        mine[dst + 64 * cb + d * sb:dst + 64 * cb + (d + 1) * sb] = pool[src + P * cb + r * sb:src + P * cb + (r + 1) * sb]
    rc, ws = O.dequant(layout, 6, mine, np.arange(n // 64, dtype=np.int32), n)
    assert rc == O.OK
    return bf16_to_f64(ws)[:slots.size]


def make_pool(layout, page_bits, slots, seed):
    """numpy pool whose every slot holds a quantised row."""
    from compress_kv_write_gb300 import synth
    x = synth.store_rows_bf16(slots, "cpu", seed, outlier_scale=8.0)
    pool = np.zeros(slots * O.bytes_per_token(layout), np.uint8)
    assert O.store(layout, page_bits, 0, x.view(torch.int16).numpy().view(np.uint16), np.arange(slots), pool) == O.OK
    return pool


def queries(n, heads, seed, std=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((n, heads, 512), generator=g) * std).to(torch.bfloat16)


def row_power(layout, rows):
    """The power of two that each row is decoded relative to (a V41 block's largest code is 2^8 to 448)."""
    if layout == FP4:
        return np.ones(rows.shape[0])
    amax = np.abs(rows).max(1)
    top = np.where(amax > 0, np.frexp(amax)[1] - 1 - 8, -127)          # the largest scale's exponent
    return np.ldexp(1.0, np.maximum(top, -40) - 7)


def reference(layout, q, rows, scale):
    """q float64 [h, 512] over rows [n, 512]: (out, lse, tol_out without the output's rounding, tol_lse)."""
    h = q.shape[0]
    if rows.shape[0] == 0:
        z = np.zeros((h, 512))
        return z, np.full(h, -math.inf), z, np.zeros(h)
    s = q @ rows.T * scale
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(1, keepdims=True)
    out = p @ rows / l
    lse = (m + np.log(l))[:, 0]
    ds = (512 * 2.0 ** -23 * abs(scale) * (np.abs(q) @ np.abs(rows).T) + 2.0 ** -22 * np.abs(s)).max(1)
    mean = p @ np.abs(rows) / l
    blocks = -(-rows.shape[0] // 64)
    rel = 2 * ds + 2.0 ** -21 + 2.0 ** -22 * (blocks + 16) + 2.0 ** -11
    t = row_power(layout, rows)
    tol = rel[:, None] * mean + 2.0 ** -25 * (p * t).max(1, keepdims=True) * (np.abs(rows) / t[:, None]).sum(0) / l
    if layout == V41:
        tol = tol + 2.0 ** -25 * (p @ t)[:, None] / l
    return out, lse, tol, ds + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse)


def check(got, lse, want, tag):
    """want: list over query tokens of reference() tuples."""
    out = got.detach().float().cpu().numpy().astype(np.float64)
    lse = None if lse is None else lse.cpu().numpy().astype(np.float64)
    rnd = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -22
    for t, (o, l, tol, tl) in enumerate(want):
        assert np.isfinite(out[t]).all(), (tag, t)
        bad = np.abs(out[t] - o) > tol + rnd * np.abs(o) + 1e-30
        assert not bad.any(), (tag, t, int(bad.sum()), np.argwhere(bad)[:4], np.abs(out[t] - o).max())
        if lse is not None:
            none = np.isneginf(l)
            assert (np.isneginf(lse[t]) == none).all(), (tag, t)
            off = np.abs(lse[t][~none] - l[~none])
            assert (off <= tl[~none]).all(), (tag, t, off.max())


class Paged:
    """A paged problem: numpy pool, table of distinct physical pages, lengths."""

    def __init__(self, layout, page_bits, lens, heads, q_len=1, seed=0, width_more=0):
        self.layout, self.pb, self.lens, self.heads, self.q_len = layout, page_bits, list(lens), heads, q_len
        P = 1 << page_bits
        need = [-(-n // P) for n in lens]
        pages = max(1, sum(need))
        self.pages = pages + 1
        self.pool = make_pool(layout, page_bits, self.pages * P, seed)
        rng = np.random.default_rng(seed)
        perm = rng.permutation(self.pages)[:pages]
        self.width = max([1] + need) + width_more
        self.table = np.full((len(lens), self.width), 1 << 30, np.int32)     # entries past a length are never read
        at = 0
        for i, k in enumerate(need):
            self.table[i, :k] = perm[at:at + k]
            at += k
        self.q = queries(len(lens) * q_len, heads, seed + 1)
        self.scale = 512 ** -0.5

    def slots(self, i, n):
        t = np.arange(n)
        return self.table[i][t >> self.pb].astype(np.int64) * (1 << self.pb) + (t & ((1 << self.pb) - 1))

    def want(self, tokens=None):
        got = []
        q = self.q.double().numpy()
        for i, n in enumerate(self.lens):
            rows = decode(self.layout, self.pb, self.pool, self.slots(i, n))
            for j in range(self.q_len):
                vis = max(0, n - (self.q_len - 1 - j))
                got.append(reference(self.layout, q[i * self.q_len + j], rows[:vis], self.scale))
        return got

    def run(self, K, out=None, q=None, table=None, req=None, kv_len=None, err=None, lse=True, ws=None):
        q = self.q.to(DEV) if q is None else q
        out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV) if out is None else out
        lse = torch.full(q.shape[:2], float("nan"), device=DEV) if lse else None
        if ws is None:   # stale contents of a workspace mean nothing
            ws = torch.full((K.attend_workspace(self.q_len * self.heads),), 0xFF, dtype=torch.uint8, device=DEV)
        table = torch.from_numpy(self.table).to(DEV) if table is None else table
        kv_len = torch.tensor(self.lens, dtype=torch.int32, device=DEV) if kv_len is None else kv_len
        K.kvq_attend(self.layout, self.pb, q, torch.from_numpy(self.pool).to(DEV), self.pages, table, kv_len, out, ws,
                     scale=self.scale, q_len=self.q_len, req=req, lse=lse, err=err)
        torch.cuda.synchronize()
        return out, lse


# --------------------------------------------------------------------------- paged

@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads,q_len,lens,pb", [
    (1, 1, [1], 6),
    (16, 1, [0], 6),
    (16, 1, [100], 6),
    (5, 1, [63, 64, 65], 6),
    (16, 1, [127, 128, 129, 0, 1], 6),
    (17, 1, [255, 256, 257], 4),
    (33, 1, [1000, 3], 2),
    (64, 1, [640, 129, 1, 0, 77], 8),
    (65, 1, [300, 128], 6),
    (128, 1, [511, 2], 6),
    (8, 4, [1, 3, 4, 5, 128, 131, 260], 6),       # sequences shorter than their query
    (7, 3, [130, 0, 2], 4),
    (64, 5, [257, 64], 6),
    (3, 70, [200, 69, 33], 6),
])
def test_paged_lengths(K, layout, heads, q_len, lens, pb):
    c = Paged(layout, pb, lens, heads, q_len, seed=heads + q_len)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = c.run(K, err=err)
    assert err.item() == 0
    check(out, lse, c.want(), "paged")


@pytest.mark.parametrize("layout", [V41, FP4])
def test_split_over_ctas_and_joined(K, layout):
    """One long sequence among short and empty ones: its blocks are split over
    many CTAs; fp32 output, twice the same bits."""
    c = Paged(layout, 6, [21001, 5, 0, 3000, 700], 20, seed=3)
    out = torch.full(c.q.shape, float("nan"), device=DEV)
    out, lse = c.run(K, out=out)
    check(out, lse, c.want(), "split")
    again, lse2 = c.run(K, out=torch.empty_like(out))
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("layout", [V41, FP4])
def test_many_sequences(K, layout):
    """More sequences than SMs and than threads of a CTA, most of them short."""
    rng = np.random.default_rng(5)
    lens = [int(n) for n in rng.integers(0, 40, 1300)]
    lens[700] = 900
    c = Paged(layout, 2, lens, 4, seed=7)
    out, lse = c.run(K)
    check(out, lse, c.want(), "many")


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads,q_len", [(16, 1), (32, 1), (64, 1), (40, 2)])
def test_many_blocks_a_cta(K, layout, heads, q_len):
    """More blocks than CTAs, in long tiles and in short ones: every ring goes round several times."""
    c = Paged(layout, 6, [64 * 152 * 12 + 5] if heads < 64 else [64 * 152 * 6 + 5, 700], heads, q_len=q_len, seed=51)
    out, lse = c.run(K)
    check(out, lse, c.want(), (heads, "long"))
    lens = [64 * (1 + (7 * i) % 9) - (i % 3) for i in range(200)]
    c = Paged(layout, 6, lens, heads, q_len=q_len, seed=53)
    out, lse = c.run(K)
    check(out, lse, c.want(), (heads, "short"))


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads", [16, 64])
def test_many_blocks_a_cta_by_slots(K, layout, heads):
    pool = make_pool(layout, 6, 2048, 57)
    g = torch.Generator().manual_seed(59)
    q = queries(200, heads, 61)
    slots = torch.randint(-1, 2048, (200, 333), generator=g, dtype=torch.int32)
    out, lse = torch.empty(q.shape, device=DEV), torch.empty(q.shape[:2], device=DEV)
    ws = torch.empty(K.attend_workspace(heads), dtype=torch.uint8, device=DEV)
    K.kvq_attend_slots(layout, 6, q.to(DEV), torch.from_numpy(pool).to(DEV), 2048, slots.to(DEV), out, ws, scale=512 ** -0.5, lse=lse)
    torch.cuda.synchronize()
    want = []
    for i in range(200):
        s = slots[i].numpy()
        want.append(reference(layout, q[i].double().numpy(), decode(layout, 6, pool, s[s >= 0]), 512 ** -0.5))
    check(out, lse, want, heads)


def test_query_and_output_layouts(K):
    """Head-major q and out, a slice of a wider projection, and a query row
    repeated by a stride of 0 give the contiguous call's bits."""
    c = Paged(V41, 6, [200, 90, 1], 6, q_len=2, seed=11)
    want, lse = c.run(K)
    check(want, lse, c.want(), "contiguous")
    q = c.q.to(DEV)
    head_major = q.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    out = torch.full((6, 6, 512), float("nan"), dtype=torch.bfloat16, device=DEV).permute(1, 0, 2)
    got, lse2 = c.run(K, q=head_major, out=out)
    assert torch.equal(got, want) and torch.equal(lse2, lse)
    wide = torch.zeros((6, 6, 576), dtype=torch.bfloat16, device=DEV)
    wide[..., 64:] = q
    owide = torch.full((6, 6, 640), 7.0, dtype=torch.bfloat16, device=DEV)
    got, _ = c.run(K, q=wide[..., 64:], out=owide[..., :512])
    assert torch.equal(got, want) and (owide[..., 512:] == 7).all()
    one = q[:, :1].expand(-1, 6, -1)
    got, _ = c.run(K, q=one)
    same, _ = c.run(K, q=one.contiguous())
    assert torch.equal(got, same)


def test_table_rows_by_index_and_wide_tables(K):
    c = Paged(FP4, 6, [130, 65, 400], 16, seed=13, width_more=9)
    want, lse = c.run(K)
    order = [2, 0, 1]
    table = torch.full((5, c.width), 1 << 30, dtype=torch.int32)
    for i, r in enumerate(order):
        table[r + 1] = torch.from_numpy(c.table[i])
    req = torch.tensor([r + 1 for r in order], dtype=torch.int32, device=DEV)
    strided = torch.full((5, c.width + 3), -1, dtype=torch.int32)
    strided[:, :c.width] = table
    got, lse2 = c.run(K, table=strided.to(DEV)[:, :c.width], req=req)
    assert torch.equal(got, want) and torch.equal(lse, lse2)


def test_rows_behind_the_last_sequence_stay(K):
    c = Paged(V41, 6, [70, 3], 16, seed=17)
    big = torch.full((6, 16, 512), 3.0, dtype=torch.bfloat16, device=DEV)
    out, _ = c.run(K, out=big[:2])
    check(out, None, c.want(), "head")
    assert (big[2:] == 3).all()


@pytest.mark.parametrize("layout", [V41, FP4])
def test_masked_places_may_hold_anything(K, layout):
    """NaN codes and scales in the rest of the last page, in unused pages and
    (q_len > 1) in query tokens that a row does not see yet."""
    c = Paged(layout, 6, [70, 129], 16, q_len=3, seed=19)
    want = c.want()
    clean, lse = c.run(K)
    check(clean, lse, want, "clean")
    bpt = O.bytes_per_token(layout)
    pool = c.pool.reshape(c.pages, -1)
    used = {int(p) for i, n in enumerate(c.lens) for p in c.table[i][:-(-n // 64)]}
    for p in range(c.pages):
        if p not in used:
            pool[p] = 0xFF
    cb = 512 if layout == V41 else 256
    sb = bpt - cb

    def poison(i, t):
        p, r = c.table[i][t >> 6], t & 63
        pool[p, r * cb:(r + 1) * cb] = 0xFF
        pool[p, 64 * cb + r * sb:64 * cb + r * sb + 16] = 0xFF
    for i, n in enumerate(c.lens):
        for t in range(n, -(-n // 64) * 64):
            poison(i, t)
    got, lse2 = c.run(K)
    assert torch.equal(got, clean) and torch.equal(lse, lse2)
    # the newest token of sequence 0 turns NaN: only its own row sees it
    poison(0, 69)
    got, lse2 = c.run(K)
    assert torch.isnan(got[2]).all() and torch.isnan(lse2[2]).all()
    rest = [0, 1, 3, 4, 5]
    check(got[rest], lse2[rest], [want[i] for i in rest], "beside a NaN")


def test_nan_query_row_stays_alone(K):
    for layout in (V41, FP4):
        c = Paged(layout, 6, [150, 40], 16, q_len=2, seed=23)
        c.q[1, 3, 100] = float("nan")
        c.q[2, 5, 7] = float("inf")
        q = c.q.to(DEV)
        out, lse = c.run(K, q=q)
        c.q[1, 3, 100] = 0
        c.q[2, 5, 7] = 0
        want = c.want()
        assert torch.isnan(out[1, 3]).all() and torch.isnan(out[2, 5]).all()
        out[1, 3], out[2, 5] = 0, 0
        lse[1, 3], lse[2, 5] = 0, 0
        for t, h in ((1, 3), (2, 5)):
            o, l, tol, tl = want[t]
            o[h], l[h], tol[h], tl[h] = 0, 0, 0, 0
        check(out, lse, want, "beside a NaN query")


def test_large_and_small_magnitudes(K):
    """Peaked rows, query rows at both ends of bf16's range, negative scale."""
    for layout in (V41, FP4):
        c = Paged(layout, 6, [300, 17], 16, seed=29)
        c.q[0] *= 40                                   # weights from 1 down to nothing
        c.q[1, :8] = (c.q[1, :8].float() * 2.0 ** -100).to(torch.bfloat16)     # all scores 0
        out, lse = c.run(K)
        check(out, lse, c.want(), "peaked")
        c.scale = -c.scale
        out, lse = c.run(K)
        check(out, lse, c.want(), "negative scale")
        c.q[:] = (queries(2, 16, 31).float() * 2.0 ** 100).to(torch.bfloat16)
        c.scale = 512 ** -0.5 * 2.0 ** -100
        out, lse = c.run(K)
        check(out, lse, c.want(), "huge queries")


def test_rows_of_many_magnitudes(K):
    """V41 tokens and blocks whose scales differ by large powers of two, down to none at all."""
    from compress_kv_write_gb300 import synth
    for span, heads in ((6, 16), (30, 16), (60, 40)):
        c = Paged(V41, 6, [200, 67, 1], heads, q_len=2, seed=37)
        x = synth.store_rows_bf16(c.pages * 64, "cpu", 41).float()
        g = torch.Generator().manual_seed(43)
        x *= torch.exp2(torch.randint(-span, span // 6 + 1, (c.pages * 64, 1), generator=g).float())
        x *= torch.exp2(torch.randint(-20, 1, (c.pages * 64, 16), generator=g).float()).repeat_interleave(32, 1)
        x[7], x[11, 32:] = 0, 0
        x = x.to(torch.bfloat16)
        assert O.store(V41, 6, 0, x.view(torch.int16).numpy().view(np.uint16), np.arange(c.pages * 64), c.pool) == O.OK
        c.q[:, ::3] = 0                                # equal weights, so that every row counts
        out, lse = c.run(K, out=torch.empty(c.q.shape, device=DEV))
        check(out, lse, c.want(), span)


def test_device_errors(K):
    c = Paged(V41, 6, [200, 90, 100, 64], 16, seed=37)
    want = c.want()
    # a bad page: its tokens are masked
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = torch.from_numpy(c.table.copy())
    table[0, 1] = c.pages
    table[1, 0] = -1
    out, lse = c.run(K, table=table.to(DEV), err=err)
    assert err.item() == 4
    q = c.q.double().numpy()
    w = list(want)
    for i, gone in ((0, range(64, 128)), (1, range(0, 64))):
        keep = np.array([t for t in range(c.lens[i]) if t not in gone])
        w[i] = reference(V41, q[i], decode(V41, 6, c.pool, c.slots(i, c.lens[i])[keep]), c.scale)
    check(out, lse, w, "bad pages")
    # bad lengths and table rows: empty sequences
    none = reference(V41, q[0], np.zeros((0, 512)), c.scale)
    err.zero_()
    lens = torch.tensor([200, -1, c.width * 64 + 1, 64], dtype=torch.int32, device=DEV)
    out, lse = c.run(K, kv_len=lens, err=err)
    assert err.item() == 64
    check(out, lse, [want[0], none, none, want[3]], "bad lengths")
    err.zero_()      # past 2^30 tokens, though the table is wide enough
    wide = torch.zeros((4, (1 << 24) + 4), dtype=torch.int32, device=DEV)
    wide[:, :c.width] = torch.from_numpy(c.table).to(DEV)
    lens = torch.tensor([200, (1 << 30) + 1, 0x7FFFFFFF, 64], dtype=torch.int32, device=DEV)
    out, lse = c.run(K, kv_len=lens, table=wide, err=err)
    assert err.item() == 64
    check(out, lse, [want[0], none, none, want[3]], "too long")
    del wide
    err.zero_()
    out, lse = c.run(K, req=torch.tensor([0, 4, 2, -1], dtype=torch.int32, device=DEV), err=err)
    assert err.item() == 32
    check(out, lse, [want[0], none, want[2], none], "bad table rows")


# --------------------------------------------------------------------------- slots

def run_slots(K, layout, pb, pool, slots_n, q, slots, out=None, err=None):
    scale = 512 ** -0.5
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV) if out is None else out
    lse = torch.full(q.shape[:2], float("nan"), device=DEV)
    ws = torch.full((K.attend_workspace(q.shape[1]),), 0xFF, dtype=torch.uint8, device=DEV)
    K.kvq_attend_slots(layout, pb, q.to(DEV), torch.from_numpy(pool).to(DEV), slots_n, slots.to(DEV), out, ws,
                       scale=scale, lse=lse, err=err)
    torch.cuda.synchronize()
    return out, lse


def want_slots(layout, pb, pool, slots_n, q, slots):
    got = []
    for t in range(q.shape[0]):
        s = slots[t].numpy().astype(np.int64)
        s = s[(s >= 0) & (s < slots_n)]
        got.append(reference(layout, q[t].double().numpy(), decode(layout, pb, pool, s), 512 ** -0.5))
    return got


@pytest.mark.parametrize("layout", [V41, FP4])
@pytest.mark.parametrize("heads,n_tok,n_sel,pb,dtype", [
    (16, 1, 1, 6, torch.int32), (16, 3, 0, 6, torch.int32), (1, 2, 127, 6, torch.int64),
    (64, 2, 128, 4, torch.int32), (32, 5, 129, 6, torch.int64), (100, 3, 1000, 2, torch.int32),
    (8, 200, 150, 8, torch.int32), (40, 1, 4096, 6, torch.int32),
])
def test_slots(K, layout, heads, n_tok, n_sel, pb, dtype):
    """Padding anywhere in the lists, a list of padding alone, a strided list
    and a repeated slot (which counts twice)."""
    slots_n = 2048
    pool = make_pool(layout, pb, slots_n, 41)
    rng = np.random.default_rng(n_sel)
    s = torch.from_numpy(rng.integers(0, slots_n, (n_tok, n_sel + 5))).to(dtype)
    s[torch.from_numpy(rng.random(s.shape) < 0.2)] = -1
    if n_sel > 3:
        s[0, 2] = s[0, 1] = 5
    if n_tok > 2:
        s[2] = -1
    s = s[:, :n_sel]
    q = queries(n_tok, heads, n_sel + 1)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = run_slots(K, layout, pb, pool, slots_n, q, s, err=err)
    assert err.item() == 0
    check(out, lse, want_slots(layout, pb, pool, slots_n, q, s), "slots")


def test_bad_slots_are_masked(K):
    slots_n = 256
    pool = make_pool(FP4, 6, slots_n, 43)
    s = torch.arange(200, dtype=torch.int64).repeat(2, 1)
    s[0, 7], s[0, 150], s[1, 3] = slots_n, -2, 1 << 40
    q = queries(2, 16, 43)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = run_slots(K, FP4, 6, pool, slots_n, q, s, err=err)
    assert err.item() == 1
    check(out, lse, want_slots(FP4, 6, pool, slots_n, q, s), "bad slots")


def test_slots_equal_paged(K):
    """The same tokens in the same order by table and by list give the same result."""
    c = Paged(FP4, 6, [333], 48, seed=47)
    out, lse = c.run(K)
    s = torch.from_numpy(c.slots(0, 333))[None]
    out2, lse2 = run_slots(K, FP4, 6, c.pool, c.pages * 64, c.q, s)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("layout", [V41, FP4])
def test_pool_offsets_past_32_bits(K, layout):
    """Rows whose byte offset is beyond 2^32: high pages and high slots."""
    bpt = O.bytes_per_token(layout)
    pages = ((1 << 32) + (1 << 28)) // (64 * bpt) + 4
    small = make_pool(layout, 6, 256, 53)
    big = torch.zeros(pages * 64 * bpt, dtype=torch.uint8, device=DEV)
    big[-256 * bpt:] = torch.from_numpy(small).to(DEV)
    first = pages - 4
    q = queries(1, 16, 53)
    want = [reference(layout, q[0].double().numpy(), decode(layout, 6, small, np.arange(250)), 512 ** -0.5)]
    out = torch.full((1, 16, 512), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(K.attend_workspace(16), dtype=torch.uint8, device=DEV)
    table = torch.arange(first, pages, dtype=torch.int32, device=DEV)[None]
    K.kvq_attend(layout, 6, q.to(DEV), big, pages, table, torch.tensor([250], dtype=torch.int32, device=DEV), out, ws,
                 scale=512 ** -0.5)
    check(out, None, want, "high pages")
    out.fill_(float("nan"))
    slots = (torch.arange(250, device=DEV) + first * 64)[None]
    K.kvq_attend_slots(layout, 6, q.to(DEV), big, pages * 64, slots, out, ws, scale=512 ** -0.5)
    check(out, None, want, "high slots")


# --------------------------------------------------------------------------- streams and graphs

def test_captured_and_replayed(K):
    """A captured call replays with the lengths and queries that its buffers
    hold then; two graphs that run in turn may share a workspace."""
    c = Paged(FP4, 6, [1500, 40, 300], 16, seed=59)
    pool = torch.from_numpy(c.pool).to(DEV)
    table = torch.from_numpy(c.table).to(DEV)
    q, lens = c.q.to(DEV), torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    ws = torch.empty(K.attend_workspace(16), dtype=torch.uint8, device=DEV)
    outs, graphs = [torch.empty_like(q) for _ in range(2)], []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            K.kvq_attend(FP4, 6, q, pool, c.pages, table, lens, o, ws, scale=c.scale)
        graphs.append(g)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    want = c.want()
    for o in outs:
        check(o, None, want, "replayed")
    lens.copy_(torch.tensor([64, 0, 299], dtype=torch.int32))
    c.lens = [64, 0, 299]
    graphs[1].replay()
    torch.cuda.synchronize()
    check(outs[1], None, c.want(), "replayed with other lengths")


def test_two_streams(K):
    """Two calls at once, each with its own workspace, on streams of their own."""
    cs = [Paged(V41, 6, [2000, 100], 16, seed=61), Paged(FP4, 6, [900, 1800], 64, seed=67)]
    made = []
    for c in cs:
        made.append((torch.from_numpy(c.pool).to(DEV), torch.from_numpy(c.table).to(DEV), c.q.to(DEV),
                     torch.tensor(c.lens, dtype=torch.int32, device=DEV),
                     torch.empty(K.attend_workspace(c.heads), dtype=torch.uint8, device=DEV),
                     torch.empty(c.q.shape, dtype=torch.bfloat16, device=DEV), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(8):
        for c, (pool, table, q, lens, ws, out, st) in zip(cs, made):
            K.kvq_attend(c.layout, 6, q, pool, c.pages, table, lens, out, ws, scale=c.scale, stream=st)
    torch.cuda.synchronize()
    for c, m in zip(cs, made):
        check(m[5], None, c.want(), "two streams")


def test_refusals_in_the_binding(K):
    c = Paged(V41, 6, [10], 16, seed=71)
    q, out = c.q.to(DEV), torch.empty((1, 16, 512), dtype=torch.bfloat16, device=DEV)
    pool, table = torch.from_numpy(c.pool).to(DEV), torch.from_numpy(c.table).to(DEV)
    lens = torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    ws = torch.empty(K.attend_workspace(16), dtype=torch.uint8, device=DEV)

    def call(q=q, pool=pool, pages=c.pages, table=table, lens=lens, out=out, ws=ws, scale=1.0, q_len=1, **kw):
        K.kvq_attend(V41, 6, q, pool, pages, table, lens, out, ws, scale=scale, q_len=q_len, **kw)
    for bad in (dict(q=q.float()), dict(out=out.half()), dict(lens=lens.long()), dict(table=table.long()),
                dict(pool=pool.cpu()), dict(lse=torch.zeros((1, 16), device=DEV, dtype=torch.float64)),
                dict(err=torch.zeros(1, device=DEV))):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(q=q[..., :500]), dict(q_len=2), dict(out=out[:, :8]), dict(pages=c.pages + 1),
                dict(lens=lens.repeat(2)), dict(lse=torch.zeros((1, 8), device=DEV)),
                dict(out=out[:, :1].expand(-1, 16, -1)), dict(req=torch.zeros(2, dtype=torch.int32, device=DEV))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(scale=float("nan")), dict(ws=ws[:8])):
        with pytest.raises(K.KVQError):
            call(**bad)


# --------------------------------------------------------------------------- a decoder step

@pytest.mark.parametrize("layout", [V41, FP4])
def test_norm_store_attend_step(K, layout):
    """The run a serving step makes: residual + RMS norm to 8 bits, a projection
    of its values to K rows, the K norm + RoPE store, attention over the pages
    just written -- by table and, for the newest tokens, by slot."""
    from compress_kv_write_gb300 import synth
    n, dim, heads = 150, 1024, 16
    g = torch.Generator().manual_seed(73)
    x = torch.randn((n, dim), generator=g).to(torch.bfloat16).to(DEV)
    res = torch.randn((n, dim), generator=g).to(torch.bfloat16).to(DEV)
    w = synth.normal((dim,), "cpu", 1, "weight", std=0.1, mean=1.0).to(DEV)
    codes = torch.empty((n, dim), dtype=torch.uint8, device=DEV)
    scales = torch.empty((n, dim // 32), dtype=torch.uint8, device=DEV)
    K.kvq_norm_quant(x, w, codes, scales, residual=res, residual_out=res)
    y = codes.view(torch.float8_e4m3fn).float().view(n, -1, 32) * torch.exp2(scales.float() - 127)[..., None]
    proj = (torch.randn((dim, 512), generator=g) / dim ** 0.5).to(DEV)
    k = (y.view(n, dim) @ proj).to(torch.bfloat16)
    pool = torch.zeros(256 * O.bytes_per_token(layout), dtype=torch.uint8, device=DEV)
    pages = torch.tensor([[2, 0, 3]], dtype=torch.int32, device=DEV)
    t = torch.arange(n, device=DEV)
    loc = pages[0].long()[t // 64] * 64 + t % 64
    kw, cs = synth.norm_weight("cpu", 2).to(DEV), synth.rope_table(256, "cpu").to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    K.kvq_store(layout, 6, K.FLAG_NORM | K.FLAG_ROPE, k, loc, pool, 256, norm_weight=kw, cos_sin=cs,
                pos=t.to(torch.int32), err=err)
    q = queries(3, heads, 79).to(DEV)
    out = torch.empty((3, heads, 512), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(K.attend_workspace(3 * heads), dtype=torch.uint8, device=DEV)
    K.kvq_attend(layout, 6, q, pool, 4, pages, torch.tensor([n], dtype=torch.int32, device=DEV), out, ws,
                 scale=512 ** -0.5, q_len=3, err=err)
    sel = torch.stack([loc[i:i + 20] for i in (0, 64, 130)])
    out2 = torch.empty_like(out)
    K.kvq_attend_slots(layout, 6, q, pool, 256, sel, out2, ws, scale=512 ** -0.5, err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    host, qn = pool.cpu().numpy(), q.double().cpu().numpy()
    # the stored rows are the normalised, rotated projections: unit variance, so every dim of a row is small
    rows = decode(layout, 6, host, loc.cpu().numpy())
    assert 0.5 < np.sqrt((rows ** 2).mean()) < 1.5
    check(out, None, [reference(layout, qn[j], rows[:n - 2 + j], 512 ** -0.5) for j in range(3)], "step")
    check(out2, None, [reference(layout, qn[j], rows[i:i + 20], 512 ** -0.5) for j, i in enumerate((0, 64, 130))],
          "step by slot")
