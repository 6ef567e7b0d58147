"""Operators that read and feed the paged V41 / V41_FP4 cache, in plain form and as the package's kernels.

attend        latent attention over a paged cache: every head of a query reads the same 512-value row of a
              token as key and as value, decoded from 8-bit (V41) or 4-bit (V41_FP4) blocks
attend_slots  the same over the tokens that a sparse selection picks, one list of slots a query token
norm_quant    RMS norm of a row plus its residual, written as e4m3 codes with one ue8m0 scale per 32 values

`own` chooses between the plain forms (elementary torch operations) and the package's entry points.
"""
import math
import random

import torch

own = False

D = 512
V41, FP4 = 1, 2
PAGE_BITS = 6
P = 1 << PAGE_BITS
CODE_BYTES = {V41: 512, FP4: 256}
SCALE_BYTES = {V41: 16, FP4: 32}
READ_BYTES = {V41: 528, FP4: 272}   # what one token's codes and scales occupy, padding left out
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one user's request, a short prompt, the heads of one of eight tensor-parallel ranks: latency
        dict(name="attend one short", op="attend", layout=FP4, n_seq=1, q_len=1, heads=16, kv=100),
        # decode batch of a rank with few heads: bound by the cache's bytes; some rows of the batch are padding
        dict(name="attend decode 8-bit", op="attend", layout=V41, n_seq=48, q_len=1, heads=16, kv=12289),
        # decode batch with 64 heads over the 4-bit cache, lengths that differ by a factor of eight
        dict(name="attend decode 4-bit", op="attend", layout=FP4, n_seq=64, q_len=1, heads=64, kv=16384),
        # two long documents with every head on this GPU: the work of one row is split over the machine
        dict(name="attend long 4-bit", op="attend", layout=FP4, n_seq=2, q_len=1, heads=128, kv=131073),
        # draft tokens verified in one step: four query tokens a request, causal among themselves
        dict(name="attend verify", op="attend", layout=V41, n_seq=17, q_len=4, heads=8, kv=4000),
        # a chunk of a prompt against the cache it was just stored into: bound by the products
        dict(name="attend chunk", op="attend", layout=V41, n_seq=2, q_len=500, heads=64, kv=4500),
        # sparse decode of one token
        dict(name="slots one", op="attend_slots", layout=FP4, n_tok=1, heads=64, topk=512, pool=65536),
        # sparse decode batch over the 8-bit cache
        dict(name="slots decode 8-bit", op="attend_slots", layout=V41, n_tok=129, heads=32, topk=2048, pool=262144),
        # sparse prefill chunk over the 4-bit cache, an odd selection width
        dict(name="slots chunk 4-bit", op="attend_slots", layout=FP4, n_tok=1024, heads=64, topk=1000, pool=262144),
        # the norm in front of a decode step's projections
        dict(name="norm one", op="norm_quant", dtype="bf16", n=1, dim=4096, residual=True),
        # an odd batch of a narrow fp32 model, without a residual
        dict(name="norm odd fp32", op="norm_quant", dtype="f32", n=1537, dim=1056, residual=False),
        # a prompt's chunk
        dict(name="norm chunk", op="norm_quant", dtype="bf16", n=16384, dim=8192, residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attend", "attend", "attend_slots", "norm_quant"))
    if op == "norm_quant":
        dim = 32 * _log(rng, 4, 512)
        n = _log(rng, 1, max(1, min(16384, 16384 * 8192 // (2 * dim))))
        return dict(op=op, dtype=rng.choice(("bf16", "f32")), n=n, dim=dim, residual=rng.random() < 0.7)
    layout = rng.choice((V41, FP4))
    heads = rng.choice((1, 5, 8, 12, 16, 24, 32, 40, 64, 96, 128))
    if op == "attend_slots":
        topk = _log(rng, 1, 2048)
        n_tok = _log(rng, 1, max(1, min(2048, 1024 * 1000 * 64 // (topk * max(heads, 16)))))
        return dict(op=op, layout=layout, n_tok=n_tok, heads=heads, topk=topk, pool=max(4096, 64 * _log(rng, 64, 4096)))
    q_len = rng.choice((1, 1, 1, 2, 3, 5, _log(rng, 6, 500)))
    kv = _log(rng, 1, 131072 if q_len == 1 else 8192)
    most = min(64, 64 * 16384 // kv, 2 * 500 * 64 * 4500 // (q_len * heads * kv))
    return dict(op=op, layout=layout, n_seq=_log(rng, 1, max(1, most)), q_len=q_len, heads=heads, kv=kv)


def _lengths(case):
    """Cached tokens of each sequence: the longest first, the others from an eighth of it up; of four or more
    sequences one holds a single token and the last is an empty row of a padded batch."""
    rng = random.Random("%(n_seq)d %(q_len)d %(kv)d" % case)
    lens = [case["kv"]] + [max(1, int(case["kv"] * math.exp(-rng.random() * math.log(8)))) for _ in range(case["n_seq"] - 1)]
    if len(lens) >= 4:
        lens[-2], lens[-1] = 1, 0
    return lens


def _selected(case):
    """How many of a query token's `topk` entries hold a slot; the others are -1."""
    return [case["topk"] - (t * 37) % (case["topk"] // 4 + 1) for t in range(case["n_tok"])]


def _pairs(case):
    """(query token, cached token) pairs that are not masked."""
    q = case["q_len"]
    return sum(max(0, n - j) for n in _lengths(case) for j in range(q))


def work(case):
    if case["op"] == "norm_quant":
        item = 2 if case["dtype"] == "bf16" else 4
        values = case["n"] * case["dim"]
        rows = (3 if case["residual"] else 1) * item
        return {"bytes": values * (rows + 1) + values // 32 + 4 * case["dim"], "flops": 8 * values}
    h = case["heads"]
    if case["op"] == "attend":
        tokens, pairs, queries = sum(_lengths(case)), _pairs(case), case["n_seq"] * case["q_len"]
    else:
        pairs, queries = sum(_selected(case)), case["n_tok"]
        tokens = min(pairs, case["pool"])  # a row that several tokens pick is read once
    return {"bytes": tokens * READ_BYTES[case["layout"]] + queries * h * (2 * 2 * D + 4), "flops": 4 * D * h * pairs}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _pool(layout, slots, g):
    """A pool of `slots` tokens with rows ~ N(0, 1), one value in a hundred ten times as large, quantised to blocks of 32."""
    pages = slots // P
    pool = torch.zeros((pages, P * (CODE_BYTES[layout] + SCALE_BYTES[layout])), dtype=torch.uint8, device="cuda")
    step = 1024
    for at in range(0, pages, step):
        k = min(step, pages - at)
        x = torch.randn((k * P, 16, 32), generator=g, device="cuda")
        x = torch.where(torch.rand(x.shape, generator=g, device="cuda") < 0.01, x * 10, x)
        amax = x.abs().amax(-1, keepdim=True)
        if layout == V41:
            e = torch.floor(torch.log2(amax)).clamp(-100, 100)
            codes = (x * torch.exp2(8 - e)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            scales = (e + 119).to(torch.uint8).view(k * P, 16)
        else:
            s = (amax / 6).to(torch.float8_e4m3fn)
            y = x / s.float().clamp_min(2.0 ** -9)
            edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
            c = torch.bucketize(y.abs(), edges).to(torch.uint8) + (y < 0).to(torch.uint8) * 8
            c = c.view(k * P, 256, 2)
            codes = c[..., 0] + c[..., 1] * 16
            scales = torch.zeros((k * P, 32), dtype=torch.uint8, device="cuda")
            scales[:, :16] = s.view(torch.uint8).view(k * P, 16)
        pool[at:at + k, :P * CODE_BYTES[layout]] = codes.reshape(k, -1)
        pool[at:at + k, P * CODE_BYTES[layout]:] = scales.reshape(k, -1)
    return pool.view(-1)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "norm_quant":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        n, dim = case["n"], case["dim"]
        x = torch.randn((n, dim), generator=g, device="cuda").to(dt)
        res = None
        if case["residual"]:
            res = (torch.randn((n, dim), generator=g, device="cuda") * 4).to(dt)
        w = 1 + 0.1 * torch.randn(dim, generator=g, device="cuda")
        return dict(case, x=x, residual=res, weight=w, eps=1e-6,
                    codes=torch.empty((n, dim), dtype=torch.uint8, device="cuda"),
                    scales=torch.empty((n, dim // 32), dtype=torch.uint8, device="cuda"),
                    total=torch.empty_like(x) if case["residual"] else None)
    h, layout = case["heads"], case["layout"]
    state = dict(case, scale=D ** -0.5)
    if case["op"] == "attend":
        lens = _lengths(case)
        width = max(1, -(-max(lens) // P))
        need = [-(-n // P) for n in lens]
        pages = max(1, sum(need))
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros((case["n_seq"], width), dtype=torch.int32, device="cuda")
        at = 0
        for s, k in enumerate(need):
            table[s, :k] = perm[at:at + k]
            at += k
        queries = case["n_seq"] * case["q_len"]
        state.update(pool=_pool(layout, pages * P, g), pages=pages, table=table,
                     kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    else:
        queries = case["n_tok"]
        state["pool"] = _pool(layout, case["pool"], g)
        state["pool_slots"] = case["pool"]
        keep = torch.tensor(_selected(case), device="cuda")
        # distinct slots a query token: an odd multiple of a running index, modulo a power of two, then folded by rank
        base = torch.randint(0, case["pool"], (queries, 1), generator=g, device="cuda")
        stride = torch.randint(0, case["pool"], (queries, 1), generator=g, device="cuda") | 1
        picks = torch.arange(case["topk"], device="cuda")[None, :]
        size = 1 << (case["pool"].bit_length() - 1)
        slots = (base + picks * stride) % size
        state["slots"] = torch.where(picks < keep[:, None], slots, -1).to(torch.int32)
    state["q"] = (2 * torch.randn((queries, h, D), generator=g, device="cuda")).to(torch.bfloat16)
    state["out"] = torch.empty_like(state["q"])
    state["lse"] = torch.empty((queries, h), dtype=torch.float32, device="cuda")
    return state


# ------------------------------------------------------------------ plain forms

def _decode(layout, codes, scales):
    """fp32 [..., 512] from code rows and scale rows."""
    if layout == V41:
        v = codes.view(torch.float8_e4m3fn).float().view(*codes.shape[:-1], 16, 32)
        s = torch.exp2(scales.float() - 127)
    else:
        lut = torch.tensor(E2M1, device=codes.device)
        both = torch.stack((codes & 15, codes >> 4), dim=-1)
        v = lut[both.int()].view(*codes.shape[:-1], 16, 32)
        s = scales[..., :16].contiguous().view(torch.float8_e4m3fn).float()
    return (v * s[..., None]).view(*codes.shape[:-1], D)


def _softmax_rows(q, kv, seen, scale):
    """Attention of q [b, r, 512] over kv [b, n, 512] where seen [b, r, n]; (out fp32, natural-log lse)."""
    s = torch.matmul(q, kv.transpose(1, 2)) * scale
    s = s.masked_fill(~seen, float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isfinite(top), top, 0.0))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, kv) / torch.where(total > 0, total, 1.0)
    return out, (top + torch.log(total)).squeeze(-1)


def _attend_plain(s):
    layout, h, q_len, n_seq = s["layout"], s["heads"], s["q_len"], s["n_seq"]
    area = P * CODE_BYTES[layout]
    pages = s["pool"].view(s["pages"], -1)[s["table"].long()]
    codes = pages[..., :area].reshape(n_seq, -1, CODE_BYTES[layout])
    scales = pages[..., area:].reshape(n_seq, -1, SCALE_BYTES[layout])
    kv = _decode(layout, codes, scales)
    j = torch.arange(q_len, device="cuda").repeat_interleave(h)
    visible = s["kv_len"][:, None] - (q_len - 1 - j)[None, :]
    seen = torch.arange(kv.shape[1], device="cuda")[None, None, :] < visible[..., None]
    out, lse = _softmax_rows(s["q"].float().view(n_seq, q_len * h, D), kv, seen, s["scale"])
    return {"out": out.view(-1, h, D).to(torch.bfloat16), "lse": lse.view(-1, h)}


def _attend_slots_plain(s):
    layout = s["layout"]
    area = P * CODE_BYTES[layout]
    pages = s["pool"].view(s["pool_slots"] // P, -1)
    slot = s["slots"].long().clamp_min(0)
    codes = pages[:, :area].reshape(-1, CODE_BYTES[layout])[slot]
    scales = pages[:, area:].reshape(-1, SCALE_BYTES[layout])[slot]
    kv = _decode(layout, codes, scales)
    out, lse = _softmax_rows(s["q"].float(), kv, (s["slots"] >= 0)[:, None, :], s["scale"])
    return {"out": out.to(torch.bfloat16), "lse": lse}


def _norm_quant_plain(s):
    z = s["x"].float()
    if s["residual"] is not None:
        z = z + s["residual"].float()
    y = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + s["eps"]) * s["weight"]
    y = y.view(s["n"], -1, 32)
    byte = ((y.abs().amax(-1, keepdim=True).view(torch.int32) >> 23) - 8).clamp_min(0)
    codes = (y * torch.exp2((127 - byte).float())).clamp(-448, 448).to(torch.float8_e4m3fn)
    got = {"codes": codes.view(s["n"], -1), "scales": byte.to(torch.uint8).view(torch.float8_e8m0fnu).view(s["n"], -1)}
    if s["residual"] is not None:
        got["total"] = z.to(s["x"].dtype)
    return got


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        import compress_kv_write_gb300 as kvq
        if s["op"] == "attend":
            ws = torch.empty(kvq.attend_workspace(s["q_len"] * s["heads"]), dtype=torch.uint8, device="cuda")
            kvq.kvq_attend(s["layout"], PAGE_BITS, s["q"], s["pool"], s["pages"], s["table"], s["kv_len"], s["out"], ws,
                           scale=s["scale"], q_len=s["q_len"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        if s["op"] == "attend_slots":
            ws = torch.empty(kvq.attend_workspace(s["heads"]), dtype=torch.uint8, device="cuda")
            kvq.kvq_attend_slots(s["layout"], PAGE_BITS, s["q"], s["pool"], s["pool_slots"], s["slots"], s["out"], ws,
                                 scale=s["scale"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        kvq.kvq_norm_quant(s["x"], s["weight"], s["codes"], s["scales"], eps=s["eps"], residual=s["residual"],
                           residual_out=s["total"])
        got = {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"].view(torch.float8_e8m0fnu)}
        if s["residual"] is not None:
            got["total"] = s["total"]
        return got
    if s["op"] == "attend":
        return _attend_plain(s)
    if s["op"] == "attend_slots":
        return _attend_slots_plain(s)
    return _norm_quant_plain(s)


# ------------------------------------------------------------------ the definition in 64 bits

def _e4m3_values():
    """The 256 e4m3 values from sign, 4 exponent bits (bias 7) and 3 mantissa bits; 0x7F and 0xFF are NaN."""
    values = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = math.nan if (e, m) == (15, 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        values.append(-v if b & 128 else v)
    return torch.tensor(values, dtype=torch.float64, device="cuda")


def _row64(pool, layout, slots):
    """Rows of the pool at int64 `slots`, in 64 bits, byte by byte from the layout's definition."""
    page, row = slots >> PAGE_BITS, slots & (P - 1)
    base = page * (P * (CODE_BYTES[layout] + SCALE_BYTES[layout]))
    dims = torch.arange(D, device="cuda")
    codes_at = base + row * CODE_BYTES[layout]
    scale_at = base + P * CODE_BYTES[layout] + row * SCALE_BYTES[layout]
    scale = pool[scale_at[:, None] + dims // 32]
    if layout == V41:
        return _e4m3_values()[pool[codes_at[:, None] + dims].int()] * torch.pow(2.0, scale.double() - 127)
    byte = pool[codes_at[:, None] + dims // 2].int()
    nibble = torch.where(dims % 2 == 0, byte % 16, byte // 16)
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    return grid[nibble] * _e4m3_values()[scale.int()]


def _one64(q, rows, count, scale):
    """q [h, 512] over the first `count` rows."""
    if count <= 0:
        return torch.zeros_like(q), torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device="cuda")
    s = (q @ rows[:count].T) * scale
    lse = torch.logsumexp(s, 1)
    return torch.exp(s - lse[:, None]) @ rows[:count], lse


def exact(case, seed):
    if case["op"] != "norm_quant" and work(case)["flops"] > 1.5e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "norm_quant":
        if case["n"] * case["dim"] > 1 << 28:
            return None
        z = s["x"].double()
        if s["residual"] is not None:
            z = z + s["residual"].double()
        y = z / torch.sqrt((z * z).sum(-1, keepdim=True) / case["dim"] + s["eps"]) * s["weight"].double()
        y = y.view(case["n"], -1, 32)
        # ue8m0 byte: the exponent of the largest magnitude less e4m3's largest exponent
        _, e = torch.frexp(y.abs().amax(-1, keepdim=True))
        scale = torch.pow(2.0, (e - 1 - 8).clamp_min(-127).double())
        u = (y / scale).clamp(-448, 448)
        # nearest e4m3 value, ties to even: a step of 2^-3 of the value's power of two, 2^-9 below 2^-6
        _, k = torch.frexp(u)
        step = torch.pow(2.0, (k - 1).clamp_min(-6).double() - 3)
        got = {"codes": (torch.round(u / step) * step).view(case["n"], -1), "scales": scale.view(case["n"], -1)}
        if s["residual"] is not None:
            got["total"] = z
        return got
    q = s["q"].double()
    outs, lses = [], []
    if case["op"] == "attend":
        for n, length in enumerate(_lengths(case)):
            at = torch.arange(length, device="cuda")
            rows = _row64(s["pool"], case["layout"], s["table"][n].long()[at >> PAGE_BITS] * P + (at & (P - 1)))
            for j in range(case["q_len"]):
                o, l = _one64(q[n * case["q_len"] + j], rows, length - (case["q_len"] - 1 - j), s["scale"])
                outs.append(o)
                lses.append(l)
    else:
        for t in range(case["n_tok"]):
            slots = s["slots"][t].long()
            slots = slots[slots >= 0]
            o, l = _one64(q[t], _row64(s["pool"], case["layout"], slots), slots.numel(), s["scale"])
            outs.append(o)
            lses.append(l)
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
