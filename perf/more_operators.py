"""Operators of a speculative, long-context decode step over the paged V41 / V41_FP4 cache, in plain form and as the
package's kernels.

rope_table  cosines and sines of every position, for frequencies that may be scaled for long contexts
rope        rotary positions of query rows, or taken back from attention's output rows: part of a head, interleaved
            pairs or halves
tree        attention of a tree of drafted tokens over the cache that already holds them, from each token's parent
mass        what weight every cached token gets in attention, over all heads and query tokens, added up step by step
evict       the tokens of most weight, with the first and the last of a sequence always among them, and their rows
            moved to pages of their own

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
        # one user's decode step: the query heads of one of eight tensor-parallel ranks, latency
        dict(name="rope one", op="rope", dtype="bf16", n=1, heads=16, dim=512, start=448, rot=64, half=False, inverse=False),
        # the rotation taken back from a prompt chunk's attention outputs, the rest of a row carried along
        dict(name="rope chunk", op="rope", dtype="bf16", n=8191, heads=64, dim=512, start=448, rot=64, half=False, inverse=True),
        # the table of a model with a short context, which a server makes when it starts
        dict(name="table short", op="rope_table", rows=8192, rot=64, factor=1.0),
        # the table of a million positions, frequencies scaled by 32 for a context that long
        dict(name="table long", op="rope_table", rows=1048576, rot=64, factor=32.0),
        # one user's request with a tree of seven drafted tokens: latency
        dict(name="tree one", op="tree", layout=FP4, n_seq=1, q_len=7, heads=16, kv=700),
        # a batch of a rank with few heads, trees of 24 tokens; one sequence is a padded row
        dict(name="tree batch 8-bit", op="tree", layout=V41, n_seq=24, q_len=24, heads=16, kv=6001),
        # wide trees with 64 heads over long documents in the 4-bit cache: bound by the products
        dict(name="tree wide 4-bit", op="tree", layout=FP4, n_seq=8, q_len=63, heads=64, kv=16384),
        # one user's decode step: weights over a short cache
        dict(name="mass one", op="mass", layout=V41, n_seq=1, q_len=1, heads=16, kv=1000, adds=True),
        # a decode batch with few heads, weights added to those of the steps before: bound by the cache's bytes
        dict(name="mass decode 8-bit", op="mass", layout=V41, n_seq=48, q_len=1, heads=16, kv=12289, adds=True),
        # the last 32 queries of three long prompts, all heads on this GPU, before their caches are cut: bound by the products
        dict(name="mass window 4-bit", op="mass", layout=FP4, n_seq=3, q_len=32, heads=64, kv=32769, adds=False),
        # one user's cache cut to half
        dict(name="evict one", op="evict", layout=FP4, n_seq=1, kv=4097, keep=2048, first=4, last=128),
        # a batch of long caches cut to one budget: some are shorter than it and stay whole
        dict(name="evict batch 8-bit", op="evict", layout=V41, n_seq=32, kv=24577, keep=8191, first=16, last=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _within(case):
    """The case with no more sequences or tokens than keep its work at or below that of the largest listed one of its kind."""
    most = max(work(c)["flops"] for c in listed() if c["op"] == case["op"])
    while work(case)["flops"] > most:
        case = dict(case, n_seq=case["n_seq"] // 2) if case["n_seq"] > 1 else dict(case, kv=case["q_len"] + (case["kv"] - case["q_len"]) // 2)
    return case


def draw(rng):
    op = rng.choice(("rope", "rope_table", "tree", "tree", "mass", "mass", "evict"))
    if op == "rope":
        dim = 16 * _log(rng, 2, 32)
        rot = min(dim, 8 * _log(rng, 1, 16))
        start = rng.choice((0, dim - rot))
        heads = _log(rng, 1, 128)
        dtype = rng.choice(("bf16", "bf16", "f32"))
        values = 8191 * 64 * 512 // (1 if dtype == "bf16" else 2)
        n = _log(rng, 1, min(16384, values // (heads * dim)))
        return dict(op=op, dtype=dtype, n=n, heads=heads, dim=dim, start=start, rot=rot, half=rng.random() < 0.5,
                    inverse=rng.random() < 0.4)
    if op == "rope_table":
        rot = 8 * _log(rng, 2, 16)
        return dict(op=op, rows=_log(rng, 128, 1048576 * 64 // max(64, rot)), rot=rot, factor=rng.choice((1.0, 4.0, 16.0, 32.0)))
    layout = rng.choice((V41, FP4))
    heads = rng.choice((1, 5, 8, 12, 16, 24, 32, 40, 64, 96, 128))
    if op == "tree":
        q_len = rng.choice((2, 5, _log(rng, 6, 64), _log(rng, 6, 130)))
        kv = q_len + _log(rng, 1, 16000)
        return _within(dict(op=op, layout=layout, n_seq=_log(rng, 1, min(64, 8 * 16384 * 4 // kv)), q_len=q_len, heads=heads, kv=kv))
    if op == "mass":
        q_len = rng.choice((1, 1, 1, 2, 4, _log(rng, 5, 64)))
        kv = q_len + _log(rng, 1, 100000 if q_len == 1 else 32000)
        return _within(dict(op=op, layout=layout, n_seq=_log(rng, 1, min(64, 48 * 12289 // kv)), q_len=q_len, heads=heads, kv=kv,
                            adds=rng.random() < 0.6))
    kv = _log(rng, 10, 131072)
    keep = max(1, int(kv * rng.uniform(0.1, 0.9)))
    first = rng.choice((0, 1, 4, 16))
    last = rng.choice((0, 1, 32, 128, 500))
    first, last = (first, last) if first + last <= keep else (0, 0)
    most = min(64, 32 * 24577 // kv, 32 * 8191 // keep)
    return dict(op=op, layout=layout, n_seq=_log(rng, 1, max(1, most)), kv=kv, keep=keep, first=first, last=last)


def _lengths(case):
    """Cached tokens of each sequence: the longest first, the others from an eighth of it up; of four or more
    sequences one is as short as can be and the last is an empty row of a padded batch."""
    rng = random.Random("%(n_seq)d %(kv)d" % case)
    least = case.get("q_len", 1)
    lens = [case["kv"]] + [max(least, int(case["kv"] * math.exp(-rng.random() * math.log(8)))) for _ in range(case["n_seq"] - 1)]
    if len(lens) >= 4:
        lens[-2], lens[-1] = least, 0
    return lens


def _causal_pairs(case):
    """(query token, cached token) pairs that a causal mask leaves."""
    return sum(max(0, n - j) for n in _lengths(case) for j in range(case["q_len"]))


def work(case):
    op = case["op"]
    if op == "rope":
        item = 2 if case["dtype"] == "bf16" else 4
        values = case["n"] * case["heads"] * case["dim"]
        return {"bytes": 2 * item * values + case["n"] * (4 + 4 * case["rot"]), "flops": 3 * case["n"] * case["heads"] * case["rot"]}
    if op == "rope_table":
        return {"bytes": 4 * case["rows"] * case["rot"] + 4 * case["rot"], "flops": case["rows"] * case["rot"]}
    lens = _lengths(case)
    if op == "evict":
        kept = sum(min(n, case["keep"]) for n in lens)
        return {"bytes": 4 * sum(lens) + kept * (2 * READ_BYTES[case["layout"]] + 4 + 4), "flops": sum(lens)}
    h, q_len, queries = case["heads"], case["q_len"], case["n_seq"] * case["q_len"]
    if op == "tree":
        # every drafted token sees what was there before the tree and, of the tree, itself and its ancestors: at least itself
        pairs = sum(q_len * (n - q_len) + q_len for n in lens if n)
        return {"bytes": sum(lens) * READ_BYTES[case["layout"]] + queries * h * (2 * 2 * D + 4) + queries * (4 + 4 + 8 * (-(-q_len // 64))),
                "flops": 4 * D * h * pairs}
    return {"bytes": sum(lens) * (READ_BYTES[case["layout"]] + 4 + 4 * case["adds"]) + queries * h * (2 * D + 4),
            "flops": 2 * D * h * _causal_pairs(case)}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 29)
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


def _frequencies(rot, factor, base=10000.0, original=4096):
    """Angles a position, slowest last.  With a factor above 1 the frequencies that turn less than once over the
    original context are divided by it, those that turn more than 32 times stay, and what lies between is blended."""
    freq = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if factor > 1:
        turns = [original * f / (2 * math.pi) for f in freq]
        stay = [min(1.0, max(0.0, math.log(max(t, 1e-300)) / math.log(32.0))) for t in turns]
        freq = [f * s + f / factor * (1 - s) for f, s in zip(freq, stay)]
    return torch.tensor(freq, dtype=torch.float64, device="cuda")


def _cache(case, g, more_pages=0):
    """A pool with the case's sequences on shuffled pages, and behind them `more_pages` pages for later; the table."""
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
    pool = _pool(case["layout"], pages * P, g)
    if more_pages:
        pool = torch.cat((pool, torch.zeros(more_pages * (pool.numel() // pages), dtype=torch.uint8, device="cuda")))
    return dict(pool=pool, pages=pages + more_pages, first_new=pages, table=table, width=width,
                kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "rope":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        rows = 65536
        x = torch.randn((case["n"], case["heads"], case["dim"]), generator=g, device="cuda").to(dt)
        angle = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * _frequencies(case["rot"], 16.0)
        table = torch.cat((torch.cos(angle), torch.sin(angle)), 1).float()
        pos = torch.randint(0, rows, (case["n"],), generator=g, device="cuda").to(torch.int32)
        return dict(case, x=x, cos_sin=table, pos=pos, out=torch.empty_like(x))
    if op == "rope_table":
        first = int(torch.randint(0, 1000, (1,), generator=g, device="cuda"))
        return dict(case, freq=_frequencies(case["rot"], case["factor"]), first=first, amplitude=1 + 0.1 * math.log(case["factor"]),
                    table=torch.empty((case["rows"], case["rot"]), dtype=torch.float32, device="cuda"))
    if op == "evict":
        width = -(-case["keep"] // P)
        need = case["n_seq"] * width
        state = dict(case, **_cache(case, g, need))
        n, most = case["n_seq"], state["width"] * P
        # weights added over many steps: a few tokens have most of it, many have none at all
        mass = torch.exp(2.5 * torch.randn((n, most), generator=g, device="cuda"))
        mass = torch.where(torch.rand((n, most), generator=g, device="cuda") < 0.3, 0.0, mass)
        new = torch.randperm(need, generator=g, device="cuda").to(torch.int32) + state["first_new"]
        state.update(mass=mass, new_table=new.view(n, width), mass_out=torch.zeros((n, case["keep"]), device="cuda"),
                     kept=torch.empty((n, case["keep"]), dtype=torch.int32, device="cuda"),
                     count=torch.empty(n, dtype=torch.int32, device="cuda"))
        return state
    h, q_len = case["heads"], case["q_len"]
    queries = case["n_seq"] * q_len
    state = dict(case, scale=D ** -0.5, **_cache(case, g))
    state["q"] = (2 * torch.randn((queries, h, D), generator=g, device="cuda")).to(torch.bfloat16)
    if op == "tree":
        # a token's parent is any token drafted before it, or what was there before the tree (-1)
        u = torch.rand((case["n_seq"], q_len), generator=g, device="cuda")
        state["parent"] = (torch.floor(u * torch.arange(1, q_len + 1, device="cuda")) - 1).to(torch.int32)
        state.update(out=torch.empty_like(state["q"]), lse=torch.empty((queries, h), dtype=torch.float32, device="cuda"),
                     mask=torch.empty((case["n_seq"], q_len, -(-q_len // 64)), dtype=torch.int64, device="cuda"),
                     pos=torch.empty((case["n_seq"], q_len), dtype=torch.int32, device="cuda"))
        return state
    # the log-sums that the step's attention left
    most = state["width"] * P
    state["lse"] = _log_sums(state)
    state["prev"] = torch.rand((case["n_seq"], most), generator=g, device="cuda") if case["adds"] else None
    state["mass"] = torch.zeros((case["n_seq"], most), device="cuda")
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


def _rows(s):
    """fp32 [n_seq, width * 64, 512]: every sequence's cached rows, in order."""
    layout, n_seq = s["layout"], s["n_seq"]
    area = P * CODE_BYTES[layout]
    pages = s["pool"].view(s["pages"], -1)[s["table"].long()]
    return _decode(layout, pages[..., :area].reshape(n_seq, -1, CODE_BYTES[layout]),
                   pages[..., area:].reshape(n_seq, -1, SCALE_BYTES[layout]))


def _causal(s):
    """[n_seq, q_len * heads, tokens]: which cached tokens a query row sees."""
    j = torch.arange(s["q_len"], device="cuda").repeat_interleave(s["heads"])
    visible = s["kv_len"][:, None] - (s["q_len"] - 1 - j)[None, :]
    return torch.arange(s["width"] * P, device="cuda")[None, None, :] < visible[..., None]


def _scores(s, seen):
    x = torch.matmul(s["q"].float().view(s["n_seq"], -1, D), _rows(s).transpose(1, 2)) * s["scale"]
    return x.masked_fill_(~seen, float("-inf"))


def _log_sums(s):
    return torch.logsumexp(_scores(s, _causal(s)), -1).view(-1, s["heads"])


def _tree_plain(s):
    n_seq, q_len, h = s["n_seq"], s["q_len"], s["heads"]
    # tokens a token descends from: the sum of all powers of "is the parent of", 0 or 1 each
    up = (s["parent"][..., None] == torch.arange(q_len, device="cuda")).float()
    eye = torch.eye(q_len, device="cuda")
    sees = torch.linalg.solve_triangular(eye - up, eye.expand(n_seq, -1, -1), upper=False) > 0.5
    words = -(-q_len // 64)
    bits = torch.nn.functional.pad(sees.long(), (0, 64 * words - q_len)).view(n_seq, q_len, words, 64)
    mask = (bits << torch.arange(64, device="cuda")).sum(-1)
    base = s["kv_len"] - q_len
    pos = (base[:, None] + sees.sum(-1) - 1).clamp_min(0).to(torch.int32)
    t = torch.arange(s["width"] * P, device="cuda")
    drafted = t[None, :] - base[:, None]
    of_tree = sees.gather(2, drafted.clamp(0, q_len - 1)[:, None, :].expand(-1, q_len, -1)) & (drafted >= 0)[:, None, :]
    seen = (of_tree | (drafted < 0)[:, None, :]) & (t[None, :] < s["kv_len"][:, None])[:, None, :]
    x = _scores(s, seen.repeat_interleave(h, 1))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isfinite(top), top, 0.0))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, _rows(s)) / torch.where(total > 0, total, 1.0)
    return {"out": out.view(-1, h, D).to(torch.bfloat16), "lse": (top + torch.log(total)).view(-1, h), "mask": mask, "pos": pos}


def _mass_plain(s):
    seen = _causal(s)
    p = torch.exp(_scores(s, seen) - s["lse"].view(s["n_seq"], -1, 1))
    total = torch.where(seen, p, 0.0).sum(1)
    if s["adds"]:
        total = total + s["prev"] * 0.98
    return {"mass": torch.where(torch.arange(s["width"] * P, device="cuda") < s["kv_len"][:, None], total, s["mass"])}


def _rope_plain(s):
    x = s["x"].float()
    a, rot = s["start"], s["rot"]
    cs = s["cos_sin"][s["pos"].long()][:, None, :]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    if s["inverse"]:
        sin = -sin
    part = x[..., a:a + rot]
    if s["half"]:
        u, v = part[..., :rot // 2], part[..., rot // 2:]
        part = torch.cat((u * cos - v * sin, v * cos + u * sin), -1)
    else:
        u, v = part[..., 0::2], part[..., 1::2]
        part = torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2)
    return {"out": torch.cat((x[..., :a], part, x[..., a + rot:]), -1).to(s["x"].dtype)}


def _rope_table_plain(s):
    pos = torch.arange(s["first"], s["first"] + s["rows"], dtype=torch.float64, device="cuda")
    angle = pos[:, None] * s["freq"]
    return {"table": (torch.cat((torch.cos(angle), torch.sin(angle)), 1) * s["amplitude"]).float()}


def _evict_plain(s):
    n, keep = s["n_seq"], s["keep"]
    t = torch.arange(s["width"] * P, device="cuda")
    lens = s["kv_len"].long()[:, None]
    key = torch.where((t < s["first"]) | (t >= lens - s["last"]), float("inf"), s["mass"])
    key = torch.where(t < lens, key, float("-inf"))
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    count = lens.clamp_max(keep)
    order = torch.nn.functional.pad(order, (0, max(0, keep - order.shape[1])))[:, :keep]
    rank = torch.arange(keep, device="cuda")
    kept = torch.where(rank < count, order, 1 << 30).sort(1).values
    live = rank < count
    at = torch.where(live, kept, 0)
    # rows go to the new pages in order; the others have a place of no use, the table's first page by itself
    layout, area = s["layout"], P * CODE_BYTES[s["layout"]]
    pages = s["pool"].view(s["pages"], -1)
    from_page = s["table"].long().gather(1, at >> PAGE_BITS)[live]
    to_page = s["new_table"].long()[:, :].gather(1, (rank >> PAGE_BITS).expand(n, -1))[live]
    from_row, to_row = (at & (P - 1))[live], (rank & (P - 1)).expand(n, -1)[live]
    codes, scales = pages[:, :area].unflatten(1, (P, CODE_BYTES[layout])), pages[:, area:].unflatten(1, (P, SCALE_BYTES[layout]))
    codes[to_page, to_row] = codes[from_page, from_row]
    scales[to_page, to_row] = scales[from_page, from_row]
    return {"kept": torch.where(live, kept, -1).to(torch.int32), "count": count.view(-1).to(torch.int32),
            "mass": torch.where(live, s["mass"].gather(1, at), s["mass_out"]), "pages": pages[s["first_new"]:]}


# ------------------------------------------------------------------ one pass

def _workspace(s, size):
    """The scratch memory that a program keeps beside its buffers."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(size(), dtype=torch.uint8, device="cuda")
    return s["workspace"]


def run(s):
    op = s["op"]
    if own:
        import compress_kv_write_gb300 as kvq
        if op == "rope":
            kvq.kvq_rope(s["x"], s["pos"], s["cos_sin"], s["out"], start=s["start"], half=s["half"], inverse=s["inverse"])
            return {"out": s["out"]}
        if op == "rope_table":
            kvq.kvq_rope_table(s["freq"], s["table"], first=s["first"], amplitude=s["amplitude"])
            return {"table": s["table"]}
        if op == "tree":
            kvq.kvq_tree_mask(s["parent"], s["mask"], kv_len=s["kv_len"], pos=s["pos"])
            kvq.kvq_attend_tree(s["layout"], PAGE_BITS, s["q"], s["pool"], s["pages"], s["table"], s["kv_len"], s["mask"],
                                s["out"], _workspace(s, lambda: kvq.attend_workspace(s["q_len"] * s["heads"])),
                                scale=s["scale"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"], "mask": s["mask"], "pos": s["pos"]}
        if op == "mass":
            kvq.kvq_attend_mass(s["layout"], PAGE_BITS, s["q"], s["lse"], s["pool"], s["pages"], s["table"], s["kv_len"],
                                s["mass"], _workspace(s, lambda: kvq.mass_workspace(s["n_seq"], s["q_len"] * s["heads"], s["width"] * P)),
                                scale=s["scale"], q_len=s["q_len"], prev=s["prev"], decay=0.98)
            return {"mass": s["mass"]}
        kvq.kvq_evict_select(s["mass"], s["kv_len"], s["kept"], s["count"], first=s["first"], last=s["last"])
        kvq.kvq_evict_move(s["layout"], PAGE_BITS, s["pool"], s["pages"], s["table"], s["new_table"], s["kept"],
                           mass=s["mass"], mass_out=s["mass_out"])
        return {"kept": s["kept"], "count": s["count"], "mass": s["mass_out"], "pages": s["pool"].view(s["pages"], -1)[s["first_new"]:]}
    if op == "rope":
        return _rope_plain(s)
    if op == "rope_table":
        return _rope_table_plain(s)
    if op == "tree":
        return _tree_plain(s)
    if op == "mass":
        return _mass_plain(s)
    return _evict_plain(s)


# ------------------------------------------------------------------ the definition in 64 bits

def _e4m3_values():
    """The 256 e4m3 values from sign, 4 exponent bits (bias 7) and 3 mantissa bits; 0x7F and 0xFF are NaN."""
    values = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = math.nan if (e, m) == (15, 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        values.append(-v if b & 128 else v)
    return torch.tensor(values, dtype=torch.float64, device="cuda")


def _row64(s, n, count):
    """The first `count` cached rows of sequence n, in 64 bits, byte by byte from the layout's definition."""
    layout, pool = s["layout"], s["pool"]
    t = torch.arange(count, device="cuda")
    page, row = s["table"][n].long()[t >> PAGE_BITS], t & (P - 1)
    base = page * (P * (CODE_BYTES[layout] + SCALE_BYTES[layout]))
    dims = torch.arange(D, device="cuda")
    codes_at = base + row * CODE_BYTES[layout]
    scale = pool[(base + P * CODE_BYTES[layout] + row * SCALE_BYTES[layout])[:, None] + dims // 32]
    if layout == V41:
        return _e4m3_values()[pool[codes_at[:, None] + dims].int()] * torch.pow(2.0, scale.double() - 127)
    byte = pool[codes_at[:, None] + dims // 2].int()
    nibble = torch.where(dims % 2 == 0, byte % 16, byte // 16)
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    return grid[nibble] * _e4m3_values()[scale.int()]


def _exact_tree(case, s):
    h, q_len = case["heads"], case["q_len"]
    q = s["q"].double()
    outs, lses, masks, places = [], [], [], []
    parents = s["parent"].tolist()
    for n, length in enumerate(_lengths(case)):
        rows = _row64(s, n, length)
        base = length - q_len
        for j in range(q_len):
            line, at = [], j
            while at >= 0:
                line.append(at)
                at = parents[n][at]
            places.append(max(0, base + len(line) - 1))
            words = [sum(1 << (k - 64 * w) for k in line if k // 64 == w) for w in range(-(-q_len // 64))]
            masks.append([w - (1 << 64) if w >> 63 else w for w in words])
            see = list(range(max(0, base))) if base < 0 else None
            picked = torch.tensor(sorted(base + k for k in line if base + k >= 0), dtype=torch.long, device="cuda")
            own_rows = rows[picked] if length else rows[:0]
            keys = own_rows if see is not None else torch.cat((rows[:base], own_rows))
            qj = q[n * q_len + j]
            if keys.shape[0] == 0:
                outs.append(torch.zeros_like(qj))
                lses.append(torch.full((h,), -math.inf, dtype=torch.float64, device="cuda"))
                continue
            x = (qj @ keys.T) * s["scale"]
            l = torch.logsumexp(x, 1)
            outs.append(torch.exp(x - l[:, None]) @ keys)
            lses.append(l)
    return {"out": torch.stack(outs), "lse": torch.stack(lses),
            "mask": torch.tensor(masks, dtype=torch.int64, device="cuda").view(s["mask"].shape),
            "pos": torch.tensor(places, dtype=torch.int32, device="cuda").view(s["pos"].shape)}


def _exact_mass(case, s):
    q_len, h = case["q_len"], case["heads"]
    got = s["mass"].double()
    for n, length in enumerate(_lengths(case)):
        rows = _row64(s, n, length)
        total = torch.zeros(length, dtype=torch.float64, device="cuda")
        for j in range(q_len):
            count = length - (q_len - 1 - j)
            if count > 0:
                at = n * q_len + j
                x = (s["q"][at].double() @ rows[:count].T) * s["scale"]
                total[:count] += torch.exp(x - s["lse"][at].double()[:, None]).sum(0)
        if case["adds"]:
            total += 0.98 * s["prev"][n, :length].double()
        got[n, :length] = total
    return {"mass": got}


def _exact_rope(case, s):
    x, out = s["x"].double(), s["x"].double().clone()
    cs = s["cos_sin"].double()[s["pos"].long()]
    r = case["rot"] // 2
    for i in range(r):
        u, v = (case["start"] + i, case["start"] + r + i) if case["half"] else (case["start"] + 2 * i, case["start"] + 2 * i + 1)
        turn = torch.complex(cs[:, i], -cs[:, r + i] if case["inverse"] else cs[:, r + i])[:, None]
        z = torch.complex(x[..., u], x[..., v]) * turn
        out[..., u], out[..., v] = z.real, z.imag
    return {"out": out}


def _exact_evict(case, s):
    kept, counts, masses = [], [], s["mass_out"].double()
    mass = s["mass"].tolist()
    for n, length in enumerate(_lengths(case)):
        row = mass[n][:length]
        sure = [t for t in range(length) if t < case["first"] or t >= length - case["last"]]
        free = [t for t in range(length) if not (t < case["first"] or t >= length - case["last"])]
        room = min(length, case["keep"]) - len(sure)
        if room < 0:
            sure, room = sure[:case["keep"]], 0
        free.sort(key=lambda t: (-row[t], t))
        got = sorted(sure + free[:room])
        masses[n, :len(got)] = torch.tensor([row[t] for t in got], dtype=torch.float64, device="cuda")
        counts.append(len(got))
        kept.append(got + [-1] * (case["keep"] - len(got)))
    return {"kept": torch.tensor(kept, dtype=torch.int32, device="cuda"), "count": torch.tensor(counts, dtype=torch.int32, device="cuda"),
            "mass": masses, "pages": None}


def exact(case, seed):
    op, todo = case["op"], work(case)
    if todo["flops"] > 1.2e12 or (op == "rope" and todo["bytes"] > 3 << 30):
        return None
    s = prepare(case, seed)
    if op == "rope":
        return _exact_rope(case, s)
    if op == "rope_table":
        # the angle in whole turns first, so that cosine and sine are of a small one
        turns = (torch.arange(case["rows"], device="cuda") + s["first"]).double()[:, None] * (s["freq"] / (2 * math.pi))[None, :]
        small = (turns - torch.round(turns)) * (2 * math.pi)
        return {"table": torch.cat((torch.cos(small), torch.sin(small)), 1) * s["amplitude"]}
    if op == "tree":
        return _exact_tree(case, s)
    if op == "mass":
        return _exact_mass(case, s)
    return _exact_evict(case, s)
