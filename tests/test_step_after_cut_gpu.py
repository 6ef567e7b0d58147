"""A speculative step over caches that were cut: positions go on from the length that a sequence would have without the cut,
while the attention and the store take the cut one.  Checked against 64 bits over caches that were never cut."""
import numpy as np
import pytest
import torch

import oracle as O
from test_attend_gpu import DEV, FP4, V41, K, check, decode, reference  # noqa: F401
from test_rope_gpu import bits, turned
from test_tree_gpu import lines, some_parents

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", [V41, FP4])
def test_step_after_a_cut(K, layout):
    n, q_len, heads, width, keep, scale = 3, 9, 16, 6, 90, 512 ** -0.5
    full = [300, 91, 40]                       # tokens before the step; the last sequence stays whole
    g = torch.Generator().manual_seed(7)
    pages = n * width + n * 2
    table = torch.randperm(n * width, generator=g).view(n, width).to(torch.int32)
    new = (n * width + torch.arange(n * 2)).view(n, 2).to(torch.int32)
    td, nd = table.to(DEV), new.to(DEV)
    cs = torch.empty((4096, 64), device=DEV)
    K.kvq_rope_table(K.rope_frequencies(64, factor=8, original=1024).to(DEV), cs)
    pool = torch.zeros(pages * 64 * O.bytes_per_token(layout), dtype=torch.uint8, device=DEV)
    # the caches: token t of a sequence is rotated by position t
    for i, m in enumerate(full):
        rows, t = torch.randn((m, 512), generator=g).to(torch.bfloat16).to(DEV), torch.arange(m)
        K.kvq_store(layout, 6, K.FLAG_ROPE, rows, (table[i].long()[t >> 6] * 64 + (t & 63)).to(DEV), pool, pages * 64, cos_sin=cs,
                    pos=t.to(torch.int32).to(DEV))
    uncut = pool.clone()
    lens = torch.tensor(full, dtype=torch.int32, device=DEV)
    mass = torch.rand((n, width * 64), generator=g).to(DEV)
    kept, count = torch.zeros((n, keep), dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
    K.kvq_evict_select(mass, lens, kept, count, first=2, last=5)
    K.kvq_evict_move(layout, 6, pool, pages, td, nd, kept)

    # a step: drafted tokens behind the uncut length in position, behind the cut one in the cache
    parent = torch.from_numpy(some_parents(n, q_len, 3)).to(DEV)
    mask, pos = torch.zeros((n, q_len, 1), dtype=torch.int64, device=DEV), torch.zeros((n, q_len), dtype=torch.int32, device=DEV)
    K.kvq_tree_mask(parent, mask, kv_len=lens + q_len, pos=pos)
    sees = [lines(p) for p in parent.tolist()]
    assert pos.tolist() == [[full[i] + len(s) - 1 for s in sees[i]] for i in range(n)]
    q = (2 * torch.randn((n * q_len, heads, 512), generator=g)).to(torch.bfloat16)
    k = torch.randn((n * q_len, 512), generator=g).to(torch.bfloat16)
    qd, out, lse = q.to(DEV), torch.zeros(q.shape, dtype=torch.bfloat16, device=DEV), torch.zeros(q.shape[:2], device=DEV)
    K.kvq_rope(qd, pos.view(-1), cs, qd, start=448)
    assert torch.equal(bits(qd), bits(turned(q, pos.view(-1).cpu(), cs.cpu(), 448, False, False)))
    for p, t, at in ((pool, nd, count), (uncut, td, lens)):
        to = (at[:, None] + torch.arange(q_len, device=DEV)).long()
        K.kvq_store(layout, 6, K.FLAG_ROPE, k.to(DEV), (t.long().gather(1, to >> 6) * 64 + (to & 63)).view(-1), p, pages * 64, cos_sin=cs,
                    pos=pos.view(-1))
    ws = torch.empty(K.attend_workspace(q_len * heads), dtype=torch.uint8, device=DEV)
    K.kvq_attend_tree(layout, 6, qd, pool, pages, nd, count + q_len, mask, out, ws, scale=scale, lse=lse)

    want, held = [], uncut.cpu().numpy()
    for i, m in enumerate(full):
        t = np.arange(m + q_len)
        rows = decode(layout, 6, held, table[i].numpy().astype(np.int64)[t >> 6] * 64 + (t & 63))
        stays = [int(x) for x in kept[i].tolist() if x >= 0]
        assert len(stays) == min(m, keep) and pos[i].min().item() > stays[-1] == m - 1
        for j in range(q_len):
            s = np.array(stays + [m + d for d in sees[i][j]])
            want.append(reference(layout, qd[i * q_len + j].cpu().double().numpy(), rows[s], scale))
    check(out, lse, want, "cut")
