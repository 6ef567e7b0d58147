"""The run a serving step makes -- norm, projection, store, attention by pages and by slots -- captured into a CUDA
graph: replayed over other inputs and lengths it gives the eager calls' bits."""
import pytest
import torch

import oracle as O
from test_attend_gpu import DEV, FP4, V41, K, queries  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", [V41, FP4])
def test_step_in_a_graph(K, layout):
    from compress_kv_write_gb300 import synth
    n, dim, heads, slots = 5, 1024, 16, 512
    g = torch.Generator().manual_seed(7)
    w = synth.normal((dim,), "cpu", 1, "weight", std=0.1, mean=1.0).to(DEV)
    proj = (torch.randn((dim, 512), generator=g) / dim ** 0.5).to(DEV)
    kw, cs = synth.norm_weight("cpu", 2).to(DEV), synth.rope_table(slots, "cpu").to(DEV)
    table = torch.tensor([[1, 3, 0, 5, 2, 7, 4, 6]], dtype=torch.int32, device=DEV).repeat(n, 1)
    x, res = (torch.zeros((n, dim), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    loc, pos = torch.zeros(n, dtype=torch.int64, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
    lens, q = torch.zeros(n, dtype=torch.int32, device=DEV), torch.zeros((n, heads, 512), dtype=torch.bfloat16, device=DEV)
    sel = torch.zeros((n, 100), dtype=torch.int64, device=DEV)
    ws, err = torch.empty(K.attend_workspace(heads), dtype=torch.uint8, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)

    def buffers():
        return dict(codes=torch.zeros((n, dim), dtype=torch.uint8, device=DEV),
                    scales=torch.zeros((n, dim // 32), dtype=torch.uint8, device=DEV), total=torch.zeros_like(res),
                    pool=torch.zeros(slots * O.bytes_per_token(layout), dtype=torch.uint8, device=DEV),
                    out=torch.zeros_like(q), lse=torch.zeros((n, heads), device=DEV), out2=torch.zeros_like(q))

    def step(b):
        K.kvq_norm_quant(x, w, b["codes"], b["scales"], residual=res, residual_out=b["total"])
        y = b["codes"].view(torch.float8_e4m3fn).float().view(n, -1, 32) * torch.exp2(b["scales"].float() - 127)[..., None]
        k = (y.view(n, dim) @ proj).to(torch.bfloat16)
        K.kvq_store(layout, 6, K.FLAG_NORM | K.FLAG_ROPE, k, loc, b["pool"], slots, norm_weight=kw, cos_sin=cs, pos=pos, err=err)
        K.kvq_attend(layout, 6, q, b["pool"], slots // 64, table, lens, b["out"], ws, scale=512 ** -0.5, lse=b["lse"], err=err)
        K.kvq_attend_slots(layout, 6, q, b["pool"], slots, sel, b["out2"], ws, scale=512 ** -0.5, err=err)

    eager, captured = buffers(), buffers()
    loc.copy_(torch.arange(n))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(buffers())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(captured)
    rows = torch.randn((slots, 512), generator=g).to(torch.bfloat16).to(DEV)
    for b in (eager, captured):      # the same cache under both
        K.kvq_store(layout, 6, 0, rows, torch.arange(slots, device=DEV), b["pool"], slots)
    for at in (3, 129, 340):
        x.copy_(torch.randn((n, dim), generator=g))
        res.copy_(torch.randn((n, dim), generator=g))
        q.copy_(queries(n, heads, at))
        t = torch.arange(n, device=DEV) + at          # the sequences share the table's pages and grow by a token each
        pos.copy_(t)
        lens.copy_(t + 1)
        loc.copy_(table[0].long()[t // 64] * 64 + t % 64)
        sel.copy_(torch.randint(-1, slots, (n, 100), generator=g))
        step(eager)
        graph.replay()
        torch.cuda.synchronize()
        assert err.item() == 0
        for name in eager:
            assert torch.equal(eager[name], captured[name]), (at, name)
        assert torch.isfinite(captured["out"]).all() and captured["out"].float().abs().amax() > 0.01
