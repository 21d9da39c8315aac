"""Graphs captured with a stream's default workspace, replayed after larger calls
on that stream have replaced it."""
import pytest
import torch

import varlen_top_select_amd as vts

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here needs the GPU
    pytest.skip("no GPU", allow_module_level=True)

DEV = "cuda"


def attention(gen, batch, draft, length, heads=32, kv=8, dim=64, page=16):
    width = -(-length // page)
    k, v = (torch.randn(batch * width, page, kv, dim, generator=gen).bfloat16().to(DEV) for _ in range(2))
    table = torch.randperm(batch * width, generator=gen).int().view(batch, width).to(DEV)
    lens = torch.full((batch,), length, dtype=torch.int32, device=DEV)
    q = torch.randn(batch, draft, heads, dim, generator=gen).bfloat16().to(DEV)
    return q, k, v, table, lens


def test_captures_of_growing_shapes():
    gen = torch.Generator().manual_seed(3)
    shapes = [attention(gen, 1, 1, 3000), attention(gen, 2, 8, 900), attention(gen, 16, 16, 200)]
    scores = torch.randn(2, 200000, generator=gen).to(DEV)
    rows = torch.full((2,), 200000, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    graphs, outs, sizes = [], [], []

    def step(shape, count):
        return (vts.tree_attention(*shape, return_lse=True)
                + vts.topk_varlen_ordered(scores[:count], rows[:count], 64))

    for i, shape in enumerate(shapes):
        count = min(i, 1) + 1
        with torch.cuda.stream(side):
            step(shape, count)
        side.synchronize()
        sizes.append(vts._WS_CACHE[(shape[0].device.index, side.cuda_stream, "decode")].numel())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(step(shape, count))
        graphs.append(g)
    assert sizes[0] < sizes[1] < sizes[2]
    # what the allocator would give to others of the replaced workspaces
    others = [torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]
    for _ in range(3):
        for i, (g, got) in enumerate(zip(graphs, outs)):
            shapes[i][0].copy_(torch.randn(shapes[i][0].shape, generator=gen).bfloat16())
            for x in got[:2]:
                x.fill_(7)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            want = step(shapes[i], min(i, 1) + 1)
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert torch.equal(got[2], want[2])
    assert all((x == 0x5A).all() for x in others)
