"""prompt_attention at the ends of what it takes: batches of no sequence, with outputs given and new."""
import math

import pytest
import torch

import varlen_top_select_amd as vts

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here needs the GPU
    pytest.skip("no GPU", allow_module_level=True)

DEV = "cuda"


@pytest.mark.parametrize("rows", [1, 20, 300])
def test_no_sequence(rows):
    gen = torch.Generator().manual_seed(930)
    q = torch.randn(rows, 4, 64, generator=gen).bfloat16().to(DEV)
    k, v = q[:, :2], q[:, 2:]
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 3.0)
    got, _ = vts.prompt_attention(q, k, v, none, out=out)
    assert got is out and (out == 3).all()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        new, lse = vts.prompt_attention(q, k, v, none, return_lse=True)
    for _ in range(3):
        new.fill_(5), lse.fill_(5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert (new == 0).all() and (lse == -math.inf).all()
