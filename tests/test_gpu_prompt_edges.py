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


def test_new_lse_beside_given_outputs():
    """Rows of no sequence get -inf in the new lse, and are left as they were in the outputs given."""
    gen = torch.Generator().manual_seed(931)
    q = torch.randn(100, 4, 64, generator=gen).bfloat16().to(DEV)
    k, v = q[:, :2], q[:, 2:]
    for cu in ([10, 40, 80], [0]):
        cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        want, want_lse = vts.prompt_attention(q, k, v, cu, return_lse=True)
        out = torch.full_like(q, 3.0)
        used = torch.full((100, 4), 5.0, device=DEV)  # (the allocator hands its memory to the lse)
        del used
        got, lse = vts.prompt_attention(q, k, v, cu, out=out, return_lse=True)
        assert torch.equal(lse, want_lse)
        assert torch.equal(got[10:80], want[10:80] if len(cu) > 1 else torch.full_like(want[10:80], 3.0))
        assert (got[:10] == 3).all() and (got[80:] == 3).all()
