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


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("front", [0, 3000])
def test_scores_that_are_not_finite(bad, front):
    """A row that sees a score of +inf or NaN gets NaN, its lse too; the rows before it do not."""
    gen = torch.Generator().manual_seed(932)
    n = 100 if front == 0 else 8
    q = torch.randn(n, 2, 64, generator=gen).bfloat16()
    q[..., 3] = q[..., 3].abs() + 0.01
    k, v = (torch.randn(front + n, 2, 64, generator=gen).bfloat16() for _ in "kv")
    at = n - 4
    k[front + at, 0, 3] = bad
    cu = [torch.tensor([0, x], dtype=torch.int32, device=DEV) for x in (n, front + n)]
    out, lse = vts.prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), cu[0], cu_seqlens_k=cu[1], return_lse=True)
    assert out[at:, 0].isnan().all() and lse[at:, 0].isnan().all()
    assert out[:at].isfinite().all() and lse[:at].isfinite().all()
    assert out[:, 1].isfinite().all() and lse[:, 1].isfinite().all()
