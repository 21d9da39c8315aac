"""Arguments of the decode-step operators at their edges, on the GPU."""
import pytest
import torch

import varlen_top_select_amd as vts

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here needs the GPU
    pytest.skip("no GPU", allow_module_level=True)

DEV = "cuda"


def step(gen, batch=2, draft=2, heads=8, kv=1, dim=64, page=16, length=70):
    width = -(-length // page)
    k, v = (torch.randn(batch * width, page, kv, dim, generator=gen).bfloat16().to(DEV) for _ in range(2))
    table = torch.randperm(batch * width, generator=gen).int().view(batch, width).to(DEV)
    lens = torch.full((batch,), length, dtype=torch.int32, device=DEV)
    q = torch.randn(batch, draft, heads, dim, generator=gen).bfloat16().to(DEV)
    return q, k, v, table, lens


def restrided(t, dim, stride):
    """t seen with another stride of a dimension of one element."""
    steps = list(t.stride())
    assert t.shape[dim] == 1
    steps[dim] = stride
    return t.as_strided(t.shape, steps)


def test_strides_of_one_element():
    gen = torch.Generator().manual_seed(80)
    q, k, v, table, lens = step(gen, draft=1)
    want, lse = vts.tree_attention(q, k, v, table, lens, return_lse=True)
    k1, v1, q1 = restrided(k, 2, 1), restrided(v, 2, 3), restrided(q, 1, 5)
    out, lse1 = vts.tree_attention(q1, k1, v1, table, lens, return_lse=True)
    assert torch.equal(out, want) and torch.equal(lse1, lse)
    weights = [torch.zeros(2, 1, 80, device=DEV) for _ in range(2)]
    vts.attention_weight_add(weights[0], q, k, table, lens, lse)
    vts.attention_weight_add(weights[1], q1, k1, table, lens, lse)
    assert torch.equal(*weights) and weights[0].any()
    moved = []
    for kk, vv in ((k, v), (k1, v1)):
        ko, vo = torch.zeros(6, 16, 1, 64, dtype=k.dtype, device=DEV), torch.zeros_like(v[:6])
        fresh = torch.arange(6, dtype=torch.int32, device=DEV).view(2, 3)
        moved.append((*vts.evict_cache(weights[0], kk, vv, table, lens, 40, restrided(ko, 2, 1), vo, fresh),
                      ko, vo))
    assert all(torch.equal(a, b) for a, b in zip(*moved))
    assert moved[0][3].any()


def test_a_table_of_one_column():
    gen = torch.Generator().manual_seed(81)
    q, k, v, table, lens = step(gen, length=16)
    column = torch.stack([table[:, 0], table[:, 0] * 0 - 1]).t()[:, :1]  # rows one apart
    assert column.stride() == (1, 2)
    want = vts.tree_attention(q, k, v, table, lens)[0]
    assert torch.equal(vts.tree_attention(q, k, v, column, lens)[0], want)


def test_empty_batch():
    gen = torch.Generator().manual_seed(82)
    _, k, v, table, _ = step(gen, kv=2)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    q = torch.zeros(0, 3, 8, 64, dtype=k.dtype, device=DEV)
    mask = torch.zeros(0, 3, dtype=torch.int64, device=DEV)
    for slots in (None, torch.zeros(0, 3, 20, dtype=torch.int32, device=DEV),
                  torch.zeros(0, 20, dtype=torch.int32, device=DEV)):
        out, lse = vts.tree_attention(q, k, v, table[:0], none, slots=slots, tree_mask=mask, return_lse=True)
        assert out.shape == q.shape and lse.shape == (0, 3, 8)
    w = vts.attention_weight_add(torch.zeros(0, 2, 80, device=DEV), q, k, table[:0], none, lse)
    kept, lens, moved = vts.evict_cache(w, k, v, table[:0], none, 16, k, v, table[:0])
    assert kept.shape == moved.shape == (0, 2, 16) and lens.shape == (0,)
    path, count, token = vts.verify_draft(torch.zeros(0, 4, 50, device=DEV),
                                          torch.zeros(0, 3, dtype=torch.int32, device=DEV),
                                          torch.zeros(0, 4, device=DEV))
    assert path.shape == (0, 3) and count.shape == token.shape == (0,)


def test_out_over_its_inputs():
    """Rows are written while others are still read: such an output is refused."""
    gen = torch.Generator().manual_seed(83)
    q, k, v, table, lens = step(gen, kv=2)
    want = vts.tree_attention(q, k, v, table, lens)[0]
    for t in (q, k, v):
        near = t.flatten()[: q.numel()].view(q.shape)
        with pytest.raises(ValueError, match="overlap"):
            vts.tree_attention(q, k, v, table, lens, out=near)
    # beside its inputs in one allocation it is none of them
    both = torch.zeros(2, *q.shape, dtype=q.dtype, device=DEV)
    both[0] = q
    out, _ = vts.tree_attention(both[0], k, v, table, lens, out=both[1])
    assert out.data_ptr() == both[1].data_ptr() and torch.equal(out, want) and torch.equal(both[0], q)


def test_weights_rows_that_coincide():
    gen = torch.Generator().manual_seed(84)
    q, k, v, table, lens = step(gen, kv=2)
    lse = vts.tree_attention(q, k, v, table, lens, return_lse=True)[1]
    for stride in ((80, 80, 1), (40, 160, 1), (0, 80, 1), (80, 0, 1)):
        w = torch.zeros(1000, device=DEV).as_strided((2, 2, 80), stride)
        with pytest.raises((ValueError, vts.VtsError)):
            vts.attention_weight_add(w, q, k, table, lens, lse)
    apart = [torch.zeros(1000, device=DEV).as_strided((2, 2, 80), s) for s in ((160, 80, 1), (80, 160, 1), (200, 90, 1))]
    for w in apart:
        vts.attention_weight_add(w, q, k, table, lens, lse)
    assert all(torch.equal(apart[0], w) for w in apart) and apart[0].any()
