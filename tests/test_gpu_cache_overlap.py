"""write_cache refuses caches whose rows lie in the same memory; rows between each other's are taken."""
import pytest
import torch

import varlen_top_select_amd as vts

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU too; every test here needs the GPU
    pytest.skip("no GPU", allow_module_level=True)

DEV = "cuda"


def test_rows_in_the_same_memory():
    gen = torch.Generator().manual_seed(940)
    q = torch.randn(6, 2, 64, generator=gen).bfloat16().to(DEV)
    slots = torch.arange(6, dtype=torch.int32, device=DEV)
    c = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    m = [torch.zeros(4, 16, 2, 32, dtype=torch.uint8, device=DEV) for _ in "kv"]
    s = [torch.zeros(4, 16, 2, 2, dtype=torch.uint8, device=DEV) for _ in "kv"]
    for k, v, ks, vs in ((c, c, None, None), (c, c.clone()[:1].expand(4, -1, -1, -1), None, None),
                         (c[:, :, :1].expand(-1, -1, 2, -1), c.clone(), None, None), (m[0], m[0], *s),
                         (*m, s[0], s[0]), (*m, s[0][:, :1].expand(-1, 16, -1, -1), s[1])):
        with pytest.raises(ValueError, match="overlap"):
            vts.write_cache(q, q, q, slots, k, v, k_scales=ks, v_scales=vs)
    assert not c.any()


def test_rows_beside_each_other():
    """K and V of one allocation, by page and by head, and a dimension of one with any step."""
    gen = torch.Generator().manual_seed(941)
    q, k, v = (torch.randn(6, 2, 64, generator=gen).bfloat16().to(DEV) for _ in "qkv")
    slots = torch.tensor([3, 17, -1, 40, 0, 63], dtype=torch.int32, device=DEV)
    both = torch.zeros(4, 2, 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    heads = torch.zeros(4, 16, 4, 64, dtype=torch.bfloat16, device=DEV)
    for kc, vc in ((both[:, 0], both[:, 1]), (heads[:, :, :2], heads[:, :, 2:])):
        vts.write_cache(q, k, v, slots, kc, vc)
        got_k, got_v = vts.read_cache(kc, vc, slots)
        there = (slots >= 0)[:, None, None]
        assert torch.equal(got_k, torch.where(there, k, 0)) and torch.equal(got_v, torch.where(there, v, 0))
    one = torch.zeros(1, 16, 1, 64, dtype=torch.bfloat16, device=DEV).as_strided((1, 16, 1, 64), (0, 64, 0, 1))
    other = torch.zeros_like(one)
    vts.write_cache(q[:, :1], k[:, :1], v[:, :1], slots, one, other)
    assert torch.equal(vts.read_cache(one, other, slots[:1])[0], k[:1, :1])
